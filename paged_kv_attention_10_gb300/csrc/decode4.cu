// Paged decode attention over a 4-bit cache (one query per request).
//
// What it computes: with the cache's values k[j] and v[j] (e2m1 codes times an e4m3 scale per 16 of them times one
// scale g per cache),  out = sum_j softmax_j(scale q . k[j]) v[j],  page lists, GQA and LSE as in the bf16 decode.
// The plan is the 8-bit decode's (quant_decode.cuh).  A position's bytes are nearly halved again, the values are as
// many, so the loop has to be lean: the conversions alone are an instruction for every two values.
//
//  * A code times its block's scale is exact in f16 (two bits times four), and the caches' scales g go into the score's
//    scale and the result's.  Both products run as f16 m16n8k16 MMAs with fp32 accumulators, Q scaled per head by a
//    power of two into f16's range as in the 8-bit decode.
//  * A product's k-slots may hold the dimensions in any order if both operands agree, and so may the rows of its
//    result.  A lane therefore takes consecutive bytes of a row: of K, a quarter of a position's row (dims 32c ..
//    32c + 31 of 128), which holds whole blocks, so that it needs two scales of the eight; of V, an eighth (dims 16g ..
//    16g + 15), one block, of the positions that its k-slots stand for.
//  * V's operand pairs two positions in a register: the codes of both are put side by side in bytes first (two
//    instructions for four pairs), then converted.
//  * Groups of up to four query heads (FEW) leave half of a product's eight columns idle, and the instructions that would
//    prepare the operands are what the loop is made of.  So the columns take the heads twice.  Of K, columns 0 to 3 see
//    Q in the dimensions of even blocks and zeros elsewhere, 4 to 7 those of odd blocks: the codes go into the product
//    unscaled (whole words of a row, by ldmatrix), and two blocks' sums come out apart and are scaled in fp32.  The two lanes
//    with the parts of the same scores add them up for half of the rows each, so a weight is formed once.  Of V, columns
//    0 to 3 sum the even dimensions and 4 to 7 the odd ones: a byte, which holds one of each of one position, is converted
//    as it is, and the weights of the other position's slots are 0.  (8 requests of 32768, 32/8 heads: 56.2 us, 58.6 as for
//    larger groups; 16 of 32000, 16/8 heads of 64: 62.0, 66.7; one KV head at page size 64: 28.3, 30.7.)
//  * The sixteen score rows of an MMA are the positions in an order in which the loads of K (two positions by four
//    quarters at a time) and of V (four positions by four eighths) meet no shared-memory bank twice, see position().
//  * A step is 64 positions of a head, four score tiles whose chains overlap: there are only two consumer warps to a
//    scheduler, since each holds O for all of its heads (32 and 64 values a lane) and the operands of a tile.  (Sixteen
//    warps with 32 positions each spill: 62 us where eight with 64 take 58; 38.6 and 34.8 with 28/4 heads.)  Of head_dim
//    64 all of that is half as much and sixteen warps with 64 positions fit.  A step with at most 32 positions left takes two tiles.
//  * Softmax weights are rounded to f16 in [0, 2^15], 11 bits of each (8 in the bf16 decode); their sum is taken before the
//    rounding, so that the LSE is that of the scores.  O and the sum carry 2^(kWeightExp), which cancels.
//
// Bound by HBM in the long run (32/8 heads of 128, page size 16: from 8 requests of 32768 positions to 8 of 98304 a
// position more costs what it does at 6.7 TB/s, 98 % of what a device copy reaches), and by about 12 us that do not
// depend on the length: the loads that come before the first stage 3, the CTAs' different speeds 2, the last stage's
// step 1.4, the grid's end 1.7, the merge 2.  8 requests of 32768 positions 56 us, 302 MB at 5.4 TB/s (80 %); 256 of 512
// to 4096 120 us, 5.7 TB/s (84 %).  DRAM reads are the cache's bytes (302 of 302 MB), the issue slots 56 % used, the conversions'
// pipe 48 %, the tensor pipe 28 %.  32 requests of 100 to 640 positions, 16/8 heads, at page size 1 11.5 us; 4 short ones of
// 14/2 heads of 64 7.5 us, a chain of latencies.  With head_dim 64 the softmax of a position, the
// scales and the loop's frame cost what they cost with 128, so the consumers do not keep up: 16 requests of 32000 positions,
// 16/8 heads 59 us at page size 32, 62 at 16, of 43.5 that their bytes take and 52 that they take to arrive.  (28/4 heads of 128,
// 64 requests of 1000 to 6000: 34.6 us, 29.6 to arrive, 19.0 for the bytes.)
#include <type_traits>

#include "quant_decode.cuh"

namespace {

using namespace pkv;

// The weights of a row are 2^((s - m) scale + kWeightExp), s a product before its scale and m one near the largest so far: m moves
// only when a score is more than kHeadroom above it, so that most steps need no maximum over lanes and no rescaling.  Weights then
// stand in [0, 2^15], the top of f16's range; one as small as 2^-32 of m's own is still counted.  The difference comes first since it
// is exact next to m, whatever the scores' size.  As an fma of s with kWeightExp - m scale, one instruction less, an exponent is
// off by a unit in the last place of the score, at 2^27 (base 2) by 16: past f16's largest, or 0.  (So, and as that fma: 8 requests
// of 32768, 32/8 heads, 56.0 and 55.8 us; 256 of 512 to 4096 118.8 both; 64 of 1000 to 6000, 28/4 heads, 34.5 both.  The fma below
// scores of 2^20 and the difference above: 56.2, 120.0 and 34.9.)
constexpr int kWeightExp = 8, kHeadroom = 7;

// The position, of eight consecutive ones, that row r of a score tile stands for.  K's loads of rows 2i and 2i + 1 and
// V's of rows 0, 2, 4, 6 and of 1, 3, 5, 7 are then free of bank conflicts.  Rows of 64 bytes, 16-byte pieces p of row t at
// p ^ (t >> 1 & 3): 0 1 3 2 4 5 7 6 where a head has the whole row, 0 1 5 4 6 7 3 2 where it has half; rows of 32 bytes:
// 0 2 1 3 6 4 7 5.
template <int D>
PKV_DEV int position(int r, bool pair) {
  if (D == 128) return r ^ ((r >> 1) & 1);
  return ((pair ? 0x23764510 : 0x57463120) >> (4 * r)) & 7;
}

template <int D, bool FEW>
struct Format4 {
  static constexpr int kDim = D, kRowBytes = D / 2, kScaleBytes = D / 16, kStep = 64, kParts = 2;
  static constexpr int kWarps = D == 64 ? 16 : 8;  // 16 requests of 32000 positions, 16/8 heads of 64: 62 us with sixteen, 75 with eight
  static constexpr bool kBoxedRows = true, kJoint = true, kScalesAnywhere = true;
  static constexpr int kRowPad = 0;
  static constexpr int kTiles = FEW ? D / 32 : D / 16;  // row tiles of O
  static constexpr int kMergeFloats = 4 + 4 * kTiles;
  template <bool>
  static __device__ void consume(const QuantDecodeArgs& a, uint8_t* stages, StageHdr* hdr, uint64_t* hdr_full,
                                 uint64_t* full, uint64_t* empty, uint64_t* meet_bar);
};

template <int N>
PKV_DEV void lds(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}

PKV_DEV uint32_t lds_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
PKV_DEV uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// D = A * B, as mma_f16_16816.
PKV_DEV void mma_f16_16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Four bytes of a and b (4 to 7), each by its nibble of `which`; with 8 added, its sign in all eight bits.
PKV_DEV uint32_t prmt(uint32_t a, uint32_t b, uint32_t which) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(which));
  return d;
}

PKV_DEV float2 half2_to_floats(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

// The product of an f16 pair with the low (high) half of another, which the instruction reads in place.
PKV_DEV uint32_t mul_f16x2_low(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 t;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 t, {l, l};\n\tmul.rn.f16x2 %0, %1, t;\n\t}"
      : "=r"(d)
      : "r"(a), "r"(b));
  return d;
}
PKV_DEV uint32_t mul_f16x2_high(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 t;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 t, {h, h};\n\tmul.rn.f16x2 %0, %1, t;\n\t}"
      : "=r"(d)
      : "r"(a), "r"(b));
  return d;
}

// ---------------------------------------------------------------------------------------------
// Consumer warps: steps of kStep positions of one KV head with its G query heads (eight of them, of groups of more).
// ---------------------------------------------------------------------------------------------
template <int D, bool FEW>
template <bool>
__device__ void Format4<D, FEW>::consume(const QuantDecodeArgs& a, uint8_t* stages, StageHdr* hdr, uint64_t* hdr_full,
                                         uint64_t* full, uint64_t* empty, uint64_t* meet_bar) {
  constexpr int RH = kRowBytes, SH = kScaleBytes, NT = kTiles;
  constexpr int NM = D / 16;          // MMAs of a score tile
  constexpr int KW = D / 32;          // words of a lane's share of a K row
  constexpr int VW = D / 64;          // ... of a V row
  constexpr int MF = kMergeFloats;    // floats per lane merged between the warps of a head
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int HC = a.HC, W = a.W, G = a.group, Ts = a.stage_tokens;
  const int HV = HC * a.nt;
  const int hv = warp % HV;
  const int hl = hv / a.nt, head0 = hv % a.nt * 8;  // KV head within the CTA's group, first of its query heads here
  const int si = warp / HV;                         // slice within a stage
  const int g = lane >> 2, c = lane & 3;
  const int NS = a.num_stages;
  const int HQU = HC * G;  // query heads per unit

  // Shared-memory places within a stage of the slice's first eight positions: of K, of V's rows 2c and 2c + 1 (the
  // lane's eighth g), and of the scales of row g.
  const int t0 = si * kStep;
  const bool pair = D == 64 && a.pair == 2;  // two heads to a box's row
  const int in_pair = pair ? hl & 1 : 0;
  const uint32_t first = (uint32_t)(((t0 / a.box_rows) * HC + hl - in_pair) * a.box_rows + t0 % a.box_rows * (pair ? 2 : 1)) * RH;
  auto piece = [&](int t, int p) -> uint32_t {  // 16-byte piece p of position t of eight, in the boxes' swizzle
    if (D == 128 || pair) return first + (uint32_t)(t * 64 + (((p + 2 * in_pair) ^ ((t >> 1) & 3)) << 4));
    return first + (uint32_t)(t * 32 + ((p ^ ((t >> 2) & 1)) << 4));
  };
  const int pk = position<D>(g, pair), pa = position<D>(2 * c, pair), pb = position<D>(2 * c + 1, pair);
  const uint32_t base = smem_u32(stages);
  // FEW: the row that the lane addresses for ldmatrix, of piece lane / 8 of four (of two, of the next eight positions'
  // row from lane 16 on).  Else its own bytes of row g.
  const int pl = position<D>(lane & 7, pair);
  const uint32_t k_at =
      base + (FEW ? D == 128 ? piece(pl, lane >> 3) : piece(pl, (lane >> 3) & 1) + (lane >= 16 ? a.eight : 0u)
                  : D == 128 ? piece(pk, c) : piece(pk, c >> 1) + (c & 1) * 8);
  const uint32_t v_at = base + a.kv_region;
  const uint32_t va_at = v_at + (D == 128 ? piece(pa, g >> 1) + (g & 1) * 8 : piece(pa, g >> 2) + (g & 3) * 4);
  const uint32_t vb_at = v_at + (D == 128 ? piece(pb, g >> 1) + (g & 1) * 8 : piece(pb, g >> 2) + (g & 3) * 4);
  const uint32_t s_at = base + 2 * a.kv_region + (uint32_t)(((t0 + pk) * HC + hl) * SH);
  const uint32_t s_eight = 8 * HC * SH;
  auto tile_off = [&](int hf) -> uint32_t { return (hf & 1) * a.sixteen + (hf >> 1) * (uint32_t)(HC * 32 * RH); };
  // two scales of a row: of the blocks 2c and 2c + 1 of eight, or twice of block c of four
  auto scales = [&](uint32_t at) -> uint32_t { return D == 128 ? lds_u16(at + 2 * c) : lds_u8(at + c) * 0x101u; };
  // FEW: which bytes of a row's scales are those of the lane's blocks, and how the weights of rows 2c and 2c + 1 of each half
  // of a tile go into B, out of the two halves' registers (a 9 takes a weight's sign, which is 0).
  const uint32_t pick = c < 2 ? 0x6420u : 0x7531u;
  const uint32_t put_a[2] = {g < 4 ? 0x9910u : 0x5499u, g < 4 ? 0x9954u : 0x1099u};
  const uint32_t put_b[2] = {g < 4 ? 0x9932u : 0x7699u, g < 4 ? 0x9976u : 0x3299u};
  constexpr int NR = FEW ? 1 : 2;        // rows of a tile that a lane has the scores of: g and g + 8, or one of them
  const int row8 = FEW && c >= 2 ? 8 : 0;  // FEW: g + 8 in the upper columns' lanes

  uint32_t qf[NM][2];
  float qs[2];       // score scale (log2 units) of the lane's two heads, positive
  float o[NT][4];
  float m[2], l[2];  // what the weights are relative to (before the scale, in the segment's steps), and the sum of the lane's own

  int stage = 0;
  uint32_t phase = 0, met_phase = 0;
  // All consumer warps (a bounded wait, unlike a hardware barrier's).
  auto meet = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(meet_bar);
    const bool ok = __all_sync(0xffffffffu, mbar_wait(meet_bar, met_phase));
    met_phase ^= 1;
    return ok;
  };
  auto wait = [&](uint64_t* bar) -> bool {
    if (__all_sync(0xffffffffu, mbar_wait(bar, phase))) return true;
    if (lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
    return false;
  };
  while (true) {
    if (!wait(&hdr_full[stage])) return;
    const StageHdr h = hdr[stage];  // the first stage of a segment, or the end
    if (h.unit < 0) return;

    {
      // q fragments.  Lane (g, c) holds head head0 + g's dims of its quarter c.  FEW: head g % 4's dims 8c .. 8c + 7 of
      // every 32, and only where they lie in the block that column g is for: the even ones for columns 0 to 3.
      const int head = FEW ? g & 3 : head0 + g;
      const bool valid = head < G && (!FEW || (g < 4) == (c < 2));
      const __nv_bfloat16* qp =
          a.q + ((int64_t)h.b * a.num_q_heads + (int64_t)(h.hg * HC + hl) * G + head) * D + c * (FEW ? 8 : D / 4);
      uint32_t raw[2 * NM];
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < NM / 2; ++i) {
        const uint4 u = valid ? ld(reinterpret_cast<const uint4*>(qp + i * (FEW ? 32 : 8))) : make_uint4(0u, 0u, 0u, 0u);
        raw[4 * i] = u.x, raw[4 * i + 1] = u.y, raw[4 * i + 2] = u.z, raw[4 * i + 3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < 2 * NM; ++i)
        amax = max(amax, max(finite_abs_bits(__uint_as_float(raw[i] << 16)),
                             finite_abs_bits(__uint_as_float(raw[i] & 0xffff0000u))));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      if (FEW) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
      // 2^e <= amax < 2^(e+1); q 2^(14 - e) goes into f16 and 2^(e - 14) into the score scale.  e is
      // held at -100 and above so that both factors are normal numbers.  The scale's sign goes into q; a scale of 0
      // (or one that is too small to be told from it) makes q 0 instead.
      const int e = max((int)(amax >> 23) - 127, -100);
      const float down = fabsf(a.scale_log2) * exp2i(e - 14);
      const float up = down == 0.f ? 0.f : copysignf(exp2i(14 - e), a.scale_log2);
      const float pos = down == 0.f ? 1.f : down;
#pragma unroll
      for (int i = 0; i < 2 * NM; ++i)
        qf[i / 2][i % 2] = pack_f16x2(__uint_as_float(raw[i] << 16) * up, __uint_as_float(raw[i] & 0xffff0000u) * up);
      // columns 2c and 2c + 1 of the tile live in lanes 8c and 8c + 4
      qs[0] = __shfl_sync(0xffffffffu, pos, 8 * c);
      qs[1] = __shfl_sync(0xffffffffu, pos, 8 * c + 4);
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][i] = 0.f;
    }

    int left = h.left;
    const int sharers = min(W, (left + kStep - 1) / kStep);  // warps of a head with positions in the segment
    while (true) {  // the segment's stages
      if (!wait(&full[stage])) return;
      const int nv = left - si * kStep;  // positions of the step, at least where it is below kStep
      // A segment's last stage is held when warps share its head: its memory carries their merge.
      const bool last = left <= Ts, hold = last && sharers > 1;
      const uint32_t at = (uint32_t)stage * a.stage_bytes;
      // A step of NH tiles of 16 positions.
      auto step = [&](auto tiles) {
        constexpr int NH = decltype(tiles)::value;
        float s[NH][2 * NR];
#pragma unroll
        for (int hf = 0; hf < NH; ++hf) {
          const uint32_t ka = k_at + at + tile_off(hf), sa = s_at + at + 2 * hf * s_eight;
          if constexpr (FEW) {
            uint32_t w[2][KW];  // rows g and g + 8: word c of each 16-byte piece
            float ks[2][KW];    // ... and the scale of its block
            if constexpr (D == 128) {
              ldsm_x4(ka, w[0][0], w[0][1], w[0][2], w[0][3]);
              ldsm_x4(ka + a.eight, w[1][0], w[1][1], w[1][2], w[1][3]);
            } else {
              ldsm_x4(ka, w[0][0], w[0][1], w[1][0], w[1][1]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t b[VW];
              lds<VW>(sa + i * s_eight, b);
              const uint32_t four = __byte_perm(b[0], VW == 2 ? b[VW - 1] : 0u, pick);
              uint32_t two[2];
              unpack_e4m3x4(four, two[0], two[1]);
#pragma unroll
              for (int j = 0; j < KW / 2; ++j) {
                const float2 f = half2_to_floats(two[j]);
                ks[i][2 * j] = f.x;
                ks[i][2 * j + 1] = f.y;
              }
            }
            float t[4];
#pragma unroll
            for (int j = 0; j < KW; ++j) {
              uint32_t x[4], y[4];
              float d[4];
              unpack_e2m1x8(w[0][j], x);
              unpack_e2m1x8(w[1][j], y);
              mma_f16_16816_zero(d, x[0], y[0], x[1], y[1], qf[2 * j][0], qf[2 * j][1]);
              mma_f16_16816(d, x[2], y[2], x[3], y[3], qf[2 * j + 1][0], qf[2 * j + 1][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) t[i] = j == 0 ? d[i] * ks[i / 2][0] : fmaf(d[i], ks[i / 2][j], t[i]);
            }
            // lanes c and c ^ 2 have the two parts of the same scores: one adds them up for row g, the other for g + 8
#pragma unroll
            for (int k = 0; k < 2; ++k)
              s[hf][k] = (row8 ? t[2 + k] : t[k]) + __shfl_xor_sync(0xffffffffu, row8 ? t[k] : t[2 + k], 2);
          } else {
            uint32_t w[2][KW];  // rows g and g + 8: codes, and the scales of the two halves of the lane's quarter
            lds<KW>(ka, w[0]);
            lds<KW>(ka + a.eight, w[1]);
            const uint32_t ks[2] = {unpack_e4m3x2(scales(sa)), unpack_e4m3x2(scales(sa + s_eight))};
#pragma unroll
            for (int j = 0; j < KW; ++j) {
              uint32_t x[4], y[4];
              unpack_e2m1x8(w[0][j], x);
              unpack_e2m1x8(w[1][j], y);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                x[i] = 2 * j < KW ? mul_f16x2_low(x[i], ks[0]) : mul_f16x2_high(x[i], ks[0]);
                y[i] = 2 * j < KW ? mul_f16x2_low(y[i], ks[1]) : mul_f16x2_high(y[i], ks[1]);
              }
              if (j == 0)
                mma_f16_16816_zero(s[hf], x[0], y[0], x[1], y[1], qf[0][0], qf[0][1]);
              else
                mma_f16_16816(s[hf], x[0], y[0], x[1], y[1], qf[2 * j][0], qf[2 * j][1]);
              mma_f16_16816(s[hf], x[2], y[2], x[3], y[3], qf[2 * j + 1][0], qf[2 * j + 1][1]);
            }
          }
        }
        uint32_t bp[NH][2];
        if (nv < 16 * NH) {
#pragma unroll
          for (int hf = 0; hf < NH; ++hf)
#pragma unroll
            for (int i = 0; i < 2 * NR; ++i)
              if (16 * hf + 8 * (i >> 1) + row8 + pk >= nv) s[hf][i] = -INFINITY;
        }
        float top[2];
        bool far = false;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          top[k] = s[0][k];
#pragma unroll
          for (int i = 1; i < NR * NH; ++i) top[k] = fmaxf(top[k], s[i / NR][2 * (i % NR) + k]);
          far |= (top[k] - m[k]) * qs[k] > (float)kHeadroom;
        }
        if (__any_sync(0xffffffffu, far)) {
#pragma unroll
          for (int off = FEW ? 2 : 4; off < 32; off <<= 1)
#pragma unroll
            for (int k = 0; k < 2; ++k) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], off));
          float corr[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float mn = fmaxf(m[k], top[k]);
            corr[k] = m[k] == -INFINITY ? 1.f : ex2((m[k] - mn) * qs[k]);  // nothing so far, or NaN: sums that stay what they are
            m[k] = mn;
            l[k] *= corr[k];
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[t][i] *= corr[i & 1];
        }
#pragma unroll
        for (int hf = 0; hf < NH; ++hf)
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            const float w0 = ex2(fmaf(s[hf][2 * i] - m[0], qs[0], (float)kWeightExp)),
                        w1 = ex2(fmaf(s[hf][2 * i + 1] - m[1], qs[1], (float)kWeightExp));
            l[0] += w0;
            l[1] += w1;
            bp[hf][i] = movmatrix_t(pack_f16x2(w0, w1));
          }
        if constexpr (FEW) {  // column g's weights of one half of the tile's rows; of the other from the lanes of column g ^ 4
#pragma unroll
          for (int hf = 0; hf < NH; ++hf) bp[hf][1] = __shfl_xor_sync(0xffffffffu, bp[hf][0], 16);
        }
#pragma unroll
        for (int hf = 0; hf < NH; ++hf) {
          const uint32_t aa = va_at + at + tile_off(hf), ab = vb_at + at + tile_off(hf);
          const uint32_t sa = s_at + at + (uint32_t)(Ts * HC * SH) + 2 * hf * s_eight;
          uint32_t wa[2][VW], wb[2][VW], vs[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            lds<VW>(aa + i * a.eight, wa[i]);
            lds<VW>(ab + i * a.eight, wb[i]);
            uint32_t two = scales(sa + i * s_eight);
            // Rows past the request's end hold unused pool slots (the boxes bring them) or what shared memory held
            // before, NaN scales among them: with a scale of 0 their values are 0, and 0 times their weight 0 stays 0.
            if (nv < 16 * NH && 16 * hf + 8 * i + pk >= nv) two = 0;
            // position g's scales of two blocks become block g's (g / 2's) scales of two positions
            vs[i] = movmatrix_t(unpack_e4m3x2(two));
          }
          if constexpr (FEW) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // row 2c's weight and row 2c + 1's, for the even dims in columns 0 to 3, for the odd ones in 4 to 7
              const uint32_t b0 = prmt(bp[hf][0], bp[hf][1], put_a[i]), b1 = prmt(bp[hf][0], bp[hf][1], put_b[i]);
#pragma unroll
              for (int j = 0; j < VW; ++j) {
                uint32_t x[4], y[4];
                unpack_e2m1x8(wa[i][j], x);
                unpack_e2m1x8(wb[i][j], y);
#pragma unroll
                for (int u = 0; u < 2; ++u)
                  mma_f16_16816(o[2 * j + u], mul_f16x2_low(x[2 * u], vs[i]), mul_f16x2_low(x[2 * u + 1], vs[i]),
                                mul_f16x2_high(y[2 * u], vs[i]), mul_f16x2_high(y[2 * u + 1], vs[i]), b0, b1);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < VW; ++j) {
              uint32_t e[2][4], f[2][4];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                // even and odd dims: byte = (row 2c, row 2c + 1)
                unpack_e2m1x8((wa[i][j] & 0x0f0f0f0fu) | ((wb[i][j] << 4) & 0xf0f0f0f0u), e[i]);
                unpack_e2m1x8(((wa[i][j] >> 4) & 0x0f0f0f0fu) | (wb[i][j] & 0xf0f0f0f0u), f[i]);
              }
#pragma unroll
              for (int u = 0; u < 4; ++u)
                mma_f16_16816(o[4 * j + u], mul_f16x2(e[0][u], vs[0]), mul_f16x2(f[0][u], vs[0]),
                              mul_f16x2(e[1][u], vs[1]), mul_f16x2(f[1][u], vs[1]), bp[hf][0], bp[hf][1]);
            }
          }
        }
      };
      if (nv > kStep / 2) step(std::integral_constant<int, kStep / 16>());
      else if (nv > 0) step(std::integral_constant<int, kStep / 32>());
      __syncwarp();
      if (!hold && lane == 0) mbar_arrive(&empty[stage]);
      if (last) break;
      left -= Ts;
      if (++stage == NS) {
        stage = 0;
        phase ^= 1;
      }
    }

#pragma unroll
    for (int k = 0; k < 2; ++k) m[k] *= qs[k];  // log2 units, as the other warps' and the LSE
    if (sharers > 1) {
      // Combine the warps that split this head's positions (all consumer warps reach the segment end on
      // the same stage).
      bool met = meet();
      float* buf = reinterpret_cast<float*>(stages + (size_t)stage * a.stage_bytes) + lane;
      // all but one at once where their states fit into the stage, else half of them, or as many as do, at a time
      const int room = (int)(a.stage_bytes / (uint32_t)(HV * MF * 128));
      for (int some = sharers; met && some > 1;) {
        const int keep = some - 1 <= room ? 1 : max(some / 2, some - room);
        if (si >= keep && si < some) {
          float* to = buf + ((si - keep) * HV + hv) * MF * 32;
          int e = 0;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            to[(e++) * 32] = m[k];
            to[(e++) * 32] = l[k];
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) to[(e++) * 32] = o[t][i];
        }
        met = meet();
        if (!met) break;
        if (si < keep) {
          for (int w = si; w < some - keep; w += keep) {
            const float* ob = buf + (w * HV + hv) * MF * 32;
            // one that has seen only NaN (or nothing) keeps its sums: they are NaN or 0
            auto weight = [](float x, float top) { return x == -INFINITY ? 1.f : ex2(x - top); };
            int e = 0;
            float fa[2], fb[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float om = ob[(e++) * 32], ol = ob[(e++) * 32];
              const float mn = fmaxf(m[k], om);
              fa[k] = weight(m[k], mn);
              fb[k] = weight(om, mn);
              l[k] = l[k] * fa[k] + ol * fb[k];
              m[k] = mn;
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[t][i] = o[t][i] * fa[i & 1] + ob[(e++) * 32] * fb[i & 1];
          }
        }
        some = keep;
        if (some > 1) met = meet();  // read before the next writes
      }
      if (!met) {
        if (lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
        return;
      }
      fence_proxy_async_smem();  // the merge's accesses, before the next async fill
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
    }
    if (si == 0) {
      const bool whole = (h.flags & kStartsUnit) && (h.flags & kEndsUnit);
#pragma unroll
      for (int off = FEW ? 2 : 4; off < 32; off <<= 1)
#pragma unroll
        for (int k = 0; k < 2; ++k) l[k] += __shfl_xor_sync(0xffffffffu, l[k], off);
      // Four consecutive dims g D/8 + 4j .. + 3 of query head `col` of the group, in r[j].
      auto store = [&](int col, const float (&r)[D / 32][4], float sum, float top, bool one) {
        if (col >= G) return;
        const int qhl = hl * G + col;
        const float inv = a.out_scale / sum, lse_v = (top + log2f(sum) - (float)kWeightExp) * kLn2;
        if (whole) {
          const int64_t qh = (int64_t)h.b * a.num_q_heads + (int64_t)h.hg * HQU + qhl;
          uint4* op = reinterpret_cast<uint4*>(a.out + qh * D + g * (D / 8));
#pragma unroll
          for (int j = 0; j < D / 32; j += 2)
            op[j / 2] = make_uint4(pack_bf16x2(r[j][0] * inv, r[j][1] * inv), pack_bf16x2(r[j][2] * inv, r[j][3] * inv),
                                   pack_bf16x2(r[j + 1][0] * inv, r[j + 1][1] * inv),
                                   pack_bf16x2(r[j + 1][2] * inv, r[j + 1][3] * inv));
          if (one && a.lse) a.lse[qh] = lse_v;
        } else {
          const int64_t row = (int64_t)h.part * HQU + qhl;
          float4* pp = reinterpret_cast<float4*>(a.part_o + row * D + g * (D / 8));
#pragma unroll
          for (int j = 0; j < D / 32; ++j) pp[j] = make_float4(r[j][0] * inv, r[j][1] * inv, r[j][2] * inv, r[j][3] * inv);
          if (one) a.part_lse[row] = lse_v;
        }
      };
      float r[D / 32][4];
      if constexpr (FEW) {
        // Tile j's rows g and g + 8 are dims 4j and 4j + 2 in columns 0 to 3, the ones behind them in 4 to 7: lanes c and
        // c ^ 2 hold the even and the odd dims of the same two heads.  The lower takes the first head, the upper the second.
        const bool up = c >= 2;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mine = up ? o[j][2 * i + 1] : o[j][2 * i], theirs = up ? o[j][2 * i] : o[j][2 * i + 1];
            const float other = __shfl_xor_sync(0xffffffffu, theirs, 2);
            r[j][2 * i] = up ? other : mine;
            r[j][2 * i + 1] = up ? mine : other;
          }
        store(2 * (c & 1) + (up ? 1 : 0), r, up ? l[1] : l[0], up ? m[1] : m[0], g == 0);
      } else {
        // tile t: row g is dim 2t, row g + 8 the one behind it
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) r[j][i] = o[2 * j + i / 2][2 * (i % 2) + k];
          store(head0 + 2 * c + k, r, l[k], m[k], g == 0);
        }
      }
      if (warp == 0 && lane == 0) {
        if (h.flags & kStartsUnit) a.unit_first[h.unit] = h.part;
        if (h.flags & kEndsUnit) a.unit_last[h.unit] = h.part;
      }
    }
    if (++stage == NS) {
      stage = 0;
      phase ^= 1;
    }
  }
}

}  // namespace

extern "C" {

size_t pkv_decode_fp4_workspace_size(int32_t batch_size, int32_t num_q_heads, int32_t num_kv_heads,
                                     int32_t head_dim) {
  if (head_dim == 128) return quant_decode_workspace<Format4<128, true>>(batch_size, num_q_heads, num_kv_heads);
  if (head_dim == 64) return quant_decode_workspace<Format4<64, true>>(batch_size, num_q_heads, num_kv_heads);
  return 0;
}

pkv_status pkv_paged_decode_fp4(const pkv_pool_fp4* pool, const void* q, int32_t batch_size,
                                int32_t num_q_heads, const int32_t* kv_indptr, const int32_t* kv_indices,
                                const int32_t* kv_lens, float sm_scale, void* out, float* lse,
                                void* workspace, size_t workspace_bytes, uint32_t* err_word,
                                int32_t max_ctas, void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_paged_decode_fp4");
  if (!pkv_host::valid_pool4(pool)) return PKV_ERR_INVALID_ARG;
  const QuantDecodeCall c = {q,   batch_size, num_q_heads, kv_indptr,       kv_indices, kv_lens,
                             out, lse,        workspace,   workspace_bytes, err_word,   max_ctas, (cudaStream_t)stream};
  const pkv_status s = check_quant_decode(c, pool->num_kv_heads, pool->head_dim);
  if (s != PKV_OK || batch_size == 0) return s;
  const float score_scale = sm_scale * pool->k_global;
  const bool few = num_q_heads / pool->num_kv_heads <= 4;
  if (pool->head_dim == 128)
    return few ? run_quant_decode<Format4<128, true>>(pool, c, score_scale, pool->v_global)
               : run_quant_decode<Format4<128, false>>(pool, c, score_scale, pool->v_global);
  return few ? run_quant_decode<Format4<64, true>>(pool, c, score_scale, pool->v_global)
             : run_quant_decode<Format4<64, false>>(pool, c, score_scale, pool->v_global);
}

}  // extern "C"
