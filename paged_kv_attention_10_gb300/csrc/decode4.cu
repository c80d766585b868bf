// Paged decode attention over a 4-bit cache (one query per request).
//
// What it computes: with the cache's values k[j] and v[j] (e2m1 codes times an e4m3 scale per 16 of them times one
// scale g per cache),  out = sum_j softmax_j(scale q . k[j]) v[j],  page lists, GQA and LSE as in the bf16 decode.
// The plan is the 8-bit decode's (quant_decode.cuh).  A position's bytes are nearly halved again, the values are as
// many, so the loop has to be lean: the conversions alone are an instruction for every two values.
//
//  * A code times its block's scale is exact in f16 (two bits times four), so the scales go into the matrix
//    operands by f16 products, and the caches' scales g into the score's scale and the result's.  Both products run
//    as f16 m16n8k16 MMAs with fp32 accumulators, Q scaled per head by a power of two into f16's range as in the 8-bit
//    decode.
//  * A product's k-slots may hold the dimensions in any order if both operands agree, and so may the rows of its
//    result.  A lane therefore takes consecutive bytes of a row: of K, a quarter of a position's row (dims 32c ..
//    32c + 31 of 128), which holds whole blocks, so that it needs two scales of the eight; of V, an eighth (dims 16g ..
//    16g + 15), one block, of the positions that its k-slots stand for.  No ldmatrix, no exchange between lanes.
//  * V's operand pairs two positions in a register: the codes of both are put side by side in bytes first (two
//    instructions for four pairs), then converted.
//  * The sixteen score rows of an MMA are the positions in an order in which the loads of K (two positions by four
//    quarters at a time) and of V (four positions by four eighths) meet no shared-memory bank twice, see position().
//  * Softmax weights are rounded to f16 in [0, 2^15]; O and the sum of the weights carry that 2^15, which cancels.
#include "quant_decode.cuh"

namespace {

using namespace pkv;

// Weights of the second product stand in [0, 2^kWeightExp], the top of f16's range: one as small as 2^-40 of the
// largest is still counted.  (A value of V is below 2^12 and the sums are fp32.)
constexpr int kWeightExp = 15;

// The position, of eight consecutive ones, that row r of a score tile stands for.  K's loads of rows 2i and 2i + 1 and
// V's of rows 0, 2, 4, 6 and of 1, 3, 5, 7 are then free of bank conflicts.  Rows of 64 bytes, 16-byte pieces p of row t at
// p ^ (t >> 1 & 3): 0 1 3 2 4 5 7 6; rows of 32 bytes: 0 2 1 3 6 4 7 5.
template <int D>
PKV_DEV int position(int r) {
  if (D == 128) return r ^ ((r >> 1) & 1);
  return (0x57463120 >> (4 * r)) & 7;
}

template <int D>
struct Format4 {
  static constexpr int kDim = D, kRowBytes = D / 2, kScaleBytes = D / 16, kWarps = 16;
  static constexpr int kMergeFloats = 4 + D / 4;
  // an odd multiple of a head's bytes, so that neighbouring rows lie in other banks
  static int row_stride(int bytes) { return bytes / kRowBytes % 2 ? bytes : bytes + kRowBytes; }
  template <bool TMA>
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

// ---------------------------------------------------------------------------------------------
// Consumer warps: 32-position steps of one KV head with its G query heads.
// ---------------------------------------------------------------------------------------------
template <int D>
template <bool TMA>
__device__ void Format4<D>::consume(const QuantDecodeArgs& a, uint8_t* stages, StageHdr* hdr, uint64_t* hdr_full,
                                    uint64_t* full, uint64_t* empty, uint64_t* meet_bar) {
  constexpr int RH = kRowBytes, SH = kScaleBytes;
  constexpr int NM = D / 16;          // MMAs of a score tile, row tiles of O
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
  const uint32_t region = a.kv_region;
  const int HQU = HC * G;  // query heads per unit

  // Shared-memory places: of the four groups of eight positions of the slice, and of the lane's positions in a group.
  // K: row g.  V: rows 2c and 2c + 1, the lane's eighth g.
  uint32_t group_off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = si * kSlice + 8 * i;
    group_off[i] = TMA ? (uint32_t)(((t / a.box_rows) * HC + hl) * a.box_rows + t % a.box_rows) * RH
                       : (uint32_t)(t * a.row_stride + hl * RH);
  }
  const int stride = TMA ? RH : a.row_stride;
  auto piece = [&](int t, int p) -> uint32_t {  // 16-byte piece p of position t of a group
    return (uint32_t)(t * stride + ((TMA && D == 128 ? p ^ ((t >> 1) & 3) : p) << 4));
  };
  const int pk = position<D>(g), pa = position<D>(2 * c), pb = position<D>(2 * c + 1);
  const uint32_t k_off = D == 128 ? piece(pk, c) : piece(pk, c >> 1) + (c & 1) * 8;
  const uint32_t va_off = D == 128 ? piece(pa, g >> 1) + (g & 1) * 8 : piece(pa, g >> 2) + (g & 3) * 4;
  const uint32_t vb_off = D == 128 ? piece(pb, g >> 1) + (g & 1) * 8 : piece(pb, g >> 2) + (g & 3) * 4;
  const uint32_t stages_u32 = smem_u32(stages);

  uint32_t qf[NM][2];
  float qs[2];        // score scale (log2 units) of the lane's heads head0 + 2c, + 1
  float o[NM][4];
  float m[2], l[2];   // running maximum of x and sum of the weights 2^(x - m + kWeightExp)

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
  while (true) {
    if (!__all_sync(0xffffffffu, mbar_wait(&hdr_full[stage], phase))) {
      if (lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
      break;
    }
    const StageHdr h = hdr[stage];
    if (h.unit < 0) break;

    if (h.flags & kSegFirst) {
      // q fragments: lane (g, c) holds the dims of its quarter c, of head head0 + g
      const int head = head0 + g;
      const bool valid = head < G;
      const uint4* qp = reinterpret_cast<const uint4*>(
          a.q + ((int64_t)h.b * a.num_q_heads + (int64_t)(h.hg * HC + hl) * G + head) * D + c * (D / 4));
      uint32_t raw[2 * NM];
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < NM / 2; ++i) {
        const uint4 u = valid ? ld(qp + i) : make_uint4(0u, 0u, 0u, 0u);
        raw[4 * i] = u.x, raw[4 * i + 1] = u.y, raw[4 * i + 2] = u.z, raw[4 * i + 3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < 2 * NM; ++i)
        amax = max(amax, max(finite_abs_bits(__uint_as_float(raw[i] << 16)),
                             finite_abs_bits(__uint_as_float(raw[i] & 0xffff0000u))));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^e <= amax < 2^(e+1); q 2^(14 - e) goes into f16 and 2^(e - 14) into the score scale.  e is
      // held at -100 and above so that both factors are normal numbers.
      const int e = max((int)(amax >> 23) - 127, -100);
      const float up = exp2i(14 - e);
      const float down = a.scale_log2 * exp2i(e - 14);
#pragma unroll
      for (int i = 0; i < 2 * NM; ++i)
        qf[i / 2][i % 2] = pack_f16x2(__uint_as_float(raw[i] << 16) * up, __uint_as_float(raw[i] & 0xffff0000u) * up);
      // heads 2c and 2c + 1 of the tile live in lanes 8c and 8c + 4
      qs[0] = __shfl_sync(0xffffffffu, down, 8 * c);
      qs[1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int t = 0; t < NM; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][i] = 0.f;
    }

    if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase))) {
      if (lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
      break;
    }
    const int nv = min(kSlice, h.ntok - si * kSlice);
    const uint32_t kb = stages_u32 + (uint32_t)stage * a.stage_bytes;
    const uint32_t vb = kb + region;
    // the scales of the slice's first position; V's lie Ts positions behind K's
    const uint8_t* sc = stages + (size_t)stage * a.stage_bytes + 2 * region + (si * kSlice * HC + hl) * SH;
    float s[2][2][4];  // [half][MMA parity]: four independent accumulation chains
    if (nv > 0) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int pr = 0; pr < 2; ++pr)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[hf][pr][i] = 0.f;
        uint32_t w[2][KW], ks[2][2];  // rows g and g + 8: codes, and the scales of the two halves of the lane's quarter
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          lds<KW>(kb + group_off[2 * hf + i] + k_off, w[i]);
          const uint8_t* p = sc + (16 * hf + 8 * i + pk) * HC * SH;
          if (D == 128) {
            const uint32_t pair = unpack_e4m3x2(*reinterpret_cast<const uint16_t*>(p + 2 * c));
            ks[i][0] = __byte_perm(pair, 0, 0x1010);
            ks[i][1] = __byte_perm(pair, 0, 0x3232);
          } else {
            const uint32_t one = unpack_e4m3x2(p[c]);
            ks[i][0] = ks[i][1] = __byte_perm(one, 0, 0x1010);
          }
        }
#pragma unroll
        for (int j = 0; j < KW; ++j) {
          uint32_t x[4], y[4];
          unpack_e2m1x8(w[0][j], x);
          unpack_e2m1x8(w[1][j], y);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = mul_f16x2(x[i], ks[0][2 * j / KW]);
            y[i] = mul_f16x2(y[i], ks[1][2 * j / KW]);
          }
          mma_f16_16816(s[hf][0], x[0], y[0], x[1], y[1], qf[2 * j][0], qf[2 * j][1]);
          mma_f16_16816(s[hf][1], x[2], y[2], x[3], y[3], qf[2 * j + 1][0], qf[2 * j + 1][1]);
        }
      }
    }
    // A segment's last stage is held when warps share a head: its memory carries their merge.
    const bool hold = (h.flags & kSegLast) && W > 1;
    __syncwarp();
    if (!hold && lane == 0) mbar_arrive(&empty[stage]);  // K is read: its buffer is free while V is still in use
    if (!__all_sync(0xffffffffu, mbar_wait(&full[NS + stage], phase))) {
      if (lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
      break;
    }
    if (nv > 0) {
      uint32_t bp[2][2];
      float x[2][4];
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = (s[hf][0][i] + s[hf][1][i]) * qs[i & 1];
          x[hf][i] = 16 * hf + 8 * (i >> 1) + pk < nv ? v : -INFINITY;
          mx[i & 1] = fmaxf(mx[i & 1], x[hf][i]);
        }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
#pragma unroll
        for (int k = 0; k < 2; ++k) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], off));
      }
      float corr[2], base[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float mn = fmaxf(m[k], mx[k]);
        // nothing but NaN so far: any finite maximum will do
        corr[k] = mn == -INFINITY ? 1.f : ex2(m[k] - mn);
        base[k] = (mn == -INFINITY ? 0.f : mn) - (float)kWeightExp;
        m[k] = mn;
        l[k] *= corr[k];
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = ex2(x[hf][i] - base[i & 1]);
          l[i & 1] += w[i];
        }
        bp[hf][0] = movmatrix_t(pack_f16x2(w[0], w[1]));
        bp[hf][1] = movmatrix_t(pack_f16x2(w[2], w[3]));
      }
      if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
        for (int t = 0; t < NM; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[t][i] *= corr[i & 1];
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        // Rows past the request's end hold unused pool slots (the boxes bring them) or what shared memory held
        // before, NaN scales among them: with a scale of 0 their values are 0, and 0 times their weight 0 stays 0.
        uint32_t va[2][VW], vo[2][VW], vs[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t wa[VW], wb[VW];
          lds<VW>(vb + group_off[2 * hf + i] + va_off, wa);
          lds<VW>(vb + group_off[2 * hf + i] + vb_off, wb);
          const int t0 = 16 * hf + 8 * i;
          const uint8_t* p = sc + (Ts + t0) * HC * SH + (D == 128 ? g : g >> 1);
          const uint32_t sa = t0 + pa < nv ? p[pa * HC * SH] : 0u, sb = t0 + pb < nv ? p[pb * HC * SH] : 0u;
          vs[i] = unpack_e4m3x2(sa | sb << 8);
#pragma unroll
          for (int j = 0; j < VW; ++j) {
            va[i][j] = (wa[j] & 0x0f0f0f0fu) | ((wb[j] << 4) & 0xf0f0f0f0u);  // even dims: byte = (position a, position b)
            vo[i][j] = ((wa[j] >> 4) & 0x0f0f0f0fu) | (wb[j] & 0xf0f0f0f0u);  // odd dims
          }
        }
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          uint32_t e0[4], e1[4], f0[4], f1[4];
          unpack_e2m1x8(va[0][j], e0);
          unpack_e2m1x8(vo[0][j], f0);
          unpack_e2m1x8(va[1][j], e1);
          unpack_e2m1x8(vo[1][j], f1);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_f16_16816(o[4 * j + i], mul_f16x2(e0[i], vs[0]), mul_f16x2(f0[i], vs[0]), mul_f16x2(e1[i], vs[1]),
                          mul_f16x2(f1[i], vs[1]), bp[hf][0], bp[hf][1]);
        }
      }
    }
    __syncwarp();
    if (!hold && lane == 0) mbar_arrive(&empty[NS + stage]);

    if (h.flags & kSegLast) {
      if (W > 1) {
        // Combine the W warps that split this head's positions (all consumer warps reach the segment end on
        // the same stage).  A warp without a position in the segment holds a maximum of -inf and sums of 0.
        bool met = meet();
        float* buf = reinterpret_cast<float*>(stages + (size_t)stage * a.stage_bytes) + lane;
        // all but one at once where their states fit into the stage, else half of them, or as many as do, at a time
        const int room = (int)(a.stage_bytes / (uint32_t)(HV * MF * 128));
        for (int left = W; met && left > 1;) {
          const int keep = left - 1 <= room ? 1 : max(left / 2, left - room);
          if (si >= keep && si < left) {
            float* to = buf + ((si - keep) * HV + hv) * MF * 32;
            int e = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              to[(e++) * 32] = m[k];
              to[(e++) * 32] = l[k];
            }
#pragma unroll
            for (int t = 0; t < NM; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) to[(e++) * 32] = o[t][i];
          }
          met = meet();
          if (!met) break;
          if (si < keep) {
            for (int w = si; w < left - keep; w += keep) {
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
              for (int t = 0; t < NM; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][i] = o[t][i] * fa[i & 1] + ob[(e++) * 32] * fb[i & 1];
            }
          }
          left = keep;
          if (left > 1) met = meet();  // read before the next writes
        }
        if (!met) {
          if (lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
          break;
        }
        fence_proxy_async_smem();  // the merge's accesses, before the next async fill
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&empty[stage]);
          mbar_arrive(&empty[NS + stage]);
        }
      }
      if (si == 0) {
        const bool whole = (h.flags & kStartsUnit) && (h.flags & kEndsUnit);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float lt = l[k];
          lt += __shfl_xor_sync(0xffffffffu, lt, 4);
          lt += __shfl_xor_sync(0xffffffffu, lt, 8);
          lt += __shfl_xor_sync(0xffffffffu, lt, 16);
          const int col = head0 + 2 * c + k;  // query head within the group
          const float inv = a.out_scale / lt;
          const float lse_v = (m[k] + log2f(lt) - (float)kWeightExp) * kLn2;
          if (col < G) {
            // tile t of O: row g is dim D / 8 g + 2t, row g + 8 the next one
            const int qhl = hl * G + col;
            if (whole) {
              const int64_t qh = (int64_t)h.hg * HQU + qhl;
              uint4* op = reinterpret_cast<uint4*>(a.out + ((int64_t)h.b * a.num_q_heads + qh) * D + g * (D / 8));
#pragma unroll
              for (int t = 0; t < NM; t += 4)
                op[t / 4] = make_uint4(pack_bf16x2(o[t][k] * inv, o[t][2 + k] * inv),
                                       pack_bf16x2(o[t + 1][k] * inv, o[t + 1][2 + k] * inv),
                                       pack_bf16x2(o[t + 2][k] * inv, o[t + 2][2 + k] * inv),
                                       pack_bf16x2(o[t + 3][k] * inv, o[t + 3][2 + k] * inv));
              if (g == 0 && a.lse) a.lse[(int64_t)h.b * a.num_q_heads + qh] = lse_v;
            } else {
              float4* pp = reinterpret_cast<float4*>(a.part_o + ((int64_t)h.part * HQU + qhl) * D + g * (D / 8));
#pragma unroll
              for (int t = 0; t < NM; t += 2)
                pp[t / 2] = make_float4(o[t][k] * inv, o[t][2 + k] * inv, o[t + 1][k] * inv, o[t + 1][2 + k] * inv);
              if (g == 0) a.part_lse[(int64_t)h.part * HQU + qhl] = lse_v;
            }
          }
        }
        if (warp == 0 && lane == 0) {
          if (h.flags & kStartsUnit) a.unit_first[h.unit] = h.part;
          if (h.flags & kEndsUnit) a.unit_last[h.unit] = h.part;
        }
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
  if (head_dim == 128) return quant_decode_workspace<Format4<128>>(batch_size, num_q_heads, num_kv_heads);
  if (head_dim == 64) return quant_decode_workspace<Format4<64>>(batch_size, num_q_heads, num_kv_heads);
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
  return pool->head_dim == 128 ? run_quant_decode<Format4<128>>(pool, c, score_scale, pool->v_global)
                               : run_quant_decode<Format4<64>>(pool, c, score_scale, pool->v_global);
}

}  // extern "C"
