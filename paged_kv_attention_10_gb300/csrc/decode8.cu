// Paged decode attention over an 8-bit cache (one query per request) and its split-KV merge.
//
// What it computes: with the cache rows k8[j] ks[j] and v8[j] vs[j] (e4m3 values and one scale per row
// and head),  out = sum_j softmax_j(scale q . k8[j] ks[j]) vs[j] v8[j],  page lists, GQA and LSE as in the
// bf16 decode.  HBM-bound: half the bytes of the bf16 cache per position, the same arithmetic, so
// the instructions per byte double and the loop is built to keep them few.
//
//  * Scales never touch the matrix operands.  ks[j] multiplies a score after the product.  vs[j] goes
//    into the softmax weights of the second product, w_j = p_j vs[j], which f16 must hold: they are
//    formed as 2^(x_j + e_j - M) m_j 2^14 with vs[j] = m_j 2^e_j and M a running maximum of x_j + e_j of its
//    own, so that they stay in [0, 2^15) whatever the scales' range.  The softmax's own sum keeps its
//    own running maximum, and the two meet when a segment ends.
//  * Both products run as f16 m16n8k16 MMAs with fp32 accumulators: e4m3 converts to f16 exactly, two
//    values per instruction.  Q, bf16, is scaled per head by a power of two into f16's range (largest
//    value in [2^14, 2^15)): exact for every value within 2^-31 of the largest.  Weights are rounded
//    to f16 (11 bits, against 8 of the bf16 decode).
//  * A product's k-slots may hold the dimensions in any order, if both operands agree, so the
//    ldmatrix of byte rows needs no rearrangement: a lane's four bytes of K are dims 4c .. 4c+3, which
//    fill slots (2c, 2c+1, 2c+8, 2c+9).  V^T through ldmatrix.trans pairs two dims of two tokens in a
//    register; one byte permute makes pairs of tokens, and the output rows g, g + 8 become the
//    neighbouring dims 2g, 2g + 1, which store as one bf16 pair.
//  * Groups of 9 to 16 query heads take two warps per KV head, eight heads each, over the same rows in
//    shared memory: one warp with both would convert once instead of twice but spills (16 heads of
//    128, 16 requests of 10000 to 20000 positions: 57 us, 42 with two).
//  * A warp takes 32 positions of one KV head at a time (the bf16 decode: 16), so the shuffles of
//    the maxima, the rescaling of O and the barrier round are paid half as often.
//  * The rest is the bf16 decode's plan: one persistent CTA per SM over an equal share of the stream
//    of slices, TMA boxes of 32, 16 or 8 rows (the largest that divides the page size) in the 128- or 64-byte
//    swizzle, copies of single rows otherwise.  K and V have a producer warp and barriers each.  The
//    scales come into the same stage: by bulk copies beside the boxes where the CTA takes every KV
//    head (a box's lie side by side then), by cp.async otherwise.
// Measured with 32/8 heads of 128 at page size 16: 8 requests of 32768 positions 90 us, 6.1 TB/s, 90 % of
// what a device copy reaches; 256 requests of 512 to 4096 positions 196 to 198 us, 93 %.  DRAM reads are the cache's
// bytes (554 MB of 554), the tensor pipe is 18 % busy, 43 % of the issue slots are used.  Small KV head counts are
// bound by the producers' issue instead: one head of 128, 720000 positions, 50 us at page size 16, 41 at
// 64 and 151 at 1 of the 28 that the bytes take; two heads at page size 1 118 of 28.
#include <atomic>

#include "quant.cuh"
#include "tc05.cuh"

namespace {

using namespace pkv;

constexpr int kSegFirst = 1;    // first stage of this CTA's segment of the unit
constexpr int kSegLast = 2;     // last stage of the segment
constexpr int kStartsUnit = 4;  // the segment starts at position 0 of the unit
constexpr int kEndsUnit = 8;    // the segment ends at the unit's last position

struct StageHdr {
  int32_t unit;  // -1: no more work
  int32_t b, hg, ntok, flags, part, pad0, pad1;
};

struct Decode8Args {
  CUtensorMap tm_k;  // pool bytes as (dim, row, head), box [D x box_rows x HC]; TMA instance only
  CUtensorMap tm_v;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* k_scale;
  const float* v_scale;
  int64_t num_pages;
  int32_t page_size, num_kv_heads;
  FastDiv page_div;  // by page_size
  const __nv_bfloat16* q;
  int32_t batch, num_q_heads;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* kv_lens;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;
  float* part_lse;
  int32_t* unit_first;
  int32_t* unit_last;
  uint32_t* err_word;
  int32_t HC;            // KV heads per CTA
  int32_t nhg;           // head groups = num_kv_heads / HC
  int32_t W;             // consumer warps per KV head
  int32_t group;         // query heads per KV head
  int32_t nt;            // warps that share a KV head's rows, eight of its query heads each
  int32_t box_rows;      // TMA instance: rows of a box (32, 16 or 8)
  int32_t row_stride;    // row-copy instance: shared-memory bytes per token row
  int32_t stage_tokens;  // 32 * W
  int32_t num_stages, num_parts;
  uint32_t kv_region;    // bytes of the K (or V) part of one stage
  uint32_t stage_bytes;  // K, V and the scales
};

// No request has more positions than the pool has rows; a longer kv_lens[b] (reported, its pages run
// out) must not take the token counter past 31 bits.
constexpr int kMaxLen = 0x7fff0000;
constexpr int kSlice = 32;  // positions of a warp's step, and the unit of the work split
constexpr int kMaxStages = 8;
// Weights of the second product stand in [0, 2^(kWeightExp + 1)), the top of f16's range: one as small as 2^-39 of
// the largest is still counted.  (In [0, 2), what is below 2^-25 of it was not: 20000 positions with weights of
// 2^-25.6 are 0.0004 of the sum.)
constexpr int kWeightExp = 14;

PKV_DEV void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
PKV_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival on the barrier when every cp.async of this thread so far has landed.
PKV_DEV void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// D = A * B + D, A 16x16 f16 (row), B 16x8 f16 (col), D 16x8 fp32.
PKV_DEV void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                           uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

PKV_DEV uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------------------------------------
// Producer warps, one for K and one for V: each walks the CTA's share of the slice stream and fills
// its part of the stages; K's also writes the headers.  A stage is a few hundred cycles of address work
// for a warp and about 1400 of memory time, so one warp for both held the stream back (8 x 32768
// positions, D 128: 105 us, 96 with two).
// ---------------------------------------------------------------------------------------------
template <int D, bool TMA>
__device__ void decode8_producer(const Decode8Args& a, uint8_t* stages, StageHdr* hdr, uint64_t* hdr_full,
                                 uint64_t* full, uint64_t* empty, bool v) {
  const int lane = threadIdx.x & 31;
  const int NS = a.num_stages, Ts = a.stage_tokens, W = a.W, HC = a.HC, nhg = a.nhg;
  const uint32_t region = a.kv_region;
  const CUtensorMap* tm = v ? &a.tm_v : &a.tm_k;
  const uint8_t* pool = v ? a.v_pool : a.k_pool;
  const float* scale = v ? a.v_scale : a.k_scale;
  // Page indices come from a register window of 96 consecutive entries (three 32-lane slices), its
  // last third loaded 32 pages before a stage can need it.  Usable while one stage spans at most
  // 33 pages.
  const bool windowed = (Ts - 1) / a.page_size + 1 <= 32;

  // the first 32 requests' numbers in one round of loads, which the walk below starts with
  const bool in0 = lane < a.batch;
  const int32_t first_len = in0 ? min(max(0, ld(a.kv_lens + lane)), kMaxLen) : 0;
  const int32_t first_p0 = in0 ? ld(a.kv_indptr + lane) : 0;
  const int32_t first_p1 = in0 ? ld(a.kv_indptr + lane + 1) : 0;
  int64_t sumS = ((int64_t)first_len + kSlice - 1) / kSlice;  // slices over all requests
  for (int i = 32 + lane; i < a.batch; i += 128) {
#pragma unroll
    for (int u = 0; u < 4; ++u)  // four loads in flight
      if (i + 32 * u < a.batch) sumS += (min(max(0, ld(a.kv_lens + i + 32 * u)), kMaxLen) + kSlice - 1) / kSlice;
  }
  sumS = warp_sum(sumS);
  const int64_t T = sumS * nhg;
  int64_t share = (T + gridDim.x - 1) / gridDim.x;
  if (share < 1) share = 1;
  const int64_t c0 = (int64_t)blockIdx.x * share;
  const int64_t c1 = min(T, c0 + share);

  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  int32_t cur_p0 = 0, cur_np = 0;  // page list of the request being streamed
  int win_b = -1, wbase = 0;
  int32_t w0 = -1, w1 = -1, w2 = -1;
  auto entry = [&](int pidx) -> int32_t {  // page-list entry of the current request; -1 past its end
    return pidx < cur_np ? ld(a.kv_indices + cur_p0 + pidx) : -1;
  };
  int nissued = 0;
  auto next_stage = [&]() {
    ++nissued;
    if (++stage == NS) {
      stage = 0;
      phase ^= 1;
    }
  };

  auto emit = [&](int unit, int b, int hg, int tok0, int ntok, int flags) -> bool {
    if (unit >= 0 && !v && (flags & kSegFirst)) {
      const int hqu = HC * a.group;  // the unit's queries, on their way to L2 before they are read
      const char* qb = reinterpret_cast<const char*>(a.q + ((int64_t)b * a.num_q_heads + (int64_t)hg * hqu) * D);
      for (int off = lane * 128; off < hqu * D * 2; off += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(qb + off));
    }
    if (unit >= 0 && windowed) {
      const int first_page = a.page_div.quot(tok0);
      if (b != win_b || first_page < wbase) {
        win_b = b;
        wbase = first_page;
        w0 = entry(wbase + lane);
        w1 = entry(wbase + 32 + lane);
        w2 = entry(wbase + 64 + lane);
      }
      while (first_page >= wbase + 32) {
        w0 = w1;
        w1 = w2;
        wbase += 32;
        w2 = entry(wbase + 64 + lane);
      }
    }
    uint64_t* bar = &full[stage];
    if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1))) return false;
    if (!v && lane == 0) {  // the consumers read the header, and a new unit's queries, while the stage is on its way
      hdr[stage] = StageHdr{unit, b, hg, ntok, flags, (int32_t)blockIdx.x + unit, 0, 0};
      mbar_arrive(&hdr_full[stage]);
    }
    if (unit >= 0) {
      uint8_t* dst = stages + (size_t)stage * a.stage_bytes + (v ? region : 0u);
      uint8_t* sdst = stages + (size_t)stage * a.stage_bytes + 2 * region + (v ? (size_t)Ts * HC * 4 : 0);
      uint32_t bad = 0;
      auto window_page = [&](uint32_t pidx) -> int32_t {  // all lanes call
        const int k = (int)pidx - wbase;  // < 64
        const int32_t v0 = __shfl_sync(0xffffffffu, w0, k & 31);
        const int32_t v1 = __shfl_sync(0xffffffffu, w1, k & 31);
        return k < 32 ? v0 : v1;
      };
      auto row_at = [&](uint32_t pidx, uint32_t in_page, int32_t page, bool in) -> int64_t {
        if (!in) return -1;
        if ((int)pidx >= cur_np) {
          bad |= PKV_DEVERR_LENGTH;
          return -1;
        }
        if (page < 0 || page >= a.num_pages) {
          bad |= PKV_DEVERR_PAGE_OOB;
          return -1;
        }
        return (int64_t)page * a.page_size + in_page;
      };
      auto copy_scales = [&](int64_t row, int j) {  // token j's HC scales, one by one
        const float* src = scale + row * a.num_kv_heads + hg * HC;
        const uint32_t sd = smem_u32(sdst) + (uint32_t)(j * HC) * 4;
        if ((HC & 3) == 0) {
          for (int i = 0; i < HC; i += 4) cp_async16(sd + 4 * i, src + i);
        } else {
          for (int i = 0; i < HC; ++i) cp_async4(sd + 4 * i, src + i);
        }
      };
      if constexpr (TMA) {
        // Lane i fetches box i, box_rows tokens inside one page, and their scales, which lie side by side when
        // the CTA takes all KV heads.  (One lookup a stage: with one per 32 tokens the eight of a stage of
        // one KV head took 4 us, and 720000 positions of it 96 us; 48 now, of the 28 that their bytes take.)
        const int sh = 31 - __clz(a.box_rows), nbox = Ts >> sh;
        const int tok = tok0 + (lane << sh);
        const bool in = lane < nbox && tok < tok0 + ntok;
        uint32_t pidx, in_page;
        a.page_div.divmod((uint32_t)(in ? tok : tok0), pidx, in_page);
        const int32_t page = windowed ? window_page(pidx) : in ? entry((int)pidx) : -1;
        const int64_t row = row_at(pidx, in_page, page, in);
        const bool side_by_side = nhg == 1;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, row >= 0));
        const uint32_t box = (uint32_t)(HC * D) << sh, sbox = (uint32_t)(HC * 4) << sh;
        if (lane == 0) mbar_expect_tx(bar, n * (box + (side_by_side ? sbox : 0u)));
        __syncwarp();
        if (row >= 0) {
          tma_load_3d(smem_u32(dst) + lane * box, tm, 0, (int)row, hg * HC, bar);
          if (side_by_side) bulk_g2s(sdst + lane * sbox, scale + row * a.num_kv_heads, sbox, bar);
        }
        if (!side_by_side) {
          for (int r = 0; r < W; ++r) {
            const int j = lane + 32 * r;
            const int first = __shfl_sync(0xffffffffu, (int)row, j >> sh);
            if (j < ntok && first >= 0) copy_scales(first + (j & (a.box_rows - 1)), j);
          }
        }
      } else {
        // One bulk copy per token row, or, for rows of 64 or 128 bytes, 16 bytes a lane: a bulk copy takes
        // about 80 cycles to issue whatever it brings.  24 requests at page size 1, D 128: one KV head and 20000
        // to 40000 positions 162 us so and 200 by bulk copies, two heads and half as many positions
        // (rows of 256 bytes) 144 and 116.  Page indices that are not in the window are loaded four rounds
        // ahead.
        const uint32_t RB = (uint32_t)(HC * D);
        const bool short_rows = RB <= 128;
        const int csh = RB == 64 ? 2 : 3;  // log2 of the 16-byte chunks of a short row
        auto ahead = [&](int r) -> int32_t {
          const int j = lane + 32 * r;
          return !windowed && j < ntok ? entry((int)a.page_div.quot((uint32_t)(tok0 + j))) : -1;
        };
        int32_t p0 = ahead(0), p1 = ahead(1), p2 = ahead(2), p3 = ahead(3);
#pragma unroll 1
        for (int r = 0; r < W; ++r) {
          const int j = lane + 32 * r;
          const bool in = j < ntok;
          uint32_t pidx, in_page;
          a.page_div.divmod((uint32_t)(tok0 + (in ? j : 0)), pidx, in_page);
          int32_t page = p0;
          if (windowed) page = window_page(pidx);
          p0 = p1, p1 = p2, p2 = p3, p3 = ahead(r + 4);
          const int64_t row = row_at(pidx, in_page, page, in);
          if (short_rows) {
            const uint32_t to = smem_u32(dst) + 32 * r * a.row_stride;
#pragma unroll 1
            for (int it = lane; it < 32 << csh; it += 32) {
              const int tk = it >> csh, ch = it & ((1 << csh) - 1);
              const int64_t from = __shfl_sync(0xffffffffu, row, tk);
              if (from >= 0)
                cp_async16(to + tk * a.row_stride + ch * 16, pool + (from * a.num_kv_heads + hg * HC) * D + ch * 16);
            }
            if (row >= 0) copy_scales(row, j);
          } else {
            const uint32_t n = __popc(__ballot_sync(0xffffffffu, row >= 0));
            if (lane == 0) mbar_expect_tx(bar, n * RB);
            __syncwarp();
            if (row >= 0) {
              bulk_g2s(dst + (size_t)j * a.row_stride, pool + (row * a.num_kv_heads + hg * HC) * D, RB, bar);
              copy_scales(row, j);
            }
          }
        }
      }
      if (bad && !v) report(a.err_word, bad);
    }
    // the arrival that lets the stage complete comes after every byte count
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    cp_async_arrive(bar);
    next_stage();
    return true;
  };

  if (c0 < c1) {
    int64_t base = 0;  // stream offset (in slices) of request b0
    for (int b0 = 0; b0 < a.batch && base < c1 && ok; b0 += 32) {
      const int b = b0 + lane;
      const bool in = b < a.batch;
      int64_t L = first_len;
      int32_t ip0 = first_p0, ip1 = first_p1;
      if (b0 > 0) {
        L = in ? min(max(0, ld(a.kv_lens + b)), kMaxLen) : 0;
        ip0 = in ? ld(a.kv_indptr + b) : 0;
        ip1 = in ? ld(a.kv_indptr + b + 1) : 0;
      }
      const int64_t S = (L + kSlice - 1) / kSlice;
      int64_t incl = S;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const int64_t rs = base + nhg * (incl - S);
      const int64_t re = base + nhg * incl;
      uint32_t mask = __ballot_sync(0xffffffffu, in && S > 0 && re > c0 && rs < c1);
      while (mask && ok) {
        const int src_lane = __ffs(mask) - 1;
        mask &= mask - 1;
        const int bb = b0 + src_lane;
        const int64_t Lb = __shfl_sync(0xffffffffu, L, src_lane);
        const int64_t Sb = __shfl_sync(0xffffffffu, S, src_lane);
        const int64_t rsb = __shfl_sync(0xffffffffu, rs, src_lane);
        cur_p0 = __shfl_sync(0xffffffffu, ip0, src_lane);
        cur_np = __shfl_sync(0xffffffffu, ip1, src_lane) - cur_p0;
        for (int hg = 0; hg < nhg && ok; ++hg) {
          const int64_t us = rsb + (int64_t)hg * Sb, ue = us + Sb;
          const int64_t s0 = max(us, c0), s1 = min(ue, c1);
          if (s0 >= s1) continue;
          const int t0 = (int)(s0 - us) * kSlice;
          const int t1 = (int)min((s1 - us) * kSlice, Lb);
          for (int t = t0; t < t1 && ok; t += Ts) {
            int flags = 0;
            if (t == t0) flags |= kSegFirst;
            if (t + Ts >= t1) flags |= kSegLast;
            if (s0 == us) flags |= kStartsUnit;
            if (s1 == ue) flags |= kEndsUnit;
            ok = emit(bb * nhg + hg, bb, hg, t, min(Ts, t1 - t), flags);
          }
        }
      }
      base += nhg * __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  ok = ok && emit(-1, 0, 0, 0, 0, 0);
  // The merge may be scheduled once every CTA has issued its last copies (it waits for this grid's
  // completion before it reads): early enough to hide its launch, late enough not to hold thread
  // slots that kernels on other streams could use.
  if (!v) pdl_trigger();
  if (!ok && lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
  // No copy into this CTA's shared memory is in flight when it exits (bounded waits; immediate on
  // the normal path, where the consumers have seen every stage complete).
  for (int k = 0; k < min(nissued, NS); ++k) {
    if (--stage < 0) {
      stage = NS - 1;
      phase ^= 1;
    }
    mbar_wait(&full[stage], phase);
  }
}

// ---------------------------------------------------------------------------------------------
// Consumer warps: 32-position steps of one KV head with its G query heads.
// ---------------------------------------------------------------------------------------------
template <int D, bool TMA>
__device__ void decode8_consumer(const Decode8Args& a, uint8_t* stages, StageHdr* hdr, uint64_t* hdr_full,
                                 uint64_t* full, uint64_t* empty, uint64_t* meet_bar) {
  constexpr int NK = D / 16;                      // 16-byte chunks of a row: k-steps of K q, row tiles of O
  constexpr int MF = 6 + NK * 4;                  // floats per lane merged between the warps of a head
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

  // ldmatrix addressing, the same for K and V: lane 8 mi + ri addresses row 8 (mi & 1) + ri of a
  // 16-row half at chunk 2 j + (mi >> 1)
  const int mi = lane >> 3, ri = lane & 7;
  uint32_t row_off[2];
  int sw[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int t = si * kSlice + h * 16 + ((mi & 1) << 3) + ri;
    if (TMA) {
      const int R = a.box_rows;
      row_off[h] = (uint32_t)(((t / R) * HC + hl) * R + t % R) * D;
      sw[h] = D == 128 ? (t & 7) : ((t >> 1) & 3);
    } else {
      row_off[h] = (uint32_t)(t * a.row_stride + hl * D);
      sw[h] = 0;
    }
  }
  const uint32_t stages_u32 = smem_u32(stages);

  uint32_t qf[NK][2];
  float qs[2];        // score scale (log2 units) of the lane's heads head0 + 2c, + 1
  float o[NK][4];
  float m[2], l[2];   // running maximum of x and sum of 2^(x - m)
  float mw[2];        // running maximum of x + e, which O is relative to

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
      // q fragments: lane (g, c) holds dims 16 ks + 4c .. + 3 of head head0 + g
      const int head = head0 + g;
      const bool valid = head < G;
      const __nv_bfloat16* qp =
          a.q + ((int64_t)h.b * a.num_q_heads + (int64_t)(h.hg * HC + hl) * G + head) * D + 4 * c;
      uint2 raw[NK];
      uint32_t amax = 0;
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        raw[ks] = valid ? ld(reinterpret_cast<const uint2*>(qp + ks * 16)) : make_uint2(0u, 0u);
        amax = max(amax, max(max(finite_abs_bits(__uint_as_float(raw[ks].x << 16)),
                                 finite_abs_bits(__uint_as_float(raw[ks].x & 0xffff0000u))),
                             max(finite_abs_bits(__uint_as_float(raw[ks].y << 16)),
                                 finite_abs_bits(__uint_as_float(raw[ks].y & 0xffff0000u)))));
      }
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^e <= amax < 2^(e+1); q 2^(14 - e) goes into f16 and 2^(e - 14) into the score scale.  e is
      // held at -100 and above so that both factors are normal numbers.
      const int e = max((int)(amax >> 23) - 127, -100);
      const float up = exp2i(14 - e);
      const float down = a.scale_log2 * exp2i(e - 14);
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        qf[ks][0] = pack_f16x2(__uint_as_float(raw[ks].x << 16) * up,
                                   __uint_as_float(raw[ks].x & 0xffff0000u) * up);
        qf[ks][1] = pack_f16x2(__uint_as_float(raw[ks].y << 16) * up,
                                   __uint_as_float(raw[ks].y & 0xffff0000u) * up);
      }
      // heads 2c and 2c + 1 of the tile live in lanes 8c and 8c + 4
      qs[0] = __shfl_sync(0xffffffffu, down, 8 * c);
      qs[1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
      m[0] = m[1] = mw[0] = mw[1] = -INFINITY;
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int kc = 0; kc < NK; ++kc)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[kc][i] = 0.f;
    }

    if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase))) {
      if (lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
      break;
    }
    const int nv = min(kSlice, h.ntok - si * kSlice);
    const uint32_t kb = stages_u32 + (uint32_t)stage * a.stage_bytes;
    const uint32_t vb = kb + region;
    const float* sc = reinterpret_cast<const float*>(stages + (size_t)stage * a.stage_bytes + 2 * region) +
                      (si * kSlice + g) * HC + hl;  // K scales of tokens g, g + 8, ... of the slice; V's Ts rows on
    float s[2][2][4];  // [half][chunk parity]: four independent accumulation chains
    float ksc[4];
    if (nv > 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ksc[i] = sc[8 * i * HC];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int pr = 0; pr < 2; ++pr)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[hf][pr][i] = 0.f;
#pragma unroll
      for (int j = 0; j < NK / 2; ++j) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t r[4];
          ldsm_x4(kb + row_off[hf] + (((2 * j + (mi >> 1)) ^ sw[hf]) << 4), r[0], r[1], r[2], r[3]);
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            uint32_t a0, a1, a2, a3;
            unpack_e4m3x4(r[2 * pr], a0, a2);
            unpack_e4m3x4(r[2 * pr + 1], a1, a3);
            mma_f16_16816(s[hf][pr], a0, a1, a2, a3, qf[2 * j + pr][0], qf[2 * j + pr][1]);
          }
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
    if (nv > 0 && nv < kSlice) {
      // rows past the request's end hold unused pool slots (the boxes bring them, possibly NaN) or
      // what shared memory held before: V rows there become 0 so that weight 0 times V stays 0
      // (scores there are masked by a select).
      uint8_t* vreg = stages + (size_t)stage * a.stage_bytes + region;
      for (int idx = lane; idx < (kSlice - nv) * NK; idx += 32) {
        const int t = si * kSlice + nv + idx / NK, ch = idx % NK;
        uint32_t off;
        if (TMA)
          off = (uint32_t)(((t / a.box_rows) * HC + hl) * a.box_rows + t % a.box_rows) * D;
        else
          off = (uint32_t)(t * a.row_stride + hl * D);
        *reinterpret_cast<uint4*>(vreg + off + ch * 16) = make_uint4(0u, 0u, 0u, 0u);  // whole rows: any order
      }
      __syncwarp();
    }
    if (nv > 0) {
      float vm[4], ve[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u = __float_as_uint(sc[(Ts + 8 * i) * HC]);
        ve[i] = (float)((int)(u >> 23) - 127);
        vm[i] = __uint_as_float((u & 0x7fffffu) | (uint32_t)(127 + kWeightExp) << 23);
      }
      uint32_t bp[2][2];
      float x[2][4];
      float mx[2] = {-INFINITY, -INFINITY}, mxe[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 2 * hf + (i >> 1);  // token g + 8 row
          const float v = (s[hf][0][i] + s[hf][1][i]) * qs[i & 1] * ksc[row];
          x[hf][i] = g + 8 * row < nv ? v : -INFINITY;
          mx[i & 1] = fmaxf(mx[i & 1], x[hf][i]);
          mxe[i & 1] = fmaxf(mxe[i & 1], x[hf][i] + ve[row]);
        }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], off));
          mxe[k] = fmaxf(mxe[k], __shfl_xor_sync(0xffffffffu, mxe[k], off));
        }
      }
      float corr[2], corrw[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float mn = fmaxf(m[k], mx[k]), wn = fmaxf(mw[k], mxe[k]);
        corr[k] = ex2(m[k] - mn);
        corrw[k] = ex2(mw[k] - wn);
        m[k] = mn;
        mw[k] = wn;
        l[k] *= corr[k];
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 2 * hf + (i >> 1), k = i & 1;
          l[k] += ex2(x[hf][i] - m[k]);
          w[i] = ex2(x[hf][i] + ve[row] - mw[k]) * vm[row];
        }
        bp[hf][0] = movmatrix_t(pack_f16x2(w[0], w[1]));
        bp[hf][1] = movmatrix_t(pack_f16x2(w[2], w[3]));
      }
#pragma unroll
      for (int kc = 0; kc < NK; ++kc) {
        o[kc][0] *= corrw[0];
        o[kc][1] *= corrw[1];
        o[kc][2] *= corrw[0];
        o[kc][3] *= corrw[1];
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int j = 0; j < NK / 2; ++j) {
          uint32_t r[4];
          ldsm_x4_t(vb + row_off[hf] + (((2 * j + (mi >> 1)) ^ sw[hf]) << 4), r[0], r[1], r[2], r[3]);
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            uint32_t a0, a1, a2, a3;
            unpack_e4m3x4(__byte_perm(r[2 * pr], 0, 0x3120), a0, a1);
            unpack_e4m3x4(__byte_perm(r[2 * pr + 1], 0, 0x3120), a2, a3);
            mma_f16_16816(o[2 * j + pr], a0, a1, a2, a3, bp[hf][0], bp[hf][1]);
          }
        }
      }
    }
    if (nv > 0 && nv < kSlice) fence_proxy_async_smem();  // zeros above, before the next async fill
    __syncwarp();
    if (!hold && lane == 0) mbar_arrive(&empty[NS + stage]);

    if (h.flags & kSegLast) {
      if (W > 1) {
        // Combine the W warps that split this head's tokens (all consumer warps reach the segment end on
        // the same stage).  A warp without a token in the segment holds
        // maxima of -inf and sums of 0.
        bool met = meet();
        float* buf = reinterpret_cast<float*>(stages + (size_t)stage * a.stage_bytes) + lane;
        // all but one at once where their states fit into the stage, else half of them at a time
        for (int left = W; met && left > 1;) {
          const int keep = (uint32_t)((left - 1) * HV * MF * 128) <= 2 * region ? 1 : left / 2;
          if (si >= keep && si < left) {
            float* to = buf + ((si - keep) * HV + hv) * MF * 32;
            int e = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              to[(e++) * 32] = m[k];
              to[(e++) * 32] = l[k];
              to[(e++) * 32] = mw[k];
            }
#pragma unroll
            for (int kc = 0; kc < NK; ++kc)
#pragma unroll
              for (int i = 0; i < 4; ++i) to[(e++) * 32] = o[kc][i];
          }
          met = meet();
          if (!met) break;
          if (si < keep) {
            for (int w = si; w < left - keep; w += keep) {
              const float* ob = buf + (w * HV + hv) * MF * 32;
              auto weight = [](float x, float top) { return x == -INFINITY ? 0.f : ex2(x - top); };
              int e = 0;
              float fa[2], fb[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float om = ob[(e++) * 32], ol = ob[(e++) * 32], ow = ob[(e++) * 32];
                const float mn = fmaxf(m[k], om), wn = fmaxf(mw[k], ow);
                l[k] = l[k] * weight(m[k], mn) + ol * weight(om, mn);
                fa[k] = weight(mw[k], wn);
                fb[k] = weight(ow, wn);
                m[k] = mn;
                mw[k] = wn;
              }
#pragma unroll
              for (int kc = 0; kc < NK; ++kc)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[kc][i] = o[kc][i] * fa[i & 1] + ob[(e++) * 32] * fb[i & 1];
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
          const float inv = ex2(mw[k] - m[k]) / lt;
          const float unit = exp2i(-kWeightExp);  // first of the two: inv can be as small as fp32 goes
          const float lse_v = (m[k] + log2f(lt)) * kLn2;
          if (col < G) {
            const int qhl = hl * G + col;
            if (whole) {
              const int64_t qh = (int64_t)h.hg * HQU + qhl;
              uint32_t* op = reinterpret_cast<uint32_t*>(a.out + ((int64_t)h.b * a.num_q_heads + qh) * D) + g;
#pragma unroll
              for (int kc = 0; kc < NK; ++kc)
                op[8 * kc] = pack_bf16x2(o[kc][k] * unit * inv, o[kc][2 + k] * unit * inv);
              if (g == 0 && a.lse) a.lse[(int64_t)h.b * a.num_q_heads + qh] = lse_v;
            } else {
              float2* pp = reinterpret_cast<float2*>(a.part_o + ((int64_t)h.part * HQU + qhl) * D) + g;
#pragma unroll
              for (int kc = 0; kc < NK; ++kc)
                pp[8 * kc] = make_float2(o[kc][k] * unit * inv, o[kc][2 + k] * unit * inv);
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

template <int D, bool TMA>
__global__ void __launch_bounds__(320, 1) paged_decode8_kernel(const __grid_constant__ Decode8Args a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int NS = a.num_stages;
  const int NC = a.HC * a.nt * a.W;
  if (TMA && (smem_u32(smem) & 1023u)) {  // the swizzled stage layout needs a 1024-byte base
    if (threadIdx.x == 0) {
      pdl_wait();
      report(a.err_word, PKV_DEVERR_INTERNAL);
    }
    return;
  }
  uint8_t* stages = smem;
  StageHdr* hdr = reinterpret_cast<StageHdr*>(smem + (size_t)NS * a.stage_bytes);
  uint64_t* hdr_full = reinterpret_cast<uint64_t*>(hdr + NS);
  uint64_t* full = hdr_full + NS;
  uint64_t* empty = full + 2 * NS;  // K's barriers, then V's
  uint64_t* meet_bar = empty + 2 * NS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(&hdr_full[s], 1);
    mbar_init(meet_bar, NC);
    for (int s = 0; s < 2 * NS; ++s) {
      mbar_init(&full[s], 1 + 32);  // a producer's go-ahead, and every lane's scale copies
      mbar_init(&empty[s], NC);
    }
    fence_mbar_init();
    if (TMA) {
      prefetch_tmap(&a.tm_k);
      prefetch_tmap(&a.tm_v);
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  pdl_wait();

  const int warp = threadIdx.x >> 5;
  if (warp == NC) {
    decode8_producer<D, TMA>(a, stages, hdr, hdr_full, full, empty, false);
  } else if (warp == NC + 1) {
    decode8_producer<D, TMA>(a, stages, hdr, hdr_full, full + NS, empty + NS, true);
  } else if (warp < NC) {
    decode8_consumer<D, TMA>(a, stages, hdr, hdr_full, full, empty, meet_bar);
  }
}

// ---------------------------------------------------------------------------------------------
// Merge of the split partials: one warp per (unit, query head), a programmatic dependent of the
// decode kernel.  Bound by latency: 4 us after 8 requests of 32768 positions, 7 after 256 requests.
// ---------------------------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) decode8_merge_kernel(const __grid_constant__ Decode8Args a) {
  pdl_trigger();
  pdl_wait();
  const int u = blockIdx.x;
  const int b = u / a.nhg, hg = u % a.nhg;
  const int HQU = a.HC * a.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qhl = blockIdx.y * 8 + warp;
  if (qhl >= HQU) return;
  constexpr int VPL = D / 32;  // values per lane
  const int64_t row = (int64_t)b * a.num_q_heads + (int64_t)hg * HQU + qhl;
  __nv_bfloat16* op = a.out + row * D + lane * VPL;
  auto store = [&](const float (&v)[VPL]) {
    if constexpr (VPL == 4)
      *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    else
      *reinterpret_cast<uint32_t*>(op) = pack_bf16x2(v[0], v[1]);
  };
  if (ld(a.kv_lens + b) <= 0) {
    if (blockIdx.y == 0 && threadIdx.x == 0) report(a.err_word, PKV_DEVERR_LENGTH);
    const float zero[VPL] = {};
    store(zero);
    if (lane == 0 && a.lse) a.lse[row] = -INFINITY;
    return;
  }
  const int first = a.unit_first[u], last = a.unit_last[u];
  if (first == last) return;  // written directly
  if (first < 0 || last >= a.num_parts || last < first) {  // a wait gave up somewhere
    if (lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
    return;
  }
  // One pass: the partials' LSEs (one per lane) and the first sixteen partial rows are loaded together,
  // so up to 32 partials cost one trip to L2; more rescale what they found.
  const float* plse = a.part_lse + qhl;
  const float* po = a.part_o + (int64_t)qhl * D + lane * VPL;
  float mx = -INFINITY, tot = 0.f;
  float acc[VPL] = {};
  for (int base = first; base <= last; base += 32) {
    const int n = min(32, last - base + 1);
    const float pl = lane < n ? ld(plse + (int64_t)(base + lane) * HQU) : -INFINITY;
    float x[16][VPL];
    auto load = [&](int i0) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float* src = po + (int64_t)(base + i0 + k) * HQU * D;
        if (i0 + k < n) {
          if constexpr (VPL == 4)
            *reinterpret_cast<float4*>(x[k]) = ld(reinterpret_cast<const float4*>(src));
          else
            *reinterpret_cast<float2*>(x[k]) = ld(reinterpret_cast<const float2*>(src));
        } else {
#pragma unroll
          for (int v = 0; v < VPL; ++v) x[k][v] = 0.f;
        }
      }
    };
    load(0);
    float mn = pl;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, s));
    mn = fmaxf(mx, mn);
    const float corr = __expf(mx - mn);  // 0 on the first round
    mx = mn;
    const float w = lane < n ? __expf(pl - mx) : 0.f;
    tot = tot * corr + w;
#pragma unroll
    for (int v = 0; v < VPL; ++v) acc[v] *= corr;
    for (int i0 = 0; i0 < n; i0 += 16) {
      if (i0 > 0) load(i0);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, (i0 + k) & 31);
#pragma unroll
        for (int v = 0; v < VPL; ++v) acc[v] += wk * x[k][v];
      }
    }
  }
  tot = warp_sum(tot);
  const float inv = 1.f / tot;
#pragma unroll
  for (int v = 0; v < VPL; ++v) acc[v] *= inv;
  store(acc);
  if (lane == 0 && a.lse) a.lse[row] = mx + logf(tot);
}

// ---------------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------------
struct Plan {
  int HC, nhg, W, G, NT, Ts, RS, R, NS, ncta;
  bool tma;
  uint32_t region, stage;
  size_t smem;
  int64_t nunits, nparts;
  size_t off_first, off_last, off_plse, off_po, ws_bytes;
};

constexpr size_t kSmemBudget = 225 * 1024;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// page_size 0: the workspace's part of the plan only.
bool make_plan(int B, int Hq, int Hkv, int D, int ncta, Plan& p, int page_size = 0, int64_t num_pages = 0) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return false;
  if (D != 64 && D != 128) return false;
  p.G = Hq / Hkv;
  if (p.G > 16) return false;
  p.NT = (p.G + 7) / 8;
  p.HC = 1;
  for (int d = 1; d <= 8 / p.NT; ++d)
    if (Hkv % d == 0) p.HC = d;
  p.nhg = Hkv / p.HC;
  p.W = 8 / (p.HC * p.NT);
  p.Ts = kSlice * p.W;
  const int RB = p.HC * D;
  p.RS = RB + 16;  // RB is a multiple of 64: rows 16 bytes off a multiple of 32 keep ldmatrix free of conflicts
  p.R = page_size % 32 == 0 ? 32 : page_size % 16 == 0 ? 16 : 8;
  p.tma = page_size > 0 && page_size % 8 == 0 && num_pages * (int64_t)page_size < 0x7fffffffLL;
  p.region = p.tma ? (uint32_t)(p.Ts * RB) : (uint32_t)(p.Ts * p.RS);
  p.stage = (2 * p.region + (uint32_t)(2 * p.Ts * p.HC * 4) + 1023u) & ~1023u;
  // the merge of a head's warps must fit into the stage that carries it
  const size_t merge = (size_t)(p.W / 2) * p.HC * p.NT * (6 + (D / 16) * 4) * 32 * 4;
  if (merge > 2 * (size_t)p.region) return false;
  const size_t per_stage = p.stage + sizeof(StageHdr) + 40;
  if (2 * per_stage + 8 > kSmemBudget) return false;
  p.NS = (int)((kSmemBudget - 8) / per_stage);
  if (p.NS > kMaxStages) p.NS = kMaxStages;
  p.smem = (size_t)p.NS * per_stage + 8;
  p.ncta = ncta;
  p.nunits = (int64_t)B * p.nhg;
  p.nparts = p.ncta + p.nunits;
  const int HQU = p.HC * p.G;
  p.off_first = 0;
  p.off_last = align256(p.off_first + (size_t)p.nunits * 4);
  p.off_plse = align256(p.off_last + (size_t)p.nunits * 4);
  p.off_po = align256(p.off_plse + (size_t)p.nparts * HQU * 4);
  p.ws_bytes = align256(p.off_po + (size_t)p.nparts * HQU * D * 4);
  return true;
}

template <int D, bool TMA>
pkv_status launch(const Plan& p, const Decode8Args& a, cudaStream_t st) {
  auto kern = paged_decode8_kernel<D, TMA>;
  // whether this instance's dynamic shared-memory limit was raised on this device (any host thread)
  static std::atomic<bool> configured[64];
  const int dev = pkv_host::current_device();
  if (dev < 0) return PKV_ERR_CUDA;
  if (dev >= 64 || !configured[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess)
      return PKV_ERR_CUDA;
    if (dev < 64) configured[dev].store(true, std::memory_order_relaxed);
  }
  const pkv_status s = pkv_host::launch_after(kern, dim3(p.ncta), (p.HC * p.NT * p.W + 2) * 32, p.smem, st, a);
  if (s != PKV_OK) return s;
  return pkv_host::launch_after(decode8_merge_kernel<D>, dim3((unsigned)p.nunits, (unsigned)((p.HC * p.G + 7) / 8)), 256, 0,
                                st, a);
}

}  // namespace

extern "C" {

size_t pkv_decode_fp8_workspace_size(int32_t batch_size, int32_t num_q_heads, int32_t num_kv_heads,
                                     int32_t head_dim) {
  Plan p;
  const int n = pkv_host::sm_count();
  if (n <= 0 || !make_plan(batch_size, num_q_heads, num_kv_heads, head_dim, n, p)) return 0;
  return p.ws_bytes;
}

pkv_status pkv_paged_decode_fp8(const pkv_pool_fp8* pool, const void* q, int32_t batch_size,
                                int32_t num_q_heads, const int32_t* kv_indptr, const int32_t* kv_indices,
                                const int32_t* kv_lens, float sm_scale, void* out, float* lse,
                                void* workspace, size_t workspace_bytes, uint32_t* err_word,
                                int32_t max_ctas, void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_paged_decode_fp8");
  if (!pkv_host::valid_pool8(pool) || batch_size < 0 || num_q_heads <= 0 || max_ctas < 0)
    return PKV_ERR_INVALID_ARG;
  if (batch_size == 0) return PKV_OK;
  if (!q || !kv_indptr || !kv_indices || !kv_lens || !out) return PKV_ERR_INVALID_ARG;
  if (!pkv_host::aligned16(q) || !pkv_host::aligned16(out)) return PKV_ERR_INVALID_ARG;
  if (num_q_heads % pool->num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  if (batch_size > 0x7fffffff / 64) return PKV_ERR_UNSUPPORTED;
  const int D = pool->head_dim;
  if ((D != 64 && D != 128) || num_q_heads / pool->num_kv_heads > 16) return PKV_ERR_UNSUPPORTED;
  int ncta = pkv_host::sm_count();
  if (ncta <= 0) return PKV_ERR_CUDA;
  if (max_ctas > 0 && max_ctas < ncta) ncta = max_ctas;  // fewer partials: the workspace still fits
  Plan p;
  if (!make_plan(batch_size, num_q_heads, pool->num_kv_heads, D, ncta, p, pool->page_size, pool->num_pages))
    return PKV_ERR_UNSUPPORTED;
  if (p.nparts > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;  // 31-bit numbers of units and partials
  if (!workspace || workspace_bytes < p.ws_bytes) return PKV_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PKV_ERR_INVALID_ARG;

  Decode8Args a;
  a.k_pool = (const uint8_t*)pool->k;
  a.v_pool = (const uint8_t*)pool->v;
  a.k_scale = pool->k_scale;
  a.v_scale = pool->v_scale;
  a.num_pages = pool->num_pages;
  a.page_size = pool->page_size;
  a.page_div = FastDiv((uint32_t)pool->page_size);
  a.num_kv_heads = pool->num_kv_heads;
  a.q = (const __nv_bfloat16*)q;
  a.batch = batch_size;
  a.num_q_heads = num_q_heads;
  a.kv_indptr = kv_indptr;
  a.kv_indices = kv_indices;
  a.kv_lens = kv_lens;
  a.scale_log2 = sm_scale * kLog2e;
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  uint8_t* ws = (uint8_t*)workspace;
  a.unit_first = (int32_t*)(ws + p.off_first);
  a.unit_last = (int32_t*)(ws + p.off_last);
  a.part_lse = (float*)(ws + p.off_plse);
  a.part_o = (float*)(ws + p.off_po);
  a.err_word = err_word;
  a.HC = p.HC;
  a.nhg = p.nhg;
  a.W = p.W;
  a.group = p.G;
  a.nt = p.NT;
  a.box_rows = p.R;
  a.row_stride = p.RS;
  a.stage_tokens = p.Ts;
  a.num_stages = p.NS;
  a.num_parts = (int32_t)p.nparts;
  a.kv_region = p.region;
  a.stage_bytes = p.stage;
  if (p.tma) {
    const uint64_t Hkv = pool->num_kv_heads;
    const uint64_t rows = (uint64_t)pool->num_pages * pool->page_size;
    if (!pkv_host::encode_tmap_3d_u8(&a.tm_k, pool->k, D, rows, Hkv, Hkv * D, D, D, p.R, p.HC) ||
        !pkv_host::encode_tmap_3d_u8(&a.tm_v, pool->v, D, rows, Hkv, Hkv * D, D, D, p.R, p.HC))
      return PKV_ERR_CUDA;
  }
  cudaStream_t st = (cudaStream_t)stream;
  if (p.tma) return D == 128 ? launch<128, true>(p, a, st) : launch<64, true>(p, a, st);
  return D == 128 ? launch<128, false>(p, a, st) : launch<64, false>(p, a, st);
}

}  // extern "C"
