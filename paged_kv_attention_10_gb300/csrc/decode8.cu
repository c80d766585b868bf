// Paged decode attention over an 8-bit cache (one query per request).
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
//    own running maximum m, and the two meet when a segment ends.  M is held as its distance to m, and a weight's exponent
//    is formed from x_j - m, exact next to m: of scores of 2^24 and more x_j + e_j would not hold e_j.  (The two maxima one after
//    the other, 16 requests of 4000 to 9000, 48/16 heads of 64: 54.6 us; as pairs in one round of shuffles 57.5.)
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
//  * The rest is the bf16 decode's plan, shared with the 4-bit cache (quant_decode.cuh), with boxes in the 128- or
//    64-byte swizzle.
// Measured with 32/8 heads of 128 at page size 16: 8 requests of 32768 positions 90 us, 6.2 TB/s, 91 % of
// what a device copy reaches; 256 requests of 512 to 4096 positions 195 to 196 us, 94 %.  DRAM reads are the cache's
// bytes (554 MB of 554), the tensor pipe is 18 % busy, 43 % of the issue slots are used.  Small KV head counts are
// bound by the producers' issue instead: one head of 128, 720000 positions, 50 us at page size 16, 41 at
// 64 and 151 at 1 of the 28 that the bytes take; two heads at page size 1 118 of 28.
#include "quant_decode.cuh"

namespace {

using namespace pkv;

template <int D>
struct Format8 {
  static constexpr int kDim = D, kRowBytes = D, kScaleBytes = 4, kWarps = 8, kStep = 32, kParts = 1;
  static constexpr bool kBoxedRows = false, kJoint = false, kScalesAnywhere = false;
  static constexpr int kMergeFloats = 6 + D / 4;
  // the bytes of a row are a multiple of 64: rows 16 bytes off a multiple of 32 keep ldmatrix free of conflicts
  static constexpr int kRowPad = 16;
  template <bool TMA>
  static __device__ void consume(const QuantDecodeArgs& a, uint8_t* stages, StageHdr* hdr, uint64_t* hdr_full,
                                 uint64_t* full, uint64_t* empty, uint64_t* meet_bar);
};

// Weights of the second product stand in [0, 2^(kWeightExp + 1)), the top of f16's range: one as small as 2^-39 of
// the largest is still counted.  (In [0, 2), what is below 2^-25 of it was not: 20000 positions with weights of
// 2^-25.6 are 0.0004 of the sum.)
constexpr int kWeightExp = 14;

// ---------------------------------------------------------------------------------------------
// Consumer warps: 32-position steps of one KV head with its G query heads.
// ---------------------------------------------------------------------------------------------
template <int D>
template <bool TMA>
__device__ void Format8<D>::consume(const QuantDecodeArgs& a, uint8_t* stages, StageHdr* hdr, uint64_t* hdr_full,
                                    uint64_t* full, uint64_t* empty, uint64_t* meet_bar) {
  constexpr int NK = D / 16;                      // 16-byte chunks of a row: k-steps of K q, row tiles of O
  constexpr int MF = Format8<D>::kMergeFloats;     // floats per lane merged between the warps of a head
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
  float mw[2];        // running maximum of x + e less m, which O is relative to beside m

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
      float mx[2] = {-INFINITY, -INFINITY}, mxe[2] = {-INFINITY, -INFINITY};  // of x, and of x + e less m
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 2 * hf + (i >> 1);  // token g + 8 row
          const float v = (s[hf][0][i] + s[hf][1][i]) * qs[i & 1] * ksc[row];
          x[hf][i] = g + 8 * row < nv ? v : -INFINITY;
          mx[i & 1] = fmaxf(mx[i & 1], x[hf][i]);
        }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int k = 0; k < 2; ++k) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], off));
      float corr[2], corrw[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float mn = fmaxf(m[k], mx[k]);
        corrw[k] = m[k] - mn + mw[k];
        corr[k] = ex2(m[k] - mn);
        m[k] = mn;
        l[k] *= corr[k];
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float d = x[hf][i] - m[i & 1];
          l[i & 1] += ex2(d);
          x[hf][i] = d + ve[2 * hf + (i >> 1)];
          mxe[i & 1] = fmaxf(mxe[i & 1], x[hf][i]);
        }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int k = 0; k < 2; ++k) mxe[k] = fmaxf(mxe[k], __shfl_xor_sync(0xffffffffu, mxe[k], off));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        mw[k] = fmaxf(corrw[k], mxe[k]);
        corrw[k] = ex2(corrw[k] - mw[k]);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 2 * hf + (i >> 1), k = i & 1;
          w[i] = ex2(x[hf][i] - mw[k]) * vm[row];
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
        // all but one at once where their states fit into the stage, else half of them, or as many as do, at a time
        const int room = (int)(2 * region / (uint32_t)(HV * MF * 128));
        for (int left = W; met && left > 1;) {
          const int keep = left - 1 <= room ? 1 : max(left / 2, left - room);
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
              auto moved = [](float m, float top, float w) { return m == -INFINITY ? -INFINITY : m - top + w; };
              int e = 0;
              float fa[2], fb[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float om = ob[(e++) * 32], ol = ob[(e++) * 32], ow = ob[(e++) * 32];
                const float mn = fmaxf(m[k], om), wa = moved(m[k], mn, mw[k]), wb = moved(om, mn, ow), wn = fmaxf(wa, wb);
                l[k] = l[k] * weight(m[k], mn) + ol * weight(om, mn);
                fa[k] = weight(wa, wn);
                fb[k] = weight(wb, wn);
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
          const float inv = ex2(mw[k]) / lt;
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

}  // namespace

extern "C" {

size_t pkv_decode_fp8_workspace_size(int32_t batch_size, int32_t num_q_heads, int32_t num_kv_heads,
                                     int32_t head_dim) {
  if (head_dim == 128) return quant_decode_workspace<Format8<128>>(batch_size, num_q_heads, num_kv_heads);
  if (head_dim == 64) return quant_decode_workspace<Format8<64>>(batch_size, num_q_heads, num_kv_heads);
  return 0;
}

pkv_status pkv_paged_decode_fp8(const pkv_pool_fp8* pool, const void* q, int32_t batch_size,
                                int32_t num_q_heads, const int32_t* kv_indptr, const int32_t* kv_indices,
                                const int32_t* kv_lens, float sm_scale, void* out, float* lse,
                                void* workspace, size_t workspace_bytes, uint32_t* err_word,
                                int32_t max_ctas, void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_paged_decode_fp8");
  if (!pkv_host::valid_pool8(pool)) return PKV_ERR_INVALID_ARG;
  const QuantDecodeCall c = {q,   batch_size, num_q_heads, kv_indptr,       kv_indices, kv_lens,
                             out, lse,        workspace,   workspace_bytes, err_word,   max_ctas, (cudaStream_t)stream};
  const pkv_status s = check_quant_decode(c, pool->num_kv_heads, pool->head_dim);
  if (s != PKV_OK || batch_size == 0) return s;
  return pool->head_dim == 128 ? run_quant_decode<Format8<128>>(pool, c, sm_scale, 1.f)
                               : run_quant_decode<Format8<64>>(pool, c, sm_scale, 1.f);
}

}  // extern "C"
