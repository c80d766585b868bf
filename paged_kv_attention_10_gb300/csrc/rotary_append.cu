// Rotary embedding of the step's new K and Q fused with the KV-cache write, for every pairing and
// width, into a bf16 or an 8-bit cache; and the 8-bit cache write without a rotation.
//
// For pair i < R/2 of the first R = rotary_dim values of a head, at position p,
//   x'[a] = x[a] cos(p, i) - x[b] sin(p, i),   x'[b] = x[b] cos(p, i) + x[a] sin(p, i),
// with (a, b) = (i, i + R/2) (half-split pairs) or (2i, 2i + 1) (neighbouring pairs), in fp32 with
// one rounding at the end; the values from R on pass through.  In the 8-bit cache a row is
// quantised from those fp32 values (quant.cuh), so K is rounded once, to e4m3.
//
// Bound by HBM.  A row of a head is held by D/16 lanes, two 16-byte chunks each: for half-split
// pairs the chunk and its partner R/2 further on, so that a pair never leaves its lane, for
// neighbouring pairs (and without a rotation) two chunks side by side.  A warp takes two such steps of
// one token, all of whose loads are issued before the token's position and slot are needed, and
// loads the token's cosines and sines once for both.  (With one chunk per lane, a shuffle for the
// partner and the table read again for every head, 8191 tokens of 32/8 heads took 43 us, 39 so, and 36
// started beside the kernel before it: 5.6 TB/s, 83 % of what a device copy of 1 GB reaches.  2304 tokens
// into an 8-bit cache, R 128: 12 us, 64 %, bound by latency, as are the few tokens of a decode step: 2.6 us.)
// Widths that are no multiple of 16 (half) or 8 (neighbours) take a
// kernel of one chunk per lane that reads its partners one by one: 8191 tokens of 32/8 heads of 80, R 20, 74 us,
// 1.7 TB/s, where R 32 takes 27.
#include "quant.cuh"

namespace {

using namespace pkv;

enum { kNone = 0, kHalf = 1, kPairs = 2 };

struct AppendArgs {
  void* k_pool;
  void* v_pool;
  float* k_scale;
  float* v_scale;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  const __nv_bfloat16* q;
  __nv_bfloat16* q_out;
  const int64_t* slots;
  const int32_t* positions;
  const float* cos_sin;
  int32_t max_position, R, interleaved;
  int32_t T, Hkv, Hq, D;
  int64_t num_slots;
  int32_t heads;     // rows of a token: Hkv K heads, Hkv V heads, Hq Q heads
  FastDiv row_div;   // general widths: by heads
  FastDiv item_div;  // by the warps of a token
  uint32_t items;    // warps (rows, for the general widths) of the call
  uint32_t* err_word;
};

PKV_DEV void unpack8(const uint4& u, float (&f)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __bfloat1622float2(h[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

PKV_DEV uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Largest finite |x| of the row, as bits, over the L lanes that hold it.
template <int L>
PKV_DEV uint32_t row_max(uint32_t m, unsigned mask) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
  return m;
}

// 8 values times 2^-k as e4m3.
PKV_DEV uint2 quantise8(float (&x)[8], int k) {
  const float inv = exp2i(-k);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= inv;
  if (k == kE4m3MaxExp) {  // keep the largest rows below 2^128: no rounding up to 256 * 2^120
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (fabsf(x[e]) > 240.f && fabsf(x[e]) < INFINITY) x[e] = copysignf(240.f, x[e]);
  }
  return make_uint2(pack_e4m3x4(x[0], x[1], x[2], x[3]), pack_e4m3x4(x[4], x[5], x[6], x[7]));
}

struct Row {
  const __nv_bfloat16* src;
  int kind;  // 0 K, 1 V, 2 Q
  int head;
};

PKV_DEV Row row_of(const AppendArgs& a, uint32_t t, int h) {
  Row r;
  r.kind = h >= 2 * a.Hkv ? 2 : h >= a.Hkv ? 1 : 0;
  r.head = h - r.kind * a.Hkv;
  r.src = r.kind == 2 ? a.q + ((int64_t)t * a.Hq + r.head) * a.D
                      : (r.kind == 1 ? a.v_new : a.k_new) + ((int64_t)t * a.Hkv + r.head) * a.D;
  return r;
}

// The token's position is usable; false (reported once, by `reporter`) skips the token.
PKV_DEV bool position_ok(const AppendArgs& a, int pos, bool reporter) {
  if (pos >= 0 && pos < a.max_position) return true;
  if (reporter) report(a.err_word, PKV_DEVERR_LENGTH);
  return false;
}
PKV_DEV bool slot_ok(const AppendArgs& a, int64_t slot, bool reporter) {
  if (slot >= 0 && slot < a.num_slots) return true;  // a negative slot is padding
  if (slot >= 0 && reporter) report(a.err_word, PKV_DEVERR_SLOT_OOB);
  return false;
}

// Steps and blocks per SM, measured on 8191 tokens of 32/8 heads at D 128, R 64 (and quantising 2304 with
// R 128): 2 steps and 4 blocks 39.0 us (15.3), 4 and 3 39.5 (16.8), 4 and 2 41.1 (17.3), 1 and 4 46.0
// (17.1); more blocks spill.  All of these before the kernel started beside the one before it, with which the
// chosen setting takes 35.9 us (12.2).  A device copy of the same bytes takes 37.1 us (16.5).
constexpr int kSteps = 2;

// L lanes hold a row (the power of two at or above its units of two chunks); a warp takes kSteps
// times 32 / L rows of one token.
template <bool FP8, int ROT, int L>
__global__ void __launch_bounds__(256, 4) append_rows_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kRows = 32 / L;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (item >= a.items) return;
  uint32_t t, part;
  a.item_div.divmod(item, t, part);
  const int u = lane & (L - 1), row0 = (int)part * kSteps * kRows + lane / L;
  const unsigned mask = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1u) << (lane & ~(L - 1));
  // this lane's chunks; the rotated ones come first, in pairs R/2 apart for half-split pairs
  const int hc = a.R / 16;
  const bool paired = ROT == kHalf && u < hc;
  const int c0 = ROT == kHalf ? (paired ? u : 2 * hc + 2 * (u - hc)) : 2 * u;
  const int c1 = paired ? u + hc : c0 + 1;
  const bool has0 = 8 * c0 < a.D, has1 = 8 * c1 < a.D;

  const int64_t slot = ld(a.slots + t);
  const int pos = ROT != kNone ? ld(a.positions + t) : 0;
  uint4 v0[kSteps], v1[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int h = row0 + i * kRows;
    v0[i] = v1[i] = make_uint4(0u, 0u, 0u, 0u);
    if (h < a.heads) {
      const uint4* src = reinterpret_cast<const uint4*>(row_of(a, t, h).src);
      if (has0) v0[i] = src[c0];
      if (has1) v1[i] = src[c1];
    }
  }
  const bool reporter = part == 0 && lane == 0;
  float co[8], si[8];  // of the lane's eight pairs
  if constexpr (ROT != kNone) {
    if (!position_ok(a, pos, reporter)) return;
    const float* cs = a.cos_sin + (int64_t)pos * a.R;
    const int p = ROT == kHalf ? 8 * c0 : 4 * c0;
    const bool lo = ROT == kHalf ? paired : 8 * c0 < a.R, hi = ROT == kHalf ? paired : 8 * c1 < a.R;
    float4 z = make_float4(1.f, 1.f, 1.f, 1.f);
    const float4 ca = lo ? ld(reinterpret_cast<const float4*>(cs + p)) : z;
    const float4 cb = hi ? ld(reinterpret_cast<const float4*>(cs + p + 4)) : z;
    z = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 sa = lo ? ld(reinterpret_cast<const float4*>(cs + a.R / 2 + p)) : z;
    const float4 sb = hi ? ld(reinterpret_cast<const float4*>(cs + a.R / 2 + p + 4)) : z;
    co[0] = ca.x, co[1] = ca.y, co[2] = ca.z, co[3] = ca.w, co[4] = cb.x, co[5] = cb.y, co[6] = cb.z, co[7] = cb.w;
    si[0] = sa.x, si[1] = sa.y, si[2] = sa.z, si[3] = sa.w, si[4] = sb.x, si[5] = sb.y, si[6] = sb.z, si[7] = sb.w;
  }
  const bool cached = slot_ok(a, slot, reporter);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int h = row0 + i * kRows;
    if (h >= a.heads) break;
    const Row r = row_of(a, t, h);
    const bool is_q = r.kind == 2;
    if (!is_q && !cached) continue;
    const bool turn0 = ROT != kNone && r.kind != 1 && (ROT == kHalf ? paired : 8 * c0 < a.R);
    const bool turn1 = ROT != kNone && r.kind != 1 && (ROT == kHalf ? paired : 8 * c1 < a.R);
    float x0[8], x1[8];
    unpack8(v0[i], x0);
    unpack8(v1[i], x1);
    if constexpr (ROT == kHalf) {
      if (turn0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float lo = x0[e], hi = x1[e];
          x0[e] = fmaf(lo, co[e], -hi * si[e]);
          x1[e] = fmaf(hi, co[e], lo * si[e]);
        }
      }
    } else if constexpr (ROT == kPairs) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (turn0) {
          const float lo = x0[2 * e], hi = x0[2 * e + 1];
          x0[2 * e] = fmaf(lo, co[e], -hi * si[e]);
          x0[2 * e + 1] = fmaf(hi, co[e], lo * si[e]);
        }
        if (turn1) {
          const float lo = x1[2 * e], hi = x1[2 * e + 1];
          x1[2 * e] = fmaf(lo, co[4 + e], -hi * si[4 + e]);
          x1[2 * e + 1] = fmaf(hi, co[4 + e], lo * si[4 + e]);
        }
      }
    }
    if (FP8 && !is_q) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, max(finite_abs_bits(x0[e]), finite_abs_bits(x1[e])));
      const int k = e4m3_scale_exp(row_max<L>(m, mask));
      const int64_t dst = slot * a.Hkv + r.head;
      uint8_t* out = (uint8_t*)(r.kind == 1 ? a.v_pool : a.k_pool) + dst * a.D;
      const uint2 p0 = quantise8(x0, k), p1 = quantise8(x1, k);
      if (has0) *reinterpret_cast<uint2*>(out + 8 * c0) = p0;
      if (has1) *reinterpret_cast<uint2*>(out + 8 * c1) = p1;
      if (u == 0) (r.kind == 1 ? a.v_scale : a.k_scale)[dst] = exp2i(k);
    } else {
      uint4* out = reinterpret_cast<uint4*>(is_q ? a.q_out + ((int64_t)t * a.Hq + r.head) * a.D
                                                 : (__nv_bfloat16*)(r.kind == 1 ? a.v_pool : a.k_pool) +
                                                       (slot * a.Hkv + r.head) * a.D);
      if (has0) out[c0] = turn0 ? pack8(x0) : v0[i];
      if (has1) out[c1] = turn1 ? pack8(x1) : v1[i];
    }
  }
}

// Any even width: one chunk per lane, L lanes per row, partners read one by one.
template <bool FP8, int L>
__global__ void __launch_bounds__(256) append_any_width_kernel(const __grid_constant__ AppendArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int c = lane & (L - 1);
  const unsigned mask = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1u) << (lane & ~(L - 1));
  const bool has = 8 * c < a.D;
  const int R = a.R, half = R / 2;
  const uint32_t row = blockIdx.x * (256 / L) + threadIdx.x / L;
  if (row >= a.items) return;
  uint32_t t, h;
  a.row_div.divmod(row, t, h);
  const Row r = row_of(a, t, (int)h);
  const bool is_q = r.kind == 2, reporter = h == 0 && c == 0;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (has) v = reinterpret_cast<const uint4*>(r.src)[c];
  const int pos = ld(a.positions + t);
  if (!position_ok(a, pos, reporter)) return;
  const int64_t slot = ld(a.slots + t);
  const bool cached = slot_ok(a, slot, reporter);
  if (!is_q && !cached) return;
  float x[8];
  unpack8(v, x);
  if (r.kind != 1 && has) {
    const float* cs = a.cos_sin + (int64_t)pos * R;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = 8 * c + e;
      if (j < R) {
        const int i = a.interleaved ? j >> 1 : (j < half ? j : j - half);
        const bool first = a.interleaved ? !(j & 1) : j < half;
        const float y = __bfloat162float(r.src[a.interleaved ? j ^ 1 : (first ? j + half : j - half)]);
        x[e] = fmaf(x[e], ld(cs + i), (first ? -y : y) * ld(cs + half + i));
      }
    }
  }
  __syncwarp(mask);  // q may be rotated in place: every lane of the row has read its partners
  if (FP8 && !is_q) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, finite_abs_bits(x[e]));
    const int k = e4m3_scale_exp(row_max<L>(m, mask));
    const int64_t dst = slot * a.Hkv + r.head;
    const uint2 p = quantise8(x, k);
    if (has) *reinterpret_cast<uint2*>((uint8_t*)(r.kind == 1 ? a.v_pool : a.k_pool) + dst * a.D + 8 * c) = p;
    if (c == 0) (r.kind == 1 ? a.v_scale : a.k_scale)[dst] = exp2i(k);
  } else if (has) {
    uint4* out = reinterpret_cast<uint4*>(is_q ? a.q_out + ((int64_t)t * a.Hq + r.head) * a.D
                                               : (__nv_bfloat16*)(r.kind == 1 ? a.v_pool : a.k_pool) +
                                                     (slot * a.Hkv + r.head) * a.D);
    out[c] = r.kind == 1 ? v : pack8(x);
  }
}

int pow2_at_least(int n) {
  int p = 1;
  while (p < n) p <<= 1;
  return p;
}

template <bool FP8, int ROT>
pkv_status launch_rows(AppendArgs a, cudaStream_t st) {
  const int hc = a.R / 16;
  const int units = ROT == kHalf ? hc + (a.D - 16 * hc + 15) / 16 : (a.D + 15) / 16;
  const int L = pow2_at_least(units);
  const int rows = kSteps * (32 / L);
  const int64_t parts = (a.heads + rows - 1) / rows;
  a.items = (uint32_t)(parts * a.T);
  a.item_div = FastDiv((uint32_t)parts);
  const unsigned g = (a.items + 7) / 8;
  switch (L) {
    case 1: return pkv_host::launch_after(append_rows_kernel<FP8, ROT, 1>, dim3(g), 256, 0, st, a);
    case 2: return pkv_host::launch_after(append_rows_kernel<FP8, ROT, 2>, dim3(g), 256, 0, st, a);
    case 4: return pkv_host::launch_after(append_rows_kernel<FP8, ROT, 4>, dim3(g), 256, 0, st, a);
    case 8: return pkv_host::launch_after(append_rows_kernel<FP8, ROT, 8>, dim3(g), 256, 0, st, a);
    default: return pkv_host::launch_after(append_rows_kernel<FP8, ROT, 16>, dim3(g), 256, 0, st, a);
  }
}

template <bool FP8>
pkv_status launch_any_width(AppendArgs a, cudaStream_t st) {
  const int L = pow2_at_least(a.D / 8);
  a.items = (uint32_t)((int64_t)a.heads * a.T);
  a.row_div = FastDiv((uint32_t)a.heads);
  const unsigned per = 256 / L, g = (a.items + per - 1) / per;
  switch (L) {
    case 1: return pkv_host::launch_after(append_any_width_kernel<FP8, 1>, dim3(g), 256, 0, st, a);
    case 2: return pkv_host::launch_after(append_any_width_kernel<FP8, 2>, dim3(g), 256, 0, st, a);
    case 4: return pkv_host::launch_after(append_any_width_kernel<FP8, 4>, dim3(g), 256, 0, st, a);
    case 8: return pkv_host::launch_after(append_any_width_kernel<FP8, 8>, dim3(g), 256, 0, st, a);
    case 16: return pkv_host::launch_after(append_any_width_kernel<FP8, 16>, dim3(g), 256, 0, st, a);
    default: return pkv_host::launch_after(append_any_width_kernel<FP8, 32>, dim3(g), 256, 0, st, a);
  }
}

bool disjoint_or_same(const void* a, const void* b, size_t bytes) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x == y || x + bytes <= y || y + bytes <= x;
}

// The checks and the launch every entry point of this file shares.  rotary: with positions and Q.
template <bool FP8>
pkv_status append_rows(AppendArgs a, int64_t num_pages, int32_t page_size, bool rotary, cudaStream_t st) {
  if (a.T < 0 || a.Hq < 0) return PKV_ERR_INVALID_ARG;
  if (rotary && (a.max_position <= 0 || a.R <= 0 || a.R % 2 != 0 || a.R > a.D)) return PKV_ERR_INVALID_ARG;
  if (a.T == 0) return PKV_OK;
  if (!a.k_new || !a.v_new || !a.slots) return PKV_ERR_INVALID_ARG;
  if (!pkv_host::aligned16(a.k_new) || !pkv_host::aligned16(a.v_new)) return PKV_ERR_INVALID_ARG;
  if (rotary) {
    if (!a.positions || !a.cos_sin || !pkv_host::aligned16(a.cos_sin)) return PKV_ERR_INVALID_ARG;
    if ((a.Hq != 0) != (a.q != nullptr) || (a.q != nullptr) != (a.q_out != nullptr)) return PKV_ERR_INVALID_ARG;
    if (a.q && (!pkv_host::aligned16(a.q) || !pkv_host::aligned16(a.q_out))) return PKV_ERR_INVALID_ARG;
    if (a.q && !disjoint_or_same(a.q, a.q_out, (size_t)a.T * a.Hq * a.D * 2)) return PKV_ERR_INVALID_ARG;
  }
  if (a.D > 256) return PKV_ERR_UNSUPPORTED;
  const int64_t heads = 2 * (int64_t)a.Hkv + a.Hq;
  if (heads * a.T > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;  // 31-bit row numbers
  a.heads = (int32_t)heads;
  a.num_slots = num_pages * page_size;
  if (!rotary) return launch_rows<FP8, kNone>(a, st);
  if (a.interleaved ? a.R % 8 != 0 : a.R % 16 != 0) return launch_any_width<FP8>(a, st);
  return a.interleaved ? launch_rows<FP8, kPairs>(a, st) : launch_rows<FP8, kHalf>(a, st);
}

AppendArgs rotary_args(const void* k_new, const void* v_new, const int64_t* slots, const int32_t* positions,
                       const float* cos_sin, int32_t max_position, int32_t rotary_dim, int32_t interleaved,
                       const void* q, void* q_out, int32_t num_q_heads, int32_t num_tokens,
                       uint32_t* err_word) {
  AppendArgs a = {};
  a.k_new = (const __nv_bfloat16*)k_new;
  a.v_new = (const __nv_bfloat16*)v_new;
  a.slots = slots;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.max_position = max_position;
  a.R = rotary_dim;
  a.interleaved = interleaved;
  a.q = (const __nv_bfloat16*)q;
  a.q_out = (__nv_bfloat16*)q_out;
  a.Hq = num_q_heads;
  a.T = num_tokens;
  a.err_word = err_word;
  return a;
}

void set_pool(AppendArgs& a, const pkv_pool_fp8* p) {
  a.k_pool = p->k;
  a.v_pool = p->v;
  a.k_scale = p->k_scale;
  a.v_scale = p->v_scale;
  a.Hkv = p->num_kv_heads;
  a.D = p->head_dim;
}

}  // namespace

extern "C" {

pkv_status pkv_rotary_kv_append(const pkv_pool* pool, const void* k_new, const void* v_new,
                                const int64_t* slot_mapping, const int32_t* positions, const float* cos_sin,
                                int32_t max_position, int32_t rotary_dim, int32_t interleaved,
                                const void* q, void* q_out, int32_t num_q_heads, int32_t num_tokens,
                                uint32_t* err_word, void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_rotary_kv_append");
  if (!pkv_host::valid_pool(pool)) return PKV_ERR_INVALID_ARG;
  AppendArgs a = rotary_args(k_new, v_new, slot_mapping, positions, cos_sin, max_position, rotary_dim,
                             interleaved, q, q_out, num_q_heads, num_tokens, err_word);
  a.k_pool = pool->k;
  a.v_pool = pool->v;
  a.Hkv = pool->num_kv_heads;
  a.D = pool->head_dim;
  return append_rows<false>(a, pool->num_pages, pool->page_size, true, (cudaStream_t)stream);
}

pkv_status pkv_rotary_kv_append_fp8(const pkv_pool_fp8* pool, const void* k_new, const void* v_new,
                                    const int64_t* slot_mapping, const int32_t* positions,
                                    const float* cos_sin, int32_t max_position, int32_t rotary_dim,
                                    int32_t interleaved, const void* q, void* q_out, int32_t num_q_heads,
                                    int32_t num_tokens, uint32_t* err_word, void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_rotary_kv_append_fp8");
  if (!pkv_host::valid_pool8(pool)) return PKV_ERR_INVALID_ARG;
  AppendArgs a = rotary_args(k_new, v_new, slot_mapping, positions, cos_sin, max_position, rotary_dim,
                             interleaved, q, q_out, num_q_heads, num_tokens, err_word);
  set_pool(a, pool);
  return append_rows<true>(a, pool->num_pages, pool->page_size, true, (cudaStream_t)stream);
}

pkv_status pkv_kv_append_fp8(const pkv_pool_fp8* pool, const void* k_new, const void* v_new,
                             const int64_t* slot_mapping, int32_t num_tokens, uint32_t* err_word,
                             void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_kv_append_fp8");
  if (!pkv_host::valid_pool8(pool)) return PKV_ERR_INVALID_ARG;
  AppendArgs a = rotary_args(k_new, v_new, slot_mapping, nullptr, nullptr, 0, 0, 0, nullptr, nullptr, 0,
                             num_tokens, err_word);
  set_pool(a, pool);
  return append_rows<true>(a, pool->num_pages, pool->page_size, false, (cudaStream_t)stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------------------------
// The cos/sin table of the rotary append, for a rotated width and a long-context scaling of the
// frequencies f_i = theta^(-2i/R).  Angles in double precision, cos and sin rounded once to fp32.
// ---------------------------------------------------------------------------------------------
namespace {

struct TableArgs {
  float* table;
  int32_t max_position, R;
  double theta, factor, orig, low, high, mscale;
  int32_t kind;
};

__device__ double scaled_frequency(const TableArgs& a, int i) {
  const double f = pow(a.theta, -2.0 * (double)i / (double)a.R);
  constexpr double kTwoPi = 6.283185307179586;
  if (a.kind == PKV_ROPE_LINEAR) return f / a.factor;
  if (a.kind == PKV_ROPE_BANDED) {
    const double turns = a.orig * f / kTwoPi;  // turns of this pair over the original context
    if (turns > a.high) return f;
    if (turns < a.low) return f / a.factor;
    const double s = (turns - a.low) / (a.high - a.low);
    return (1.0 - s) * f / a.factor + s * f;
  }
  if (a.kind == PKV_ROPE_YARN) {
    const double d = 2.0 * log(a.theta);
    double lo = floor(a.R * log(a.orig / (a.high * kTwoPi)) / d);  // pairs below turn more than `high` times
    double hi = ceil(a.R * log(a.orig / (a.low * kTwoPi)) / d);    // pairs above turn less than `low` times
    lo = fmax(lo, 0.0);
    hi = fmin(hi, (double)a.R - 1.0);
    if (hi == lo) hi += 0.001;
    const double ramp = fmin(fmax(((double)i - lo) / (hi - lo), 0.0), 1.0);
    return f / a.factor * ramp + f * (1.0 - ramp);
  }
  return f;
}

// A thread keeps one pair's frequency and walks the positions.
__global__ void __launch_bounds__(128) rotary_table_kernel(const __grid_constant__ TableArgs a) {
  const int half = a.R / 2;
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    const double f = scaled_frequency(a, i);
    for (int64_t p = blockIdx.x; p < a.max_position; p += gridDim.x) {
      double s, c;
      sincos((double)p * f, &s, &c);
      a.table[p * a.R + i] = (float)(c * a.mscale);
      a.table[p * a.R + half + i] = (float)(s * a.mscale);
    }
  }
}

}  // namespace

extern "C" pkv_status pkv_rotary_cos_sin_table(float* table, int32_t max_position, int32_t rotary_dim,
                                               double theta, const pkv_rope_scaling* scaling, void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_rotary_cos_sin_table");
  const double kInf = (double)INFINITY;
  if (max_position < 0 || rotary_dim <= 0 || rotary_dim % 2 != 0 || !(theta > 0.0) || !(theta < kInf))
    return PKV_ERR_INVALID_ARG;
  TableArgs a = {};
  a.table = table;
  a.max_position = max_position;
  a.R = rotary_dim;
  a.theta = theta;
  a.mscale = 1.0;
  if (scaling && scaling->kind != PKV_ROPE_UNSCALED) {
    const pkv_rope_scaling& s = *scaling;
    a.kind = s.kind;
    a.factor = s.factor;
    a.orig = s.original_max_position;
    a.low = s.low;
    a.high = s.high;
    if (!(s.factor >= 1.0) || !(s.factor < kInf)) return PKV_ERR_INVALID_ARG;
    if (s.kind == PKV_ROPE_BANDED || s.kind == PKV_ROPE_YARN) {
      if (!(s.original_max_position > 0.0) || !(s.original_max_position < kInf) || !(s.low > 0.0) ||
          !(s.high > s.low) || !(s.high < kInf))
        return PKV_ERR_INVALID_ARG;
    } else if (s.kind != PKV_ROPE_LINEAR) {
      return PKV_ERR_INVALID_ARG;
    }
    if (s.kind == PKV_ROPE_YARN) {
      if (!(theta > 1.0) || !(s.attention_factor > 0.0) || !(s.attention_factor < kInf))
        return PKV_ERR_INVALID_ARG;
      a.mscale = s.attention_factor;
    }
  }
  if (max_position == 0) return PKV_OK;
  if (!table) return PKV_ERR_INVALID_ARG;
  const int64_t cap = (int64_t)pkv_host::sm_count() * 16;
  const int64_t blocks = cap > 0 && max_position > cap ? cap : max_position;
  rotary_table_kernel<<<(unsigned)blocks, 128, 0, (cudaStream_t)stream>>>(a);
  return pkv_host::launch_status();
}
