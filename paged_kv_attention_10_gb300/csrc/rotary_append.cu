// Rotary embedding of the step's new K and Q fused with the KV-cache write, for every pairing and
// width, into a bf16 or an 8-bit cache; and the 8-bit cache write without a rotation.
//
// For pair i < R/2 of the first R = rotary_dim values of a head, at position p,
//   x'[a] = x[a] cos(p, i) - x[b] sin(p, i),   x'[b] = x[b] cos(p, i) + x[a] sin(p, i),
// with (a, b) = (i, i + R/2) (half-split pairs) or (2i, 2i + 1) (neighbouring pairs), in fp32 with
// one rounding at the end; the values from R on pass through.  In the 8-bit cache a row is
// quantised from those fp32 values (quant.cuh), so K is rounded once, to e4m3.
//
// Bound by HBM: a thread holds one 16-byte chunk of a (token, head) row, D/8 lanes of a warp hold a
// row, and consecutive groups take consecutive heads, so loads and stores are whole lines.  The
// half-split partner comes from another lane of the row by shuffle and the row's maximum by
// xor-shuffles, so every value is read once.
#include "quant.cuh"

namespace {

using namespace pkv;

enum { kNone = 0, kHalf = 1, kPairs = 2, kAnyWidth = 3 };

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
  uint32_t rows;   // T * heads
  FastDiv heads;   // rows of a token: Hkv K heads, Hkv V heads, Hq Q heads
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

// Chunk c (8 values) of a row rotated.  All lanes of the row call it together (shuffles); `src` is
// the row, for the general widths.
template <int ROT>
PKV_DEV void rotate_chunk(const AppendArgs& a, const __nv_bfloat16* src, const float* cs, int c, int lane0,
                          unsigned mask, const uint4& u, float (&x)[8]) {
  const int R = a.R, half = R / 2;
  if constexpr (ROT == kHalf) {  // R a multiple of 16: the partner is the same place of another chunk
    const int hc = R / 16;
    const int partner = c < hc ? c + hc : c < 2 * hc ? c - hc : c;
    uint4 w;
    w.x = __shfl_sync(mask, u.x, lane0 + partner);
    w.y = __shfl_sync(mask, u.y, lane0 + partner);
    w.z = __shfl_sync(mask, u.z, lane0 + partner);
    w.w = __shfl_sync(mask, u.w, lane0 + partner);
    if (c < 2 * hc) {
      float y[8];
      unpack8(w, y);
      const int p = 8 * (c < hc ? c : c - hc);
      const float sign = c < hc ? -1.f : 1.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 co = __ldg(reinterpret_cast<const float4*>(cs + p + 4 * h));
        const float4 si = __ldg(reinterpret_cast<const float4*>(cs + half + p + 4 * h));
        x[4 * h + 0] = fmaf(x[4 * h + 0], co.x, sign * y[4 * h + 0] * si.x);
        x[4 * h + 1] = fmaf(x[4 * h + 1], co.y, sign * y[4 * h + 1] * si.y);
        x[4 * h + 2] = fmaf(x[4 * h + 2], co.z, sign * y[4 * h + 2] * si.z);
        x[4 * h + 3] = fmaf(x[4 * h + 3], co.w, sign * y[4 * h + 3] * si.w);
      }
    }
  } else if constexpr (ROT == kPairs) {  // R a multiple of 8: four whole pairs in the chunk
    if (8 * c < R) {
      const float4 co = __ldg(reinterpret_cast<const float4*>(cs + 4 * c));
      const float4 si = __ldg(reinterpret_cast<const float4*>(cs + half + 4 * c));
      const float cv[4] = {co.x, co.y, co.z, co.w}, sv[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = x[2 * i], hi = x[2 * i + 1];
        x[2 * i] = fmaf(lo, cv[i], -hi * sv[i]);
        x[2 * i + 1] = fmaf(hi, cv[i], lo * sv[i]);
      }
    }
  } else if constexpr (ROT == kAnyWidth) {  // any even R: partners read one by one
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = 8 * c + e;
      if (j < R) {
        const int i = a.interleaved ? j >> 1 : (j < half ? j : j - half);
        const bool first = a.interleaved ? !(j & 1) : j < half;
        const int pj = a.interleaved ? j ^ 1 : (first ? j + half : j - half);
        const float y = __bfloat162float(src[pj]);
        x[e] = fmaf(x[e], __ldg(cs + i), (first ? -y : y) * __ldg(cs + half + i));
      }
    }
  }
}

// LPR lanes hold one row: the power of two at or above D / 8.
template <bool FP8, int ROT, int LPR>
__global__ void __launch_bounds__(256) append_rows_kernel(const __grid_constant__ AppendArgs a) {
  const int lane = threadIdx.x & 31;
  const int c = lane & (LPR - 1), lane0 = lane & ~(LPR - 1);
  const unsigned mask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << lane0;
  const bool has = 8 * c < a.D;
  const uint32_t step = gridDim.x * (256 / LPR);
  for (uint32_t r = (blockIdx.x * 256 + threadIdx.x) / LPR; r < a.rows; r += step) {
    uint32_t t, h;
    a.heads.divmod(r, t, h);
    const bool is_q = h >= 2u * a.Hkv, is_v = !is_q && h >= (uint32_t)a.Hkv;
    const int hh = (int)h - (is_q ? 2 * a.Hkv : is_v ? a.Hkv : 0);
    // the row, its position and its slot are loaded together
    const __nv_bfloat16* src = is_q ? a.q + ((int64_t)t * a.Hq + hh) * a.D
                                    : (is_v ? a.v_new : a.k_new) + ((int64_t)t * a.Hkv + hh) * a.D;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (has) u = *reinterpret_cast<const uint4*>(src + 8 * c);
    const int64_t slot = is_q ? 0 : __ldg(a.slots + t);
    int pos = 0;
    if constexpr (ROT != kNone) {
      pos = __ldg(a.positions + t);
      if (pos < 0 || pos >= a.max_position) {
        if (h == 0 && c == 0) report(a.err_word, PKV_DEVERR_LENGTH);
        continue;
      }
    }
    if (slot < 0) continue;  // padding token
    if (slot >= a.num_slots) {
      if (h == 0 && c == 0) report(a.err_word, PKV_DEVERR_SLOT_OOB);
      continue;
    }
    float x[8];
    unpack8(u, x);
    if (ROT != kNone && !is_v) {
      rotate_chunk<ROT>(a, src, a.cos_sin + (int64_t)pos * a.R, c, lane0, mask, u, x);
      if constexpr (ROT == kAnyWidth) __syncwarp(mask);  // q may be rotated in place: partners are read before stores
    }
    if (FP8 && !is_q) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, finite_abs_bits(x[e]));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
      const int k = e4m3_scale_exp(m);
      const float inv = exp2i(-k);
      const int64_t dst = slot * a.Hkv + hh;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= inv;
      if (k == kE4m3MaxExp) {  // keep the largest rows below 2^128: no rounding up to 256 * 2^120
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (fabsf(x[e]) > 240.f && fabsf(x[e]) < INFINITY) x[e] = copysignf(240.f, x[e]);
      }
      if (has) {
        uint2 p;
        p.x = pack_e4m3x4(x[0], x[1], x[2], x[3]);
        p.y = pack_e4m3x4(x[4], x[5], x[6], x[7]);
        *reinterpret_cast<uint2*>((uint8_t*)(is_v ? a.v_pool : a.k_pool) + dst * a.D + 8 * c) = p;
      }
      if (c == 0) (is_v ? a.v_scale : a.k_scale)[dst] = exp2i(k);
    } else if (has) {
      uint4 p = u;
      if (!is_v && (ROT != kNone) && 8 * c < a.R)
        p = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
      __nv_bfloat16* dst = is_q ? a.q_out + ((int64_t)t * a.Hq + hh) * a.D
                                : (__nv_bfloat16*)(is_v ? a.v_pool : a.k_pool) + (slot * a.Hkv + hh) * a.D;
      *reinterpret_cast<uint4*>(dst + 8 * c) = p;
    }
  }
}

template <bool FP8, int ROT>
pkv_status launch_rows(const AppendArgs& a, cudaStream_t st) {
  const int chunks = a.D / 8;
  int lpr = 1;
  while (lpr < chunks) lpr <<= 1;
  const int64_t per_block = 256 / lpr;
  int64_t blocks = (a.rows + per_block - 1) / per_block;
  const int64_t cap = (int64_t)pkv_host::sm_count() * 16;
  if (cap > 0 && blocks > cap) blocks = cap;
  const unsigned g = (unsigned)blocks;
  switch (lpr) {
    case 1: append_rows_kernel<FP8, ROT, 1><<<g, 256, 0, st>>>(a); break;
    case 2: append_rows_kernel<FP8, ROT, 2><<<g, 256, 0, st>>>(a); break;
    case 4: append_rows_kernel<FP8, ROT, 4><<<g, 256, 0, st>>>(a); break;
    case 8: append_rows_kernel<FP8, ROT, 8><<<g, 256, 0, st>>>(a); break;
    case 16: append_rows_kernel<FP8, ROT, 16><<<g, 256, 0, st>>>(a); break;
    default: append_rows_kernel<FP8, ROT, 32><<<g, 256, 0, st>>>(a); break;
  }
  return pkv_host::launch_status();
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
  a.rows = (uint32_t)(heads * a.T);
  a.heads = FastDiv((uint32_t)heads);
  a.num_slots = num_pages * page_size;
  if (!rotary) return launch_rows<FP8, kNone>(a, st);
  if (a.interleaved ? a.R % 8 != 0 : a.R % 16 != 0) return launch_rows<FP8, kAnyWidth>(a, st);
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
