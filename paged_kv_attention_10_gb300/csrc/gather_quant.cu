// Read-back of an 8-bit or a 4-bit paged cache: every request's rows in position order as bf16.
//
// bf16(x8 * scale) per value, exact for the power-of-two scales the append writes; bf16(x4 * scale * global) with one
// scale per 16 values.  Bound by HBM (one byte, or a little over half of one, in, two out).  A CTA takes a tile of
// consecutive output rows: a thread a row finds its request by binary search over out_indptr and its slot, then
// all threads copy 8 bytes at a time, K and V, with the loads of four chunks each in flight.  The search is a chain of
// loads that the copies of other CTAs hide, so a CTA takes one tile and no more, and the tile is just large enough for
// the four chunks.  64 requests of 1 to 4096 positions, 8 heads of 128: 124 us (8 bits), 106 (4 bits), 97 and 96 % of what a
// device copy reaches (with tiles of sixteen rows taken in turn by eight CTAs an SM 135 and 117; with twice the rows
// a tile 127 and 109); 16 requests 34 and 29 us (36 and 31; 38 and 34).
#include "quant.cuh"

namespace {

using namespace pkv;

constexpr int kThreads = 256;
constexpr int kMostRows = 128;  // of a tile

struct GatherArgs {
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const void* k_scale;
  const void* v_scale;
  float k_global, v_global;  // 4 bits: the caches' scales
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* kv_lens;
  const int32_t* out_indptr;
  int32_t batch, num_out_rows, page_size, Hkv;
  int64_t num_pages;
  int32_t rows;  // of a tile
  int32_t rows_at_32;  // whether k_out and v_out are 32-byte aligned
  FastDiv page_div;
  FastDiv cpr;   // 8-byte chunks of a token row
  FastDiv cph;   // ... of a head
  uint4* k_out;
  uint4* v_out;
  uint32_t* err_word;
};

// What an 8-byte chunk's scale is, and the chunk's values as bf16.
struct Bits8 {
  static constexpr int kWords = 1;  // 16-byte words that a chunk becomes
  using Scale = float;
  // one per head
  static PKV_DEV int64_t scale_at(const GatherArgs& a, int64_t slot, uint32_t c) {
    return slot * a.Hkv + a.cph.quot(c);
  }
  static PKV_DEV void store(const GatherArgs&, uint4* to, uint2 u, float s, float) {
    uint32_t h[4], r[4];
    unpack_e4m3x4(u.x, h[0], h[1]);
    unpack_e4m3x4(u.y, h[2], h[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      r[i] = pack_bf16x2(f.x * s, f.y * s);
    }
    to[0] = make_uint4(r[0], r[1], r[2], r[3]);
  }
};

struct Bits4 {
  static constexpr int kWords = 2;
  using Scale = uint8_t;
  // one per chunk
  static PKV_DEV int64_t scale_at(const GatherArgs& a, int64_t slot, uint32_t c) { return slot * a.cpr.d + c; }
  static PKV_DEV void store(const GatherArgs& a, uint4* to, uint2 u, uint8_t s8, float g) {
    const uint32_t s = unpack_e4m3x2(s8 | s8 << 8);
    uint32_t h[4], r[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      unpack_e2m1x8(j ? u.y : u.x, h);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = mul_f16x2(h[i], s);  // exact
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
        r[4 * j + i] = pack_bf16x2(f.x * g, f.y * g);
      }
    }
    if (!a.rows_at_32) {
      to[0] = make_uint4(r[0], r[1], r[2], r[3]);
      to[1] = make_uint4(r[4], r[5], r[6], r[7]);
      return;
    }
    // one store of 32 bytes: in two of 16, each instruction fills half of every sector that it touches (16 requests of up to
    // 4096 positions: 48 us where one store took 32)
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  }
};

// Slot of output row `row`, or -1: a row of no request, behind its request's end, or of a bad page.
PKV_DEV int64_t find_slot(const GatherArgs& a, int32_t row) {
  int lo = 0, hi = a.batch;  // the last b in [0, batch] with out_indptr[b] <= row
  if (row < ld(a.out_indptr)) return -1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ld(a.out_indptr + mid) <= row) lo = mid;
    else hi = mid - 1;
  }
  if (lo == a.batch) return -1;
  const int32_t o0 = ld(a.out_indptr + lo), len = ld(a.kv_lens + lo), p0 = ld(a.kv_indptr + lo);  // in one round of loads
  const int32_t np = ld(a.kv_indptr + lo + 1) - p0, j = row - o0;
  if (j < 0 || j >= len) return -1;
  uint32_t pidx, in_page;
  a.page_div.divmod((uint32_t)j, pidx, in_page);
  if ((int32_t)pidx >= np || !a.kv_indices) {
    report(a.err_word, PKV_DEVERR_LENGTH);
    return -1;
  }
  const int32_t page = ld(a.kv_indices + p0 + pidx);
  if (page < 0 || page >= a.num_pages) {
    report(a.err_word, PKV_DEVERR_PAGE_OOB);
    return -1;
  }
  return (int64_t)page * a.page_size + in_page;
}

template <class F>
__global__ void __launch_bounds__(kThreads) paged_gather_quant_kernel(const __grid_constant__ GatherArgs a) {
  __shared__ int64_t s_slot[kMostRows];
  const int kRows = a.rows;
  pdl_trigger();
  pdl_wait();
  // what the copies below cannot see: a request whose rows do not hold its length, or lie outside out
  for (int b = blockIdx.x * kThreads + threadIdx.x; b < a.batch; b += gridDim.x * kThreads) {
    const int64_t o0 = ld(a.out_indptr + b), o1 = ld(a.out_indptr + b + 1);
    const int32_t n = ld(a.kv_lens + b);
    if (n < 0 || n > o1 - o0) report(a.err_word, PKV_DEVERR_LENGTH);
    if (n > 0 && (o0 < 0 || o0 + n > a.num_out_rows)) report(a.err_word, PKV_DEVERR_ROW_OOB);
  }
  const uint32_t cpr = a.cpr.d;
  using Scale = typename F::Scale;
  const uint2* k_in = reinterpret_cast<const uint2*>(a.k_pool);
  const uint2* v_in = reinterpret_cast<const uint2*>(a.v_pool);
  const Scale* k_scale = reinterpret_cast<const Scale*>(a.k_scale);
  const Scale* v_scale = reinterpret_cast<const Scale*>(a.v_scale);
  const int32_t row0 = blockIdx.x * kRows;
  if ((int)threadIdx.x < kRows)
    s_slot[threadIdx.x] = row0 + (int)threadIdx.x < a.num_out_rows ? find_slot(a, row0 + threadIdx.x) : -1;
  __syncthreads();
  const uint32_t n = kRows * cpr;
  for (uint32_t i0 = threadIdx.x; i0 < n; i0 += 4 * kThreads) {
    uint2 k[4], v[4];
    Scale ks[4], vs[4];
    bool on[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t i = i0 + u * kThreads;
      uint32_t r, c;
      a.cpr.divmod(i < n ? i : 0, r, c);
      const int64_t slot = s_slot[r];
      on[u] = i < n && slot >= 0;
      if (on[u]) {
        const int64_t src = slot * cpr + c;
        k[u] = ld(k_in + src);
        v[u] = ld(v_in + src);
        const int64_t hs = F::scale_at(a, slot, c);
        ks[u] = ld(k_scale + hs);
        vs[u] = ld(v_scale + hs);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (on[u]) {
        const int64_t dst = ((int64_t)row0 * cpr + i0 + u * kThreads) * F::kWords;
        F::store(a, a.k_out + dst, k[u], ks[u], a.k_global);
        F::store(a, a.v_out + dst, v[u], vs[u], a.v_global);
      }
    }
  }
}

// row_bytes: of a head in the pool
template <class F, class Pool>
pkv_status gather(const Pool* pool, int32_t row_bytes, float k_global, float v_global, const int32_t* kv_indptr,
                  const int32_t* kv_indices, const int32_t* kv_lens, int32_t batch_size, const int32_t* out_indptr,
                  int32_t num_out_rows, void* k_out, void* v_out, uint32_t* err_word, void* stream) {
  if (batch_size < 0 || num_out_rows < 0) return PKV_ERR_INVALID_ARG;
  if (batch_size == 0 || num_out_rows == 0) return PKV_OK;
  if (!kv_indptr || !kv_lens || !out_indptr || !k_out || !v_out) return PKV_ERR_INVALID_ARG;
  if (!pkv_host::aligned16(k_out) || !pkv_host::aligned16(v_out)) return PKV_ERR_INVALID_ARG;
  const int64_t cpr = (int64_t)pool->num_kv_heads * (row_bytes / 8);
  if (cpr > 0x7fffffffLL / kMostRows || num_out_rows > 0x7fffffff - kMostRows) return PKV_ERR_UNSUPPORTED;
  // Four rows, or as many as give every thread four chunks: a tile's slots are looked up before its copies start.
  int rows = 4;
  while (rows < kMostRows && rows * cpr < 4 * kThreads) rows *= 2;
  GatherArgs a;
  a.k_pool = (const uint8_t*)pool->k;
  a.v_pool = (const uint8_t*)pool->v;
  a.k_scale = pool->k_scale;
  a.v_scale = pool->v_scale;
  a.k_global = k_global;
  a.v_global = v_global;
  a.kv_indptr = kv_indptr;
  a.kv_indices = kv_indices;
  a.kv_lens = kv_lens;
  a.out_indptr = out_indptr;
  a.batch = batch_size;
  a.num_out_rows = num_out_rows;
  a.page_size = pool->page_size;
  a.Hkv = pool->num_kv_heads;
  a.num_pages = pool->num_pages;
  a.rows = rows;
  a.rows_at_32 = (((uintptr_t)k_out | (uintptr_t)v_out) & 31) == 0;
  a.page_div = FastDiv((uint32_t)pool->page_size);
  a.cpr = FastDiv((uint32_t)cpr);
  a.cph = FastDiv((uint32_t)(row_bytes / 8));
  a.k_out = (uint4*)k_out;
  a.v_out = (uint4*)v_out;
  a.err_word = err_word;
  const int64_t blocks = ((int64_t)num_out_rows + rows - 1) / rows;
  return pkv_host::launch_after(paged_gather_quant_kernel<F>, dim3((unsigned)blocks), kThreads, 0,
                                (cudaStream_t)stream, a);
}

}  // namespace

extern "C" {

pkv_status pkv_paged_gather_fp8(const pkv_pool_fp8* pool, const int32_t* kv_indptr, const int32_t* kv_indices,
                                const int32_t* kv_lens, int32_t batch_size, const int32_t* out_indptr,
                                int32_t num_out_rows, void* k_out, void* v_out, uint32_t* err_word,
                                void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_paged_gather_fp8");
  if (!pkv_host::valid_pool8(pool)) return PKV_ERR_INVALID_ARG;
  return gather<Bits8>(pool, pool->head_dim, 1.f, 1.f, kv_indptr, kv_indices, kv_lens, batch_size, out_indptr,
                       num_out_rows, k_out, v_out, err_word, stream);
}

pkv_status pkv_paged_gather_fp4(const pkv_pool_fp4* pool, const int32_t* kv_indptr, const int32_t* kv_indices,
                                const int32_t* kv_lens, int32_t batch_size, const int32_t* out_indptr,
                                int32_t num_out_rows, void* k_out, void* v_out, uint32_t* err_word,
                                void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_paged_gather_fp4");
  if (!pkv_host::valid_pool4(pool)) return PKV_ERR_INVALID_ARG;
  return gather<Bits4>(pool, pool->head_dim / 2, pool->k_global, pool->v_global, kv_indptr, kv_indices, kv_lens,
                       batch_size, out_indptr, num_out_rows, k_out, v_out, err_word, stream);
}

}  // extern "C"
