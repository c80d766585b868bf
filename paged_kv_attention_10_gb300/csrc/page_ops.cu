// Movements of rows within a paged cache of any format, in many tensors (the K, V and scale tensors of all layers) at
// once: copies of whole or begun pages, and the accepted tokens of drafted trees moved behind their prefix.
//
// Nothing is computed: bytes move, in pieces of the largest power of two up to 16 that divides a tensor's address and its
// bytes per slot.  Bound by HBM for many pages, by latency for a few.
#include <algorithm>
#include <utility>

#include "quant.cuh"

namespace {

using namespace pkv;

// The tensors of a call.  N: how many it has room for; a call of a few (one layer) does not carry the room of all layers
// through its launch (a copy of 4 pages 2.1 us, 2.4 with all of it).
template <int N>
struct Planes {
  void* base[N];
  uint32_t slot_bytes[N];
  uint8_t piece[N];   // bytes of a lane's copy
  uint32_t first[N];  // of the plane's tiles (chunks), counted from those of plane 0 (see each kernel)
  int32_t count;
};
constexpr int kFewPlanes = 8, kMaxPlanes = 256;

// The plane of tile (chunk) r: the last whose first is not behind r.
template <int N>
PKV_DEV int plane_of(const Planes<N>& p, uint32_t r) {
  int lo = 0, hi = p.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.first[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Pieces that a lane has in flight, and so the tile of a warp.  With eight, four, two and one: 256 pages of 16 slots of a 4-bit
// cache, 8 heads of 128, 36 layers, among the sources pages that several copies read, 48.7, 48.4, 51.5 and 68.2 us; of a bf16
// cache, 8 heads of 64, every page once, 91.5, 91.2, 92.6 and 115.9; 4 pages of bf16, one layer, on the device alone, 2.0, 1.7, 1.5 and 1.5.
constexpr int kFlight = 4;

// ---------------------------------------------------------------------------------------------
// Copies of pages.  A warp takes a tile of one page of one tensor: 32 lanes times kFlight pieces.
// ---------------------------------------------------------------------------------------------
template <int N>
struct CopyArgs {
  Planes<N> planes;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* rows;
  int64_t num_pages;
  int32_t page_size;
  FastDiv tile_div;  // by the tiles of a page in all tensors
  uint32_t items;
  uint32_t* err_word;
};

template <typename V>
PKV_DEV void copy_tile(const char* from, char* to, uint32_t bytes, uint32_t tile) {
  const uint32_t n = bytes / sizeof(V), at = tile * 32 * kFlight + (threadIdx.x & 31);
  const V* s = reinterpret_cast<const V*>(from);
  V* d = reinterpret_cast<V*>(to);
  V v[kFlight];
#pragma unroll
  for (int u = 0; u < kFlight; ++u)
    if (at + 32 * u < n) v[u] = ld(s + at + 32 * u);
#pragma unroll
  for (int u = 0; u < kFlight; ++u)
    if (at + 32 * u < n) d[at + 32 * u] = v[u];
}

template <int N>
__global__ void __launch_bounds__(256) copy_pages_kernel(const __grid_constant__ CopyArgs<N> a) {
  pdl_trigger();
  pdl_wait();
  const uint32_t item = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (item >= a.items) return;
  uint32_t i, r;
  a.tile_div.divmod(item, i, r);
  const int32_t dst = ld(a.dst + i), src = ld(a.src + i);
  const int32_t rows = a.rows ? ld(a.rows + i) : a.page_size;
  if (dst < 0) return;  // padding
  const bool pages_ok = src >= 0 && src < a.num_pages && dst < a.num_pages, rows_ok = rows >= 0 && rows <= a.page_size;
  if (!pages_ok || !rows_ok) {
    if (r == 0 && (threadIdx.x & 31) == 0)
      report(a.err_word, (pages_ok ? 0u : PKV_DEVERR_PAGE_OOB) | (rows_ok ? 0u : PKV_DEVERR_LENGTH));
    return;
  }
  if (src == dst) return;
  const int p = plane_of(a.planes, r);
  const uint32_t tile = r - a.planes.first[p], slot = a.planes.slot_bytes[p], bytes = rows * slot;
  const int64_t page = (int64_t)slot * a.page_size;
  const char* from = (const char*)a.planes.base[p] + src * page;
  char* to = (char*)a.planes.base[p] + dst * page;
  switch (a.planes.piece[p]) {
    case 16: copy_tile<uint4>(from, to, bytes, tile); break;
    case 8: copy_tile<uint2>(from, to, bytes, tile); break;
    case 4: copy_tile<uint32_t>(from, to, bytes, tile); break;
    case 2: copy_tile<uint16_t>(from, to, bytes, tile); break;
    default: copy_tile<uint8_t>(from, to, bytes, tile);
  }
}

// ---------------------------------------------------------------------------------------------
// Compaction.  Row k of a request's accepted tokens moves from position prefix + accepted[k] to prefix + k.  With
// accepted ascending, no row is written before it is read as long as rows are taken in order: what row k writes
// (prefix + k) is not the source of a later row j (prefix + accepted[j], accepted[j] >= j > k).  A warp takes a run of
// chunks, 32 pieces side by side in one tensor, of one request's rows: it looks the rows' slots up once.  Of narrow rows it
// takes several at a time: it reads a group of rows, then writes it.
// ---------------------------------------------------------------------------------------------
template <int N>
struct CompactArgs {
  Planes<N> planes;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* prefix_lens;
  const int32_t* accepted_indptr;
  const int32_t* accepted;
  int64_t num_pages;
  int32_t page_size, num_accepted;
  FastDiv item_div;  // by the warps of a request
  FastDiv page_div;
  uint32_t chunks, run;  // of a request in all tensors, and of a warp
  uint32_t* err_word;
};

// The slot of position `pos` of a request with np pages from p0 on; -1 and a bit in bad where there is none.
template <int N>
PKV_DEV int64_t slot_at(const CompactArgs<N>& a, int32_t p0, int32_t np, int64_t pos, uint32_t& bad) {
  uint32_t pidx = 0, in_page = 0;
  if (pos <= 0x7fffffff) a.page_div.divmod((uint32_t)pos, pidx, in_page);
  if (pos > 0x7fffffff || (int64_t)pidx >= np) {
    bad |= PKV_DEVERR_LENGTH;
    return -1;
  }
  const int32_t page = ld(a.kv_indices + p0 + pidx);
  if (page < 0 || page >= a.num_pages) {
    bad |= PKV_DEVERR_PAGE_OOB;
    return -1;
  }
  return (int64_t)page * a.page_size + in_page;
}

// A warp's pieces `chunk` (32 side by side) of the n rows of lane l's (source, target) slots, kMoves pieces a lane in
// flight: four, with 32 warps an SM (64 trees in 36 layers: two 17.6 us, four 15.8, eight with 24 warps 16.0).
constexpr int kMoves = 4;

template <typename V, typename Slot>
PKV_DEV void move_rows(char* base, uint32_t slot_bytes, uint32_t chunk, Slot src, Slot dst, int n) {
  const int lane = threadIdx.x & 31;
  const int cols = min(32, (int)(slot_bytes / sizeof(V)) - 32 * (int)chunk);
  const int sh = 32 - __clz(cols - 1);  // lanes of a row: the power of two at or above cols
  const int col = lane & ((1 << sh) - 1), sub = lane >> sh, step = 32 >> sh;
  char* at = base + (32 * (int64_t)chunk + col) * sizeof(V);
#pragma unroll 1
  for (int k0 = 0; k0 < n; k0 += step * kMoves) {
    V v[kMoves];
    uint32_t on = 0;
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      const int k = k0 + u * step + sub;
      const Slot s = __shfl_sync(0xffffffffu, src, k & 31);
      if (k < n && col < cols && s >= 0) {
        v[u] = ld(reinterpret_cast<const V*>(at + (int64_t)s * slot_bytes));
        on |= 1u << u;
      }
    }
    __syncwarp();  // read by every lane before any writes
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      const Slot d = __shfl_sync(0xffffffffu, dst, (k0 + u * step + sub) & 31);
      if (on >> u & 1) *reinterpret_cast<V*>(at + (int64_t)d * slot_bytes) = v[u];
    }
    __syncwarp();  // a group's rows are written before the next group's are read
  }
}

// kWide: every tensor moves in pieces of 16 bytes, and slots have 31-bit numbers.  Blocks of one warp, 32 an SM: requests
// have different numbers of rows, and a block keeps its place until its last warp is done (64 trees in 36 layers: eight
// warps 17.4 us, two 17.0, one 15.5).
constexpr int kCompactWarps = 32;
constexpr int kRun = 4;  // chunks of a warp, at most
template <int N, bool kWide>
__global__ void __launch_bounds__(32, kWide ? kCompactWarps : kCompactWarps / 2) compact_accepted_kernel(const __grid_constant__ CompactArgs<N> a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x;
  uint32_t b, part;
  a.item_div.divmod(blockIdx.x, b, part);
  const int32_t i0 = ld(a.accepted_indptr + b), i1 = ld(a.accepted_indptr + b + 1), prefix = ld(a.prefix_lens + b);
  const int32_t p0 = ld(a.kv_indptr + b), np = ld(a.kv_indptr + b + 1) - p0;
  if (i0 < 0 || i1 > a.num_accepted || prefix < 0) {
    if (part == 0 && lane == 0) report(a.err_word, prefix < 0 ? PKV_DEVERR_LENGTH : PKV_DEVERR_ROW_OOB);
    return;
  }
  const uint32_t r0 = part * a.run, r1 = min(r0 + a.run, a.chunks);
  for (int k0 = 0; k0 < i1 - i0; k0 += 32) {
    const int k = k0 + lane, n = min(32, i1 - i0 - k0);
    int64_t src = -1, dst = -1;
    if (lane < n) {
      const int32_t node = ld(a.accepted + i0 + k), before = k > 0 ? ld(a.accepted + i0 + k - 1) : -1;
      uint32_t bad = node <= before ? PKV_DEVERR_LENGTH : 0u;
      if (!bad && node > k) {  // else it is in its place
        src = slot_at(a, p0, np, (int64_t)prefix + node, bad);
        dst = slot_at(a, p0, np, (int64_t)prefix + k, bad);
        if (dst < 0) src = -1;
      }
      if (bad && part == 0) report(a.err_word, bad);
    }
    uint32_t moving = __ballot_sync(0xffffffffu, src >= 0);
    if (!moving) continue;
    int p = plane_of(a.planes, r0);
    if constexpr (kWide) {
      // Row by row, with the loads of all of the run's chunks together.  A lane reads and writes the same columns only, so its
      // own order of loads and stores is all that is needed.  (64 trees in 36 layers 14.3 us, chunk by chunk 15.5; over
      // inputs that L2 does not hold 16.6 and 17.0; two rows at a time with 24 warps an SM 14.2 and 16.2.)  Where no chunk is
      // whole several rows at a time are better (2 heads of 64, 32 rows a tree: 16 us, 29 row by row).
      char* at[kRun];
      uint32_t slot[kRun];
      bool whole = false;
      int q = p;
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        at[j] = nullptr;
        slot[j] = 0;
        if (r0 + j < r1) {
          if (q + 1 < a.planes.count && a.planes.first[q + 1] <= r0 + j) ++q;
          const uint32_t chunk = r0 + j - a.planes.first[q], column = 512 * chunk + 16 * lane;
          slot[j] = a.planes.slot_bytes[q];
          whole = whole || slot[j] >= 512 * (chunk + 1);
          if (column < slot[j]) at[j] = (char*)a.planes.base[q] + column;
        }
      }
      if (whole) {
        while (moving) {
          const int row = __ffs(moving) - 1;
          moving &= moving - 1;
          const int64_t s = __shfl_sync(0xffffffffu, (int32_t)src, row), d = __shfl_sync(0xffffffffu, (int32_t)dst, row);
          uint4 v[kRun];
#pragma unroll
          for (int j = 0; j < kRun; ++j)
            if (at[j]) v[j] = ld(reinterpret_cast<const uint4*>(at[j] + s * slot[j]));
#pragma unroll
          for (int j = 0; j < kRun; ++j)
            if (at[j]) *reinterpret_cast<uint4*>(at[j] + d * slot[j]) = v[j];
        }
        continue;
      }
    }
    for (uint32_t r = r0; r < r1; ++r) {
      if (p + 1 < a.planes.count && a.planes.first[p + 1] <= r) ++p;
      const uint32_t chunk = r - a.planes.first[p], slot = a.planes.slot_bytes[p];
      char* base = (char*)a.planes.base[p];
      if constexpr (kWide) {
        move_rows<uint4, int32_t>(base, slot, chunk, (int32_t)src, (int32_t)dst, n);
      } else {
        switch (a.planes.piece[p]) {
          case 16: move_rows<uint4>(base, slot, chunk, src, dst, n); break;
          case 8: move_rows<uint2>(base, slot, chunk, src, dst, n); break;
          case 4: move_rows<uint32_t>(base, slot, chunk, src, dst, n); break;
          case 2: move_rows<uint16_t>(base, slot, chunk, src, dst, n); break;
          default: move_rows<uint8_t>(base, slot, chunk, src, dst, n);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------------
uint32_t piece_bytes(const pkv_plane& p) {
  uint32_t v = 16;
  while (((uintptr_t)p.base | (uintptr_t)p.slot_bytes) % v) v >>= 1;
  return v;
}

pkv_status check_planes(const pkv_plane* planes, int32_t num_planes, int64_t num_pages, int32_t page_size) {
  if (num_planes < 0 || num_pages <= 0 || page_size <= 0 || (num_planes > 0 && !planes)) return PKV_ERR_INVALID_ARG;
  for (int32_t i = 0; i < num_planes; ++i) {
    if (!planes[i].base || planes[i].slot_bytes <= 0) return PKV_ERR_INVALID_ARG;
    // 31-bit numbers of the bytes and pieces of a page
    if (planes[i].slot_bytes > 0x7fffffff / page_size) return PKV_ERR_UNSUPPORTED;
  }
  return num_planes > kMaxPlanes ? PKV_ERR_UNSUPPORTED : PKV_OK;
}

// Whether two tensors share bytes: those would move twice, and a compaction would read what it has overwritten.
bool overlap(const pkv_plane* planes, int32_t num_planes, int64_t num_pages, int32_t page_size) {
  std::pair<uintptr_t, uintptr_t> at[kMaxPlanes];  // first byte, and the one behind the last
  for (int32_t i = 0; i < num_planes; ++i) {
    const uint64_t first = (uintptr_t)planes[i].base, page = (uint64_t)planes[i].slot_bytes * page_size;  // 31 bits
    if ((uint64_t)num_pages > (UINT64_MAX - first) / page) return true;  // no such tensor
    at[i] = {first, first + num_pages * page};
  }
  if (!std::is_sorted(at, at + num_planes)) std::sort(at, at + num_planes);
  for (int32_t i = 1; i < num_planes; ++i)
    if (at[i].first < at[i - 1].second) return true;
  return false;
}

// Fills the planes, items(i) of each; the sum of those, or -1 where it passes 31 bits.
template <int N, typename Items>
int64_t fill_planes(Planes<N>& to, const pkv_plane* planes, int32_t num_planes, Items items) {
  int64_t sum = 0;
  to.count = num_planes;
  for (int32_t i = 0; i < num_planes; ++i) {
    to.base[i] = planes[i].base;
    to.slot_bytes[i] = (uint32_t)planes[i].slot_bytes;
    to.piece[i] = (uint8_t)piece_bytes(planes[i]);
    to.first[i] = (uint32_t)sum;
    sum += items(planes[i]);
    if (sum > 0x7fffffffLL) return -1;
  }
  return sum;
}

template <int N>
pkv_status copy_pages(const pkv_plane* planes, int32_t num_planes, int64_t num_pages, int32_t page_size,
                      const int32_t* src, const int32_t* dst, const int32_t* rows, int32_t num_copies,
                      uint32_t* err_word, cudaStream_t st) {
  CopyArgs<N> a;
  const int64_t tiles = fill_planes(a.planes, planes, num_planes, [&](const pkv_plane& p) {
    const int64_t tile = 32 * kFlight * piece_bytes(p);
    return (p.slot_bytes * page_size + tile - 1) / tile;
  });
  if (tiles < 0 || tiles * num_copies > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  a.src = src;
  a.dst = dst;
  a.rows = rows;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.tile_div = FastDiv((uint32_t)tiles);
  a.items = (uint32_t)(tiles * num_copies);
  a.err_word = err_word;
  return pkv_host::launch_after(copy_pages_kernel<N>, dim3((a.items + 7) / 8), 256, 0, st, a);
}

template <int N>
pkv_status compact(const pkv_plane* planes, int32_t num_planes, int64_t num_pages, int32_t page_size,
                   const int32_t* kv_indptr, const int32_t* kv_indices, const int32_t* prefix_lens, int32_t batch,
                   const int32_t* accepted_indptr, const int32_t* accepted, int32_t num_accepted, uint32_t* err_word,
                   cudaStream_t st) {
  CompactArgs<N> a;
  const int64_t chunks = fill_planes(a.planes, planes, num_planes, [&](const pkv_plane& p) {
    return (p.slot_bytes / piece_bytes(p) + 31) / 32;
  });
  if (chunks < 0 || chunks * batch > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  // Runs of up to four chunks, so that one round of warps takes them all where it can (64 trees in 36 layers: one chunk
  // 21.0 us, two 15.8, three 15.9, four 15.5).
  const int64_t places = (int64_t)std::max(1, pkv_host::sm_count()) * kCompactWarps;
  const int64_t run = std::min<int64_t>(kRun, (chunks * batch + places - 1) / places);
  const int64_t warps = (chunks + run - 1) / run;
  a.kv_indptr = kv_indptr;
  a.kv_indices = kv_indices;
  a.prefix_lens = prefix_lens;
  a.accepted_indptr = accepted_indptr;
  a.accepted = accepted;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.num_accepted = num_accepted;
  a.item_div = FastDiv((uint32_t)warps);
  a.page_div = FastDiv((uint32_t)page_size);
  a.chunks = (uint32_t)chunks;
  a.run = (uint32_t)run;
  a.err_word = err_word;
  const dim3 grid((unsigned)(warps * batch));
  bool wide = num_pages * page_size <= 0x7fffffffLL;
  for (int32_t i = 0; i < num_planes; ++i) wide = wide && a.planes.piece[i] == 16;
  return wide ? pkv_host::launch_after(compact_accepted_kernel<N, true>, grid, 32, 0, st, a)
              : pkv_host::launch_after(compact_accepted_kernel<N, false>, grid, 32, 0, st, a);
}

}  // namespace

extern "C" {

pkv_status pkv_copy_pages(const pkv_plane* planes, int32_t num_planes, int64_t num_pages, int32_t page_size,
                          const int32_t* src_pages, const int32_t* dst_pages, const int32_t* rows,
                          int32_t num_copies, uint32_t* err_word, void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_copy_pages");
  const pkv_status s = check_planes(planes, num_planes, num_pages, page_size);
  if (s != PKV_OK) return s;
  if (num_copies < 0) return PKV_ERR_INVALID_ARG;
  if (num_copies == 0 || num_planes == 0) return PKV_OK;
  if (!src_pages || !dst_pages || overlap(planes, num_planes, num_pages, page_size)) return PKV_ERR_INVALID_ARG;
  return num_planes <= kFewPlanes
             ? copy_pages<kFewPlanes>(planes, num_planes, num_pages, page_size, src_pages, dst_pages, rows, num_copies,
                                      err_word, (cudaStream_t)stream)
             : copy_pages<kMaxPlanes>(planes, num_planes, num_pages, page_size, src_pages, dst_pages, rows, num_copies,
                                      err_word, (cudaStream_t)stream);
}

pkv_status pkv_compact_accepted(const pkv_plane* planes, int32_t num_planes, int64_t num_pages, int32_t page_size,
                                const int32_t* kv_indptr, const int32_t* kv_indices, const int32_t* prefix_lens,
                                int32_t batch_size, const int32_t* accepted_indptr, const int32_t* accepted,
                                int32_t num_accepted, uint32_t* err_word, void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_compact_accepted");
  const pkv_status s = check_planes(planes, num_planes, num_pages, page_size);
  if (s != PKV_OK) return s;
  if (batch_size < 0 || num_accepted < 0) return PKV_ERR_INVALID_ARG;
  if (batch_size == 0 || num_accepted == 0 || num_planes == 0) return PKV_OK;
  if (!kv_indptr || !kv_indices || !prefix_lens || !accepted_indptr || !accepted) return PKV_ERR_INVALID_ARG;
  if (overlap(planes, num_planes, num_pages, page_size)) return PKV_ERR_INVALID_ARG;
  return num_planes <= kFewPlanes
             ? compact<kFewPlanes>(planes, num_planes, num_pages, page_size, kv_indptr, kv_indices, prefix_lens,
                                   batch_size, accepted_indptr, accepted, num_accepted, err_word, (cudaStream_t)stream)
             : compact<kMaxPlanes>(planes, num_planes, num_pages, page_size, kv_indptr, kv_indices, prefix_lens,
                                   batch_size, accepted_indptr, accepted, num_accepted, err_word, (cudaStream_t)stream);
}

}  // extern "C"
