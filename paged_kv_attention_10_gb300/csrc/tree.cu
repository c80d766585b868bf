// Attention of a tree of drafted tokens over a paged cache (speculative verification).
//
// What it computes: request b's T_b drafted tokens sit behind its P_b cached positions, their K/V in
// the pool like an extend's; drafted token i sees every position j < P_b, and position P_b + t for
// each bit t of its mask row (its ancestors and itself, or whatever the caller allows).  GQA, page
// lists and LSE as in the other attention calls; a row that sees nothing gives 0 and -inf.
//
// A few query rows over a long cache: bound by reading K and V once.  The extend's pipeline (two
// producer warps, QK and PV issued by two threads, P over S in TMEM, a softmax thread per row, two CTAs an SM)
// with what the shape asks for besides:
//  * Persistent CTAs, two per SM, each over an equal share of the stream of 64-position KV tiles of
//    all units (request, KV head, 128-row Q tile), so that one tree over a long context fills the GPU
//    as well as many trees do.  A unit cut by a share's border leaves fp32 partial states, merged by
//    log-sum-exp in a programmatic dependent launch.  The CTA takes its segments one after the other, with
//    all warps meeting between them; the other CTA of the SM fills the gap.
//  * Where a request may have more rows than a Q tile, CTAs 2 c and 2 c + 1 take the same share with a Q
//    tile each, so that K and V come from DRAM once for both (each its own share: 4 requests of 64
//    tokens over 32700 positions 178 us, 127 so).  Whether it may have follows from max_tree_len, not from the
//    trees: a pass of one Q tile is then one CTA's of the pair (in turn over a request's units), the other
//    passes it by.  A bound above a Q tile over smaller trees so costs 64 requests of 1 to 16 tokens 119 us for
//    109, 16 of 8 tokens over 4000 positions 64 for 51, and 64 of 8 over 4000 with one KV head (where every
//    second CTA is left without work) 46 for 39, at D 64 and group 8 37 for 27.
//  * P goes to the second product in bf16 (the type of V, which the MMA asks for), so a result is divided by the
//    sum of the rounded weights: a rounding that a row's weights share cancels (values of 1 give 1; 0.996
//    with the fp32 sum, which the LSE keeps).  The second sum costs 4 requests of 64 tokens 3 to 5 %.
//  * Only tiles that reach past the prefix are masked.  There the V rows behind the last position
//    and the infinities and NaNs of drafted tokens become 0 in shared memory (weight 0 times them
//    would be NaN for rows that do not see them); rows that do see them get them added when they are
//    written, which is what a sum with a non-zero weight would give.
// Measured with 32/8 heads of 128 at page size 16: 64 requests of 1 to 16 tokens over 512 to 4096 positions
// 109 us, 5.6 TB/s, 83 % of what a device copy reaches (K and V once from DRAM; the rest is the start, the
// shares' uneven ends and the merge); 4 requests of 64 tokens over 32700 positions 129 to 144 us, 0.95 to 1.07
// PFLOP/s, 55 to 62 % of the bytes' floor (two slots of product, softmax, product an SM; the tensor pipe is 51 %
// busy and 58 % of the issue slots are used); one request of 8 tokens over 1000 positions 12 us, all
// latency.  Page size 1 (29 requests of 8 tokens over 6000 positions, 8 heads): 146 us at D 128, 92 at D 64.
#include <atomic>

#include "quant.cuh"
#include "tc05.cuh"

namespace {

using namespace pkv;

constexpr int kBM = 128;  // Q tile rows: (token, group head) pairs
constexpr int kBN = 64;   // KV positions per tile
// warp 0 the walk and K, warp 1 QK MMAs, warps 2..5 softmax (one per TMEM lane quadrant, a thread per
// row), warp 6 V, warp 7 PV MMAs
constexpr int kSoftmaxWarps = 4;
constexpr int kVWarp = 2 + kSoftmaxWarps;
constexpr int kPVWarp = kVWarp + 1;
constexpr int kThreads = (kPVWarp + 1) * 32;
constexpr int kMaxNodes = 1024;  // drafted tokens of a request
constexpr int kUnitCost = 4;     // a unit's start and epilogue, in KV tiles of the work split (2, 4, 6, 9 tried: 64
                                 // requests of up to 16 tokens 111.8, 109.0, 109.1, 109.0 us)
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColO = 128;  // O at columns [128, 128 + D); S buffers at [0, 64) and [64, 128)
constexpr uint32_t kQHalf = kBM * 128;   // one 64-dim half of the Q tile, 16 KB
constexpr uint32_t kKVHalf = kBN * 128;  // 64 positions x 64 dims, 8 KB

// Operands are 64-dim halves of 128-byte swizzled rows.
template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kKVStage = kHalves * kKVHalf;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffK = kOffQ + kHalves * kQHalf;
  static constexpr uint32_t kOffV = kOffK + 2 * kKVStage;
  static constexpr uint32_t kOffCtl = kOffV + 2 * kKVStage;
};

// A run of KV tiles of one unit that this CTA computes.
struct Seg {
  int32_t q0;      // first row of the request in q and out
  int32_t T, P;    // drafted tokens (covered), cached positions
  int32_t p0, np;  // page list
  int32_t h;       // KV head
  int32_t t0;      // first token of the unit
  int32_t j0, n;   // first KV tile, number of tiles (0: no more work)
  int32_t part;    // partial state's slot, or -1: the segment is the whole unit
};

struct Ctl {
  Seg seg;
  uint32_t tmem_base;
  uint32_t failed;   // a wait gave up
  uint32_t bad_any;
  uint32_t bad[kMaxNodes / 32];  // drafted tokens of this segment whose V is not finite
  uint32_t pad;
  uint64_t q_full;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], s_free[2];  // S buffer b: QK written / its P consumed by PV
  uint64_t p_full[2];             // P written, V cleaned
  uint64_t qk_done, pv_done;      // every MMA of the issuing thread has completed (exit path)
  float inv[kBM];                 // 1 / (sum of P) of each row, 0 for a row that saw nothing
};
static_assert(kMaxNodes / 32 == 32, "a warp clears the notes");

// The unit that a CTA's share ends in the middle of, for the merge: its parts are the slots
// 2c + 1, 2(c + 1), 2(c + 2), ... (paired: 2c + 1, 2(c + 2), 2(c + 4), ...)
struct Cut {
  int32_t parts;  // 0: none
  int32_t q0, T, t0, h;
  int32_t pad[3];
};

struct TreeArgs {
  CUtensorMap tm_q, tm_k, tm_v;
  const int32_t* qo_indptr;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* prefix_lens;
  const uint32_t* mask;  // [num_q_tokens, words]
  int32_t words;
  const __nv_bfloat16* v_pool;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* err_word;
  int64_t num_pages;
  int32_t page_size, box_rows;
  FastDiv page_div;  // by page_size
  int32_t num_kv_heads, num_q_heads, group;
  int32_t tpt;       // tokens per Q tile
  int32_t paired;    // CTAs 2 c and 2 c + 1 take the same share, a Q tile each
  int32_t batch, num_q_tokens, max_nodes;
  float scale_log2;
  Cut* cut;          // [CTAs]
  float* part_o;     // [2 CTAs][D / 4][128 rows][4]: a warp's rows lie side by side
  float* part_lse;   // [2 CTAs][128 rows]
};

// ---------------------------------------------------------------------------------------------
// The walk over this CTA's share of the stream (warp 0)
// ---------------------------------------------------------------------------------------------
// What a request asks for: its rows, its KV, its units and their tiles.
struct Req {
  int32_t q0, T, P, p0, np;
  int32_t passes, tiles;  // over its KV by a head's Q tiles, KV tiles (0: nothing to do)
  int32_t cost;           // of a unit in the stream: its tiles and what an epilogue costs
};

__device__ Req load_req(const TreeArgs& a, int b, bool check) {
  Req r;
  r.q0 = ld(a.qo_indptr + b);
  const int32_t rows = ld(a.qo_indptr + b + 1) - r.q0;
  r.P = ld(a.prefix_lens + b);
  r.p0 = ld(a.kv_indptr + b);
  r.np = ld(a.kv_indptr + b + 1) - r.p0;
  r.T = min(max(rows, 0), a.max_nodes);
  r.passes = r.tiles = r.cost = 0;
  uint32_t bad = 0;
  if (rows < 0 || rows > a.max_nodes || r.P < 0 || r.P > 0x7fffffff - kMaxNodes - kBN) bad = PKV_DEVERR_LENGTH;
  if (rows > 0 && (r.q0 < 0 || r.q0 > a.num_q_tokens - rows)) bad |= PKV_DEVERR_ROW_OOB;
  if (bad && check) report(a.err_word, bad);
  if (r.T > 0 && r.P >= 0 && r.P <= 0x7fffffff - kMaxNodes - kBN && !(bad & PKV_DEVERR_ROW_OOB)) {
    const int per = a.paired ? 2 * a.tpt : a.tpt;  // tokens of a pass
    r.passes = (r.T + per - 1) / per;
    r.tiles = (r.P + r.T + kBN - 1) / kBN;
    r.cost = r.tiles + kUnitCost;
  }
  return r;
}

struct Walk {
  int64_t c, c1;     // next stream position, end of the share
  int64_t share;
  int64_t base;      // stream offset of request b0
  int32_t b0;
  Req r;             // of request b0 + lane
  int64_t len, incl; // its units' length in the stream, and up to its end from `base`
  Cut cut;
};

__device__ void walk_scan(const TreeArgs& a, Walk& w) {
  w.len = (int64_t)w.r.passes * w.r.cost * a.num_kv_heads;
  w.incl = w.len;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, w.incl, o);
    if ((int)(threadIdx.x & 31) >= o) w.incl += t;
  }
}

__device__ void walk_start(const TreeArgs& a, Walk& w) {
  const int lane = threadIdx.x & 31;
  w.r = Req{};
  if (lane < a.batch) w.r = load_req(a, lane, blockIdx.x == 0);
  int64_t total = (int64_t)w.r.passes * w.r.cost;
  for (int i = 32 + lane; i < a.batch; i += 128) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {  // four requests' loads in flight
      if (i + 32 * u < a.batch) {
        const Req r = load_req(a, i + 32 * u, blockIdx.x == 0);
        total += (int64_t)r.passes * r.cost;
      }
    }
  }
  total = warp_sum(total) * a.num_kv_heads;
  const int shares = gridDim.x >> a.paired;
  w.share = (total + shares - 1) / shares;
  if (w.share < 1) w.share = 1;
  w.c = (int64_t)(blockIdx.x >> a.paired) * w.share;
  w.c1 = min(total, w.c + w.share);
  w.base = 0;
  w.b0 = 0;
  w.cut = Cut{};
  walk_scan(a, w);
}

// The next segment of the share (all lanes); n = 0 when there is none.
__device__ Seg walk_next(const TreeArgs& a, Walk& w) {
  const int lane = threadIdx.x & 31;
  Seg s{};
  while (w.c < w.c1) {
    const int64_t group = __shfl_sync(0xffffffffu, w.incl, 31);
    if (w.c >= w.base + group) {  // (not past the last request: c lies in the stream)
      w.base += group;
      w.b0 += 32;
      w.r = Req{};
      if (w.b0 + lane < a.batch) w.r = load_req(a, w.b0 + lane, false);
      walk_scan(a, w);
      if (w.b0 >= a.batch) break;
      continue;
    }
    const int64_t rs = w.base + w.incl - w.len;
    const uint32_t hit = __ballot_sync(0xffffffffu, w.len > 0 && rs <= w.c && w.c < rs + w.len);
    if (!hit) break;
    const int src = __ffs(hit) - 1;
    const int64_t r0 = __shfl_sync(0xffffffffu, rs, src);
    const int tiles = __shfl_sync(0xffffffffu, w.r.tiles, src);
    const int cost = __shfl_sync(0xffffffffu, w.r.cost, src);
    const int passes = __shfl_sync(0xffffffffu, w.r.passes, src);
    s.q0 = __shfl_sync(0xffffffffu, w.r.q0, src);
    s.T = __shfl_sync(0xffffffffu, w.r.T, src);
    s.P = __shfl_sync(0xffffffffu, w.r.P, src);
    s.p0 = __shfl_sync(0xffffffffu, w.r.p0, src);
    s.np = __shfl_sync(0xffffffffu, w.r.np, src);
    const int u = (int)((w.c - r0) / cost);  // units in the order (KV head, pass)
    const int64_t us = r0 + (int64_t)u * cost;
    const int off = (int)(w.c - us);
    if (off >= tiles) {  // the rest of the unit is its epilogue's time
      w.c = us + cost;
      continue;
    }
    s.h = u / passes;
    s.j0 = off;
    s.n = (int)min((int64_t)(tiles - off), w.c1 - w.c);
    w.c += s.n;
    s.t0 = (u % passes) * a.tpt << a.paired;
    if (a.paired) {  // the pass's only Q tile goes to one CTA of the pair, taking turns
      const int parity = blockIdx.x & 1;
      if (s.t0 + a.tpt < s.T)
        s.t0 += parity * a.tpt;
      else if ((u & 1) != parity)
        continue;
    }
    s.part = s.n == tiles ? -1 : 2 * (int)blockIdx.x + (off == 0 ? 1 : 0);
    if (off == 0 && s.n < tiles)
      w.cut = Cut{(int32_t)((us + tiles - 1) / w.share) - (int)(blockIdx.x >> a.paired) + 1, s.q0, s.T, s.t0, s.h, {0, 0, 0}};
    return s;
  }
  s.n = 0;
  return s;
}

// ---------------------------------------------------------------------------------------------
// K / V producers.  t0: tiles of this CTA before the segment.
// ---------------------------------------------------------------------------------------------
// No copy of this warp is left in flight after a wait that gave up (bounded waits).
PKV_DEV void drain(uint64_t* fulls, uint32_t issued) {
  for (uint32_t t = issued < 2 ? 0 : issued - 2; t < issued; ++t) mbar_wait(&fulls[t & 1], (t >> 1) & 1);
}

// TMA boxes of min(page_size, 64) rows, lane i box i; the page indices come from a register window of 64
// page-list entries whose upper half is loaded 32 pages before it is needed.
template <int D>
__device__ bool tree_load_boxes(const TreeArgs& a, Ctl* ctl, uint32_t sb, const Seg& s, uint32_t t, bool v) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  const int R = a.box_rows, nbox = kBN / R, kv_end = s.P + s.T;
  uint64_t* fulls = v ? ctl->v_full : ctl->k_full;
  uint64_t* empties = v ? ctl->v_empty : ctl->k_empty;
  const CUtensorMap* tm = v ? &a.tm_v : &a.tm_k;
  const uint32_t base = sb + (v ? C::kOffV : C::kOffK);
  auto entry = [&](int pidx) -> int32_t {
    return (pidx >= 0 && pidx < s.np) ? ld(a.kv_indices + s.p0 + pidx) : -1;
  };
  int wbase = (int)a.page_div.quot((uint32_t)(s.j0 * kBN));
  int32_t w0 = entry(wbase + lane), w1 = entry(wbase + 32 + lane);
  for (int j = s.j0; j < s.j0 + s.n; ++j, ++t) {
    while ((int)a.page_div.quot((uint32_t)(j * kBN)) >= wbase + 32) {
      w0 = w1;
      wbase += 32;
      w1 = entry(wbase + 32 + lane);
    }
    const int pos = j * kBN + min(lane, nbox - 1) * R;
    const int pidx = (int)a.page_div.quot((uint32_t)pos), k = pidx - wbase;  // < 64: a tile spans at most 8 pages
    const int32_t v0 = __shfl_sync(0xffffffffu, w0, k & 31);
    const int32_t v1 = __shfl_sync(0xffffffffu, w1, k & 31);
    const int32_t page = k < 32 ? v0 : v1;
    int row = -1;
    if (lane < nbox && pos < kv_end) {
      if (pidx >= s.np)
        report(a.err_word, PKV_DEVERR_LENGTH);
      else if (page < 0 || page >= a.num_pages)
        report(a.err_word, PKV_DEVERR_PAGE_OOB);
      else
        row = page * a.page_size + (pos - pidx * a.page_size);
    }
    const uint32_t nload = __popc(__ballot_sync(0xffffffffu, row >= 0));
    const int st = t & 1;
    if (!__all_sync(0xffffffffu, mbar_wait(&empties[st], ((t >> 1) & 1) ^ 1))) {
      drain(fulls, t);
      return false;
    }
    if (lane == 0) mbar_arrive_expect_tx(&fulls[st], nload * R * 128 * C::kHalves);
    __syncwarp();
    if (row >= 0) {
#pragma unroll
      for (int hf = 0; hf < C::kHalves; ++hf)
        tma_load_3d(base + st * C::kKVStage + hf * kKVHalf + lane * R * 128, tm, hf * 64, s.h, row, &fulls[st]);
    }
    __syncwarp();
  }
  return true;
}

// Page sizes that are not a power of two of at least 8: a lane gathers four rows at a time (tile::gather4), one
// copy per 64-dim half, their pages loaded a tile ahead.  Positions behind the end repeat the last
// one and a bad page's (reported) read the pool's row 0: neither is seen by a row whose result means
// anything.
template <int D>
__device__ bool tree_load_rows(const TreeArgs& a, Ctl* ctl, uint32_t sb, const Seg& s, uint32_t t, bool v) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  const int kv_end = s.P + s.T;
  uint64_t* fulls = v ? ctl->v_full : ctl->k_full;
  uint64_t* empties = v ? ctl->v_empty : ctl->k_empty;
  const CUtensorMap* tm = v ? &a.tm_v : &a.tm_k;
  const uint32_t base = sb + (v ? C::kOffV : C::kOffK);
  const int quad = lane & 15, half = lane >> 4;  // four rows, and their 64-dim half (D 64: lanes 0..15)
  int32_t page[4];
  uint32_t in_page[4];
  bool listed[4];
  auto load_pages = [&](int j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t pidx;
      a.page_div.divmod((uint32_t)min(j * kBN + 4 * quad + i, kv_end - 1), pidx, in_page[i]);
      listed[i] = (int)pidx < s.np;
      page[i] = listed[i] ? ld(a.kv_indices + s.p0 + pidx) : 0;
    }
  };
  load_pages(s.j0);
  for (int j = s.j0; j < s.j0 + s.n; ++j, ++t) {
    int row[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = page[i] >= 0 && page[i] < a.num_pages;
      if (!listed[i] || !in) report(a.err_word, !listed[i] ? PKV_DEVERR_LENGTH : PKV_DEVERR_PAGE_OOB);
      row[i] = listed[i] && in ? page[i] * a.page_size + (int)in_page[i] : 0;
    }
    if (j + 1 < s.j0 + s.n) load_pages(j + 1);
    const int st = t & 1;
    if (!__all_sync(0xffffffffu, mbar_wait(&empties[st], ((t >> 1) & 1) ^ 1))) {
      drain(fulls, t);
      return false;
    }
    if (lane == 0) mbar_arrive_expect_tx(&fulls[st], C::kKVStage);
    __syncwarp();
    if (half < C::kHalves)
      tma_gather4(base + st * C::kKVStage + half * kKVHalf + quad * 512, tm, s.h * D + half * 64, row[0], row[1], row[2],
                  row[3], &fulls[st]);
    __syncwarp();
  }
  return true;
}

// ---------------------------------------------------------------------------------------------
// MMA issuers: one thread each.
// ---------------------------------------------------------------------------------------------
template <int D>
__device__ bool tree_mma_qk(Ctl* ctl, uint32_t sb, uint32_t tmem, const Seg& s, uint32_t seg, uint32_t t) {
  using C = Cfg<D>;
  constexpr uint32_t idesc = umma_idesc_bf16(kBM, kBN, false);
  const uint64_t qdesc = smem_desc_sw128(sb + C::kOffQ, 16, 1024);
  const uint64_t kdesc0 = smem_desc_sw128(sb + C::kOffK, 16, 1024);
  if (!mbar_wait(&ctl->q_full, seg & 1)) return false;
  for (int j = 0; j < s.n; ++j, ++t) {
    const int st = t & 1;
    const uint32_t ph = (t >> 1) & 1;
    if (!mbar_wait(&ctl->k_full[st], ph)) return false;
    if (!mbar_wait(&ctl->s_free[st], ph ^ 1)) return false;
    tc_fence_after();
    const uint64_t kdesc = kdesc0 + ((st * C::kKVStage) >> 4);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const uint32_t qoff = ((ks >> 2) * kQHalf + (ks & 3) * 32) >> 4;
      const uint32_t koff = ((ks >> 2) * kKVHalf + (ks & 3) * 32) >> 4;
      umma_ss(tmem + st * 64, qdesc + qoff, kdesc + koff, idesc, ks > 0);
    }
    umma_commit(&ctl->s_full[st]);
    umma_commit(&ctl->k_empty[st]);
  }
  return true;
}

template <int D>
__device__ bool tree_mma_pv(Ctl* ctl, uint32_t sb, uint32_t tmem, const Seg& s, uint32_t t) {
  using C = Cfg<D>;
  constexpr uint32_t idesc = umma_idesc_bf16(kBM, D, true);
  const uint64_t vdesc0 = smem_desc_sw128(sb + C::kOffV, kKVHalf, 1024);
  for (int j = 0; j < s.n; ++j, ++t) {
    const int st = t & 1;
    const uint32_t ph = (t >> 1) & 1;
    if (!mbar_wait(&ctl->p_full[st], ph)) return false;
    if (!mbar_wait(&ctl->v_full[st], ph)) return false;
    tc_fence_after();
    const uint64_t vdesc = vdesc0 + ((st * C::kKVStage) >> 4);
#pragma unroll
    for (int ks = 0; ks < kBN / 16; ++ks) {
      const uint32_t pa = tmem + st * 64 + (ks >> 1) * 32 + (ks & 1) * 8;
      umma_ts(tmem + kColO, pa, vdesc + ((ks * 2048) >> 4), idesc, j > 0 || ks > 0);
    }
    umma_commit(&ctl->v_empty[st]);
    umma_commit(&ctl->s_free[st]);  // P consumed; also marks this PV done
  }
  return true;
}

// A row's mask words: the first four in registers (loaded before they are needed), others from memory.
struct MaskRow {
  const uint32_t* m;  // nullptr: an unused row
  int32_t words;
  uint32_t w[4];
};

PKV_DEV void load_mask(MaskRow& k) {
#pragma unroll
  for (int i = 0; i < 4; ++i) k.w[i] = k.m && i < k.words ? ld(k.m + i) : 0u;
}

// Which of the 32 positions of drafted-token offsets t0 .. t0 + 31 (t0 may be negative: the prefix)
// the row sees, T drafted tokens in all.
PKV_DEV uint32_t visible(const MaskRow& k, int T, int t0) {
  if (t0 <= -32) return 0xffffffffu;
  if (t0 >= T) return 0u;
  auto word = [&](int i) -> uint32_t {
    if (i < 0) return 0xffffffffu;
    if (i < 4) return i < 2 ? (i == 0 ? k.w[0] : k.w[1]) : (i == 2 ? k.w[2] : k.w[3]);
    return k.m && i < k.words ? ld(k.m + i) : 0u;
  };
  const int w = t0 >> 5, sh = t0 & 31;
  uint32_t v = __funnelshift_r(word(w), sh ? word(w + 1) : 0u, sh);
  if (T - t0 < 32) v &= (1u << (T - t0)) - 1u;
  return v;
}

// A pair of bf16 values with the non-finite ones replaced by 0.
PKV_DEV uint32_t finite_bf16x2(uint32_t u) {
  if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
  if ((u & 0x7f800000u) == 0x7f800000u) u &= 0x0000ffffu;
  return u;
}
// Non-zero where a pair holds an infinity or a NaN: an exponent of ones carries into the sign's place.
PKV_DEV uint32_t nonfinite_bits(uint32_t u) { return ((u & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }


// What no weight may touch in a tile of V becomes zeros: the rows behind the last position, and the
// infinities and NaNs of drafted tokens, which are noted.  By the four softmax warps, a thread per 64-dim
// half of a row; the prefix's rows are left alone.
template <int D>
__device__ void clean_v(uint8_t* vtile, Ctl* ctl, const Seg& s, int pos0, int tid) {
  using C = Cfg<D>;
  const int row = tid & (kBN - 1), half = tid / kBN;
  const int t = pos0 + row - s.P;
  if (half < C::kHalves && t >= 0) {
    uint8_t* at = vtile + half * kKVHalf + row * 128;
    auto chunk = [&](int i) { return reinterpret_cast<uint4*>(at + (((i + row) & 7) << 4)); };  // spread over the banks
    if (t >= s.T) {
#pragma unroll
      for (int i = 0; i < 8; ++i) *chunk(i) = make_uint4(0u, 0u, 0u, 0u);
    } else {
      uint32_t bad = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 u = *chunk(i);
        bad |= nonfinite_bits(u.x) | nonfinite_bits(u.y) | nonfinite_bits(u.z) | nonfinite_bits(u.w);
      }
      if (bad) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const uint4 u = *chunk(i);
          *chunk(i) = make_uint4(finite_bf16x2(u.x), finite_bf16x2(u.y), finite_bf16x2(u.z), finite_bf16x2(u.w));
        }
        atomicOr(&ctl->bad[t >> 5], 1u << (t & 31));
        ctl->bad_any = 1u;
      }
    }
  }
  fence_proxy_async_smem();  // before the MMA reads the tile
}

PKV_DEV float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
PKV_DEV float max32(const float (&v)[32]) {
  float a[11];
#pragma unroll
  for (int i = 0; i < 10; ++i) a[i] = max3f(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
  a[10] = fmaxf(v[30], v[31]);
  return fmaxf(max3f(max3f(a[0], a[1], a[2]), max3f(a[3], a[4], a[5]), max3f(a[6], a[7], a[8])), fmaxf(a[9], a[10]));
}

// Packed pairs of fp32.
PKV_DEV uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
PKV_DEV void split_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
PKV_DEV uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
PKV_DEV uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// acc + (float)(low or high bf16 half of v), one rounding
PKV_DEV float add_bf16_lo(uint32_t v, float acc) {
  float r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tadd.rn.f32.bf16 %0, lo, %2;\n\t}" : "=f"(r) : "r"(v), "f"(acc));
  return r;
}
PKV_DEV float add_bf16_hi(uint32_t v, float acc) {
  float r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tadd.rn.f32.bf16 %0, hi, %2;\n\t}" : "=f"(r) : "r"(v), "f"(acc));
  return r;
}

// A thread owns a row of the tile.
template <int D>
__device__ bool tree_softmax(const TreeArgs& a, uint8_t* smem, Ctl* ctl, uint32_t tmem, const Seg& s, uint32_t t) {
  using C = Cfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wq = warp & 3;       // TMEM lane quadrant this warp may access
  const int r = wq * 32 + lane;  // tile row == TMEM lane
  const int tid = (warp - 2) * 32 + lane;
  const uint32_t taddr = tmem + ((uint32_t)(wq * 32) << 16);
  const int G = a.group;
  const int rt = r / G, g = r - rt * G;  // token of the tile, head of the group
  const int tok = s.t0 + rt;
  const bool valid = rt < a.tpt && tok < s.T;
  const bool warp_live = __any_sync(0xffffffffu, valid);
  const bool pos_scale = a.scale_log2 > 0.f;
  const float sc = pos_scale ? a.scale_log2 : 1.f;
  MaskRow mask{valid ? a.mask + (int64_t)(s.q0 + tok) * a.words : nullptr, a.words, {0u, 0u, 0u, 0u}};
  if ((s.j0 + s.n) * kBN > s.P) load_mask(mask);
  float m_used = -INFINITY;  // running max of the scaled (log2) scores
  float l = 0.f;             // sum of the weights (for the LSE)
  float lr = 0.f;            // ... as rounded to bf16 for the PV MMA (for O: a rounding that they share cancels)

  for (int j = 0; j < s.n; ++j, ++t) {
    const int st = t & 1;
    const uint32_t ph = (t >> 1) & 1;
    const int pos0 = (s.j0 + j) * kBN;
    const bool special = pos0 + kBN > s.P;
    if (!__all_sync(0xffffffffu, mbar_wait(&ctl->s_full[st], ph))) return false;
    tc_fence_after();
    if (warp_live) {
      float s0[32], s1[32];  // the row's scores, positions [0, 32) and [32, 64) of the tile
      uint32_t see0 = 0xffffffffu, see1 = 0xffffffffu;
      if (special) {
        see0 = visible(mask, s.T, pos0 - s.P);
        see1 = visible(mask, s.T, pos0 + 32 - s.P);
      }
      __syncwarp();
      tmem_fetch32(taddr + st * 64, s0);
      tmem_fetch32(taddr + st * 64 + 32, s1);
      tmem_wait_ld32(s0);
      tmem_wait_ld32(s1);
      if (!pos_scale) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          s0[c] *= a.scale_log2;
          s1[c] *= a.scale_log2;
        }
      }
      if (special) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          s0[c] = (see0 >> c) & 1u ? s0[c] : -INFINITY;
          s1[c] = (see1 >> c) & 1u ? s1[c] : -INFINITY;
        }
      }
      const float m_new = fmaxf(m_used, fmaxf(max32(s0), max32(s1)) * sc);
      // the maximum moves only when it grows by more than 2^8, so that O is seldom rescaled
      const bool resc = m_new > m_used + 8.f;
      const float m_ref = resc ? m_new : m_used;
      const float corr = resc ? ex2(m_used - m_ref) : 1.f;
      const float neg = m_ref == -INFINITY ? 0.f : -m_ref;  // nothing seen so far: every weight is 0
      const uint64_t sc2 = f32x2(sc, sc), nm2 = f32x2(neg, neg);
      float tot = 0.f, rtot = 0.f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float(&sv)[32] = hf ? s1 : s0;
        uint32_t pk[16];
        uint64_t acc_a = f32x2(0.f, 0.f), acc_b = f32x2(0.f, 0.f);
        float rs0 = 0.f, rs1 = 0.f, rs2 = 0.f, rs3 = 0.f;
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          float x0, x1, x2, x3;
          split_f32x2(fma_f32x2(f32x2(sv[2 * c], sv[2 * c + 1]), sc2, nm2), x0, x1);
          split_f32x2(fma_f32x2(f32x2(sv[2 * c + 2], sv[2 * c + 3]), sc2, nm2), x2, x3);
          const float p0 = ex2(x0), p1 = ex2(x1), p2 = ex2(x2), p3 = ex2(x3);
          acc_a = add_f32x2(acc_a, f32x2(p0, p1));
          acc_b = add_f32x2(acc_b, f32x2(p2, p3));
          pk[c] = pack_bf16x2(p0, p1);
          pk[c + 1] = pack_bf16x2(p2, p3);
          rs0 = add_bf16_lo(pk[c], rs0);
          rs1 = add_bf16_hi(pk[c], rs1);
          rs2 = add_bf16_lo(pk[c + 1], rs2);
          rs3 = add_bf16_hi(pk[c + 1], rs3);
        }
        float e0, e1;
        split_f32x2(add_f32x2(acc_a, acc_b), e0, e1);
        tot += e0 + e1;
        rtot += (rs0 + rs1) + (rs2 + rs3);
        // P (bf16 pairs) over the first 16 columns of each 32-column half of the S buffer
        tmem_st16(taddr + st * 64 + hf * 32, pk);
      }
      l = l * corr + tot;
      lr = lr * corr + rtot;
      m_used = m_ref;
      if (j > 0 && __any_sync(0xffffffffu, resc)) {
        // O is rescaled only after the previous tile's PV is done
        if (!__all_sync(0xffffffffu, mbar_wait(&ctl->s_free[(t - 1) & 1], ((t - 1) >> 1) & 1))) return false;
        tc_fence_after();
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          float o[32];
          tmem_fetch32(taddr + kColO + ch * 32, o);
          tmem_wait_ld32(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= corr;
          tmem_st32(taddr + kColO + ch * 32, o);
        }
      }
      tmem_wait_st();
    }
    if (special) {
      if (!__all_sync(0xffffffffu, mbar_wait(&ctl->v_full[st], ph))) return false;
      clean_v<D>(smem + C::kOffV + st * C::kKVStage, ctl, s, pos0, tid);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->p_full[st]);
    __syncwarp();
  }
  // the last PV is done
  const uint32_t last = t - 1;
  if (!__all_sync(0xffffffffu, mbar_wait(&ctl->s_free[last & 1], (last >> 1) & 1))) return false;
  ctl->inv[r] = l == 0.f ? 0.f : 1.f / lr;  // (NaN among the scores: in every dim)
  if (valid) {
    const float lse_v = (m_used + log2f(l)) * kLn2;
    if (s.part >= 0)
      a.part_lse[(int64_t)s.part * kBM + r] = lse_v;
    else if (a.lse)
      a.lse[(int64_t)(s.q0 + tok) * a.num_q_heads + (int64_t)s.h * G + g] = lse_v;
  }
  return true;
}

// Adds the non-finite values of 32 dims from d0 on of the noted drafted tokens that the row sees to o.
template <int D>
PKV_DEV void add_nonfinite(const TreeArgs& a, const Ctl* ctl, const Seg& s, const uint32_t* m, int d0, float (&o)[32]) {
  for (int w = 0; w < (s.T + 31) / 32; ++w) {
    uint32_t hit = ctl->bad[w] & (w < a.words ? ld(m + w) : 0u);
    while (hit) {
      const int t = 32 * w + __ffs(hit) - 1;
      hit &= hit - 1;
      const int pos = s.P + t, pidx = pos / a.page_size;
      if (pidx >= s.np) continue;
      const int32_t page = ld(a.kv_indices + s.p0 + pidx);
      if (page < 0 || page >= a.num_pages) continue;
      const __nv_bfloat16* src =
          a.v_pool + (((int64_t)page * a.page_size + pos % a.page_size) * a.num_kv_heads + s.h) * D + d0;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float x = __bfloat162float(src[i]);
        if (!(fabsf(x) < INFINITY)) o[i] += x;
      }
    }
  }
}

// Epilogue, by all eight warps: warp w reads TMEM lane quadrant w % 4, the softmax warps the first 64
// dims of their rows, the others the second 64 (D 64: the softmax warps alone).  A whole unit's rows are
// staged over the Q buffer and leave by coalesced 16-byte stores; a part's go to scratch in fp32.
template <int D>
__device__ void tree_epilogue(const TreeArgs& a, uint8_t* smem, Ctl* ctl, uint32_t tmem, const Seg& s) {
  using C = Cfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wq = warp & 3;
  const int r = wq * 32 + lane;
  const bool softmax_warp = warp >= 2 && warp < 2 + kSoftmaxWarps;
  const int G = a.group;
  const int rt = r / G, tok = s.t0 + rt;
  const bool valid = rt < a.tpt && tok < s.T;
  uint8_t* stage = smem + C::kOffQ;
  tc_fence_after();
  if ((softmax_warp || C::kHalves == 2) && __any_sync(0xffffffffu, valid)) {
    const int hf = softmax_warp ? 0 : 1;
    const float inv = ctl->inv[r];
    const bool any_bad = ctl->bad_any != 0u;
#pragma unroll 1
    for (int ch = 0; ch < 2; ++ch) {
      float o[32];
      __syncwarp();
      tmem_fetch32(tmem + ((uint32_t)(wq * 32) << 16) + kColO + hf * 64 + ch * 32, o);
      tmem_wait_ld32(o);
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = inv == 0.f ? 0.f : o[e] * inv;
      if (any_bad && valid) add_nonfinite<D>(a, ctl, s, a.mask + (int64_t)(s.q0 + tok) * a.words, hf * 64 + ch * 32, o);
      if (s.part < 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(stage + hf * kQHalf + r * 128 + (((ch * 4 + q) ^ (r & 7)) << 4)) =
              make_uint4(pack_bf16x2(o[8 * q], o[8 * q + 1]), pack_bf16x2(o[8 * q + 2], o[8 * q + 3]),
                         pack_bf16x2(o[8 * q + 4], o[8 * q + 5]), pack_bf16x2(o[8 * q + 6], o[8 * q + 7]));
      } else if (valid) {
        float4* dst = reinterpret_cast<float4*>(a.part_o) + ((int64_t)s.part * (D / 4) + hf * 16 + ch * 8) * kBM + r;
#pragma unroll
        for (int q = 0; q < 8; ++q) dst[q * kBM] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      }
    }
  }
  if (s.part < 0) {
    __syncthreads();
    constexpr int kCh = D / 8;  // 16-byte chunks of a row
    const int rows = min(a.tpt, s.T - s.t0) * G;
    for (int i = threadIdx.x; i < rows * kCh; i += kThreads) {
      const int row = i / kCh, c = i % kCh;
      const int tr = row / G;
      const int64_t orow = (int64_t)(s.q0 + s.t0 + tr) * a.num_q_heads + (int64_t)s.h * G + (row - tr * G);
      reinterpret_cast<uint4*>(a.out + orow * D)[c] = *reinterpret_cast<const uint4*>(
          stage + (c >> 3) * kQHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4));
    }
  }
  fence_proxy_async_smem();  // the staged rows, before the next Q lands on them
}

template <int D, bool kRows>
__global__ void __launch_bounds__(kThreads, 2) paged_tree_kernel(const __grid_constant__ TreeArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  if (sb & 1023u) {  // the swizzled layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) {
      pdl_wait();
      report(a.err_word, PKV_DEVERR_INTERNAL);
      a.cut[blockIdx.x] = Cut{};
    }
    return;
  }
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::kOffCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 64) {
    mbar_init(&ctl->q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->k_full[i], 1);
      mbar_init(&ctl->k_empty[i], 1);
      mbar_init(&ctl->v_full[i], 1);
      mbar_init(&ctl->v_empty[i], 1);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->s_free[i], 1);
      mbar_init(&ctl->p_full[i], kSoftmaxWarps);
    }
    mbar_init(&ctl->qk_done, 1);
    mbar_init(&ctl->pv_done, 1);
    ctl->failed = 0u;
    ctl->bad_any = 0u;
    for (int i = 0; i < kMaxNodes / 32; ++i) ctl->bad[i] = 0u;
    fence_mbar_init();
    prefetch_tmap(&a.tm_q);
    prefetch_tmap(&a.tm_k);
    prefetch_tmap(&a.tm_v);
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  Walk walk;
  if (warp == 0) {
    walk_start(a, walk);
    const Seg s = walk_next(a, walk);
    if (lane == 0) ctl->seg = s;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  uint32_t tiles = 0;  // of this CTA so far
  for (uint32_t i = 0;; ++i) {
    const Seg s = ctl->seg;
    if (s.n == 0) break;
    bool ok = true;
    if (threadIdx.x == 0) {
      // [64 dims x G heads x tokens] boxes; rows behind the request's are read along and not used
      mbar_arrive_expect_tx(&ctl->q_full, C::kHalves * a.tpt * a.group * 128);
#pragma unroll
      for (int hf = 0; hf < C::kHalves; ++hf)
        tma_load_3d(sb + C::kOffQ + hf * kQHalf, &a.tm_q, hf * 64, s.h * a.group, s.q0 + s.t0, &ctl->q_full);
    }
    __syncwarp();
    if (warp == 0 || warp == kVWarp) {
      ok = kRows ? tree_load_rows<D>(a, ctl, sb, s, tiles, warp == kVWarp) : tree_load_boxes<D>(a, ctl, sb, s, tiles, warp == kVWarp);
      if (!ok && warp == 0) mbar_wait(&ctl->q_full, i & 1);
    } else if (warp == 1) {
      if (lane == 0) ok = tree_mma_qk<D>(ctl, sb, tmem, s, i, tiles);
      __syncwarp();
    } else if (warp == kPVWarp) {
      if (lane == 0) ok = tree_mma_pv<D>(ctl, sb, tmem, s, tiles);
      __syncwarp();
    } else {
      ok = tree_softmax<D>(a, smem, ctl, tmem, s, tiles);
    }
    if (!ok) {
      report(a.err_word, PKV_DEVERR_TIMEOUT);
      ctl->failed = 1u;
    }
    tc_fence_before();
    __syncthreads();  // every warp is done with the segment; O is complete unless a wait gave up
    if (ctl->failed) {  // no copy is left in flight (bounded waits)
      if (warp == 0) drain(ctl->k_full, tiles + s.n);
      if (warp == kVWarp) drain(ctl->v_full, tiles + s.n);
      break;
    }
    tree_epilogue<D>(a, smem, ctl, tmem, s);
    tiles += s.n;
    Seg next{};
    if (warp == 0) next = walk_next(a, walk);
    tc_fence_before();
    __syncthreads();  // the epilogue has read O, the notes and the staged rows
    tc_fence_after();
    if (warp == 0) {
      if (ctl->bad_any) {
        ctl->bad[lane] = 0u;
        __syncwarp();
        if (lane == 0) ctl->bad_any = 0u;
      }
      if (lane == 0) ctl->seg = next;
    }
    __syncthreads();
  }
  if (warp == 0) {
    if (lane == 0) a.cut[blockIdx.x] = walk.cut;
    pdl_trigger();
  }
  // every MMA has completed before TMEM is released (immediate on the normal path)
  if (warp == 1 || warp == kPVWarp) {
    if (lane == 0) {
      uint64_t* done = warp == 1 ? &ctl->qk_done : &ctl->pv_done;
      umma_commit(done);
      if (!mbar_wait(done, 0)) report(a.err_word, PKV_DEVERR_TIMEOUT);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------------------------
// Merge: block (c, y) joins rows 32 y .. 32 y + 31 of the unit that CTA c began and did not finish.  A
// lane is a row, a warp every eighth group of four dims, so a part's rows are read as whole lines; the
// states are joined in one pass with a running maximum, the loads of four parts in flight.  5 us after
// 64 requests of up to 16 tokens, about 9 after 4 of 64 (23 MB of states, which L2 holds).
// ---------------------------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int kGroups = D / 32;  // groups of four dims of a thread
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x;
  const Cut cut = a.cut[c];
  if (cut.parts <= 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int prow = blockIdx.y * 32 + lane;
  const int tok = cut.t0 + prow / a.group;
  if (prow >= a.group * a.tpt || tok >= cut.T) return;
  auto slot = [&](int p) -> int64_t { return (int64_t)2 * (c + (p << a.paired)) + (p == 0 ? 1 : 0); };
  float mx = -INFINITY, tot = 0.f;
  float acc[kGroups][4] = {};
  for (int p0 = 0; p0 < cut.parts; p0 += 4) {
    float pl[4];
    float4 x[4][kGroups];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool on = p0 + k < cut.parts;
      const int64_t at = slot(on ? p0 + k : p0);
      pl[k] = on ? ld(a.part_lse + at * kBM + prow) : -INFINITY;
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        x[k][i] = ld(reinterpret_cast<const float4*>(a.part_o) + (at * (D / 4) + warp + 8 * i) * kBM + prow);
    }
    const float mn = fmaxf(fmaxf(fmaxf(pl[0], pl[1]), fmaxf(pl[2], pl[3])), mx);
    if (mn > mx) {  // (not while every part so far is empty)
      const float corr = __expf(mx - mn);
      tot *= corr;
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][v] *= corr;
      mx = mn;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (pl[k] == -INFINITY) continue;  // an empty part, or none
      const float w = __expf(pl[k] - mx);
      tot += w;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        acc[i][0] = fmaf(w, x[k][i].x, acc[i][0]);
        acc[i][1] = fmaf(w, x[k][i].y, acc[i][1]);
        acc[i][2] = fmaf(w, x[k][i].z, acc[i][2]);
        acc[i][3] = fmaf(w, x[k][i].w, acc[i][3]);
      }
    }
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  const int64_t orow = (int64_t)(cut.q0 + tok) * a.num_q_heads + (int64_t)cut.h * a.group + prow % a.group;
#pragma unroll
  for (int i = 0; i < kGroups; ++i)
    *reinterpret_cast<uint2*>(a.out + orow * D + (warp + 8 * i) * 4) =
        make_uint2(pack_bf16x2(acc[i][0] * inv, acc[i][1] * inv), pack_bf16x2(acc[i][2] * inv, acc[i][3] * inv));
  if (warp == 0 && a.lse) a.lse[orow] = tot == 0.f ? -INFINITY : mx + logf(tot);
}

// ---------------------------------------------------------------------------------------------
// The mask of a tree given by parents: row i has the bits of i and its ancestors.
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(128) tree_mask_kernel(const int32_t* parents, const int32_t* qo_indptr,
                                                        int32_t num_tokens, int32_t max_nodes, int32_t words,
                                                        uint32_t* mask, uint32_t* err_word) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y;
  const int32_t q0 = ld(qo_indptr + b), rows = ld(qo_indptr + b + 1) - q0;
  const bool first = blockIdx.x == 0 && threadIdx.x == 0;
  if (rows < 0 || rows > max_nodes) {
    if (first) report(err_word, PKV_DEVERR_LENGTH);
    if (rows < 0) return;
  }
  if (q0 < 0 || q0 > num_tokens - rows) {
    if (first) report(err_word, PKV_DEVERR_ROW_OOB);
    return;
  }
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= rows || t >= max_nodes) return;
  uint32_t* row = mask + (int64_t)(q0 + t) * words;
  int cur = t;  // strictly falling, so the walk ends
  for (int w = words - 1; w >= 0; --w) {
    uint32_t bits = 0;
    while (cur >= 0 && (cur >> 5) == w) {
      bits |= 1u << (cur & 31);
      const int p = ld(parents + q0 + cur);
      if (p >= cur) {  // a parent comes before its children
        report(err_word, PKV_DEVERR_LENGTH);
        cur = -1;
      } else {
        cur = p;
      }
    }
    row[w] = bits;
  }
}

// ---------------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------------
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Plan {
  int G, tpt, ncta;
  size_t off_lse, off_o, ws_bytes;
};

bool make_plan(int B, int Hq, int Hkv, int D, int max_nodes, int sms, Plan& p) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || max_nodes < 0 || max_nodes > kMaxNodes) return false;
  if (D != 64 && D != 128) return false;
  p.G = Hq / Hkv;
  if (p.G > 16) return false;
  p.tpt = kBM / p.G;
  p.ncta = 2 * sms;  // two per SM
  p.off_lse = align256((size_t)p.ncta * sizeof(Cut));
  p.off_o = align256(p.off_lse + (size_t)2 * p.ncta * kBM * 4);
  p.ws_bytes = align256(p.off_o + (size_t)2 * p.ncta * kBM * D * 4);
  return true;
}

template <int D, bool kRows>
pkv_status launch(const Plan& p, const TreeArgs& a, cudaStream_t st) {
  auto kern = paged_tree_kernel<D, kRows>;
  constexpr uint32_t smem = Cfg<D>::kOffCtl + sizeof(Ctl);
  static std::atomic<bool> configured[64];
  const int dev = pkv_host::current_device();
  if (dev < 0) return PKV_ERR_CUDA;
  if (dev >= 64 || !configured[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
      return PKV_ERR_CUDA;
    if (dev < 64) configured[dev].store(true, std::memory_order_relaxed);
  }
  const pkv_status s = pkv_host::launch_after(kern, dim3(p.ncta), kThreads, smem, st, a);
  if (s != PKV_OK) return s;
  return pkv_host::launch_after(tree_merge_kernel<D>, dim3((unsigned)p.ncta, kBM / 32), 256, 0, st, a);
}

}  // namespace

extern "C" {

size_t pkv_tree_workspace_size(int32_t batch_size, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                               int32_t max_tree_len) {
  Plan p;
  const int n = pkv_host::sm_count();
  if (n <= 0 || !make_plan(batch_size, num_q_heads, num_kv_heads, head_dim, max_tree_len, n, p)) return 0;
  return p.ws_bytes;
}

pkv_status pkv_paged_tree_attention(const pkv_pool* pool, const void* q, int32_t num_q_tokens,
                                    const int32_t* qo_indptr, int32_t batch_size, int32_t num_q_heads,
                                    const int32_t* kv_indptr, const int32_t* kv_indices,
                                    const int32_t* prefix_lens, const void* tree_mask, int32_t mask_words,
                                    int32_t max_tree_len, float sm_scale, void* out, float* lse,
                                    void* workspace, size_t workspace_bytes, uint32_t* err_word,
                                    void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_paged_tree_attention");
  if (!pkv_host::valid_pool(pool) || batch_size < 0 || num_q_heads <= 0 || num_q_tokens < 0 || max_tree_len < 0 ||
      mask_words < 0 || (int64_t)mask_words * 32 < max_tree_len)
    return PKV_ERR_INVALID_ARG;
  if (batch_size == 0 || num_q_tokens == 0 || max_tree_len == 0) return PKV_OK;
  if (!q || !qo_indptr || !kv_indptr || !kv_indices || !prefix_lens || !tree_mask || !out) return PKV_ERR_INVALID_ARG;
  if (!pkv_host::aligned16(q) || !pkv_host::aligned16(out)) return PKV_ERR_INVALID_ARG;
  if (num_q_heads % pool->num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  if (pool->num_pages * (int64_t)pool->page_size > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  const int D = pool->head_dim;
  const int sms = pkv_host::sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  Plan p;
  if (!make_plan(batch_size, num_q_heads, pool->num_kv_heads, D, max_tree_len, sms, p)) return PKV_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < p.ws_bytes) return PKV_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PKV_ERR_INVALID_ARG;

  TreeArgs a;
  const int ps = pool->page_size;
  const bool rows_path = ps < 8 || (ps & (ps - 1)) != 0;
  const uint64_t Hq = num_q_heads, Hkv = pool->num_kv_heads;
  const uint64_t rows = (uint64_t)pool->num_pages * ps;
  const uint64_t Db = (uint64_t)D * 2;
  a.box_rows = rows_path ? 8 : (ps < kBN ? ps : kBN);
  a.tpt = p.tpt;
  a.paired = max_tree_len > p.tpt ? 1 : 0;
  if (!pkv_host::encode_tmap_3d(&a.tm_q, q, D, Hq, (uint64_t)num_q_tokens, Db, Hq * Db, 64, p.G, a.tpt) ||
      !(rows_path ? pkv_host::encode_tmap_rows(&a.tm_k, pool->k, Hkv * D, rows, D) &&
                        pkv_host::encode_tmap_rows(&a.tm_v, pool->v, Hkv * D, rows, D)
                  : pkv_host::encode_tmap_head(&a.tm_k, pool->k, D, Hkv, rows, a.box_rows) &&
                        pkv_host::encode_tmap_head(&a.tm_v, pool->v, D, Hkv, rows, a.box_rows)))
    return PKV_ERR_CUDA;
  a.qo_indptr = qo_indptr;
  a.kv_indptr = kv_indptr;
  a.kv_indices = kv_indices;
  a.prefix_lens = prefix_lens;
  a.mask = (const uint32_t*)tree_mask;
  a.words = mask_words;
  a.v_pool = (const __nv_bfloat16*)pool->v;
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  a.err_word = err_word;
  a.num_pages = pool->num_pages;
  a.page_size = ps;
  a.page_div = FastDiv((uint32_t)ps);
  a.num_kv_heads = pool->num_kv_heads;
  a.num_q_heads = num_q_heads;
  a.group = p.G;
  a.batch = batch_size;
  a.num_q_tokens = num_q_tokens;
  a.max_nodes = max_tree_len;
  a.scale_log2 = sm_scale * kLog2e;
  uint8_t* ws = (uint8_t*)workspace;
  a.cut = (Cut*)ws;
  a.part_lse = (float*)(ws + p.off_lse);
  a.part_o = (float*)(ws + p.off_o);
  cudaStream_t st = (cudaStream_t)stream;
  if (rows_path) return D == 128 ? launch<128, true>(p, a, st) : launch<64, true>(p, a, st);
  return D == 128 ? launch<128, false>(p, a, st) : launch<64, false>(p, a, st);
}

pkv_status pkv_tree_mask_from_parents(const int32_t* parents, const int32_t* qo_indptr, int32_t batch_size,
                                      int32_t num_tokens, int32_t max_tree_len, int32_t mask_words,
                                      void* tree_mask, uint32_t* err_word, void* stream) {
  pkv_host::NvtxRange nvtx_range("pkv_tree_mask_from_parents");
  if (batch_size < 0 || num_tokens < 0 || max_tree_len < 0 || mask_words < 0 ||
      (int64_t)mask_words * 32 < max_tree_len)
    return PKV_ERR_INVALID_ARG;
  if (batch_size == 0 || num_tokens == 0 || max_tree_len == 0) return PKV_OK;
  if (!parents || !qo_indptr || !tree_mask) return PKV_ERR_INVALID_ARG;
  if (batch_size > 65535 || max_tree_len > kMaxNodes) return PKV_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)((max_tree_len + 127) / 128), (unsigned)batch_size, 1);
  return pkv_host::launch_after(tree_mask_kernel, grid, 128, 0, (cudaStream_t)stream, parents, qo_indptr, num_tokens,
                                max_tree_len, mask_words, (uint32_t*)tree_mask, err_word);
}

}  // extern "C"
