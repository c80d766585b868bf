// Attention of a tree of drafted tokens over a paged cache (speculative verification).
//
// What it computes: request b's T_b drafted tokens sit behind its P_b cached positions, their K/V in
// the pool like an extend's; drafted token i sees every position j < P_b, and position P_b + t for
// each bit t of its mask row (its ancestors and itself, or whatever the caller allows).  GQA, page
// lists and LSE as in the other attention calls; a row that sees nothing gives 0 and -inf.
//
// A few query rows over a long cache: bound by reading K and V once.  What the shape asks for:
//  * One persistent CTA per SM over an equal share of the stream of 128-position KV tiles of all
//    (request, KV head) units, so that one tree over a long context fills the GPU as well as many
//    trees do.  A unit cut by a share's border leaves partial states, merged by log-sum-exp in a
//    programmatic dependent launch.
//  * The rows of a unit are (token, group head) pairs, up to two 128-row Q tiles.  S = Q K^T and
//    O += P V run as tcgen05.mma (M 128, N 128), accumulators in TMEM: two slots, each an S buffer of
//    128 columns (P, bf16, is written over it) and an O of 128.  With two Q tiles a slot is a Q
//    tile and each K/V tile in shared memory serves both; with one Q tile the slots take alternate
//    KV tiles, so that one slot's softmax runs beside the other's MMAs, and their states are joined
//    when the segment ends.
//  * A thread owns a row, and a warp can read only its quarter of TMEM's lanes, so a unit of at most 32
//    (64) rows would leave three (two) of a slot's four softmax warps idle while the busy ones took
//    128 columns of every tile each, and that chain, not memory, would set the pace.  The rows are
//    therefore loaded four times (twice) into the tile, the MMA's rows being there anyway: each
//    copy takes 32 (64) of the tile's columns, writes zeros for P elsewhere, and ends up with a state
//    of its own; the copies' states are joined in the epilogue.
//  * Twelve warps: K producer (which also walks the stream and publishes the segments), QK issuer, PV
//    issuer, V and Q producer, and four softmax warps per slot, one thread per row.
//  * Only tiles that reach past the prefix are masked.  There the V rows behind the last position
//    and the infinities and NaNs of drafted tokens become 0 in shared memory (weight 0 times them
//    would be NaN for rows that do not see them); rows that do see them get them added when they are
//    written, which is what a sum with a non-zero weight would give.
// Measured with 32/8 heads of 128 at page size 16: 64 requests of 1 to 16 tokens over 512 to 4096 positions
// 111 us, 5.5 TB/s, 81 % of what a device copy reaches (bound by memory and by the ends of segments,
// about 3 us each); 4 requests of 64 tokens over 32700 positions 129 us, 1.06 PFLOP/s, 62 % of the bytes' floor
// and 56 % of the tensor cores' (bound by the chain of a slot: product, softmax, product, about 1.85 us a
// tile, of which the tensor cores work 1.33); one request of 8 tokens over 1000 positions 13 us, all latency.
#include <atomic>

#include "quant.cuh"
#include "tc05.cuh"

namespace {

using namespace pkv;

constexpr int kBM = 128;              // Q tile rows
constexpr int kBN = 128;              // KV positions per tile
constexpr int kThreads = 384;
constexpr int kSoftmaxWarp0 = 4;      // warps 4..7 slot 0, 8..11 slot 1
constexpr int kMaxNodes = 1024;       // drafted tokens of a request
constexpr int kSegRing = 4;
constexpr int kMaxRing = 9;
constexpr int kUnitCost = 3;          // a unit's start and epilogue, in KV tiles of the work split (1 to 4
                                      // tried: 64 requests of up to 16 tokens 118.9, 115.7, 114.7, 115.5 us)
constexpr uint32_t kHalfTile = 128 * 128;  // 128 rows of one 64-dim half, 16 KB
constexpr uint32_t kColO = 0, kColS = 256;  // O of slot s at 128 s, S at 256 + 128 s

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kTile = kHalves * kHalfTile;
  static constexpr uint32_t kOffQ = 0;
  // One ring for K and V tiles, K of tile j at place 2 j and V at 2 j + 1: a buffer that K's product
  // frees soon is the next V's, and the loads run 2.5 tiles ahead.  (Two K and three V buffers of their own
  // left K's reload little more than a tile's time.)
  static constexpr int kRing = D == 128 ? 5 : 9;
  static constexpr uint32_t kOffRing = kOffQ + 2 * kTile;
  // the epilogue's exchange between replicas, 2 slots x 3 x 32 rows x 32 dims fp32: at D 128 it is the
  // second Q buffer, which one Q tile leaves free
  static constexpr uint32_t kScratch = 2 * 3 * 32 * 32 * 4;
  static constexpr bool kShared = kTile >= kScratch;
  static constexpr uint32_t kOffScratch = kShared ? kOffQ + kTile : kOffRing + kRing * kTile;
  static constexpr uint32_t kOffCtl = kOffRing + kRing * kTile + (kShared ? 0 : kScratch);
};

// A run of KV tiles of one unit that this CTA computes.
struct Seg {
  int32_t q0;      // first row of the request in q and out
  int32_t T, P;    // drafted tokens (covered), cached positions
  int32_t p0, np;  // page list
  int32_t h;       // KV head
  int32_t t0;      // first token of the unit's first Q tile
  int32_t nq;      // Q tiles of the unit (1 or 2); 0: no more work
  int32_t j0, n;   // first KV tile, number of tiles
  int32_t part;    // partial state's slot, or -1: the segment is the whole unit
  int32_t rep;     // copies of the Q rows in the tile (1, 2 or 4)
};

struct Ctl {
  Seg seg[kSegRing];
  uint64_t seg_full[kSegRing], seg_empty[kSegRing];
  uint64_t q_full[2], q_empty[2];
  uint64_t full[kMaxRing], empty[kMaxRing];  // the K / V ring
  uint64_t s_full[2];  // QK written
  uint64_t qk_issued[2];
  uint64_t p_full[2];  // P written, V cleaned
  uint64_t s_free[2];  // PV done
  uint64_t o_free;     // O read by the epilogue
  uint64_t x_full, x_free;  // the slots' exchange of row states
  uint32_t epilogues;       // warps done with the scratch, counted over all segments
  uint64_t qk_done, pv_done;
  uint32_t tmem_base;
  uint32_t bad_any;
  uint32_t bad[kMaxNodes / 32];  // drafted tokens of this segment whose V is not finite
  float xm[2][kBM], xl[2][kBM];  // row maxima and sums of the slots
};
constexpr uint32_t kSmemLimit = 227 * 1024;
static_assert(kMaxNodes / 32 == 32, "a warp clears the notes");
static_assert(Cfg<128>::kOffCtl + sizeof(Ctl) <= kSmemLimit, "shared memory");

// The unit that a CTA's share ends in the middle of, for the merge: its parts are the slots
// 2c + 1, 2(c + 1), 2(c + 2), ...
struct Cut {
  int32_t parts;  // 0: none
  int32_t q0, T, t0, h, nq;
  int32_t pad[2];
};

struct TreeArgs {
  CUtensorMap tm_q[3];  // box of the tokens of 128, 64 and 32 rows
  CUtensorMap tm_k, tm_v;
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
  int32_t tpt;        // tokens per Q tile
  int32_t tpt2, tpt4; // ... of which 2 or 4 copies fit into the tile
  int32_t batch, num_q_tokens, max_nodes;
  float scale_log2;
  Cut* cut;           // [CTAs]
  float* part_o;      // [2 CTAs][D / 4][part_rows][4]: a warp's rows lie side by side
  float* part_lse;    // [2 CTAs][part_rows]
  int32_t part_rows;
};

// ---------------------------------------------------------------------------------------------
// Segment ring
// ---------------------------------------------------------------------------------------------
// Next segment for a whole warp (all lanes wait and read), then released by lane 0.  False: a wait gave up.
PKV_DEV bool next_seg(Ctl* ctl, int i, Seg& s) {
  const int r = i % kSegRing;
  if (!__all_sync(0xffffffffu, mbar_wait(&ctl->seg_full[r], (i / kSegRing) & 1))) return false;
  s = ctl->seg[r];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&ctl->seg_empty[r]);
  return true;
}

// ---------------------------------------------------------------------------------------------
// K / V producers
// ---------------------------------------------------------------------------------------------
// Copies the tiles of segments into the ring.  kRows: gathers of four rows, for page sizes that are not
// a power of two of at least 8; else TMA boxes of min(page_size, 128) rows.
template <int D, bool kRows>
struct Producer {
  using C = Cfg<D>;
  const TreeArgs& a;
  uint64_t* fulls;
  uint64_t* empties;
  const CUtensorMap* tm;
  uint32_t base;  // of the ring, shared address
  int item;       // place of the next tile in the ring's order: even K, odd V

  __device__ Producer(const TreeArgs& args, Ctl* ctl, uint32_t sb, bool v)
      : a(args), fulls(ctl->full), empties(ctl->empty), tm(v ? &args.tm_v : &args.tm_k),
        base(sb + C::kOffRing), item(v ? 1 : 0) {}

  // Waits until the next tile's buffer is free.
  __device__ bool acquire() {
    return __all_sync(0xffffffffu, mbar_wait(&empties[item % C::kRing], ((item / C::kRing) & 1) ^ 1)) != 0;
  }

  // Row of the pool that holds position pos, or -1 (reported).
  __device__ int64_t row_of(int pos, int32_t page, int np) {
    const int pidx = (int)a.page_div.quot((uint32_t)pos);
    if (pidx >= np) {
      report(a.err_word, PKV_DEVERR_LENGTH);
      return -1;
    }
    if (page < 0 || page >= a.num_pages) {
      report(a.err_word, PKV_DEVERR_PAGE_OOB);
      return -1;
    }
    return (int64_t)page * a.page_size + (pos - pidx * a.page_size);
  }

  __device__ bool run(const Seg& s) {
    return kRows ? run_rows(s) : run_boxes(s);
  }

  __device__ bool run_boxes(const Seg& s) {
    const int lane = threadIdx.x & 31;
    const int R = a.box_rows, nbox = kBN / R, kv_end = s.P + s.T;
    const int box = lane % nbox, half = lane / nbox;  // lane issues one half of one box
    auto entry = [&](int pidx) -> int32_t {
      return (pidx >= 0 && pidx < s.np) ? ld(a.kv_indices + s.p0 + pidx) : -1;
    };
    int wbase = (int)a.page_div.quot((uint32_t)(s.j0 * kBN));
    int32_t w0 = entry(wbase + lane), w1 = entry(wbase + 32 + lane);
    for (int j = s.j0; j < s.j0 + s.n; ++j) {
      while ((int)a.page_div.quot((uint32_t)(j * kBN)) >= wbase + 32) {  // the upper half was loaded 32 pages ago
        w0 = w1;
        wbase += 32;
        w1 = entry(wbase + 32 + lane);
      }
      const int pos = j * kBN + box * R;
      const int k = (int)a.page_div.quot((uint32_t)pos) - wbase;  // < 64: a tile spans at most 16 pages
      const int32_t v0 = __shfl_sync(0xffffffffu, w0, k & 31);
      const int32_t v1 = __shfl_sync(0xffffffffu, w1, k & 31);
      const bool in = half < C::kHalves && pos < kv_end;
      const int64_t row = in ? row_of(pos, k < 32 ? v0 : v1, s.np) : -1;
      const uint32_t nload = __popc(__ballot_sync(0xffffffffu, row >= 0));
      if (!acquire()) return false;
      const int stage = item % C::kRing;
      if (lane == 0) mbar_arrive_expect_tx(&fulls[stage], nload * R * 128);
      __syncwarp();
      if (row >= 0)
        tma_load_3d(base + stage * C::kTile + half * kHalfTile + box * R * 128, tm, half * 64, s.h, (int)row,
                    &fulls[stage]);
      item += 2;
    }
    return true;
  }

  // A lane gathers four rows at a time (tile::gather4), its positions 4 lane .. 4 lane + 3 of the tile, one
  // copy per 64-dim half; their pages are loaded a tile ahead.  Positions behind the end repeat the
  // last one and a bad page's (reported) read the pool's row 0: neither is seen by a row whose result
  // means anything.  29 requests of about 6000 positions, 8 heads at page size 1: 208 us at D 128 and 128 at
  // D 64; 16-byte cp.async copies with the same look-ahead 262 and 251, gathers whose pages were
  // loaded when needed 286 and 207.
  __device__ bool run_rows(const Seg& s) {
    const int lane = threadIdx.x & 31;
    const int kv_end = s.P + s.T;
    int32_t page[4];
    uint32_t in_page[4];
    bool listed[4];
    auto load_pages = [&](int j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t pidx;
        a.page_div.divmod((uint32_t)min(j * kBN + 4 * lane + i, kv_end - 1), pidx, in_page[i]);
        listed[i] = (int)pidx < s.np;
        page[i] = listed[i] ? ld(a.kv_indices + s.p0 + pidx) : 0;
      }
    };
    load_pages(s.j0);
    for (int j = s.j0; j < s.j0 + s.n; ++j) {
      int row[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = page[i] >= 0 && page[i] < a.num_pages;
        if (!listed[i] || !in) report(a.err_word, !listed[i] ? PKV_DEVERR_LENGTH : PKV_DEVERR_PAGE_OOB);
        row[i] = listed[i] && in ? page[i] * a.page_size + (int)in_page[i] : 0;
      }
      if (j + 1 < s.j0 + s.n) load_pages(j + 1);
      if (!acquire()) return false;
      const int stage = item % C::kRing;
      if (lane == 0) mbar_arrive_expect_tx(&fulls[stage], C::kTile);
      __syncwarp();
#pragma unroll
      for (int hf = 0; hf < C::kHalves; ++hf)
        tma_gather4(base + stage * C::kTile + hf * kHalfTile + lane * 512, tm, s.h * D + hf * 64, row[0], row[1], row[2],
                    row[3], &fulls[stage]);
      item += 2;
    }
    return true;
  }

  // No copy of this warp is in flight when the CTA exits.  With every tile issued (`all`, the normal
  // path) the last kRing places of the order, K's and V's, are the buffers' last occupants, and the
  // consumers have seen them land.  A place before those has been landed on, consumed and used again,
  // and its phase could no longer be waited for.  After a wait that gave up, every buffer's is tried
  // (bounded waits).
  __device__ void drain(bool all) {
    const int end = (item & ~1);  // places issued in all, if the other warp has come as far
    for (int i = item - 2; i >= max(0, all ? end - C::kRing : item - 2 * C::kRing); i -= 2)
      mbar_wait(&fulls[i % C::kRing], (i / C::kRing) & 1);
  }
};

// What a request asks for: its rows, its KV, its units and their tiles.
struct Req {
  int32_t q0, T, P, p0, np;
  int32_t pairs, tiles;  // Q tile pairs, KV tiles (0: nothing to do)
  int32_t cost;          // of a unit in the stream: its tiles and what an epilogue costs
};

__device__ Req load_req(const TreeArgs& a, int b, bool check) {
  Req r;
  r.q0 = ld(a.qo_indptr + b);
  const int32_t rows = ld(a.qo_indptr + b + 1) - r.q0;
  r.P = ld(a.prefix_lens + b);
  r.p0 = ld(a.kv_indptr + b);
  r.np = ld(a.kv_indptr + b + 1) - r.p0;
  r.T = min(max(rows, 0), a.max_nodes);
  r.pairs = r.tiles = r.cost = 0;
  uint32_t bad = 0;
  if (rows < 0 || rows > a.max_nodes || r.P < 0 || r.P > 0x7fffffff - kMaxNodes - kBN) bad = PKV_DEVERR_LENGTH;
  if (rows > 0 && (r.q0 < 0 || r.q0 > a.num_q_tokens - rows)) bad |= PKV_DEVERR_ROW_OOB;
  if (bad && check) report(a.err_word, bad);
  if (r.T > 0 && r.P >= 0 && r.P <= 0x7fffffff - kMaxNodes - kBN && !(bad & PKV_DEVERR_ROW_OOB)) {
    r.pairs = (r.T + 2 * a.tpt - 1) / (2 * a.tpt);
    r.tiles = (r.P + r.T + kBN - 1) / kBN;
    r.cost = r.tiles + kUnitCost;
  }
  return r;
}

// Length of the stream (K producer warp, before the set-up barrier); first: this lane's of the first 32
// requests, which the walk starts with.
__device__ int64_t tree_stream_length(const TreeArgs& a, Req& first) {
  const int lane = threadIdx.x & 31;
  first = Req{};
  if (lane < a.batch) first = load_req(a, lane, blockIdx.x == 0);
  int64_t total = (int64_t)first.pairs * first.cost;
  for (int i = 32 + lane; i < a.batch; i += 128) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {  // four requests' loads in flight
      if (i + 32 * u < a.batch) {
        const Req r = load_req(a, i + 32 * u, blockIdx.x == 0);
        total += (int64_t)r.pairs * r.cost;
      }
    }
  }
  return warp_sum(total) * a.num_kv_heads;
}

// K producer warp: walks this CTA's share of the stream, publishes each segment and loads its K.
template <int D, bool kRows>
__device__ void tree_walk(const TreeArgs& a, Ctl* ctl, uint32_t sb, int64_t total, const Req& first) {
  const int lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  Producer<D, kRows> k(a, ctl, sb, false);
  int64_t share = (total + gridDim.x - 1) / gridDim.x;
  if (share < 1) share = 1;
  const int64_t c0 = cta * share, c1 = min(total, c0 + share);

  bool ok = true;
  int nseg = 0;
  Cut cut = {};
  auto publish = [&](const Seg& s) -> bool {
    const int r = nseg % kSegRing;
    if (!__all_sync(0xffffffffu, mbar_wait(&ctl->seg_empty[r], ((nseg / kSegRing) & 1) ^ 1))) return false;
    if (lane == 0) {
      ctl->seg[r] = s;
      mbar_arrive(&ctl->seg_full[r]);
    }
    ++nseg;
    return true;
  };

  int64_t base = 0;  // stream offset of request b0
  for (int b0 = 0; b0 < a.batch && base < c1 && ok; b0 += 32) {
    Req r = first;
    if (b0 > 0) {
      r = Req{};
      if (b0 + lane < a.batch) r = load_req(a, b0 + lane, false);
    }
    const int64_t len = (int64_t)r.pairs * r.cost * a.num_kv_heads;
    int64_t incl = len;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const int64_t rs = base + incl - len;
    uint32_t hit = __ballot_sync(0xffffffffu, len > 0 && rs + len > c0 && rs < c1);
    while (hit && ok) {
      const int src = __ffs(hit) - 1;
      hit &= hit - 1;
      Seg s;
      s.q0 = __shfl_sync(0xffffffffu, r.q0, src);
      s.T = __shfl_sync(0xffffffffu, r.T, src);
      s.P = __shfl_sync(0xffffffffu, r.P, src);
      s.p0 = __shfl_sync(0xffffffffu, r.p0, src);
      s.np = __shfl_sync(0xffffffffu, r.np, src);
      const int pairs = __shfl_sync(0xffffffffu, r.pairs, src);
      const int tiles = __shfl_sync(0xffffffffu, r.tiles, src);
      const int64_t r0 = __shfl_sync(0xffffffffu, rs, src);
      const int cost = __shfl_sync(0xffffffffu, r.cost, src);
      const int units = pairs * a.num_kv_heads;
      // units in the order (KV head, pair): the first that reaches into the share
      for (int u = (int)max((int64_t)0, (c0 - r0) / cost); u < units && ok; ++u) {
        const int64_t us = r0 + (int64_t)u * cost, ue = us + tiles;  // (the rest is the epilogue's time)
        if (us >= c1) break;
        const int64_t s0 = max(us, c0), s1 = min(ue, c1);
        if (s0 >= s1) continue;
        s.h = u / pairs;
        s.t0 = (u % pairs) * 2 * a.tpt;
        s.nq = s.T - s.t0 > a.tpt ? 2 : 1;
        s.j0 = (int)(s0 - us);
        s.n = (int)(s1 - s0);
        s.part = s0 == us && s1 == ue ? -1 : 2 * cta + (us >= c0 ? 1 : 0);
        s.rep = s.nq == 2 ? 1 : s.T - s.t0 <= a.tpt4 ? 4 : s.T - s.t0 <= a.tpt2 ? 2 : 1;
        if (us >= c0 && ue > c1) cut = Cut{(int32_t)((ue - 1) / share) - cta + 1, s.q0, s.T, s.t0, s.h, s.nq, {0, 0}};
        ok = publish(s);
        ok = ok && k.run(s);
      }
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (ok) {
    Seg end = {};
    ok = publish(end);
  }
  if (lane == 0) a.cut[cta] = cut;
  // The merge may be scheduled once every CTA has issued its last K (it waits for this grid's
  // completion before it reads): early enough to hide its launch, late enough not to hold thread
  // slots that kernels on other streams could use.
  pdl_trigger();
  if (!ok && lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
  k.drain(ok);
}

// V and Q producer warp.  One Q tile always takes the first Q buffer, so that the second is free for
// the epilogue's scratch; two Q tiles wait until that is no longer read.
template <int D, bool kRows>
__device__ void tree_load_v(const TreeArgs& a, Ctl* ctl, uint32_t sb) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  Producer<D, kRows> v(a, ctl, sb, true);
  int uses[2] = {0, 0};
  Seg s;
  bool ok = true;
  for (int i = 0; ok; ++i) {
    ok = next_seg(ctl, i, s);
    if (!ok || s.nq == 0) break;
    if (C::kShared && s.nq == 2) {
      const uint64_t t0 = globaltimer_ns();
      while (ok && atomicAdd(&ctl->epilogues, 0u) < 8u * (uint32_t)i) ok = globaltimer_ns() - t0 <= kWaitLimitNs;
      ok = __all_sync(0xffffffffu, ok);
    }
    const int level = s.rep == 1 ? 0 : s.rep == 2 ? 1 : 2;
    const int tokens = level == 0 ? a.tpt : level == 1 ? a.tpt2 : a.tpt4;
    for (int q = 0; q < s.nq && ok; ++q, ++uses[q - 1]) {
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl->q_empty[q], (uses[q] & 1) ^ 1));
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&ctl->q_full[q], C::kHalves * s.rep * tokens * a.group * 128);
      __syncwarp();
      if (lane < C::kHalves * s.rep) {
        const int hf = lane % C::kHalves, copy = lane / C::kHalves;
        tma_load_3d(sb + C::kOffQ + q * C::kTile + hf * kHalfTile + copy * (kBM / s.rep) * 128, &a.tm_q[level], hf * 64,
                    s.h * a.group, s.q0 + s.t0 + q * a.tpt, &ctl->q_full[q]);
      }
    }
    ok = ok && v.run(s);
  }
  if (!ok && lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
  v.drain(ok);
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (uses[q] > 0) mbar_wait(&ctl->q_full[q], (uses[q] - 1) & 1);
}

// ---------------------------------------------------------------------------------------------
// MMA issuers: one thread each.  A tile of a segment goes to slot (tile & 1) with one Q tile, and to
// both slots with two.
// ---------------------------------------------------------------------------------------------
PKV_DEV bool next_seg_thread(Ctl* ctl, int i, Seg& s) {
  const int r = i % kSegRing;
  if (!mbar_wait(&ctl->seg_full[r], (i / kSegRing) & 1)) return false;
  s = ctl->seg[r];
  mbar_arrive(&ctl->seg_empty[r]);
  return true;
}

template <int D>
__device__ bool tree_mma_qk(Ctl* ctl, uint32_t sb, uint32_t tmem) {
  using C = Cfg<D>;
  constexpr uint32_t idesc = umma_idesc_bf16(kBM, kBN, false);
  const uint64_t qdesc0 = smem_desc_sw128(sb + C::kOffQ, 16, 1024);
  const uint64_t kdesc0 = smem_desc_sw128(sb + C::kOffRing, 16, 1024);
  uint32_t kt = 0, qt[2] = {0, 0}, used[2] = {0, 0};  // K tiles, uses of the Q buffers and the slots so far
  Seg s;
  for (int i = 0;; ++i) {
    if (!next_seg_thread(ctl, i, s)) return false;
    if (s.nq == 0) return true;
    for (int q = 0; q < s.nq; ++q)
      if (!mbar_wait(&ctl->q_full[q], qt[q] & 1)) return false;
    for (int j = 0; j < s.n; ++j, ++kt) {
      const uint32_t st = (2 * kt) % C::kRing;
      if (!mbar_wait(&ctl->full[st], ((2 * kt) / C::kRing) & 1)) return false;
      const uint64_t kdesc = kdesc0 + ((st * C::kTile) >> 4);
      for (int q = 0; q < s.nq; ++q) {
        const int slot = s.nq == 2 ? q : (j & 1);
        if (!mbar_wait(&ctl->s_free[slot], (used[slot] & 1) ^ 1)) return false;
        tc_fence_after();
        const uint64_t qdesc = qdesc0 + ((q * C::kTile) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * kHalfTile + (ks & 3) * 32) >> 4;
          umma_ss(tmem + kColS + slot * 128, qdesc + off, kdesc + off, idesc, ks > 0);
        }
        umma_commit(&ctl->s_full[slot]);
        mbar_arrive(&ctl->qk_issued[slot]);
        ++used[slot];
      }
      umma_commit(&ctl->empty[st]);
    }
    for (int q = 0; q < s.nq; ++q, ++qt[q - 1]) umma_commit(&ctl->q_empty[q]);
  }
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
// infinities and NaNs of drafted tokens, which are noted.  By one warp, a row per lane at a time; the
// prefix's rows are left alone.
template <int D>
__device__ void clean_v(uint8_t* vtile, Ctl* ctl, const Seg& s, int pos0) {
  using C = Cfg<D>;
  constexpr int kChunks = C::kHalves * 8;
  const int lane = threadIdx.x & 31;
  for (int r = max(0, s.P - pos0) + lane; r < kBN; r += 32) {
    const int t = pos0 + r - s.P;
    uint8_t* row = vtile + r * 128;
    auto at = [&](int i) {  // chunks in an order that spreads the lanes over the banks
      return reinterpret_cast<uint4*>(row + (i >> 3) * kHalfTile + (((i + r) & 7) << 4));
    };
    if (t >= s.T) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) *at(i) = make_uint4(0u, 0u, 0u, 0u);
    } else {
      uint32_t bad = 0;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const uint4 u = *at(i);
        bad |= nonfinite_bits(u.x) | nonfinite_bits(u.y) | nonfinite_bits(u.z) | nonfinite_bits(u.w);
      }
      if (bad) {
#pragma unroll 1
        for (int i = 0; i < kChunks; ++i) {
          const uint4 u = *at(i);
          *at(i) = make_uint4(finite_bf16x2(u.x), finite_bf16x2(u.y), finite_bf16x2(u.z), finite_bf16x2(u.w));
        }
        atomicOr(&ctl->bad[t >> 5], 1u << (t & 31));
        ctl->bad_any = 1u;
      }
    }
  }
  fence_proxy_async_smem();  // before the MMA reads the tile
  __syncwarp();
}

// PV warp.  Its first lane issues; the whole warp cleans the V tiles that reach past the prefix, while
// the softmax is still at work on their scores.
template <int D>
__device__ bool tree_mma_pv(Ctl* ctl, uint8_t* smem, uint32_t tmem) {
  using C = Cfg<D>;
  constexpr uint32_t idesc = umma_idesc_bf16(kBM, D, true);
  const int lane = threadIdx.x & 31;
  const uint64_t vdesc0 = smem_desc_sw128(smem_u32(smem) + C::kOffRing, kHalfTile, 1024);
  uint32_t vt = 0, used[2] = {0, 0};
  auto wait = [](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0; };
  Seg s;
  for (int i = 0;; ++i) {
    if (!next_seg(ctl, i, s)) return false;
    if (s.nq == 0) return true;
    if (!wait(&ctl->o_free, (i & 1) ^ 1)) return false;  // the last segment's O and notes have been read
    if (ctl->bad_any) {
      ctl->bad[lane] = 0u;
      __syncwarp();
      if (lane == 0) ctl->bad_any = 0u;
      __syncwarp();
    }
    for (int j = 0; j < s.n; ++j, ++vt) {
      const uint32_t st = (2 * vt + 1) % C::kRing;
      const uint64_t vdesc = vdesc0 + ((st * C::kTile) >> 4);
      const int pos0 = (s.j0 + j) * kBN;
      if (!wait(&ctl->full[st], ((2 * vt + 1) / C::kRing) & 1)) return false;
      if (pos0 + kBN > s.P) clean_v<D>(smem + C::kOffRing + st * C::kTile, ctl, s, pos0);
      for (int q = 0; q < s.nq; ++q) {
        const int slot = s.nq == 2 ? q : (j & 1);
        const bool first = s.nq == 2 ? j == 0 : j < 2;
        if (!wait(&ctl->p_full[slot], used[slot] & 1)) return false;
        // With two Q tiles the order is PV 0, QK 0, PV 1, QK 1, so that each slot's products run beside the
        // other's softmax; left to themselves the slots fall into step and both products wait for both
        // softmaxes (4 requests of 64 tokens over 32700 positions: 134 us, 129 so).
        if (s.nq == 2 && (q == 0 || j + 1 < s.n) && !wait(&ctl->qk_issued[q ^ 1], used[q ^ 1] & 1)) return false;
        tc_fence_after();
        if (lane == 0) {
#pragma unroll
          for (int ks = 0; ks < kBN / 16; ++ks)
            umma_ts(tmem + kColO + slot * 128, tmem + kColS + slot * 128 + ks * 8, vdesc + ((ks * 2048) >> 4), idesc,
                    !first || ks > 0);
          umma_commit(&ctl->s_free[slot]);
        }
        __syncwarp();
        ++used[slot];
      }
      if (lane == 0) umma_commit(&ctl->empty[st]);
    }
    if (lane == 0) mbar_arrive(&ctl->x_full);  // this segment's notes are made
  }
}

// ---------------------------------------------------------------------------------------------
// Softmax and epilogue
// ---------------------------------------------------------------------------------------------
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

// Adds the non-finite values of dims [d0, d0 + n) of the noted drafted tokens that the row sees to what
// this thread has written at `to` (the rest of them is in it already).
template <int D, typename T>
__device__ __noinline__ void add_nonfinite(const TreeArgs& a, const Ctl* ctl, int P, int nodes, int p0, int np, int h,
                                           const uint32_t* m, int d0, int n, T* to) {
  for (int w = 0; w < (nodes + 31) / 32; ++w) {
    uint32_t hit = ctl->bad[w] & (w < a.words ? ld(m + w) : 0u);
    while (hit) {
      const int t = 32 * w + __ffs(hit) - 1;
      hit &= hit - 1;
      const int pos = P + t, pidx = pos / a.page_size;
      if (pidx >= np) continue;
      const int32_t page = ld(a.kv_indices + p0 + pidx);
      if (page < 0 || page >= a.num_pages) continue;
      const __nv_bfloat16* src =
          a.v_pool + (((int64_t)page * a.page_size + pos % a.page_size) * a.num_kv_heads + h) * D + d0;
      for (int i = 0; i < n; ++i) {
        const float x = __bfloat162float(src[i]);
        if (!(fabsf(x) < INFINITY)) to[i] = (T)((float)to[i] + x);
      }
    }
  }
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

// The weights 2^(v sc + neg) of 32 scores as bf16 pairs, and their sum.
PKV_DEV float weights32(const float (&v)[32], float sc, float neg, uint32_t (&pk)[16]) {
  const uint64_t sc2 = f32x2(sc, sc), neg2 = f32x2(neg, neg);
  uint64_t t0 = f32x2(0.f, 0.f), t1 = t0;
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    float x0, x1, x2, x3;
    split_f32x2(fma_f32x2(f32x2(v[2 * e], v[2 * e + 1]), sc2, neg2), x0, x1);
    split_f32x2(fma_f32x2(f32x2(v[2 * e + 2], v[2 * e + 3]), sc2, neg2), x2, x3);
    const float p0 = ex2(x0), p1 = ex2(x1), p2 = ex2(x2), p3 = ex2(x3);
    t0 = add_f32x2(t0, f32x2(p0, p1));
    t1 = add_f32x2(t1, f32x2(p2, p3));
    pk[e] = pack_bf16x2(p0, p1);
    pk[e + 1] = pack_bf16x2(p2, p3);
  }
  float lo, hi;
  split_f32x2(add_f32x2(t0, t1), lo, hi);
  return lo + hi;
}

// A row's N chunks of 32 scores from chunk ch0 on, in TMEM at ts: the new reference maximum, the factor of
// what was summed under the old one m, P written over S as bf16 pairs, the other chunks' P zeroed, and
// the sum of the weights.  Two passes over the scores, the next chunk's load in flight while one is
// worked on; the first chunk stays in registers between them.
template <int N>
PKV_DEV float softmax_tile(uint32_t ts, int ch0, float sc, float m, float& m_ref, float& corr) {
  float a[32], b[32];  // odd and even chunks
  const uint32_t s0 = ts + ch0 * 32, p0 = ts + ch0 * 16;
  float mx = -INFINITY;
  if constexpr (N == 1) {
    tmem_ld32(s0, b);
    tmem_wait_ld32(b);
    mx = max32(b);
  } else {
    tmem_ld32(s0 + (N - 1) * 32, a);
    tmem_wait_ld32(a);
    if constexpr (N == 4) {
      tmem_ld32(s0 + 64, b);
      mx = max32(a);
      tmem_wait_ld32(b);
      tmem_ld32(s0 + 32, a);
      mx = fmaxf(mx, max32(b));
      tmem_wait_ld32(a);
    }
    tmem_ld32(s0, b);
    mx = N == 4 ? fmaxf(mx, max32(a)) : max32(a);
    tmem_wait_ld32(b);
    mx = fmaxf(mx, max32(b));
  }
  const float m_new = fmaxf(m, mx * sc);
  // the maximum moves only when it grows by more than 2^8, so that O is seldom rescaled
  const bool resc = m_new > m + 8.f;
  m_ref = resc ? m_new : m;
  corr = resc ? ex2(m - m_ref) : 1.f;
  const float neg = m_ref == -INFINITY ? 0.f : -m_ref;  // nothing seen so far: every weight is 0
  // P of chunk c goes over columns of S of chunk c / 2, which has been read by then
  uint32_t pk[16];
  float tot;
  if constexpr (N == 1) {
    tot = weights32(b, sc, neg, pk);
    tmem_st16(p0, pk);
  } else {
    tmem_ld32(s0 + 32, a);
    tot = weights32(b, sc, neg, pk);
    tmem_wait_ld32(a);
    tmem_st16(p0, pk);
    if constexpr (N == 4) tmem_ld32(s0 + 64, b);
    tot += weights32(a, sc, neg, pk);
    if constexpr (N == 4) tmem_wait_ld32(b);
    tmem_st16(p0 + 16, pk);
    if constexpr (N == 4) {
      tmem_ld32(s0 + 96, a);
      tot += weights32(b, sc, neg, pk);
      tmem_wait_ld32(a);
      tmem_st16(p0 + 32, pk);
      tot += weights32(a, sc, neg, pk);
      tmem_st16(p0 + 48, pk);
    }
  }
  if constexpr (N < 4) {
#pragma unroll
    for (int e = 0; e < 16; ++e) pk[e] = 0u;
#pragma unroll 1
    for (int c = N; c < 4; ++c) tmem_st16(ts + ((ch0 + c) & 3) * 16, pk);
  }
  return tot;
}

template <int D>
__device__ void tree_softmax(const TreeArgs& a, uint8_t* smem, Ctl* ctl, uint32_t tmem) {
  using C = Cfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = (warp - kSoftmaxWarp0) >> 2;
  const int wq = warp & 3;       // TMEM lane quadrant
  const int r = wq * 32 + lane;  // tile row
  const uint32_t tq = tmem + ((uint32_t)(wq * 32) << 16);
  const uint32_t ts = tq + kColS + slot * 128;
  const uint32_t to = tq + kColO + slot * 128;
  const int G = a.group;
  const bool pos_scale = a.scale_log2 > 0.f;
  const float sc = pos_scale ? a.scale_log2 : 1.f;
  uint32_t used[2] = {0, 0};  // uses of both slots before this segment
  bool ok = true;

  for (int i = 0; ok; ++i) {
    Seg s;
    if (!next_seg(ctl, i, s)) {
      ok = false;
      break;
    }
    if (s.nq == 0) break;
    const bool two = s.nq == 2;
    // the thread's row among the distinct ones, and its copy's share of a tile's four 32-column chunks
    const int rr = s.rep == 4 ? lane : s.rep == 2 ? r & 63 : r;
    const int copy = s.rep == 4 ? wq : s.rep == 2 ? wq >> 1 : 0;
    const int nch = 4 / s.rep, ch0 = copy * nch;
    const int rt = rr / G, g = rr - rt * G;  // token of the tile, head of the group
    const int tok = s.t0 + (two ? slot * a.tpt : 0) + rt;
    const bool valid = rt < (s.rep == 4 ? a.tpt4 : s.rep == 2 ? a.tpt2 : a.tpt) && tok < s.T;
    const bool warp_live = __any_sync(0xffffffffu, valid);
    MaskRow mask{valid ? a.mask + (int64_t)(s.q0 + tok) * a.words : nullptr, a.words, {0u, 0u, 0u, 0u}};
    if ((s.j0 + s.n) * kBN > s.P) load_mask(mask);
    float m = -INFINITY, l = 0.f;  // running maximum of the scaled (log2) scores, sum of weights
    uint32_t n_used = used[slot];

    for (int jj = two ? 0 : slot; jj < s.n && ok; jj += two ? 1 : 2, ++n_used) {
      const int pos0 = (s.j0 + jj) * kBN;
      const bool special = pos0 + kBN > s.P;
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl->s_full[slot], n_used & 1));
      if (!ok) break;
      tc_fence_after();
      if (warp_live) {
        if (special || !pos_scale) {  // masked (and scaled) scores take the place of the scores
#pragma unroll 1
          for (int ch = ch0; ch < ch0 + nch; ++ch) {
            float v[32];
            tmem_ld32(ts + ch * 32, v);
            const uint32_t vis = special ? visible(mask, s.T, pos0 + 32 * ch - s.P) : 0xffffffffu;
            const float mul = pos_scale ? 1.f : a.scale_log2;
            tmem_wait_ld32(v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (vis >> e) & 1u ? v[e] * mul : -INFINITY;
            tmem_st32(ts + ch * 32, v);
          }
          tmem_wait_st();
        }
        float m_ref, corr, tot;
        if (nch == 1)
          tot = softmax_tile<1>(ts, ch0, sc, m, m_ref, corr);
        else if (nch == 2)
          tot = softmax_tile<2>(ts, ch0, sc, m, m_ref, corr);
        else
          tot = softmax_tile<4>(ts, ch0, sc, m, m_ref, corr);
        const bool resc = m_ref > m;
        l = l * corr + tot;
        m = m_ref;
        const bool later = two ? jj > 0 : jj > 1;  // O holds earlier tiles (whose PV is done: S was free)
        if (later && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            float v[32];
            tmem_ld32(to + ch * 32, v);
            tmem_wait_ld32(v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= corr;
            tmem_st32(to + ch * 32, v);
          }
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->p_full[slot]);
    }
    if (!ok) break;

    // every PV of the segment is done, in both slots
    if (two) {
      used[0] += s.n;
      used[1] += s.n;
    } else {
      used[0] += (s.n + 1) / 2;
      used[1] += s.n / 2;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (used[k] > 0) ok = ok && __all_sync(0xffffffffu, mbar_wait(&ctl->s_free[k], (used[k] - 1) & 1));
    // the row states of slots and copies change hands (the previous segment's have been read)
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&ctl->x_free, (i & 1) ^ 1));
    if (!ok) break;
    ctl->xm[slot][r] = m;
    ctl->xl[slot][r] = l;
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->x_full);
    ok = __all_sync(0xffffffffu, mbar_wait(&ctl->x_full, i & 1));
    if (!ok) break;
    // From here to the end of the segment nothing can give up: all eight warps have come this far.
    tc_fence_after();
    const bool any_bad = ctl->bad_any != 0u;
    float mt = m, lt = l, om = -INFINITY;  // over every state of the row; the other slot's of this thread
    if (!two) {
      const int step = kBM / s.rep;
      float km[8], kl[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool on = (k >> 1) < s.rep;
        km[k] = on ? ctl->xm[k & 1][rr + (k >> 1) * step] : -INFINITY;
        kl[k] = on ? ctl->xl[k & 1][rr + (k >> 1) * step] : 0.f;
      }
      om = ctl->xm[slot ^ 1][r];
      mt = max3f(max3f(km[0], km[1], km[2]), max3f(km[3], km[4], km[5]), fmaxf(km[6], km[7]));
      lt = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) lt += kl[k] * (km[k] == -INFINITY ? 0.f : ex2(km[k] - mt));
    }
    const float inv = lt == 0.f ? 0.f : 1.f / lt;
    const float f_mine = m == -INFINITY ? 0.f : ex2(m - mt) * inv;
    const float f_other = om == -INFINITY ? 0.f : ex2(om - mt) * inv;
    const bool nan = !(lt == lt);  // a NaN among the scores: in every dim
    // (a slot or copy that saw nothing may hold anything: its O must not be used)
    const bool plain = __all_sync(0xffffffffu, !valid || (f_mine > 0.f && (two || f_other > 0.f)));
    const int64_t orow = (int64_t)(s.q0 + tok) * a.num_q_heads + (int64_t)s.h * G + g;
    const int prow = (two ? slot * kBM : 0) + rr;
    // Two Q tiles: all dims of the thread's own O.  One: half of the dims, from both slots' O; of 32 dims
    // a copy finishes 32 / rep, for which the other copies leave theirs in scratch, so it reads its
    // groups of 8 dims rotated: the first 4 / rep are its own.
    const int c0 = two ? 0 : slot * (D / 64), c1 = two ? D / 32 : c0 + D / 64;
    const int own = 4 / s.rep, rot = copy * own;
    float* scratch = reinterpret_cast<float*>(smem + C::kOffScratch) + slot * 3 * 32 * 32 + lane;
#pragma unroll 1
    for (int ch = c0; ch < c1; ++ch) {
      float o[32];
      if (two) {
        tmem_ld32(to + ch * 32, o);
        tmem_wait_ld32(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = plain || f_mine > 0.f ? o[e] * f_mine : 0.f;
      } else {
        float x[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t col = ch * 32 + ((j + rot) & 3) * 8;
          tmem_ld8(to + col, o + 8 * j);
          tmem_ld8(tq + kColO + (slot ^ 1) * 128 + col, x + 8 * j);
        }
        tmem_wait_ld32(o);
        tmem_wait_ld32(x);
        if (plain) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = fmaf(x[e], f_other, o[e] * f_mine);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = (f_mine > 0.f ? o[e] * f_mine : 0.f) + (f_other > 0.f ? x[e] * f_other : 0.f);
        }
      }
      if (nan) {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = lt;
      }
      // scratch: areas of [8 dims][32 rows]; with four copies area 3 d + j - 1 is for copy d from the copy j
      // before it, with two area 4 (row block) + 2 d + j - 2 for copy d's group j - 2
      if (s.rep == 4) {
#pragma unroll
        for (int j = 1; j < 4; ++j) {
          float* to_copy = scratch + (3 * ((copy + j) & 3) + j - 1) * 256;
#pragma unroll
          for (int e = 0; e < 8; ++e) to_copy[e * 32] = o[8 * j + e];
        }
        named_bar_sync(1 + slot, 128);
#pragma unroll
        for (int j = 1; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += scratch[(3 * copy + j - 1) * 256 + e * 32];
        named_bar_sync(1 + slot, 128);
      } else if (s.rep == 2) {
        float* block = scratch + (wq & 1) * 4 * 256;
#pragma unroll
        for (int j = 2; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) block[(2 * (copy ^ 1) + j - 2) * 256 + e * 32] = o[8 * j + e];
        named_bar_sync(1 + slot, 128);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) o[8 * j + e] += block[(2 * copy + j) * 256 + e * 32];
        named_bar_sync(1 + slot, 128);
      }
      if (valid) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= own) continue;
          const int d0 = ch * 32 + ((j + rot) & 3) * 8;
          const int e = 8 * j;
          if (s.part < 0) {
            __nv_bfloat16* dst = a.out + orow * D + d0;
            *reinterpret_cast<uint4*>(dst) =
                make_uint4(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]),
                           pack_bf16x2(o[e + 4], o[e + 5]), pack_bf16x2(o[e + 6], o[e + 7]));
            if (any_bad) add_nonfinite<D>(a, ctl, s.P, s.T, s.p0, s.np, s.h, mask.m, d0, 8, dst);
          } else {
            float* dst = a.part_o + (((int64_t)s.part * (D / 4) + d0 / 4) * a.part_rows + prow) * 4;
            float* dst1 = dst + (int64_t)a.part_rows * 4;
            *reinterpret_cast<float4*>(dst) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            *reinterpret_cast<float4*>(dst1) = make_float4(o[e + 4], o[e + 5], o[e + 6], o[e + 7]);
            if (any_bad) {
              add_nonfinite<D>(a, ctl, s.P, s.T, s.p0, s.np, s.h, mask.m, d0, 4, dst);
              add_nonfinite<D>(a, ctl, s.P, s.T, s.p0, s.np, s.h, mask.m, d0 + 4, 4, dst1);
            }
          }
        }
      }
    }
    if (valid && copy == 0 && (two || slot == 0)) {
      const float lse_v = (mt + log2f(lt)) * kLn2;
      if (s.part >= 0)
        a.part_lse[(int64_t)s.part * a.part_rows + prow] = lse_v;
      else if (a.lse)
        a.lse[orow] = lse_v;
    }
    tc_fence_before();
    fence_proxy_async_smem();  // the scratch may become a Q tile
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&ctl->o_free);
      mbar_arrive(&ctl->x_free);
      __threadfence_block();
      atomicAdd(&ctl->epilogues, 1u);
    }
  }
  if (!ok && lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
}

template <int D, bool kRows>
__global__ void __launch_bounds__(kThreads, 1) paged_tree_kernel(const __grid_constant__ TreeArgs a) {
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
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(&ctl->seg_full[i], 1);
      mbar_init(&ctl->seg_empty[i], 3 + 8);  // V producer, QK, PV, softmax warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], 1);
      mbar_init(&ctl->q_empty[i], 1);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->qk_issued[i], 1);
      mbar_init(&ctl->p_full[i], 4);
      mbar_init(&ctl->s_free[i], 1);
    }
    for (int i = 0; i < kMaxRing; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    mbar_init(&ctl->o_free, 8);
    mbar_init(&ctl->x_full, 8 + 1);  // and the PV warp's notes
    mbar_init(&ctl->x_free, 8);
    mbar_init(&ctl->qk_done, 1);
    mbar_init(&ctl->pv_done, 1);
    ctl->bad_any = 0u;
    ctl->epilogues = 0u;
    for (int i = 0; i < kMaxNodes / 32; ++i) ctl->bad[i] = 0u;
    fence_mbar_init();
    for (int i = 0; i < 3; ++i) prefetch_tmap(&a.tm_q[i]);
    prefetch_tmap(&a.tm_k);
    prefetch_tmap(&a.tm_v);
  }
  int64_t total = 0;
  Req first;
  if (warp == 0) {
    pdl_wait();
    total = tree_stream_length(a, first);
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 0) {
    tree_walk<D, kRows>(a, ctl, sb, total, first);
  } else if (warp == 3) {
    tree_load_v<D, kRows>(a, ctl, sb);
  } else if (warp == 1) {
    if (lane == 0) {
      if (!tree_mma_qk<D>(ctl, sb, tmem)) report(a.err_word, PKV_DEVERR_TIMEOUT);
      umma_commit(&ctl->qk_done);  // its MMAs have completed before TMEM is released
      if (!mbar_wait(&ctl->qk_done, 0)) report(a.err_word, PKV_DEVERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == 2) {
    const bool ok = tree_mma_pv<D>(ctl, smem, tmem);
    if (lane == 0) {
      if (!ok) report(a.err_word, PKV_DEVERR_TIMEOUT);
      umma_commit(&ctl->pv_done);
      if (!mbar_wait(&ctl->pv_done, 0)) report(a.err_word, PKV_DEVERR_TIMEOUT);
    }
    __syncwarp();
  } else {
    tree_softmax<D>(a, smem, ctl, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------------------------
// Merge: block (c, y) joins rows 32 y .. 32 y + 31 of the unit that CTA c began and did not finish.  A
// lane is a row, a warp every eighth group of four dims, so a part's rows are read as whole lines; the
// states are joined in one pass with a running maximum, the loads of four parts in flight.  5 us after
// 64 requests of up to 16 tokens, 9 after 4 of 64 (23 MB of states, which L2 holds).
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
  const int r = prow & (kBM - 1), tile = prow / kBM;
  const int tok = cut.t0 + tile * a.tpt + r / a.group;
  if (tile >= cut.nq || r >= a.group * a.tpt || tok >= cut.T) return;
  auto slot = [&](int p) -> int64_t { return (int64_t)2 * (c + p) + (p == 0 ? 1 : 0); };
  float mx = -INFINITY, tot = 0.f;
  float acc[kGroups][4] = {};
  for (int p0 = 0; p0 < cut.parts; p0 += 4) {
    float pl[4];
    float4 x[4][kGroups];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool on = p0 + k < cut.parts;
      const int64_t at = slot(on ? p0 + k : p0);
      pl[k] = on ? ld(a.part_lse + at * a.part_rows + prow) : -INFINITY;
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        x[k][i] = ld(reinterpret_cast<const float4*>(a.part_o) + (at * (D / 4) + warp + 8 * i) * a.part_rows + prow);
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
  const int64_t orow = (int64_t)(cut.q0 + tok) * a.num_q_heads + (int64_t)cut.h * a.group + r % a.group;
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
  int G, tpt, part_rows, ncta;
  size_t off_lse, off_o, ws_bytes;
};

bool make_plan(int B, int Hq, int Hkv, int D, int max_nodes, int ncta, Plan& p) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || max_nodes < 0 || max_nodes > kMaxNodes) return false;
  if (D != 64 && D != 128) return false;
  p.G = Hq / Hkv;
  if (p.G > 16) return false;
  p.tpt = kBM / p.G;
  p.part_rows = max_nodes > p.tpt ? 2 * kBM : kBM;
  p.ncta = ncta;
  p.off_lse = align256((size_t)ncta * sizeof(Cut));
  p.off_o = align256(p.off_lse + (size_t)2 * ncta * p.part_rows * 4);
  p.ws_bytes = align256(p.off_o + (size_t)2 * ncta * p.part_rows * D * 4);
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
  return pkv_host::launch_after(tree_merge_kernel<D>, dim3((unsigned)p.ncta, (unsigned)(p.part_rows / 32)), 256, 0, st, a);
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
  const int ncta = pkv_host::sm_count();
  if (ncta <= 0) return PKV_ERR_CUDA;
  Plan p;
  if (!make_plan(batch_size, num_q_heads, pool->num_kv_heads, D, max_tree_len, ncta, p)) return PKV_ERR_UNSUPPORTED;
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
  a.tpt2 = 64 / p.G;
  a.tpt4 = 32 / p.G;
  if (!pkv_host::encode_tmap_3d(&a.tm_q[0], q, D, Hq, (uint64_t)num_q_tokens, Db, Hq * Db, 64, p.G, a.tpt) ||
      !pkv_host::encode_tmap_3d(&a.tm_q[1], q, D, Hq, (uint64_t)num_q_tokens, Db, Hq * Db, 64, p.G, a.tpt2) ||
      !pkv_host::encode_tmap_3d(&a.tm_q[2], q, D, Hq, (uint64_t)num_q_tokens, Db, Hq * Db, 64, p.G, a.tpt4) ||
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
  a.part_rows = p.part_rows;
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
