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
//  * Twelve warps: K producer (which also walks the stream and publishes the segments), QK issuer, PV
//    issuer, V producer, and four softmax warps per slot, one thread per row.
//  * Only tiles that reach past the prefix are masked.  There the V rows behind the last position
//    and the infinities and NaNs of drafted tokens become 0 in shared memory (weight 0 times them
//    would be NaN for rows that do not see them); rows that do see them get them added when they are
//    written, which is what a sum with a non-zero weight would give.
#include <atomic>

#include "tc05.cuh"

namespace {

using namespace pkv;

constexpr int kBM = 128;              // Q tile rows
constexpr int kBN = 128;              // KV positions per tile
constexpr int kThreads = 384;
constexpr int kSoftmaxWarp0 = 4;      // warps 4..7 slot 0, 8..11 slot 1
constexpr int kMaxNodes = 1024;       // drafted tokens of a request
constexpr int kSegRing = 4;
constexpr int kKStages = 2, kVStages = 3;
constexpr uint32_t kHalfTile = 128 * 128;  // 128 rows of one 64-dim half, 16 KB
constexpr uint32_t kColO = 0, kColS = 256;  // O of slot s at 128 s, S at 256 + 128 s

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kTile = kHalves * kHalfTile;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffK = kOffQ + 2 * kTile;
  static constexpr uint32_t kOffV = kOffK + kKStages * kTile;
  static constexpr uint32_t kOffCtl = kOffV + kVStages * kTile;
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
  int32_t pad;
};

struct Ctl {
  Seg seg[kSegRing];
  uint64_t seg_full[kSegRing], seg_empty[kSegRing];
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2];  // QK written
  uint64_t p_full[2];  // P written, V cleaned
  uint64_t s_free[2];  // PV done
  uint64_t o_free;     // O read by the epilogue
  uint64_t x_full, x_free;  // the slots' exchange of row states
  uint64_t qk_done, pv_done;
  uint32_t tmem_base;
  uint32_t bad_any;
  uint32_t bad[kMaxNodes / 32];  // drafted tokens of this segment whose V is not finite
  float xm[2][kBM], xl[2][kBM];  // row maxima and sums of the slots
};
constexpr uint32_t kSmemLimit = 227 * 1024;
static_assert(Cfg<128>::kOffCtl + sizeof(Ctl) <= kSmemLimit, "shared memory");

// The unit that a CTA's share ends in the middle of, for the merge: its parts are the slots
// 2c + 1, 2(c + 1), 2(c + 2), ...
struct Cut {
  int32_t parts;  // 0: none
  int32_t q0, T, t0, h, nq;
  int32_t pad[2];
};

struct TreeArgs {
  CUtensorMap tm_q, tm_k, tm_v;
  const int32_t* qo_indptr;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* prefix_lens;
  const uint32_t* mask;  // [num_q_tokens, words]
  int32_t words;
  const __nv_bfloat16* k_pool;
  const __nv_bfloat16* v_pool;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* err_word;
  int64_t num_pages;
  int32_t page_size, box_rows;
  int32_t num_kv_heads, num_q_heads, group;
  int32_t tpt;        // tokens per Q tile
  int32_t rows_used;  // group * tpt
  int32_t batch, num_q_tokens, max_nodes;
  float scale_log2;
  Cut* cut;           // [CTAs]
  float* part_o;      // [2 CTAs][part_rows][D]
  float* part_lse;    // [2 CTAs][part_rows]
  int32_t part_rows;
};

PKV_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

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
// Copies the tiles of segments into a ring.  kRows: one row at a time by cp.async, for page sizes
// that are not a power of two of at least 8; else TMA boxes of min(page_size, 128) rows.
template <int D, bool kRows>
struct Producer {
  using C = Cfg<D>;
  const TreeArgs& a;
  uint64_t* fulls;
  uint64_t* empties;
  const CUtensorMap* tm;
  const __nv_bfloat16* pool;
  uint32_t base;  // of the ring, shared address
  int stages;
  int stage = 0;
  uint32_t phase = 0;
  int issued = 0;
  int unpublished = -1;  // kRows: the stage whose copies are not announced yet

  __device__ Producer(const TreeArgs& args, Ctl* ctl, uint32_t sb, bool v)
      : a(args), fulls(v ? ctl->v_full : ctl->k_full), empties(v ? ctl->v_empty : ctl->k_empty),
        tm(v ? &args.tm_v : &args.tm_k), pool(v ? args.v_pool : args.k_pool),
        base(sb + (v ? C::kOffV : C::kOffK)), stages(v ? kVStages : kKStages) {}

  __device__ void advance() {
    ++issued;
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }

  // Row of the pool that holds position pos, or -1 (reported).
  __device__ int64_t row_of(int pos, int32_t page, int np) {
    const int pidx = pos / a.page_size;
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
      return (pidx >= 0 && pidx < s.np) ? __ldg(a.kv_indices + s.p0 + pidx) : -1;
    };
    int wbase = s.j0 * kBN / a.page_size;
    int32_t w0 = entry(wbase + lane), w1 = entry(wbase + 32 + lane);
    for (int j = s.j0; j < s.j0 + s.n; ++j) {
      while (j * kBN / a.page_size >= wbase + 32) {  // the upper half was loaded 32 pages ago
        w0 = w1;
        wbase += 32;
        w1 = entry(wbase + 32 + lane);
      }
      const int pos = j * kBN + box * R;
      const int k = pos / a.page_size - wbase;  // < 64: a tile spans at most 16 pages
      const int32_t v0 = __shfl_sync(0xffffffffu, w0, k & 31);
      const int32_t v1 = __shfl_sync(0xffffffffu, w1, k & 31);
      const bool in = half < C::kHalves && pos < kv_end;
      const int64_t row = in ? row_of(pos, k < 32 ? v0 : v1, s.np) : -1;
      const uint32_t nload = __popc(__ballot_sync(0xffffffffu, row >= 0));
      if (!__all_sync(0xffffffffu, mbar_wait(&empties[stage], phase ^ 1))) return false;
      if (lane == 0) mbar_arrive_expect_tx(&fulls[stage], nload * R * 128);
      __syncwarp();
      if (row >= 0)
        tma_load_3d(base + stage * C::kTile + half * kHalfTile + box * R * 128, tm, half * 64, s.h, (int)row,
                    &fulls[stage]);
      advance();
    }
    return true;
  }

  // The previous stage's copies have landed: make them visible to the tensor cores, announce them.
  __device__ void publish(bool all) {
    if (unpublished < 0) return;
    if (all)
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&fulls[unpublished]);
    unpublished = -1;
  }

  __device__ bool run_rows(const Seg& s) {
    const int lane = threadIdx.x & 31;
    const int kv_end = s.P + s.T;
    auto slot_of = [&](int j, int r) -> int64_t {
      const int pos = j * kBN + r;
      if (j >= s.j0 + s.n || pos >= kv_end) return -1;
      const int pidx = pos / a.page_size;
      return row_of(pos, pidx < s.np ? __ldg(a.kv_indices + s.p0 + pidx) : -1, s.np);
    };
    int64_t next[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) next[i] = slot_of(s.j0, lane + 32 * i);
    for (int j = s.j0; j < s.j0 + s.n; ++j) {
      // no free stage yet: announce the pending one now instead of behind the next issue
      if (!__all_sync(0xffffffffu, mbar_test(&empties[stage], phase ^ 1))) publish(true);
      if (!__all_sync(0xffffffffu, mbar_wait(&empties[stage], phase ^ 1))) return false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (next[i] < 0) continue;
        const int row = lane + 32 * i;
        const char* src = reinterpret_cast<const char*>(pool + (next[i] * a.num_kv_heads + s.h) * D);
        const uint32_t dst = base + stage * C::kTile + row * 128;
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
#pragma unroll
          for (int c = 0; c < 8; ++c)
            cp_async16(dst + hf * kHalfTile + ((c ^ (row & 7)) << 4), src + hf * 128 + c * 16);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      const int mine = stage;
      advance();
#pragma unroll
      for (int i = 0; i < 4; ++i) next[i] = slot_of(j + 1, lane + 32 * i);  // while these copies fly
      publish(false);
      unpublished = mine;
    }
    publish(true);
    return true;
  }

  // No copy of this warp is in flight when the CTA exits (bounded; immediate on the normal path).
  __device__ void drain() {
    if (kRows) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      publish(true);
    }
    for (int k = 0; k < min(issued, stages); ++k) {
      if (--stage < 0) {
        stage = stages - 1;
        phase ^= 1;
      }
      mbar_wait(&fulls[stage], phase);
    }
  }
};

// What a request asks for: its rows, its KV, its units and their tiles.
struct Req {
  int32_t q0, T, P, p0, np;
  int32_t pairs, tiles;  // Q tile pairs, KV tiles (0: nothing to do)
};

__device__ Req load_req(const TreeArgs& a, int b, bool check) {
  Req r;
  r.q0 = __ldg(a.qo_indptr + b);
  const int32_t rows = __ldg(a.qo_indptr + b + 1) - r.q0;
  r.P = __ldg(a.prefix_lens + b);
  r.p0 = __ldg(a.kv_indptr + b);
  r.np = __ldg(a.kv_indptr + b + 1) - r.p0;
  r.T = min(max(rows, 0), a.max_nodes);
  r.pairs = r.tiles = 0;
  uint32_t bad = 0;
  if (rows < 0 || rows > a.max_nodes || r.P < 0 || r.P > 0x7fffffff - kMaxNodes - kBN) bad = PKV_DEVERR_LENGTH;
  if (rows > 0 && (r.q0 < 0 || r.q0 > a.num_q_tokens - rows)) bad |= PKV_DEVERR_ROW_OOB;
  if (bad && check) report(a.err_word, bad);
  if (r.T > 0 && r.P >= 0 && r.P <= 0x7fffffff - kMaxNodes - kBN && !(bad & PKV_DEVERR_ROW_OOB)) {
    r.pairs = (r.T + 2 * a.tpt - 1) / (2 * a.tpt);
    r.tiles = (r.P + r.T + kBN - 1) / kBN;
  }
  return r;
}

// K producer warp: walks this CTA's share of the stream, publishes each segment, loads its Q and K.
template <int D, bool kRows>
__device__ void tree_walk(const TreeArgs& a, Ctl* ctl, uint32_t sb) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  Producer<D, kRows> k(a, ctl, sb, false);
  int64_t total = 0;
  for (int i = lane; i < a.batch; i += 32) {
    const Req r = load_req(a, i, cta == 0);
    total += (int64_t)r.pairs * r.tiles;
  }
  total = warp_sum(total) * a.num_kv_heads;
  int64_t share = (total + gridDim.x - 1) / gridDim.x;
  if (share < 1) share = 1;
  const int64_t c0 = cta * share, c1 = min(total, c0 + share);

  bool ok = true;
  int nseg = 0, nqt = 0;
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
    Req r = {};
    if (b0 + lane < a.batch) r = load_req(a, b0 + lane, false);
    const int64_t len = (int64_t)r.pairs * r.tiles * a.num_kv_heads;
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
      const int units = pairs * a.num_kv_heads;
      // units in the order (KV head, pair): the first that reaches into the share
      for (int u = (int)max((int64_t)0, (c0 - r0) / tiles); u < units && ok; ++u) {
        const int64_t us = r0 + (int64_t)u * tiles, ue = us + tiles;
        if (us >= c1) break;
        const int64_t s0 = max(us, c0), s1 = min(ue, c1);
        if (s0 >= s1) continue;
        s.h = u / pairs;
        s.t0 = (u % pairs) * 2 * a.tpt;
        s.nq = s.T - s.t0 > a.tpt ? 2 : 1;
        s.j0 = (int)(s0 - us);
        s.n = (int)(s1 - s0);
        s.part = s0 == us && s1 == ue ? -1 : 2 * cta + (us >= c0 ? 1 : 0);
        s.pad = 0;
        if (us >= c0 && ue > c1) cut = Cut{(int32_t)((ue - 1) / share) - cta + 1, s.q0, s.T, s.t0, s.h, s.nq, {0, 0}};
        ok = publish(s);
        for (int i = 0; i < s.nq && ok; ++i, ++nqt) {
          const int qb = nqt & 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&ctl->q_empty[qb], ((nqt >> 1) & 1) ^ 1));
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(&ctl->q_full[qb], C::kHalves * a.rows_used * 128);
#pragma unroll
            for (int hf = 0; hf < C::kHalves; ++hf)
              tma_load_3d(sb + C::kOffQ + qb * C::kTile + hf * kHalfTile, &a.tm_q, hf * 64, s.h * a.group,
                          s.q0 + s.t0 + i * a.tpt, &ctl->q_full[qb]);
          }
          __syncwarp();
        }
        ok = ok && k.run(s);
      }
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (ok) {
    Seg end = {};
    ok = publish(end);
  }
  if (!ok && lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
  if (lane == 0) a.cut[cta] = cut;
  k.drain();
  for (int i = max(0, nqt - 2); i < nqt; ++i) mbar_wait(&ctl->q_full[i & 1], (i >> 1) & 1);
}

template <int D, bool kRows>
__device__ void tree_load_v(const TreeArgs& a, Ctl* ctl, uint32_t sb) {
  Producer<D, kRows> v(a, ctl, sb, true);
  Seg s;
  for (int i = 0;; ++i) {
    if (!next_seg(ctl, i, s) || (s.nq > 0 && !v.run(s))) {
      if ((threadIdx.x & 31) == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
      break;
    }
    if (s.nq == 0) break;
  }
  v.drain();
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
  const uint64_t kdesc0 = smem_desc_sw128(sb + C::kOffK, 16, 1024);
  uint32_t kt = 0, nqt = 0, used[2] = {0, 0};  // K tiles, Q tiles, uses of each slot so far
  Seg s;
  for (int i = 0;; ++i) {
    if (!next_seg_thread(ctl, i, s)) return false;
    if (s.nq == 0) return true;
    for (int q = 0; q < s.nq; ++q)
      if (!mbar_wait(&ctl->q_full[(nqt + q) & 1], ((nqt + q) >> 1) & 1)) return false;
    for (int j = 0; j < s.n; ++j, ++kt) {
      const uint32_t st = kt % kKStages;
      if (!mbar_wait(&ctl->k_full[st], (kt / kKStages) & 1)) return false;
      const uint64_t kdesc = kdesc0 + ((st * C::kTile) >> 4);
      for (int q = 0; q < s.nq; ++q) {
        const int slot = s.nq == 2 ? q : (j & 1);
        if (!mbar_wait(&ctl->s_free[slot], (used[slot] & 1) ^ 1)) return false;
        tc_fence_after();
        const uint64_t qdesc = qdesc0 + ((((nqt + q) & 1) * C::kTile) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * kHalfTile + (ks & 3) * 32) >> 4;
          umma_ss(tmem + kColS + slot * 128, qdesc + off, kdesc + off, idesc, ks > 0);
        }
        umma_commit(&ctl->s_full[slot]);
        ++used[slot];
      }
      umma_commit(&ctl->k_empty[st]);
    }
    for (int q = 0; q < s.nq; ++q, ++nqt) umma_commit(&ctl->q_empty[nqt & 1]);
  }
}

template <int D>
__device__ bool tree_mma_pv(Ctl* ctl, uint32_t sb, uint32_t tmem) {
  using C = Cfg<D>;
  constexpr uint32_t idesc = umma_idesc_bf16(kBM, D, true);
  const uint64_t vdesc0 = smem_desc_sw128(sb + C::kOffV, kHalfTile, 1024);
  uint32_t vt = 0, used[2] = {0, 0};
  Seg s;
  for (int i = 0;; ++i) {
    if (!next_seg_thread(ctl, i, s)) return false;
    if (s.nq == 0) return true;
    if (!mbar_wait(&ctl->o_free, (i & 1) ^ 1)) return false;
    for (int j = 0; j < s.n; ++j, ++vt) {
      const uint32_t st = vt % kVStages;
      const uint64_t vdesc = vdesc0 + ((st * C::kTile) >> 4);
      for (int q = 0; q < s.nq; ++q) {
        const int slot = s.nq == 2 ? q : (j & 1);
        const bool first = s.nq == 2 ? j == 0 : j < 2;
        if (!mbar_wait(&ctl->p_full[slot], used[slot] & 1)) return false;
        if (!mbar_wait(&ctl->v_full[st], (vt / kVStages) & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < kBN / 16; ++ks)
          umma_ts(tmem + kColO + slot * 128, tmem + kColS + slot * 128 + ks * 8, vdesc + ((ks * 2048) >> 4), idesc,
                  !first || ks > 0);
        umma_commit(&ctl->s_free[slot]);
        ++used[slot];
      }
      umma_commit(&ctl->v_empty[st]);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Softmax and epilogue
// ---------------------------------------------------------------------------------------------
// Which of the 32 positions of drafted-token offsets t0 .. t0 + 31 (t0 may be negative: the prefix)
// a row with mask words m (nullptr: an unused row) sees.
PKV_DEV uint32_t visible(const uint32_t* m, int words, int T, int t0) {
  if (t0 <= -32) return 0xffffffffu;
  if (t0 >= T) return 0u;
  auto word = [&](int w) -> uint32_t { return w < 0 ? 0xffffffffu : (m && w < words ? __ldg(m + w) : 0u); };
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

// What no weight may touch in a tile of V becomes zeros: the rows behind the last position, and the
// infinities and NaNs of drafted tokens, which are noted.  One thread per row; the prefix's rows are
// left alone.
template <int D>
__device__ void clean_v(uint8_t* vtile, Ctl* ctl, const Seg& s, int pos0, int r) {
  using C = Cfg<D>;
  const int t = pos0 + r - s.P;
  if (t < 0) return;
  uint8_t* row = vtile + r * 128;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < C::kHalves * 8; ++i) {
    uint4* at = reinterpret_cast<uint4*>(row + (i >> 3) * kHalfTile + (((i + r) & 7) << 4));
    if (t >= s.T) {
      *at = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const uint4 u = *at;
      const uint4 f = make_uint4(finite_bf16x2(u.x), finite_bf16x2(u.y), finite_bf16x2(u.z), finite_bf16x2(u.w));
      if (f.x != u.x || f.y != u.y || f.z != u.z || f.w != u.w) {
        *at = f;
        bad = true;
      }
    }
  }
  if (bad) {
    atomicOr(&ctl->bad[t >> 5], 1u << (t & 31));
    ctl->bad_any = 1u;
  }
}

// Adds the non-finite values of dims [d0, d0 + 32) of the noted drafted tokens that the row sees.
template <int D>
__device__ void add_nonfinite(const TreeArgs& a, const Ctl* ctl, const Seg& s, const uint32_t* m, int d0,
                              float (&v)[32]) {
  for (int w = 0; w < (s.T + 31) / 32; ++w) {
    uint32_t hit = ctl->bad[w] & (m && w < a.words ? __ldg(m + w) : 0u);
    while (hit) {
      const int t = 32 * w + __ffs(hit) - 1;
      hit &= hit - 1;
      const int pos = s.P + t, pidx = pos / a.page_size;
      if (pidx >= s.np) continue;
      const int32_t page = __ldg(a.kv_indices + s.p0 + pidx);
      if (page < 0 || page >= a.num_pages) continue;
      const __nv_bfloat16* src =
          a.v_pool + (((int64_t)page * a.page_size + pos % a.page_size) * a.num_kv_heads + s.h) * D + d0;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float x = __bfloat162float(src[i]);
        if (!(fabsf(x) < INFINITY)) v[i] += x;
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
  const int rt = r / G, g = r - rt * G;  // token of the tile, head of the group
  const bool pos_scale = a.scale_log2 > 0.f;
  const float sc = pos_scale ? a.scale_log2 : 1.f;
  uint32_t used[2] = {0, 0};  // uses of both slots before this segment
  uint32_t vt0 = 0;           // V tiles before this segment
  bool ok = true;

  for (int i = 0; ok; ++i) {
    Seg s;
    if (!next_seg(ctl, i, s)) {
      ok = false;
      break;
    }
    if (s.nq == 0) break;
    const bool two = s.nq == 2;
    const int tok = s.t0 + (two ? slot * a.tpt : 0) + rt;
    const bool valid = r < a.rows_used && tok < s.T;
    const bool warp_live = __any_sync(0xffffffffu, valid);
    const uint32_t* mrow = valid ? a.mask + (int64_t)(s.q0 + tok) * a.words : nullptr;
    float m = -INFINITY, l = 0.f;  // running maximum of the scaled (log2) scores, sum of weights
    uint32_t n_used = used[slot];

    for (int jj = two ? 0 : slot; jj < s.n && ok; jj += two ? 1 : 2, ++n_used) {
      const int pos0 = (s.j0 + jj) * kBN;
      const bool special = pos0 + kBN > s.P;
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl->s_full[slot], n_used & 1));
      if (!ok) break;
      tc_fence_after();
      if (warp_live) {
        uint32_t vis[4];
        float mx = -INFINITY;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          float v[32];
          tmem_ld32(ts + ch * 32, v);
          vis[ch] = special ? visible(mrow, a.words, s.T, pos0 + 32 * ch - s.P) : 0xffffffffu;
          tmem_wait_ld();
          if (!pos_scale) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= a.scale_log2;
          }
          if (special) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (vis[ch] >> e) & 1u ? v[e] : -INFINITY;
          }
          mx = fmaxf(mx, max32(v));
        }
        mx *= sc;
        const float m_new = fmaxf(m, mx);
        // the maximum moves only when it grows by more than 2^8, so that O is seldom rescaled
        const bool resc = m_new > m + 8.f;
        const float m_ref = resc ? m_new : m;
        const float corr = resc ? ex2(m - m_ref) : 1.f;
        const float neg = m_ref == -INFINITY ? 0.f : -m_ref;  // nothing seen so far: every weight is 0
        float tot = 0.f;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          float v[32];
          tmem_ld32(ts + ch * 32, v);
          tmem_wait_ld();
          if (!pos_scale) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= a.scale_log2;
          }
          if (special) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (vis[ch] >> e) & 1u ? v[e] : -INFINITY;
          }
          uint32_t pk[16];
          float t0 = 0.f, t1 = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p0 = ex2(fmaf(v[2 * e], sc, neg)), p1 = ex2(fmaf(v[2 * e + 1], sc, neg));
            t0 += p0;
            t1 += p1;
            pk[e] = pack_bf16x2(p0, p1);
          }
          tot += t0 + t1;
          tmem_st16(ts + ch * 16, pk);  // over scores that are read: P of chunk ch lies in S of chunk ch / 2
        }
        l = l * corr + tot;
        m = m_ref;
        const bool later = two ? jj > 0 : jj > 1;  // O holds earlier tiles (whose PV is done: S was free)
        if (later && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            float o[32];
            tmem_ld32(to + ch * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= corr;
            tmem_st32(to + ch * 32, o);
          }
        }
        tmem_wait_st();
      }
      if (special && (!two || slot == 0)) {  // slot 0's PV of a tile is issued before slot 1's
        const uint32_t vt = vt0 + jj;
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl->v_full[vt % kVStages], (vt / kVStages) & 1));
        if (!ok) break;
        clean_v<D>(smem + C::kOffV + (vt % kVStages) * C::kTile, ctl, s, pos0, r);
        fence_proxy_async_smem();
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
    vt0 += s.n;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (used[k] > 0) ok = ok && __all_sync(0xffffffffu, mbar_wait(&ctl->s_free[k], (used[k] - 1) & 1));
    // the slots' row states change hands (the previous segment's have been read)
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&ctl->x_free, (i & 1) ^ 1));
    if (!ok) break;
    ctl->xm[slot][r] = m;
    ctl->xl[slot][r] = l;
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->x_full);
    ok = __all_sync(0xffffffffu, mbar_wait(&ctl->x_full, i & 1));
    if (!ok) break;
    tc_fence_after();
    const bool any_bad = ctl->bad_any != 0u;
    float f_mine = 1.f, f_other = 0.f, lt = l, mt = m;
    if (!two) {
      const float om = ctl->xm[slot ^ 1][r], ol = ctl->xl[slot ^ 1][r];
      mt = fmaxf(m, om);
      f_mine = m == -INFINITY ? 0.f : ex2(m - mt);
      f_other = om == -INFINITY ? 0.f : ex2(om - mt);
      lt = l * f_mine + ol * f_other;
    }
    const float inv = lt == 0.f ? 0.f : 1.f / lt;
    const float lse_v = (mt + log2f(lt)) * kLn2;
    const int64_t orow = (int64_t)(s.q0 + tok) * a.num_q_heads + (int64_t)s.h * G + g;
    const int prow = (two ? slot * kBM : 0) + r;
    if (warp_live) {
      // two Q tiles: all dims of the thread's own O; one: half of the dims, from both slots' O
      const int c0 = two ? 0 : slot * (D / 64), c1 = two ? D / 32 : c0 + D / 64;
#pragma unroll 1
      for (int ch = c0; ch < c1; ++ch) {
        float o[32];
        tmem_ld32(to + ch * 32, o);
        if (!two) {
          float x[32];
          tmem_ld32(tq + kColO + (slot ^ 1) * 128 + ch * 32, x);
          tmem_wait_ld();
          // a slot that took no tile holds nothing: its factor is 0 and its O is not read
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = (f_mine > 0.f ? o[e] * f_mine : 0.f) + (f_other > 0.f ? x[e] * f_other : 0.f);
        } else {
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = inv == 0.f ? 0.f : o[e] * inv;
        if (valid) {
          if (any_bad) add_nonfinite<D>(a, ctl, s, mrow, ch * 32, o);
          if (s.part < 0) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + orow * D + ch * 32);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              dst[q] = make_uint4(pack_bf16x2(o[8 * q], o[8 * q + 1]), pack_bf16x2(o[8 * q + 2], o[8 * q + 3]),
                                  pack_bf16x2(o[8 * q + 4], o[8 * q + 5]), pack_bf16x2(o[8 * q + 6], o[8 * q + 7]));
          } else {
            float4* dst = reinterpret_cast<float4*>(a.part_o + ((int64_t)s.part * a.part_rows + prow) * D + ch * 32);
#pragma unroll
            for (int q = 0; q < 8; ++q) dst[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          }
        }
      }
      if (valid && (two || slot == 0)) {
        if (s.part >= 0)
          a.part_lse[(int64_t)s.part * a.part_rows + prow] = lse_v;
        else if (a.lse)
          a.lse[orow] = lse_v;
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&ctl->o_free);
      mbar_arrive(&ctl->x_free);
    }
    if (any_bad) {  // the notes are cleared between everyone's last reading and the next segment's first note
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl->x_free, i & 1));
      if (!ok) break;
      if (slot == 0) {
        if (r < kMaxNodes / 32) ctl->bad[r] = 0u;
        if (r == 0) ctl->bad_any = 0u;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
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
      report(a.err_word, PKV_DEVERR_INTERNAL);
      a.cut[blockIdx.x] = Cut{};
    }
    return;
  }
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::kOffCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(&ctl->seg_full[i], 1);
      mbar_init(&ctl->seg_empty[i], 3 + 8);  // V producer, QK, PV, softmax warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], 1);
      mbar_init(&ctl->q_empty[i], 1);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], 4);
      mbar_init(&ctl->s_free[i], 1);
    }
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&ctl->k_full[i], 1);
      mbar_init(&ctl->k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&ctl->v_full[i], 1);
      mbar_init(&ctl->v_empty[i], 1);
    }
    mbar_init(&ctl->o_free, 8);
    mbar_init(&ctl->x_full, 8);
    mbar_init(&ctl->x_free, 8);
    mbar_init(&ctl->qk_done, 1);
    mbar_init(&ctl->pv_done, 1);
    ctl->bad_any = 0u;
    for (int i = 0; i < kMaxNodes / 32; ++i) ctl->bad[i] = 0u;
    fence_mbar_init();
    prefetch_tmap(&a.tm_q);
    prefetch_tmap(&a.tm_k);
    prefetch_tmap(&a.tm_v);
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 0) {
    tree_walk<D, kRows>(a, ctl, sb);
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
    if (lane == 0) {
      if (!tree_mma_pv<D>(ctl, sb, tmem)) report(a.err_word, PKV_DEVERR_TIMEOUT);
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
  // The merge may be scheduled from here on (it waits for this grid's completion before it reads).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------------------------------------
// Merge: block (c, y) joins rows 8y .. 8y + 7 of the unit that CTA c began and did not finish, one
// warp per row.
// ---------------------------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const Cut cut = a.cut[c];
  if (cut.parts <= 0) return;
  const int lane = threadIdx.x & 31;
  const int prow = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int r = prow & (kBM - 1), tile = prow / kBM;
  const int tok = cut.t0 + tile * a.tpt + r / a.group;
  if (tile >= cut.nq || r >= a.rows_used || tok >= cut.T) return;
  constexpr int VPL = D / 32;
  auto slot = [&](int p) -> int64_t { return ((int64_t)2 * (c + p) + (p == 0 ? 1 : 0)) * a.part_rows + prow; };
  float mx = -INFINITY;
  for (int p = lane; p < cut.parts; p += 32) mx = fmaxf(mx, __ldg(a.part_lse + slot(p)));
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
  float acc[VPL] = {};
  float tot = 0.f;
  for (int p0 = 0; p0 < cut.parts; p0 += 32) {
    const int n = min(32, cut.parts - p0);
    const float pl = lane < n ? __ldg(a.part_lse + slot(p0 + lane)) : -INFINITY;
    const float w = pl == -INFINITY ? 0.f : __expf(pl - mx);
    tot += w;
    for (int i0 = 0; i0 < n; i0 += 8) {  // eight partials in flight
      float x[8][VPL];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) x[k][v] = 0.f;
        if (i0 + k < n) {
          const float* src = a.part_o + slot(p0 + i0 + k) * D + lane * VPL;
          if constexpr (VPL == 4)
            *reinterpret_cast<float4*>(x[k]) = __ldg(reinterpret_cast<const float4*>(src));
          else
            *reinterpret_cast<float2*>(x[k]) = __ldg(reinterpret_cast<const float2*>(src));
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, (i0 + k) & 31);
        if (wk != 0.f) {
#pragma unroll
          for (int v = 0; v < VPL; ++v) acc[v] += wk * x[k][v];
        }
      }
    }
  }
  tot = warp_sum(tot);
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  const int64_t orow = (int64_t)(cut.q0 + tok) * a.num_q_heads + (int64_t)cut.h * a.group + r % a.group;
  __nv_bfloat16* op = a.out + orow * D + lane * VPL;
  if constexpr (VPL == 4)
    *reinterpret_cast<uint2*>(op) =
        make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(op) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lane == 0 && a.lse) a.lse[orow] = tot == 0.f ? -INFINITY : mx + logf(tot);
}

// ---------------------------------------------------------------------------------------------
// The mask of a tree given by parents: row i has the bits of i and its ancestors.
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(128) tree_mask_kernel(const int32_t* __restrict__ parents,
                                                        const int32_t* __restrict__ qo_indptr,
                                                        int32_t num_tokens, int32_t words,
                                                        uint32_t* __restrict__ mask, uint32_t* err_word) {
  const int b = blockIdx.y;
  const int32_t q0 = __ldg(qo_indptr + b), rows = __ldg(qo_indptr + b + 1) - q0;
  const bool first = blockIdx.x == 0 && threadIdx.x == 0;
  if (rows < 0 || rows > 32 * words) {
    if (first) report(err_word, PKV_DEVERR_LENGTH);
    if (rows < 0) return;
  }
  if (q0 < 0 || q0 > num_tokens - rows) {
    if (first) report(err_word, PKV_DEVERR_ROW_OOB);
    return;
  }
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= rows || t >= 32 * words) return;
  uint32_t* row = mask + (int64_t)(q0 + t) * words;
  int cur = t;  // strictly falling, so the walk ends
  for (int w = words - 1; w >= 0; --w) {
    uint32_t bits = 0;
    while (cur >= 0 && (cur >> 5) == w) {
      bits |= 1u << (cur & 31);
      const int p = __ldg(parents + q0 + cur);
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
  kern<<<p.ncta, kThreads, smem, st>>>(a);
  const pkv_status s = pkv_host::launch_status();
  if (s != PKV_OK) return s;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.ncta, (unsigned)(p.part_rows / 8), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, a) != cudaSuccess) return PKV_ERR_CUDA;
  return pkv_host::launch_status();
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
  if (!pkv_host::encode_tmap_3d(&a.tm_q, q, D, Hq, (uint64_t)num_q_tokens, Db, Hq * Db, 64, p.G, p.tpt) ||
      !pkv_host::encode_tmap_3d(&a.tm_k, pool->k, D, Hkv, rows, Db, Hkv * Db, 64, 1, a.box_rows) ||
      !pkv_host::encode_tmap_3d(&a.tm_v, pool->v, D, Hkv, rows, Db, Hkv * Db, 64, 1, a.box_rows))
    return PKV_ERR_CUDA;
  a.qo_indptr = qo_indptr;
  a.kv_indptr = kv_indptr;
  a.kv_indices = kv_indices;
  a.prefix_lens = prefix_lens;
  a.mask = (const uint32_t*)tree_mask;
  a.words = mask_words;
  a.k_pool = (const __nv_bfloat16*)pool->k;
  a.v_pool = (const __nv_bfloat16*)pool->v;
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  a.err_word = err_word;
  a.num_pages = pool->num_pages;
  a.page_size = ps;
  a.num_kv_heads = pool->num_kv_heads;
  a.num_q_heads = num_q_heads;
  a.group = p.G;
  a.tpt = p.tpt;
  a.rows_used = p.G * p.tpt;
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
  tree_mask_kernel<<<grid, 128, 0, (cudaStream_t)stream>>>(parents, qo_indptr, num_tokens, mask_words,
                                                           (uint32_t*)tree_mask, err_word);
  return pkv_host::launch_status();
}

}  // extern "C"
