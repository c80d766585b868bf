// Paged decode attention over a quantised cache (one query per request): what the 8-bit and the 4-bit kernels
// share, which is all but a consumer warp: its arithmetic on its positions, and the join of the warps of a head, whose states differ.
//
//  * One persistent CTA per SM over an equal share of the stream of slices of 32 positions of all (request,
//    head group) units; one or two producer warps each for K and for V fill a ring of stages, eight or sixteen consumer
//    warps read them, a second kernel merges the units that the shares cut.
//  * K and V come in TMA boxes of 32, 16 or 8 rows (the largest that divides the page size), by copies of single
//    rows for other page sizes.  The scales come into the same stage: by bulk copies beside the boxes where the
//    CTA takes every KV head (a box's lie side by side then) and there are enough of them, by cp.async otherwise.
//
// A format F is a struct with kDim (head_dim), kRowBytes and kScaleBytes (of one head of one position), kWarps
// (consumer warps), kStep (positions of a warp's step), kParts (producer warps each for K and V), kJoint (whether K
// and V share a stage's barriers), kMergeFloats (of a lane's state, see consume), kBoxedRows (whether row copies make boxes of
// 32 rows of a head in the boxes' swizzle, or whole rows kRowPad bytes apart), kScalesAnywhere (whether the pool's scales
// need not be 16-byte aligned), and consume<TMA>, a consumer warp.
#pragma once

#include <atomic>

#include "quant.cuh"
#include "tc05.cuh"

namespace pkv {

constexpr int kSegFirst = 1;    // first stage of this CTA's segment of the unit
constexpr int kSegLast = 2;     // last stage of the segment
constexpr int kStartsUnit = 4;  // the segment starts at position 0 of the unit
constexpr int kEndsUnit = 8;    // the segment ends at the unit's last position

struct StageHdr {
  int32_t unit;  // -1: no more work
  int32_t b, hg, ntok, flags, part;
  int32_t left;  // positions of the segment from this stage on
  int32_t pad;
};

struct QuantDecodeArgs {
  CUtensorMap tm_k;  // pool bytes as (byte of a head, row, head), box [row bytes x box_rows x HC]; TMA instance only
  CUtensorMap tm_v;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  int64_t num_pages;
  int32_t page_size, num_kv_heads;
  FastDiv page_div;  // by page_size
  const __nv_bfloat16* q;
  int32_t batch, num_q_heads;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* kv_lens;
  float scale_log2;
  float out_scale;       // of the values of V, for the whole cache
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
  FastDiv piece_div;     // boxed rows: by the 16-byte pieces of a row of HC heads
  int32_t scale_piece;   // bytes of one copy of a row's scales by a lane: 16, 8 or 4
  int32_t scales_at_16;  // whether k_scale and v_scale are 16-byte aligned, and so the scales of every box
  int32_t pair;          // KV heads side by side in a box's row: 1 or, of 32-byte rows, 2
  uint32_t eight, sixteen;  // shared-memory bytes from positions 0 .. 7 of a slice to the next eight, and to the next sixteen
  int32_t stage_tokens;  // kStep * W
  int32_t num_stages, num_parts;
  uint32_t kv_region;    // bytes of the K (or V) part of one stage
  uint32_t stage_bytes;  // K, V and the scales
};

// No request has more positions than the pool has rows; a longer kv_lens[b] (reported, its pages run
// out) must not take the token counter past 31 bits.
constexpr int kMaxLen = 0x7fff0000;
constexpr int kSlice = 32;  // positions: the unit of the work split
constexpr int kMaxStages = 8;

PKV_DEV void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
PKV_DEV void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
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

// Copies of 32 rows of PIECES 16-byte pieces, HC heads of RH bytes (a power of two of them), and their scales, into the
// places of a box of 32 rows, [head][row] with swizzled pieces, and [row][head].  Lane t has row t's first piece's number in
// the pool in `from` (~0: no row).  Neighbouring lanes copy neighbouring pieces; everything but the row's address is fixed
// when the loop is unrolled (with the general loop below, 64 requests of 1000 to 6000 positions of 32/8 heads of 128 at
// page size 1 took 96 us; 58 now).
template <int RH, int PIECES>
PKV_DEV void copy_round(uint32_t from, const uint8_t* pool, const uint8_t* scale, uint32_t to, uint32_t sto) {
  constexpr int HP = RH / 16, kStep = 32 / PIECES;  // pieces of a head, rows of a round of copies
  const uint32_t lane = threadIdx.x & 31, ch = lane % PIECES, t0 = lane / PIECES, pc = ch % HP;
  const uint8_t* src = pool + ch * 16;
  const uint32_t at = to + ch / HP * (32 * RH) + t0 * RH;
#pragma unroll
  for (int k = 0; k < PIECES; ++k) {
    const uint32_t t = t0 + k * kStep;
    const uint32_t f = __shfl_sync(0xffffffffu, from, t);
    const uint32_t swz = RH == 64 ? pc ^ ((t >> 1) & 3) : pc ^ ((t >> 2) & 1);
    if (f != ~0u) cp_async16(at + k * kStep * RH + swz * 16, src + (uint64_t)f * 16);
  }
  constexpr int kScales = 2 * PIECES, kPiece = kScales < 16 ? kScales : 16, kCount = kScales / kPiece;  // bytes of a row's
  const uint32_t sch = lane % kCount * kPiece, s0 = lane / kCount;
#pragma unroll
  for (int k = 0; k < kCount; ++k) {
    const uint32_t t = s0 + k * (32 / kCount);
    const uint32_t f = __shfl_sync(0xffffffffu, from, t);
    const uint32_t sd = sto + t * kScales + sch;
    const uint8_t* sp = scale + (uint64_t)f * 2 + sch;  // a piece of 32 codes has two scales
    if (f != ~0u) {
      if (kPiece == 16) cp_async16(sd, sp);
      else if (kPiece == 8) cp_async8(sd, sp);
      else cp_async4(sd, sp);
    }
  }
}

// Slices of each of n CTAs, of a stream of T.
PKV_DEV int64_t share_of(int64_t T, uint32_t n) {
  const uint64_t x = (uint64_t)(T + n - 1);
  return max((int64_t)1, (int64_t)(x >> 32 ? x / n : (uint32_t)x / n));
}

// ---------------------------------------------------------------------------------------------
// Producer warps, one for K and one for V: each walks the CTA's share of the slice stream and fills
// its part of the stages; K's also writes the headers.  A stage is a few hundred cycles of address work
// for a warp and about 1400 of memory time, so one warp for both held the stream back (8 x 32768
// positions, D 128: 105 us, 96 with two).
// ---------------------------------------------------------------------------------------------
template <class F, bool TMA>
__device__ void quant_decode_producer(const QuantDecodeArgs& a, uint8_t* stages, StageHdr* hdr, uint64_t* hdr_full,
                                 uint64_t* full, uint64_t* empty, bool v, int part) {
  constexpr int D = F::kDim, RH = F::kRowBytes, SH = F::kScaleBytes;  // bytes of a head's row and of its scales
  constexpr int P = F::kParts;
  const int lane = threadIdx.x & 31;
  const int NS = a.num_stages, Ts = a.stage_tokens, HC = a.HC, nhg = a.nhg;
  const int W = Ts / kSlice;  // rounds of 32 positions
  constexpr bool kManyBoxes = F::kWarps * F::kStep > 256 * P;  // a stage may have more boxes than the tensor's warps have lanes
  const uint32_t region = a.kv_region;
  const CUtensorMap* tm = v ? &a.tm_v : &a.tm_k;
  const uint8_t* pool = v ? a.v_pool : a.k_pool;
  const uint8_t* scale = v ? a.v_scale : a.k_scale;
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
  const int64_t share = share_of(T, gridDim.x);
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
  // boxed rows: the pages of the lane's positions in this warp's next four rounds of 32, and the round behind them
  int32_t p0 = -1, p1 = -1, p2 = -1, p3 = -1;
  int ahead_tok = 0, ahead_round = 0;
  auto ahead_page = [&]() -> int32_t {
    const int32_t page = entry((int)a.page_div.quot((uint32_t)(ahead_tok + 32 * ahead_round + lane)));
    ahead_round += P;
    if (ahead_round >= W) {
      ahead_round = part;
      ahead_tok += Ts;
    }
    return page;
  };
  const FastDiv pieces_div = a.piece_div;
  int nissued = 0;
  auto next_stage = [&]() {
    ++nissued;
    if (++stage == NS) {
      stage = 0;
      phase ^= 1;
    }
  };

  auto emit = [&](int unit, int b, int hg, int tok0, int ntok, int left, int flags) -> bool {
    const bool first = !v && part == 0;  // of the warps: the one that writes headers and reports
    if (unit >= 0 && first && (flags & kSegFirst)) {
      const int hqu = HC * a.group;  // the unit's queries, on their way to L2 before they are read
      const char* qb = reinterpret_cast<const char*>(a.q + ((int64_t)b * a.num_q_heads + (int64_t)hg * hqu) * D);
      for (int off = lane * 128; off < hqu * D * 2; off += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(qb + off));
    }
    if (unit >= 0 && (F::kBoxedRows && !TMA ? false : windowed)) {
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
    if (first && lane == 0) {  // the consumers read the header, and a new unit's queries, while the stage is on its way
      hdr[stage] = StageHdr{unit, b, hg, ntok, flags, (int32_t)blockIdx.x + unit, left, 0};
      mbar_arrive(&hdr_full[stage]);
    }
    if (unit >= 0) {
      uint8_t* dst = stages + (size_t)stage * a.stage_bytes + (v ? region : 0u);
      uint8_t* sdst = stages + (size_t)stage * a.stage_bytes + 2 * region + (v ? (size_t)Ts * HC * SH : 0);
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
      auto copy_piece = [&](uint32_t to, const uint8_t* from) {  // of scales
        if (a.scale_piece == 16) cp_async16(to, from);
        else if (a.scale_piece == 8) cp_async8(to, from);
        else cp_async4(to, from);
      };
      auto copy_scales = [&](int64_t row, int j) {  // token j's scales of HC heads
        const int n = HC * SH;
        const uint8_t* src = scale + (row * a.num_kv_heads + hg * HC) * SH;
        const uint32_t sd = smem_u32(sdst) + (uint32_t)(j * n);
        if (F::kScalesAnywhere) {
          for (int i = 0; i < n; i += a.scale_piece) copy_piece(sd + i, src + i);
        } else if ((n & 15) == 0) {
          for (int i = 0; i < n; i += 16) cp_async16(sd + i, src + i);
        } else {
          for (int i = 0; i < n; i += 4) cp_async4(sd + i, src + i);
        }
      };
      if constexpr (TMA) {
        // Lane i fetches box i, box_rows tokens inside one page, and their scales, which lie side by side when
        // the CTA takes all KV heads.  (One lookup a stage: with one per 32 tokens the eight of a stage of
        // one KV head took 4 us, and 720000 positions of it 96 us; 48 now, of the 28 that their bytes take.)
        // Only boxes of 8 rows in a stage of 1024 positions (one KV head of 64, 4 bits) are more than the two warps' lanes.
        const int sh = 31 - __clz(a.box_rows), nbox = Ts >> sh;
        // Side by side, and enough of them for a bulk copy, which costs about 65 cycles of the copy unit whatever it
        // brings (4 bits: one head of 128 at page size 16, 720000 positions, 36.1 us with copies of 128 bytes and 34.2 with
        // 16 bytes a lane; eight heads of 64, 512000 positions, 62.0 with copies of 512 bytes and 65.1).
        const bool side_by_side =
            nhg == 1 && (!F::kScalesAnywhere || (a.scales_at_16 && (HC * SH << (31 - __clz(a.box_rows))) >= 512));
        const uint32_t box = (uint32_t)(HC * RH) << sh, sbox = (uint32_t)(HC * SH) << sh;
#pragma unroll 1
        for (int i0 = 0; i0 < (kManyBoxes ? nbox : 1); i0 += 32 * P) {
          const int box_i = i0 + P * lane + part, tok = tok0 + (box_i << sh);
          const bool in = box_i < nbox && tok < tok0 + ntok;
          uint32_t pidx, in_page;
          a.page_div.divmod((uint32_t)(in ? tok : tok0), pidx, in_page);
          const int32_t page = windowed ? window_page(pidx) : in ? entry((int)pidx) : -1;
          const int64_t row = row_at(pidx, in_page, page, in);
          const uint32_t n = __popc(__ballot_sync(0xffffffffu, row >= 0));
          if (lane == 0) mbar_expect_tx(bar, n * (box + (side_by_side ? sbox : 0u)));
          __syncwarp();
          if (row >= 0) {
            tma_load_3d(smem_u32(dst) + box_i * box, tm, 0, (int)row, (hg * HC) >> (a.pair - 1), bar);
            if (side_by_side) bulk_g2s(sdst + box_i * sbox, scale + row * a.num_kv_heads * SH, sbox, bar);
          }
          if (!side_by_side) {
            if (F::kScalesAnywhere && nhg == 1 && a.scales_at_16 && (sbox & (sbox - 1)) == 0) {
              // 16 bytes a lane of this warp's boxes' scales
              const int psh = 27 - __clz(sbox), mine = min((nbox - i0 + P - 1) / P, 32);
              for (int r = 0; r < mine << psh; r += 32) {
                const int k = r + lane, bi = k >> psh;
                const int first_row = __shfl_sync(0xffffffffu, (int)row, bi & 31);
                const uint32_t off = (uint32_t)(k & ((1 << psh) - 1)) * 16;
                if (bi < mine && first_row >= 0)
                  cp_async16(smem_u32(sdst) + (i0 + P * bi + part) * sbox + off,
                             scale + (int64_t)first_row * a.num_kv_heads * SH + off);
              }
              continue;
            }
            // lane by lane the rows of this warp's boxes
            const int rounds = kManyBoxes ? min((nbox - i0 + P - 1) / P, 32) << sh : Ts / P;
            for (int r = 0; r < rounds; r += 32) {
              const int k = r + lane, j = (i0 + P * (k >> sh) + part) * a.box_rows + (k & (a.box_rows - 1));
              const int first_row = __shfl_sync(0xffffffffu, (int)row, (k >> sh) & 31);
              if (k < rounds && j < ntok && first_row >= 0) copy_scales(first_row + (k & (a.box_rows - 1)), j);
            }
          }
        }
      } else if constexpr (F::kBoxedRows) {
        // Single rows, 16 bytes a lane, into the places that a box of 32 rows has: [slice][head][row], pieces swizzled.
        constexpr int HP = RH / 16;  // pieces of a head's row
        if (flags & kSegFirst) {
          ahead_tok = tok0;
          ahead_round = part;
          p0 = ahead_page(), p1 = ahead_page(), p2 = ahead_page(), p3 = ahead_page();
        }
        const int pieces = HC * HP, spieces = HC * SH / a.scale_piece;
        // a power of two, and the scales' place allows the pieces that copy_round takes
        const bool native = (pieces & (pieces - 1)) == 0 && a.scale_piece == min(2 * pieces, 16);
        const bool narrow = a.num_pages * a.page_size * (int64_t)(a.num_kv_heads * HP) < 0xffffffffLL;  // 32-bit piece numbers
#pragma unroll 1
        for (int r = part; r < W; r += P) {
          const int j = lane + 32 * r;
          const bool in = j < ntok;
          uint32_t pidx, in_page;
          a.page_div.divmod((uint32_t)(tok0 + (in ? j : 0)), pidx, in_page);
          const int32_t page = p0;
          p0 = p1, p1 = p2, p2 = p3, p3 = ahead_page();
          const int64_t row = row_at(pidx, in_page, page, in);
          const int64_t from = row < 0 ? -1 : row * a.num_kv_heads + hg * HC;  // in heads
          const uint32_t to = smem_u32(dst) + (uint32_t)(r * HC * 32) * RH;
          const uint32_t sto = smem_u32(sdst) + (uint32_t)(r * 32 * HC) * SH;
          if (narrow && native) {
            const uint32_t f = row < 0 ? ~0u : (uint32_t)(from * HP);
            switch (HC) {
              case 1: copy_round<RH, HP>(f, pool, scale, to, sto); break;
              case 2: copy_round<RH, 2 * HP>(f, pool, scale, to, sto); break;
              case 4: copy_round<RH, 4 * HP>(f, pool, scale, to, sto); break;
              default: copy_round<RH, 8 * HP>(f, pool, scale, to, sto);
            }
          } else {
#pragma unroll 4
            for (int it = lane; it < 32 * pieces; it += 32) {
              uint32_t t, ch;
              pieces_div.divmod((uint32_t)it, t, ch);
              const int64_t f = __shfl_sync(0xffffffffu, from, t);
              const uint32_t hd = ch / HP, pc = ch % HP;
              const uint32_t swz = RH == 64 ? pc ^ ((t >> 1) & 3) : pc ^ ((t >> 2) & 1);
              if (f >= 0) cp_async16(to + (hd * 32 + t) * RH + swz * 16, pool + f * RH + ch * 16);
            }
#pragma unroll 1
            for (int it = lane; it < 32 * spieces; it += 32) {
              const uint32_t t = (uint32_t)it / (uint32_t)spieces, ch = (uint32_t)it % (uint32_t)spieces;
              const int64_t f = __shfl_sync(0xffffffffu, from, t);
              if (f >= 0) copy_piece(sto + t * HC * SH + ch * a.scale_piece, scale + f * SH + ch * a.scale_piece);
            }
          }
        }
      } else {
        // One bulk copy per token row, or, for rows of 64 or 128 bytes, 16 bytes a lane: a bulk copy takes
        // about 80 cycles to issue whatever it brings.  24 requests at page size 1, D 128: one KV head and 20000
        // to 40000 positions 162 us so and 200 by bulk copies, two heads and half as many positions
        // (rows of 256 bytes) 144 and 116.  Page indices that are not in the window are loaded four rounds
        // ahead.
        const uint32_t RB = (uint32_t)(HC * RH);
        const bool short_rows = RB <= 128 && (RB & (RB - 1)) == 0;
        const int csh = 27 - __clz(RB);  // log2 of the 16-byte chunks of a short row
        auto ahead = [&](int r) -> int32_t {
          const int j = lane + 32 * r;
          return !windowed && j < ntok ? entry((int)a.page_div.quot((uint32_t)(tok0 + j))) : -1;
        };
        p0 = ahead(0), p1 = ahead(1), p2 = ahead(2), p3 = ahead(3);
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
                cp_async16(to + tk * a.row_stride + ch * 16, pool + (from * a.num_kv_heads + hg * HC) * RH + ch * 16);
            }
            if (row >= 0) copy_scales(row, j);
          } else {
            const uint32_t n = __popc(__ballot_sync(0xffffffffu, row >= 0));
            if (lane == 0) mbar_expect_tx(bar, n * RB);
            __syncwarp();
            if (row >= 0) {
              bulk_g2s(dst + (size_t)j * a.row_stride, pool + (row * a.num_kv_heads + hg * HC) * RH, RB, bar);
              copy_scales(row, j);
            }
          }
        }
      }
      if (bad && !v) report(a.err_word, bad);  // K's warps see every row
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
            ok = emit(bb * nhg + hg, bb, hg, t, min(Ts, t1 - t), t1 - t, flags);
          }
        }
      }
      base += nhg * __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  ok = ok && emit(-1, 0, 0, 0, 0, 0, 0);
  // The merge may be scheduled once every CTA has issued its last copies (it waits for this grid's
  // completion before it reads): early enough to hide its launch, late enough not to hold thread
  // slots that kernels on other streams could use.
  if (!v && part == 0) pdl_trigger();
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

template <class F, bool TMA>
__global__ void __launch_bounds__((F::kWarps + 2 * F::kParts) * 32, 1) quant_decode_kernel(const __grid_constant__ QuantDecodeArgs a) {
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
  uint64_t* empty = full + 2 * NS;  // K's barriers, then V's (joint: those alone)
  uint64_t* meet_bar = empty + 2 * NS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(&hdr_full[s], 1);
    mbar_init(meet_bar, NC);
    for (int s = 0; s < 2 * NS; ++s) {
      mbar_init(&full[s], 33 * F::kParts * (F::kJoint ? 2 : 1));  // each producer's go-ahead, and every lane's copies
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
  if (warp >= NC) {
    const int p = warp - NC;  // K's and V's in turn
    const bool v = p & 1;
    uint64_t *v_full = F::kJoint ? full : full + NS, *v_empty = F::kJoint ? empty : empty + NS;
    // One producer each: the code twice, each for its tensor (8 bits, one KV head at page size 16, 720000 positions: 49.4 us, 51.7
    // with one for both).  Two each: once, since four warps in two copies of it miss the instruction cache (4 bits, 64 requests of
    // 1000 to 6000, 32/8 heads, page size 1: 58 us, 65 with two; 8 of 200 to 900 of one head 8.2, 9.2).
    if constexpr (F::kParts == 1) {
      if (v) quant_decode_producer<F, TMA>(a, stages, hdr, hdr_full, v_full, v_empty, true, 0);
      else quant_decode_producer<F, TMA>(a, stages, hdr, hdr_full, full, empty, false, 0);
    } else {
      quant_decode_producer<F, TMA>(a, stages, hdr, hdr_full, v ? v_full : full, v ? v_empty : empty, v, p >> 1);
    }
  } else {
    F::template consume<TMA>(a, stages, hdr, hdr_full, full, empty, meet_bar);
  }
}

// ---------------------------------------------------------------------------------------------
// Merge of the split partials, a programmatic dependent of the decode kernel: S warps per (unit, query head), each over
// every S-th partial.  Bound by latency, so a warp's loads are issued together, and where a unit can be split
// among 16 CTAs and more eight warps share its partials (4 bits, one request of 4000 positions, 32/8 heads of 128: 8.8 us
// in all with eight, 13.4 with one; 8 requests of 32768: 57.1, 58.3; 8 of 300, which are split less: 8.3, 7.9), else one
// does (16 requests of 16384: 57.7, 59.2 with eight; 64 of 1000: 21.3, 31.1).
// ---------------------------------------------------------------------------------------------
template <class F, int S>
__global__ void __launch_bounds__(256) quant_decode_merge_kernel(const __grid_constant__ QuantDecodeArgs a) {
  constexpr int D = F::kDim;
  constexpr int VPL = D / 32;  // values per lane
  pdl_trigger();
  const int u = blockIdx.x;
  const int b = u / a.nhg, hg = u % a.nhg;
  const int HQU = a.HC * a.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const int part = warp % S;
  const int qhl = (int)blockIdx.y * (8 / S) + warp / S;
  const bool in = qhl < HQU;
  if (S == 1 && !in) return;
  const int64_t row = (int64_t)b * a.num_q_heads + (int64_t)hg * HQU + qhl;
  auto store = [&](const float (&v)[VPL]) {
    __nv_bfloat16* op = a.out + row * D + lane * VPL;
    if constexpr (VPL == 4)
      *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    else
      *reinterpret_cast<uint32_t*>(op) = pack_bf16x2(v[0], v[1]);
  };
  const int len = ld(a.kv_lens + b), first = ld(a.unit_first + u), last = ld(a.unit_last + u);  // in one round of loads
  if (len <= 0) {
    if (blockIdx.y == 0 && threadIdx.x == 0) report(a.err_word, PKV_DEVERR_LENGTH);
    if (in && part == 0) {
      const float zero[VPL] = {};
      store(zero);
      if (lane == 0 && a.lse) a.lse[row] = -INFINITY;
    }
    return;
  }
  if (first == last) return;  // written directly
  if (first < 0 || last >= a.num_parts || last < first) {  // a wait gave up somewhere
    if (lane == 0) report(a.err_word, PKV_DEVERR_TIMEOUT);
    return;
  }
  // One pass: the partials' LSEs (one per lane) and the first sixteen partial rows are loaded together,
  // so up to 16 partials a warp cost one trip to L2; more rescale what they found.
  const float* plse = a.part_lse + qhl;
  const float* po = a.part_o + (int64_t)qhl * D + lane * VPL;
  float mx = -INFINITY, tot = 0.f;
  float acc[VPL] = {};
  for (int base = first + part; in && base <= last; base += 32 * S) {
    const int n = min(32, (last - base) / S + 1);
    const float pl = lane < n ? ld(plse + (int64_t)(base + S * lane) * HQU) : -INFINITY;
    float x[16][VPL];
    auto load = [&](int i0) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float* src = po + (int64_t)(base + S * (i0 + k)) * HQU * D;
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
    const float corr = mx == mn ? 1.f : __expf(mx - mn);  // 0 on the first round
    mx = mn;
    const float w = lane < n && pl != -INFINITY ? __expf(pl - mx) : 0.f;
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
  if constexpr (S > 1) {
    // the first of a head's warps joins them; one without a partial has mx = -inf and sums of 0
    __shared__ float joined[8][2 + VPL][32];
    if (part > 0) {
      joined[warp][0][lane] = mx;
      joined[warp][1][lane] = tot;
#pragma unroll
      for (int v = 0; v < VPL; ++v) joined[warp][2 + v][lane] = acc[v];
    }
    __syncthreads();
    if (part > 0) return;
    float m[S], top = mx;
    m[0] = mx;
#pragma unroll
    for (int w = 1; w < S; ++w) top = fmaxf(top, m[w] = joined[warp + w][0][lane]);
    const float corr = mx == -INFINITY ? 1.f : __expf(mx - top);
    tot *= corr;
#pragma unroll
    for (int v = 0; v < VPL; ++v) acc[v] *= corr;
#pragma unroll
    for (int w = 1; w < S; ++w) {
      const float f = m[w] == -INFINITY ? 1.f : __expf(m[w] - top);
      tot += joined[warp + w][1][lane] * f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) acc[v] += joined[warp + w][2 + v][lane] * f;
    }
    mx = top;
  }
  if (!in) return;
  const float inv = 1.f / tot;
#pragma unroll
  for (int v = 0; v < VPL; ++v) acc[v] *= inv;
  store(acc);
  if (lane == 0 && a.lse) a.lse[row] = mx + logf(tot);
}

// ---------------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------------
struct QuantDecodePlan {
  int HC, nhg, W, G, NT, Ts, RS, R, NS, ncta;
  bool tma;
  uint32_t region, stage;
  size_t smem;
  int64_t nunits, nparts;
  int merge_warps;
  size_t off_first, off_last, off_plse, off_po, ws_bytes;
};

// page_size 0: the workspace's part of the plan only.
template <class F>
bool make_plan(int B, int Hq, int Hkv, int ncta, QuantDecodePlan& p, int page_size = 0, int64_t num_pages = 0) {
  constexpr size_t kSmemBudget = 225 * 1024;
  auto align256 = [](size_t x) { return (x + 255) & ~size_t(255); };
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return false;
  p.G = Hq / Hkv;
  if (p.G > 16) return false;
  p.NT = (p.G + 7) / 8;
  p.HC = 1;
  for (int d = 1; d <= 8 / p.NT; ++d)
    if (Hkv % d == 0) p.HC = d;
  p.nhg = Hkv / p.HC;
  p.W = F::kWarps / (p.HC * p.NT);
  p.Ts = F::kStep * p.W;
  const int RB = p.HC * F::kRowBytes;
  p.RS = RB + F::kRowPad;
  p.R = page_size % 32 == 0 ? 32 : page_size % 16 == 0 ? 16 : 8;
  p.tma = page_size > 0 && page_size % 8 == 0 && num_pages * (int64_t)page_size < 0x7fffffffLL;
  p.region = p.tma ? (uint32_t)(p.Ts * RB) : (uint32_t)(p.Ts * p.RS);
  p.stage = (2 * p.region + (uint32_t)(2 * p.Ts * p.HC * F::kScaleBytes) + 1023u) & ~1023u;
  if (p.W > 1) {
    // the stage carries the merge of a head's warps, at least one of them at a time
    const uint32_t state = (uint32_t)(p.HC * p.NT * F::kMergeFloats * 128);
    if (state > p.stage) p.stage = (state + 1023u) & ~1023u;
  }
  const size_t per_stage = p.stage + sizeof(StageHdr) + 40;
  if (2 * per_stage + 8 > kSmemBudget) return false;
  p.NS = (int)((kSmemBudget - 8) / per_stage);
  if (p.NS > kMaxStages) p.NS = kMaxStages;
  p.smem = (size_t)p.NS * per_stage + 8;
  p.ncta = ncta;
  p.nunits = (int64_t)B * p.nhg;
  p.nparts = p.ncta + p.nunits;
  const int HQU = p.HC * p.G;
  p.merge_warps = p.ncta / 16 >= p.nunits ? 8 : 1;
  p.off_first = 0;
  p.off_last = align256(p.off_first + (size_t)p.nunits * 4);
  p.off_plse = align256(p.off_last + (size_t)p.nunits * 4);
  p.off_po = align256(p.off_plse + (size_t)p.nparts * HQU * 4);
  p.ws_bytes = align256(p.off_po + (size_t)p.nparts * HQU * F::kDim * 4);
  return true;
}

// What a call gives besides the pool.
struct QuantDecodeCall {
  const void* q;
  int32_t batch, num_q_heads;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* kv_lens;
  void* out;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
  uint32_t* err_word;
  int32_t max_ctas;
  cudaStream_t stream;
};

template <class F, bool TMA>
pkv_status launch_quant_decode(const QuantDecodePlan& p, const QuantDecodeArgs& a, cudaStream_t st) {
  auto kern = quant_decode_kernel<F, TMA>;
  // whether this instance's dynamic shared-memory limit was raised on this device (any host thread)
  static std::atomic<bool> configured[64];
  const int dev = pkv_host::current_device();
  if (dev < 0) return PKV_ERR_CUDA;
  if (dev >= 64 || !configured[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess) {
      cudaGetLastError();  // not left for a later call's check to find
      return PKV_ERR_CUDA;
    }
    if (dev < 64) configured[dev].store(true, std::memory_order_relaxed);
  }
  const pkv_status s = pkv_host::launch_after(kern, dim3(p.ncta), (p.HC * p.NT * p.W + 2 * F::kParts) * 32, p.smem, st, a);
  if (s != PKV_OK) return s;
  const dim3 grid((unsigned)p.nunits, (unsigned)((p.HC * p.G * p.merge_warps + 7) / 8));
  if (p.merge_warps == 8) return pkv_host::launch_after(quant_decode_merge_kernel<F, 8>, grid, 256, 0, st, a);
  return pkv_host::launch_after(quant_decode_merge_kernel<F, 1>, grid, 256, 0, st, a);
}

// The checks that the entry points of both formats share, before head_dim chooses the instance.
inline pkv_status check_quant_decode(const QuantDecodeCall& c, int32_t num_kv_heads, int32_t head_dim) {
  if (c.batch < 0 || c.num_q_heads <= 0 || c.max_ctas < 0) return PKV_ERR_INVALID_ARG;
  if (c.batch == 0) return PKV_OK;
  if (!c.q || !c.kv_indptr || !c.kv_indices || !c.kv_lens || !c.out) return PKV_ERR_INVALID_ARG;
  if (!pkv_host::aligned16(c.q) || !pkv_host::aligned16(c.out)) return PKV_ERR_INVALID_ARG;
  if (c.num_q_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  if (c.batch > 0x7fffffff / 64) return PKV_ERR_UNSUPPORTED;
  if ((head_dim != 64 && head_dim != 128) || c.num_q_heads / num_kv_heads > 16) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

// pool: any of the quantised pools; score_scale multiplies q . k, out_scale the result.
template <class F, class Pool>
pkv_status run_quant_decode(const Pool* pool, const QuantDecodeCall& c, float score_scale, float out_scale) {
  int ncta = pkv_host::sm_count();
  if (ncta <= 0) return PKV_ERR_CUDA;
  if (c.max_ctas > 0 && c.max_ctas < ncta) ncta = c.max_ctas;  // fewer partials: the workspace still fits
  QuantDecodePlan p;
  if (!make_plan<F>(c.batch, c.num_q_heads, pool->num_kv_heads, ncta, p, pool->page_size, pool->num_pages))
    return PKV_ERR_UNSUPPORTED;
  if (p.nparts > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;  // 31-bit numbers of units and partials
  if (!c.workspace || c.workspace_bytes < p.ws_bytes) return PKV_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(c.workspace) & 255u) != 0) return PKV_ERR_INVALID_ARG;

  QuantDecodeArgs a;
  a.k_pool = (const uint8_t*)pool->k;
  a.v_pool = (const uint8_t*)pool->v;
  a.k_scale = (const uint8_t*)pool->k_scale;
  a.v_scale = (const uint8_t*)pool->v_scale;
  a.num_pages = pool->num_pages;
  a.page_size = pool->page_size;
  a.page_div = FastDiv((uint32_t)pool->page_size);
  a.num_kv_heads = pool->num_kv_heads;
  a.q = (const __nv_bfloat16*)c.q;
  a.batch = c.batch;
  a.num_q_heads = c.num_q_heads;
  a.kv_indptr = c.kv_indptr;
  a.kv_indices = c.kv_indices;
  a.kv_lens = c.kv_lens;
  a.scale_log2 = score_scale * kLog2e;
  a.out_scale = out_scale;
  a.out = (__nv_bfloat16*)c.out;
  a.lse = c.lse;
  uint8_t* ws = (uint8_t*)c.workspace;
  a.unit_first = (int32_t*)(ws + p.off_first);
  a.unit_last = (int32_t*)(ws + p.off_last);
  a.part_lse = (float*)(ws + p.off_plse);
  a.part_o = (float*)(ws + p.off_po);
  a.err_word = c.err_word;
  a.HC = p.HC;
  a.nhg = p.nhg;
  a.W = p.W;
  a.group = p.G;
  a.nt = p.NT;
  a.box_rows = p.R;
  a.row_stride = p.RS;
  a.piece_div = FastDiv((uint32_t)(p.HC * F::kRowBytes / 16));
  // a piece divides a row's scales and the addresses of all of them
  const uintptr_t places = (uintptr_t)pool->k_scale | (uintptr_t)pool->v_scale;
  const uintptr_t pieces = places | (uintptr_t)(p.HC * F::kScaleBytes);
  if (pieces & 3) return PKV_ERR_INVALID_ARG;
  a.scale_piece = pieces % 16 == 0 ? 16 : pieces % 8 == 0 ? 8 : 4;
  a.scales_at_16 = places % 16 == 0;
  if (!p.tma && F::kBoxedRows) p.R = a.box_rows = kSlice;
  const bool boxed = p.tma || F::kBoxedRows;
  // The copy unit takes a box row by row: rows of 64 bytes, two heads' codes, where the heads pair up (16 requests of 32000
  // positions, 16/8 heads of 64, 4 bits, page size 16: 67 us with rows of 32 bytes, 63 so; page size 32: 62 and 61).
  const int pair = p.tma && F::kRowBytes == 32 && p.HC % 2 == 0 ? 2 : 1;
  a.pair = pair;
  a.eight = boxed ? (uint32_t)(8 * F::kRowBytes * (p.R == 8 ? p.HC : pair)) : (uint32_t)(8 * p.RS);
  a.sixteen = boxed ? (uint32_t)(16 * F::kRowBytes * (p.R <= 16 ? p.HC : pair)) : (uint32_t)(16 * p.RS);
  a.stage_tokens = p.Ts;
  a.num_stages = p.NS;
  a.num_parts = (int32_t)p.nparts;
  a.kv_region = p.region;
  a.stage_bytes = p.stage;
  if (p.tma) {
    const uint64_t Hkv = pool->num_kv_heads / pair, RH = F::kRowBytes * pair;
    const uint64_t rows = (uint64_t)pool->num_pages * pool->page_size;
    if (!pkv_host::encode_tmap_3d_u8(&a.tm_k, pool->k, RH, rows, Hkv, Hkv * RH, RH, RH, p.R, p.HC / pair) ||
        !pkv_host::encode_tmap_3d_u8(&a.tm_v, pool->v, RH, rows, Hkv, Hkv * RH, RH, RH, p.R, p.HC / pair))
      return PKV_ERR_CUDA;
  }
  return p.tma ? launch_quant_decode<F, true>(p, a, c.stream) : launch_quant_decode<F, false>(p, a, c.stream);
}

template <class F>
size_t quant_decode_workspace(int32_t batch_size, int32_t num_q_heads, int32_t num_kv_heads) {
  QuantDecodePlan p;
  const int n = pkv_host::sm_count();
  if (n <= 0 || !make_plan<F>(batch_size, num_q_heads, num_kv_heads, n, p)) return 0;
  return p.ws_bytes;
}

}  // namespace pkv
