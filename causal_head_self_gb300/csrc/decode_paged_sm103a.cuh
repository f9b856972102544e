// decode_paged_sm103a.cuh -- one decode step over a paged key-value cache, on
// the 5th-generation tensor cores (sm_103a).
//
// For sequence b of L = seqlens[b] keys and query head h of K/V head g,
//   s_t = scale q_h . k_t,  p = softmax over t in [lo, L),  o_h = sum_t p_t v_t,
// with row t of the sequence in page table[b, t / page] at row t % page.  The
// step reads every visible K and V row once for a few FLOPs per byte, so it is
// bound by HBM bandwidth; everything here serves to keep loads in flight.
//
// Work split.  The lengths are known only on the device and differ from
// sequence to sequence, so a split fixed on the host leaves SMs idle.  Instead
// the tiles (kKeys keys) of all units (sequence, K/V head, block of 128 query
// heads) form one line, in unit order, and CTA c of the grid (one per SM) takes
// places [c * share, (c + 1) * share) of it, whatever units they belong to.  A
// unit's first place holds no tile: it stands for the cost of starting and
// ending a unit, about that of a tile, so that a CTA of many short units gets
// fewer keys.  A unit is cut only where a CTA's share ends.  The part of a unit that a
// CTA holds is a segment; the segment of CTA c and unit u has the number u + c
// (along the line one of the two grows from segment to segment, so no two
// share a number), which is its place in the partial results.  A second kernel
// joins the segments of each unit.
//
// Pipeline.  Four warps load (TMA), one issues the tensor-core work, four run
// the softmax.  Q and K tiles pass through one ring of slots (Q, K0, K1, ... of
// each segment), V tiles through another, and the loading warps run ahead into
// the next segments.  Q moves on to tensor memory at once (tcgen05.cp), so its
// slot is soon free again.  A page holds `page` rows of one head in a row,
// so a tile is gathered in boxes of box_rows = gcd(page, kKeys) rows, each of
// them in one page.
//
// Softmax.  A warp reaches only its own 32 lanes (rows) of tensor memory.  A
// group of up to 32 query heads is therefore copied four times into the 128
// rows (REP = 4), and warp w works on keys [w kKeys / 4, (w + 1) kKeys / 4) of
// the tile for its copy, with P = 0 at the other keys: a quarter of the work
// each, and four partial results per segment.  Larger groups use every row
// (REP = 1).
//
// P meets V in bf16, the tensor core's operand type, which alone would cost 2^-8 of
// each weight, as much as the output's own rounding.  A group of up to 16 heads has
// room to spare in its 32 rows: rows 16 .. 31 of a copy hold the same heads again.  The
// first 16 have the upper 16 bits of p, a bf16 number, the others those of what is
// left; the two rows' products add up to those of p to 2^-14.  They are added where
// the partial results are joined.  It costs 1 % of a step (29.9 -> 30.4 us for 8 x 32
// heads of 64; a second product per tile instead, 32.5).  Larger groups round P.
//
// Short form (SHORT).  Where the table has room for few tiles a unit, starting up
// and joining cost more than reading.  A unit then belongs to a cluster of up to
// eight CTAs, each with an equal part of its tiles; the partial results stay in
// shared memory, the CTAs read each other's there, and the step is one launch
// without a workspace (but for the scores, with weights).  One sequence of 1024
// keys with 8 K/V heads: 9.1 -> 7.8 us on the GPU, 21 -> 15 us on the host.
//
// Rows outside [lo, L) are never used: boxes without a visible row are not
// loaded (their table entries may hold anything), scores of invisible rows are
// replaced by -inf, and their V rows are zeroed in shared memory before the
// product (stale rows may hold NaN, and 0 * NaN is NaN).
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>

#include "sm103a_ptx.cuh"

namespace chs {

constexpr int kPagedTwoParts = 16;   // query heads per K/V head with P in two parts, at most

struct DecodePagedParams {
  int B, Hq, Hkv, G, window;
  int num_pages, page, cols;   // pool pages, rows per page, table columns
  int box_rows;                // rows per TMA box
  int row_blocks;              // blocks of 128 query heads per K/V head
  int ctas;                    // CTAs of the grid
  int split;                   // SHORT: CTAs per unit, a cluster
  int score_stride;            // row length of `scores`
  float scale_log2;
  int accumulate;
  const int* seqlens;          // [B], device
  const int* table;            // [B, cols], device
  float* o_part;               // [segments, REP, rows, DH] unnormalised; with up to 16 heads
                               // [segments, 2, REP, rows, DH], from both parts of P
  float* m_part;               // [segments, REP, rows]     (log2 domain)
  float* l_part;               // [segments, REP, rows]
  int2* unit_ctas;             // [units]: first and last CTA of a unit
  float* scores;               // [B, Hq, score_stride] raw q . k, or null
  float* weights;              // [B, Hkv, weights_stride], or null
  int weights_stride;
  __nv_bfloat16* o;            // [B, Hq, 1, DH]
  int* error_word;
  int fault;                   // test hook: 3 = the first K tile is never loaded
};

template <int DH>
struct DecodePagedCfg {
  static constexpr int kKeys = DH <= 128 ? 128 : 64;   // keys per tile
  static constexpr int kBoxes = DH / 64;               // 64-column boxes per row
  static constexpr int kKvBox = kKeys * 128;           // bytes: kKeys rows of 64 columns
  static constexpr int kQBox = 128 * 128;              // bytes: 128 rows of 64 columns
  static constexpr int kSlot = kBoxes * kKvBox;        // ring slot: one K or V tile
  static constexpr int kQSlots = kBoxes * kQBox / kSlot;   // slots that Q takes: 1, at Dh 256 2
  static constexpr int kSlots = 224 * 1024 / kSlot;    // 14 (Dh 64) or 7
  static constexpr int kSlotsV = kSlots / 2, kSlotsK = kSlots - kSlotsV;
  // warps 0-3 softmax, 4 MMA, 5-8 loads
  static constexpr int kThreads = 288;
  static constexpr int kWarpIssuer = 4, kWarpProducer = 5;
  // tensor memory: S0, S1 | Q | O
  static constexpr uint32_t kColQ = DH == 256 ? 128 : 384, kColO = 256, kCols = 512;
  static_assert(2 * kKeys <= 256 && kColO + DH <= (DH == 256 ? 512u : kColQ), "tensor memory");
};

template <int DH>
struct DecodePagedSmem {
  using Cfg = DecodePagedCfg<DH>;
  uint8_t slot[Cfg::kSlots][Cfg::kSlot];
  uint64_t full[Cfg::kSlots], empty[Cfg::kSlots];
  uint64_t s_full[2], p_full[2], pv_done, o_final, qt_free, mma_done;
  uint32_t tmem_base;
  int abort_flag;
};

// Keys that a sequence may hold at most.
__device__ __forceinline__ int paged_rows(const DecodePagedParams& p) { return p.cols * p.page; }

// A sequence's visible keys [lo, L) and its tiles: n of them from tile `first`
// on (tile i holds positions kKeys * i ...).  None for a length of 0 or one
// outside [0, cols * page].
struct PagedSeq {
  int L, lo, first, n;
};
template <int KEYS>
__device__ __forceinline__ PagedSeq paged_seq(const DecodePagedParams& p, int b) {
  PagedSeq s;
  s.L = __ldcg(p.seqlens + b);
  if (s.L < 0 || s.L > paged_rows(p)) s.L = 0;
  s.lo = p.window > 0 ? max(0, s.L - p.window) : 0;
  s.first = s.lo / KEYS;
  s.n = (s.L + KEYS - 1) / KEYS - s.first;
  return s;
}

// One segment: tiles [tile0, tile0 + count) of unit gi (K/V head and row
// block) of sequence b.
struct PagedSegment {
  int b, gi, L, lo, tile0, count;
  bool starts;        // holds the unit's first tile
  int unit, last_cta;
};

// SHORT: the CTA of rank r in its unit's cluster holds a split-th of its tiles.
template <int KEYS>
struct PagedShortWalk {
  int b, gi, from, to;   // tiles [from, to) of the unit's, none once they are taken
  PagedSeq seq;

  __device__ __forceinline__ void init(const DecodePagedParams& p, int cta) {
    const int unit = cta / p.split, rank = cta - unit * p.split;
    b = unit / p.Hkv;
    gi = unit - b * p.Hkv;
    seq = paged_seq<KEYS>(p, b);
    from = seq.n * rank / p.split;   // (a few tiles)
    to = seq.n * (rank + 1) / p.split;
  }

  __device__ __forceinline__ bool next(const DecodePagedParams& p, PagedSegment& s) {
    if (from == to) return false;
    s = {b, gi, seq.L, seq.lo, seq.first + from, to - from, from == 0, b * p.Hkv + gi, 0};
    from = to;
    return true;
  }
};

// The segments of one CTA in order.  Every warp walks them for itself.
template <int KEYS>
struct PagedLineWalk {
  int cur, end, share;   // places on the line
  int b, gi, at;         // next segment: unit and place in it (0: before its tiles)
  PagedSeq seq;

  // places of a unit of n tiles
  static __device__ __forceinline__ int places(int n) { return n > 0 ? n + 1 : 0; }

  // Places [cur, end) of CTA `cta`.  One whole warp.
  __device__ __forceinline__ void init(const DecodePagedParams& p, int cta) {
    const int lane = threadIdx.x % 32;
    const int per_seq = p.Hkv * p.row_blocks;   // units per sequence
    // the first 32 sequences (mostly all of them) are read once and kept
    PagedSeq held = {0, 0, 0, 0};
    if (lane < p.B) held = paged_seq<KEYS>(p, lane);
    int total = places(held.n) * per_seq;
    for (int bb = 32 + lane; bb < p.B; bb += 32) total += places(paged_seq<KEYS>(p, bb).n) * per_seq;
    total = __reduce_add_sync(0xffffffffu, total);
    share = max(1, (total + p.ctas - 1) / p.ctas);
    cur = (int)min((long long)total, (long long)cta * share);
    end = min(total, cur + share);
    b = gi = at = 0;
    if (cur >= end) return;
    int before = 0;   // places of the sequences before b0
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      if (b0 > 0) {
        held = {0, 0, 0, 0};
        if (b0 + lane < p.B) held = paged_seq<KEYS>(p, b0 + lane);
      }
      const int mine = places(held.n) * per_seq;
      int upto = mine;   // inclusive scan
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, before + upto > cur);
      if (past) {
        const int from = __ffs(past) - 1;
        b = b0 + from;
        const int offset = cur - before - __shfl_sync(0xffffffffu, upto - mine, from);
        seq.L = __shfl_sync(0xffffffffu, held.L, from);
        seq.lo = __shfl_sync(0xffffffffu, held.lo, from);
        seq.first = __shfl_sync(0xffffffffu, held.first, from);
        seq.n = __shfl_sync(0xffffffffu, held.n, from);
        gi = offset / places(seq.n);
        at = offset - gi * places(seq.n);
        return;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }

  __device__ __forceinline__ bool next(const DecodePagedParams& p, PagedSegment& s) {
    const int per_seq = p.Hkv * p.row_blocks;
    while (cur < end) {
      if (gi == per_seq) {
        gi = 0;
        do {
          seq = paged_seq<KEYS>(p, ++b);
        } while (seq.n == 0);
      }
      const int take = min(seq.n + 1 - at, end - cur);   // places of this unit
      const int skip = max(at - 1, 0);                   // its tiles before them
      s.b = b;
      s.gi = gi;
      s.L = seq.L;
      s.lo = seq.lo;
      s.tile0 = seq.first + skip;
      s.count = at == 0 ? take - 1 : take;
      s.starts = skip == 0;
      s.unit = b * per_seq + gi;
      s.last_cta = (cur - at + seq.n) / share;           // the CTA of its last tile
      cur += take;
      at += take;
      if (at == seq.n + 1) {
        at = 0;
        ++gi;
      }
      if (s.count > 0) return true;
    }
    return false;
  }
};

template <int KEYS, bool SHORT>
using PagedWalk = std::conditional_t<SHORT, PagedShortWalk<KEYS>, PagedLineWalk<KEYS>>;

// SHORT: one segment's partial results, in the ring's place once nothing of it is
// in use.  Row copy * G + head; four floats more per row keep neighbouring rows in
// different banks.
template <int DH>
struct PagedPart {
  float o[128][DH + 4];         // with up to 16 heads P's second part from row 4 G on
  float m[128], l[128];
  float m_all[32], l_all[32];   // of the four copies together
  float share[32][8];           // [head][CTA]: its part of the head's result
  float top[32], inv[32];
};

// A place in a ring of slots [FIRST, FIRST + N): slot and parity of its current
// use.  Whoever waits on a ring's barriers passes every use of every slot in
// turn, so that it is never more than one phase off and the parity is enough.
template <int FIRST, int N>
struct PagedRing {
  int slot = FIRST;
  uint32_t par = 0;
  __device__ __forceinline__ void step() {
    if (++slot == FIRST + N) {
      slot = FIRST;
      par ^= 1u;
    }
  }
};
template <int DH>
using PagedRingK = PagedRing<0, DecodePagedCfg<DH>::kSlotsK>;
template <int DH>
using PagedRingV = PagedRing<DecodePagedCfg<DH>::kSlotsK, DecodePagedCfg<DH>::kSlotsV>;

// Loading warps: two load Q and K, two V, each (`part`) every other box (64
// columns of box_rows rows; at most 32 per tile: 128 rows / 8 x 2, 64 rows / 8 x
// 4), one lane per box.  A warp takes about 90 cycles to issue one
// copy, so at a page of 16 rows one warp alone is slower than the memory:
// B = 8, 32 heads of 64, 4096 keys ran at 4470 GB/s with one loading warp
// (page 8: 3041).
template <int DH, int REP, bool SHORT, bool V>
__device__ __forceinline__ void decode_paged_producer(DecodePagedSmem<DH>& sm,
                                                      const DecodePagedParams& p,
                                                      const CUtensorMap* map_q,
                                                      const CUtensorMap* map_kv,
                                                      PagedWalk<DecodePagedCfg<DH>::kKeys, SHORT> walk,
                                                      int part, int lane, volatile int* abort) {
  using Cfg = DecodePagedCfg<DH>;
  const uint64_t once = policy_evict_first();   // each cached row is read by one CTA
  const int boxes = Cfg::kKeys / p.box_rows;
  const int mine = 2 * lane + part;   // of the tile's boxes
  const int box = mine % boxes, half = mine / boxes;
  const bool has_box = half < Cfg::kBoxes;
  const int box_bytes = p.box_rows * 128;
  // tiles per group (below), and the table columns and rows of one
  const int group = 32 / boxes;
  const int cols_per_group = group * Cfg::kKeys / p.page;
  const int rows_per_group = group * Cfg::kKeys % p.page;
  const uint32_t dst_off = (uint32_t)(half * Cfg::kKvBox + box * box_bytes);
  std::conditional_t<V, PagedRingV<DH>, PagedRingK<DH>> r;
  uint32_t loaded = 0, pars = 0;
  bool ok = true, first = true;
  auto wait_slot = [&]() -> bool {
    return __all_sync(0xffffffffu, mbar_wait(&sm.empty[r.slot], r.par ^ 1u, abort));
  };
  auto mark_slot = [&] {
    loaded |= 1u << r.slot;
    pars = (pars & ~(1u << r.slot)) | (r.par << r.slot);
    r.step();
  };
  PagedSegment s;
  while (ok && walk.next(p, s)) {
    const int g = s.gi / p.row_blocks, rb = s.gi - g * p.row_blocks;
    if (!SHORT && !V && part == 0 && lane == 0 && s.starts)
      p.unit_ctas[s.unit] = make_int2(blockIdx.x, s.last_cta);
    const int* row = p.table + (size_t)s.b * p.cols;
    // The table is read for `group` tiles at a time, a group ahead: lane l holds
    // the entry of box l % boxes of the group's tile l / boxes.  (Under load an
    // entry takes longer to arrive than a tile takes to load.)
    int pos = (s.tile0 + lane / boxes) * Cfg::kKeys + (lane % boxes) * p.box_rows;
    int col = pos / p.page, c1 = pos - col * p.page;
    const int end = min(s.L, (s.tile0 + s.count) * Cfg::kKeys);
    auto in_use = [&] { return pos < end && pos + p.box_rows > s.lo; };
    bool group_use = in_use();
    int group_c1 = c1, group_id = group_use ? __ldcg(row + col) : 0;
    bool next_use = false;
    int next_c1 = 0, next_id = 0;
    // Q: the group's rows (128, or the 32 that are copied four times on their way to
    // tensor memory), with up to 16 heads twice
    constexpr int kBoxesPerSlot = Cfg::kBoxes / Cfg::kQSlots;
    const int rep = REP == 4 && p.G <= kPagedTwoParts ? 2 : 1, rows = 128 / REP / rep;
    const int copies = kBoxesPerSlot * rep;   // per slot, shared by two warps
    for (int e = 0; !V && ok && e < Cfg::kQSlots; ++e) {
      if (!(ok = wait_slot())) break;
      // (checked builds: query heads of this K/V head)
      const bool in = attn_check(s.b >= 0 && s.b < p.B && g >= 0 && g < p.Hkv && 128 * rb < p.G,
                                 p.error_word);
      if (lane == 0)
        mbar_arrive_expect_tx(&sm.full[r.slot],
                              in ? (copies + 1 - part) / 2 * (rows * 128) : 0);
      __syncwarp();
      if (in && mine < copies) {
        const int bx = mine / rep, copy = mine % rep;
        tma_load_3d(sm.slot[r.slot] + bx * Cfg::kQBox + copy * rows * 128, map_q,
                    &sm.full[r.slot], (e * kBoxesPerSlot + bx) * 64, 128 * rb, s.b * p.Hkv + g);
      }
      mark_slot();
    }
    for (int j = 0; ok && j < s.count; ++j) {
      const int in_group = j & (group - 1);   // (group is a power of two)
      if (in_group == 0) {
        if (j > 0) {
          group_use = next_use;
          group_c1 = next_c1;
          group_id = next_id;
        }
        pos += group * Cfg::kKeys;
        col += cols_per_group;
        c1 += rows_per_group;
        if (c1 >= p.page) {
          c1 -= p.page;
          ++col;
        }
        next_use = in_use();
        next_c1 = c1;
        next_id = next_use ? __ldcg(row + col) : 0;
      }
      const int from = in_group * boxes + box;
      bool load = __shfl_sync(0xffffffffu, (int)group_use, from) != 0 && has_box;
      int id = __shfl_sync(0xffffffffu, group_id, from);
      const int row_in_page = __shfl_sync(0xffffffffu, group_c1, from);
      if (load && (id < 0 || id >= p.num_pages)) {
        atomicExch(p.error_word, 1);   // ATTN_ERR_INVALID_ARG: no such page
        id = 0;
      }
      const int c2 = id * p.Hkv + g;
      // (checked builds: a box lies inside one page of the pool)
      load = load && attn_check(id < p.num_pages && row_in_page >= 0 &&
                                    row_in_page + p.box_rows <= p.page && g < p.Hkv,
                                p.error_word);
      const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, load)) * box_bytes);
      if (!(ok = wait_slot())) break;
      if (!V && first && p.fault == 3) {   // (the test hook withholds one tile)
        r.step();
      } else {
        if (lane == 0) mbar_arrive_expect_tx(&sm.full[r.slot], bytes);
        __syncwarp();
        if (load)
          tma_load_3d_hint(sm.slot[r.slot] + dst_off, map_kv, &sm.full[r.slot], half * 64,
                           row_in_page, c2, once);
        mark_slot();
      }
      first = false;
    }
  }
  // every copy this warp started has landed before the CTA may exit
  if (lane == 0)
    for (int i = 0; i < Cfg::kSlots; ++i)
      if (loaded & (1u << i)) mbar_wait_drain(&sm.full[i], (pars >> i) & 1u);
}

// Tensor-core warp.  Per segment: Q to tensor memory, S of the first two tiles,
// then per tile P.V and the S two tiles on, into the buffer that P came from.
template <int DH, int REP, bool SHORT>
__device__ __forceinline__ void decode_paged_issuer(DecodePagedSmem<DH>& sm,
                                                    const DecodePagedParams& p, uint32_t tbase,
                                                    PagedWalk<DecodePagedCfg<DH>::kKeys, SHORT> walk,
                                                    volatile int* abort) {
  using Cfg = DecodePagedCfg<DH>;
  constexpr uint32_t idesc_qk = idesc_bf16_f32(128, Cfg::kKeys, false, false);
  constexpr uint32_t idesc_pv = idesc_bf16_f32(128, DH, false, true);
  // (a shared address of a cluster's CTA has its rank above the descriptor's bits)
  const uint64_t base = (smem_u32(sm.slot[0]) >> 4) & 0x3FFFu;
  const uint64_t kmajor = smem_desc_sw128(0, 16, 1024) | base;
  const uint64_t mnmajor = smem_desc_sw128(0, Cfg::kKvBox, 1024) | base;
  const uint32_t dO = tbase + Cfg::kColO;
  auto wait = [&](uint64_t* bar, uint32_t par) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, par, abort));
  };
  PagedRingK<DH> rk;               // next Q or K
  PagedRingV<DH> rv;               // next V
  uint32_t t = 0;                  // tiles so far, over all segments
  uint32_t nseg = 0;
  bool ok = true;
  PagedSegment s;
  while (ok && walk.next(p, s)) {
    if (nseg > 0 && !(ok = wait(&sm.qt_free, (nseg - 1) & 1u))) break;
    for (int e = 0; ok && e < Cfg::kQSlots; ++e, rk.step()) {
      if (!(ok = wait(&sm.full[rk.slot], rk.par))) break;
      tc_fence_after_sync();
      constexpr int kSteps = DH / 16 / Cfg::kQSlots;
      const uint64_t q = kmajor + (uint64_t)rk.slot * (Cfg::kSlot >> 4);
#pragma unroll
      for (int kk = 0; kk < kSteps; ++kk) {
        const uint32_t to = tbase + Cfg::kColQ + 8 * (e * kSteps + kk);
        const uint64_t from = q + (((kk / 4) * Cfg::kQBox + (kk % 4) * 32) >> 4);
        if constexpr (REP == 4) {
          tmem_cp_32x128b_x4_warp(to, from);
          tmem_cp_32x128b_x4_warp(to + 4, from + 1);
        } else {
          tmem_cp_128x256b_warp(to, from);
        }
      }
      mma_commit_warp(&sm.empty[rk.slot]);
    }
    if (!ok) break;
    ++nseg;
    auto issue_s = [&](uint32_t tt) -> bool {
      if (!wait(&sm.full[rk.slot], rk.par)) return false;
      tc_fence_after_sync();
      const uint32_t dS = tbase + (uint32_t)Cfg::kKeys * (tt & 1u);
      const uint64_t k = kmajor + (uint64_t)rk.slot * (Cfg::kSlot >> 4);
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk)
        mma_bf16_ts_warp(dS, tbase + Cfg::kColQ + 8 * kk,
                         k + (((kk / 4) * Cfg::kKvBox + (kk % 4) * 32) >> 4), idesc_qk,
                         kk > 0 ? 1u : 0u);
      mma_commit_warp(&sm.s_full[tt & 1u]);
      mma_commit_warp(&sm.empty[rk.slot]);
      rk.step();
      return true;
    };
    if (!(ok = issue_s(t))) break;
    if (s.count > 1 && !(ok = issue_s(t + 1))) break;
    if (s.count <= 2) mma_commit_warp(&sm.qt_free);
    for (int j = 0; j < s.count; ++j, ++t) {
      if (!(ok = wait(&sm.full[rv.slot], rv.par))) break;
      if (!(ok = wait(&sm.p_full[t & 1u], (t >> 1) & 1u))) break;
      tc_fence_after_sync();
      const uint32_t dP = tbase + (uint32_t)Cfg::kKeys * (t & 1u);
      const uint64_t v = mnmajor + (uint64_t)rv.slot * (Cfg::kSlot >> 4);
#pragma unroll
      for (int kk = 0; kk < Cfg::kKeys / 16; ++kk)
        mma_bf16_ts_warp(dO, dP + kk * 8, v + kk * (2048 >> 4), idesc_pv,
                         (j > 0 || kk > 0) ? 1u : 0u);
      mma_commit_warp(&sm.pv_done);
      mma_commit_warp(&sm.empty[rv.slot]);
      rv.step();
      if (j + 2 < s.count) {
        if (!(ok = issue_s(t + 2))) break;
        if (j + 3 == s.count) mma_commit_warp(&sm.qt_free);
      }
    }
    if (ok) mma_commit_warp(&sm.o_final);
  }
  // nothing of this warp's may still run on the tensor core at teardown
  mma_commit_warp(&sm.mma_done);
  mbar_wait_drain(&sm.mma_done, 0);
}

// The bf16 number of x's upper 16 bits: x rounded towards zero.
__device__ __forceinline__ float top_half(float x) {
  return __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}

// Softmax warps: thread t owns row t (tensor-memory lane t).  With REP = 4 row
// 32 w + i is query head i of the block, for the keys of quarter w; with up to 16
// heads rows 32 w + 16 + i are the same, for the rest of P.
template <int DH, int REP, bool SHORT>
__device__ __forceinline__ void decode_paged_softmax(DecodePagedSmem<DH>& sm,
                                                     const DecodePagedParams& p, uint32_t tbase,
                                                     PagedWalk<DecodePagedCfg<DH>::kKeys, SHORT> walk,
                                                     int warp, int lane, int active_warps,
                                                     volatile int* abort) {
  using Cfg = DecodePagedCfg<DH>;
  constexpr int kMine = Cfg::kKeys / REP;             // keys of a tile per warp
  constexpr int kChunk = kMine < 32 ? kMine : 32;     // columns per load
  constexpr int kChunks = kMine / kChunk;
  const int col0 = REP == 4 ? warp * kMine : 0;
  const bool twice = REP == 4 && p.G <= kPagedTwoParts;
  const bool rest = twice && lane >= kPagedTwoParts;
  // in the block of query heads
  const int head = REP != 4 ? warp * 32 + lane : twice ? lane % kPagedTwoParts : lane;
  const float2 part2 = rest ? make_float2(-1.f, -1.f) : make_float2(0.f, 0.f);
  const int copy = REP == 4 ? warp : 0;
  const int tid = warp * 32 + lane;
  const uint32_t lane_addr = tbase + ((uint32_t)(warp * 32) << 16);
  const uint32_t colO = lane_addr + Cfg::kColO;
  const float sl2 = p.scale_log2;
  PagedRingV<DH> r;           // the current tile's V
  uint32_t t = 0;             // tiles so far, over all segments
  uint32_t nseg = 0;
  bool ok = true;
  // the partial results of the segment before: still in tensor memory, m and l here
  bool pending = false, pend_rows = false;
  float pend_m = 0.f, pend_l = 0.f;
  size_t pend_at = 0;
  // a segment's rows: those of m and l, and of O twice as many where P has two parts
  const int part_rows = REP == 4 ? 4 * p.G : 128, pend_row = copy * p.G + head;
  const int rest_rows = rest ? part_rows : 0;
  auto flush = [&]() -> bool {
    // (o_final, not pv_done: two P.V may still be running here, and the parity of
    // a barrier tells only one phase from the next)
    if (!mbar_wait(&sm.o_final, nseg++ & 1u, abort)) return false;
    tc_fence_after_sync();
    PagedPart<DH>& part = *reinterpret_cast<PagedPart<DH>*>(sm.slot[0]);
    float* dst = p.o_part + (twice ? 2 * pend_at - pend_row + rest_rows : pend_at) * DH;
#pragma unroll 1
    for (int c = 0; c < DH / 64; ++c) {
      uint32_t o[2][32];
      tmem_ld_32x32b_x32(colO + 64 * c, o[0]);
      tmem_ld_32x32b_x32(colO + 64 * c + 32, o[1]);
      tmem_ld_wait(o[0]);
      tmem_ld_wait(o[1]);
      if (SHORT && pend_rows) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t* x = &o[e / 8][4 * (e % 8)];
          *reinterpret_cast<uint4*>(&part.o[pend_at + rest_rows][64 * c + 4 * e]) =
              make_uint4(x[0], x[1], x[2], x[3]);
        }
      } else if (pend_rows) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint32_t w8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w8[i] = o[e / 4][8 * (e % 4) + i];
          st_global_v8(dst + 64 * c + 8 * e, w8);
        }
      }
    }
    if (pend_rows && !rest) {
      (SHORT ? part.m : p.m_part)[pend_at] = pend_m;
      (SHORT ? part.l : p.l_part)[pend_at] = pend_l;
    }
    pending = false;
    return true;
  };
  PagedSegment s;
  while (ok && walk.next(p, s)) {
    const int g = s.gi / p.row_blocks, rb = s.gi - g * p.row_blocks;
    const int rows = min(128, p.G - 128 * rb);
    const bool real = head < rows;
    const size_t bh = (size_t)s.b * p.Hq + (size_t)g * p.G + 128 * rb + head;
    float m_run = -INFINITY, l_run = 0.f;
    for (int j = 0; j < s.count; ++j, ++t) {
      const int pos0 = (s.tile0 + j) * Cfg::kKeys;
      const int clo = max(0, s.lo - pos0), chi = min(Cfg::kKeys, s.L - pos0);   // visible columns
      const bool partial = clo > 0 || chi < Cfg::kKeys;
      if (!(ok = mbar_wait(&sm.s_full[t & 1u], (t >> 1) & 1u, abort))) break;
      tc_fence_after_sync();
      const uint32_t colS = lane_addr + (uint32_t)Cfg::kKeys * (t & 1u);
      float x[kMine];
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint32_t y[kChunk];
        if constexpr (kChunk == 32) tmem_ld_32x32b_x32(colS + col0 + 32 * c, y);
        else tmem_ld_32x32b_x16(colS + col0 + 16 * c, y);
        tmem_ld_wait(y);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) x[kChunk * c + e] = __uint_as_float(y[e]);
      }
      if (partial) {
        // invisible keys become -inf, whatever was there
#pragma unroll
        for (int e = 0; e < kMine; ++e)
          x[e] = keep_if_le(x[e], (uint32_t)(col0 + e - clo), (uint32_t)(chi - 1 - clo));
      }
      if (p.scores != nullptr && real && !rest) {
        // raw scores (rows of the buffer are whole tiles, 32-byte aligned)
        float* dst = p.scores + bh * (size_t)p.score_stride + pos0 + col0;
#pragma unroll
        for (int e = 0; e < kMine / 8; ++e) {
          uint32_t w8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w8[i] = __float_as_uint(x[8 * e + i]);
          st_global_v8(dst + 8 * e, w8);
        }
      }
      float mx[2] = {x[0], x[1]};
#pragma unroll
      for (int e = 2; e + 3 < kMine; e += 4) {
        mx[0] = fmax3(mx[0], x[e], x[e + 1]);
        mx[1] = fmax3(mx[1], x[e + 2], x[e + 3]);
      }
      mx[0] = fmax3(mx[0], x[kMine - 2], x[kMine - 1]);
      const float m_tile = fmaxf(mx[0], mx[1]) * sl2;
      // lazy maximum (raised only past +8 in log2 units; exact either way)
      const float m_new = fmaxf(m_run, m_tile);
      const bool fresh = m_run == -INFINITY;
      const bool upd = fresh || (m_new > m_run + 8.0f);
      const float m_use = upd ? m_new : m_run;
      const float corr = (upd && !fresh) ? ex2_approx(m_run - m_new) : 1.0f;
      const float msub = (m_use == -INFINITY) ? 0.f : m_use;
      const float2 scale2 = make_float2(sl2, sl2), neg_m2 = make_float2(-msub, -msub);
      float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      // P in bf16 (both parts of it, or a rounding of 2^-8 relative per weight at most;
      // the sum l is of p itself) over the first kKeys / 2 columns of S, zero at the keys
      // of the other quarters.  Those columns hold scores of this warp's rows only, which
      // are all read by now.
      if constexpr (REP == 4) {
        uint32_t zero[kMine / 2];
#pragma unroll
        for (int e = 0; e < kMine / 2; ++e) zero[e] = 0u;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c == warp) continue;
          if constexpr (kMine == 32) tmem_st_32x32b_x16(colS + 16 * c, zero);
          else tmem_st_32x32b_x8(colS + 8 * c, zero);
        }
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint32_t pk[kChunk / 2];
#pragma unroll
        for (int e = 0; e < kChunk / 2; ++e) {
          const int i = kChunk * c + 2 * e;
          const float2 xs = __ffma2_rn(make_float2(x[i], x[i + 1]), scale2, neg_m2);
          const float2 pp = make_float2(ex2_approx(xs.x), ex2_approx(xs.y));
          ls[e & 1] = __fadd2_rn(ls[e & 1], pp);
          if (twice) {
            const float2 v = __ffma2_rn(make_float2(top_half(pp.x), top_half(pp.y)), part2, pp);
            pk[e] = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
          } else {
            pk[e] = pack_bf16x2(pp.x, pp.y);
          }
        }
        if constexpr (kChunk == 32) tmem_st_32x32b_x16(colS + col0 / 2 + 16 * c, pk);
        else tmem_st_32x32b_x8(colS + col0 / 2 + 8 * c, pk);
      }
      const float lsum = (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
      // a raised maximum rescales the row's O once P.V of the tile before has
      // written it (none before the segment's first tile)
      if (j > 0 && __any_sync(0xffffffffu, corr != 1.0f)) {
        if (!(ok = mbar_wait(&sm.pv_done, (t - 1) & 1u, abort))) break;
        tc_fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < DH / 16; ++c) {
          uint32_t o[16];
          tmem_ld_32x32b_x16(colO + 16 * c, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
          tmem_st_32x32b_x16(colO + 16 * c, o);
        }
      }
      l_run = l_run * corr + lsum;
      m_run = m_use;
      if (partial) {
        // zero the V rows outside [clo, chi): never loaded, or stale.  (A row's
        // 128 bytes per box are swizzled among themselves.)
        if (!(ok = mbar_wait(&sm.full[r.slot], r.par, abort))) break;
        const uint32_t vbase = smem_u32(sm.slot[r.slot]);
        const int out_rows = clo + Cfg::kKeys - chi;
        for (int i = tid; i < out_rows * Cfg::kBoxes * 8; i += 32 * active_warps) {
          const int c16 = i % 8, bx = (i / 8) % Cfg::kBoxes, k = i / (8 * Cfg::kBoxes);
          const int row = k < clo ? k : chi + (k - clo);
          st_shared_v4(vbase + bx * Cfg::kKvBox + row * 128 + c16 * 16, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      // the first P.V of a segment overwrites O, which must have been read out
      if (j == 0 && pending && !(ok = flush())) break;
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(&sm.p_full[t & 1u]);
      r.step();
    }
    if (!ok) break;
    // the segment's results are read out beside the next segment's first tile
    pend_rows = real;
    pend_m = m_run;
    pend_l = l_run;
    pend_at = SHORT ? pend_row : (size_t)(s.unit + blockIdx.x) * part_rows + pend_row;
    pending = true;
  }
  if (ok && pending) {
    flush();
  } else if (SHORT && head < p.G && !rest) {   // no tile: nothing of this CTA's counts
    reinterpret_cast<PagedPart<DH>*>(sm.slot[0])->m[copy * p.G + head] = -INFINITY;
  }
}

// *x in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ float paged_peer(const float* x, int rank) {
  uint32_t at;
  float y;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(x)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(y) : "r"(at) : "memory");
  return y;
}

// SHORT: joins the four copies of this CTA's partial results, into the first.
template <int DH>
__device__ __forceinline__ void decode_paged_short_copies(PagedPart<DH>& part,
                                                          const DecodePagedParams& p) {
  const bool twice = p.G <= kPagedTwoParts;
  for (int i = threadIdx.x; i < p.G * DH; i += DecodePagedCfg<DH>::kThreads) {
    const int h = i / DH, d = i % DH;
    float m[4], lc[4], oc[4], rest[4], M = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {   // (the loads together)
      m[c] = part.m[c * p.G + h];
      lc[c] = part.l[c * p.G + h];
      oc[c] = part.o[c * p.G + h][d];
      rest[c] = twice ? part.o[(4 + c) * p.G + h][d] : 0.f;
      M = fmaxf(M, m[c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // (where the CTA has no tile only m was written)
      const float f = m[c] == -INFINITY ? 0.f : ex2_approx(m[c] - M);
      if (f != 0.f) {
        l = fmaf(f, lc[c], l);
        o = fmaf(f, oc[c] + rest[c], o);
      }
    }
    part.o[h][d] = o;   // (this thread alone reads these columns)
    if (d == 0) {
      part.m_all[h] = M;
      part.l_all[h] = l;
    }
  }
}

// SHORT: joins the unit's partial results (as attn_decode_paged_join does), each
// CTA of the cluster a part of the outputs and, with weights, those of its keys.
template <int DH>
__device__ __forceinline__ void decode_paged_short_join(PagedPart<DH>& part,
                                                        const DecodePagedParams& p) {
  using Cfg = DecodePagedCfg<DH>;
  const int tid = threadIdx.x;
  PagedShortWalk<Cfg::kKeys> walk;
  walk.init(p, blockIdx.x);
  const int rank = (int)blockIdx.x % p.split;
  const size_t bh0 = (size_t)walk.b * p.Hq + (size_t)walk.gi * p.G;   // the unit's first head
  if (walk.seq.n == 0) {
    // no keys: zero; a length that no sequence can have is an error
    if (rank > 0) return;
    for (int i = tid; i < p.G * DH; i += Cfg::kThreads) p.o[bh0 * DH + i] = __float2bfloat16(0.f);
    if (tid == 0 && __ldcg(p.seqlens + walk.b) != 0) atomicExch(p.error_word, 1);   // ATTN_ERR_INVALID_ARG
    return;
  }
  // eight lanes per head, one for each CTA
  const int head = tid / 8, from = tid % 8;
  static_assert(Cfg::kThreads >= 8 * 32, "all heads at once");
  float m = -INFINITY, l = 0.f;
  if (head < p.G && from < p.split) {
    m = paged_peer(&part.m_all[head], from);
    l = paged_peer(&part.l_all[head], from);
  }
  float M = m;
#pragma unroll
  for (int d = 4; d > 0; d /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  const float f = m == -INFINITY ? 0.f : ex2_approx(m - M);
  l *= f;
#pragma unroll
  for (int d = 4; d > 0; d /= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
  if (head < p.G) {
    part.share[head][from] = f / l;
    if (from == 0) {
      part.top[head] = M;
      part.inv[head] = 1.0f / l;
    }
  }
  __syncthreads();
  for (int i = rank * Cfg::kThreads + tid; i < p.G * DH; i += p.split * Cfg::kThreads) {
    const int h = i / DH, d = i % DH;
    float x[8], o = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r] = r < p.split ? paged_peer(&part.o[h][d], r) : 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) o = fmaf(part.share[h][r], x[r], o);
    p.o[bh0 * DH + i] = __float2bfloat16(o);
  }
  if (p.weights == nullptr) return;
  float* out = p.weights + ((size_t)walk.b * p.Hkv + walk.gi) * p.weights_stride;
  const int first = walk.seq.first * Cfg::kKeys;   // of a tile
  const int end = min(walk.seq.L, first + walk.to * Cfg::kKeys);
  for (int t = first + walk.from * Cfg::kKeys + tid; t < end; t += Cfg::kThreads) {
    if (t < walk.seq.lo) continue;
    const float* src = p.scores + bh0 * p.score_stride + t;
    float w = 0.f;
#pragma unroll 4
    for (int h = 0; h < p.G; ++h)
      w = fmaf(ex2_approx(fmaf(__ldcg(src + (size_t)h * p.score_stride), p.scale_log2,
                               -part.top[h])),
               part.inv[h], w);
    out[t] = p.accumulate ? out[t] + w : w;
  }
  if (!p.accumulate && rank == 0)   // keys before the window
    for (int t = tid; t < walk.seq.lo; t += Cfg::kThreads) out[t] = 0.f;
}

template <int DH, int REP, bool SHORT>
__global__ void __launch_bounds__(288, 1)
    attn_decode_paged_sm103a(const __grid_constant__ CUtensorMap map_q,
                             const __grid_constant__ CUtensorMap map_k,
                             const __grid_constant__ CUtensorMap map_v,
                             const DecodePagedParams p) {
  using Cfg = DecodePagedCfg<DH>;
  using Smem = DecodePagedSmem<DH>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~uintptr_t(1023));
  volatile int* abort = &sm.abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int active_warps = REP == 4 ? 4 : (min(128, p.G) + 31) / 32;
  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    for (int i = 0; i < Cfg::kSlots; ++i) {
      mbar_init(&sm.full[i], 2);   // two loading warps
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 32 * active_warps);
    }
    mbar_init(&sm.pv_done, 1);
    mbar_init(&sm.o_final, 1);
    mbar_init(&sm.qt_free, 1);
    mbar_init(&sm.mma_done, 1);
    fence_mbarrier_init();
  }
  if (warp == Cfg::kWarpIssuer) {
    tmem_alloc(&sm.tmem_base, Cfg::kCols);
    tmem_relinquish();
  }
  if (warp == Cfg::kWarpProducer && lane == 0) {
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = sm.tmem_base;
  // the lengths, the table and the cache may come from the previous kernel
  griddep_wait();
  // the join kernel's blocks may be placed beside this grid's (every CTA of
  // which is running by then): they wait for the whole grid, but not for a launch
  if (!SHORT && threadIdx.x == 0) griddep_launch_dependents();
  PagedWalk<Cfg::kKeys, SHORT> walk;
  walk.init(p, blockIdx.x);
  if (warp >= Cfg::kWarpProducer + 2)
    decode_paged_producer<DH, REP, SHORT, true>(sm, p, &map_q, &map_v, walk, warp & 1, lane, abort);
  else if (warp >= Cfg::kWarpProducer)
    decode_paged_producer<DH, REP, SHORT, false>(sm, p, &map_q, &map_k, walk, warp & 1, lane, abort);
  else if (warp == Cfg::kWarpIssuer)
    decode_paged_issuer<DH, REP, SHORT>(sm, p, tbase, walk, abort);
  else if (warp < active_warps)
    decode_paged_softmax<DH, REP, SHORT>(sm, p, tbase, walk, warp, lane, active_warps, abort);
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == Cfg::kWarpIssuer) {
    tc_fence_after_sync();
    tmem_dealloc(tbase, Cfg::kCols);
  }
  if (threadIdx.x == 0 && sm.abort_flag) atomicExch(p.error_word, 4);   // ATTN_ERR_TIMEOUT
  if constexpr (SHORT) {
    // (all waits before this one are bounded, so every thread of the cluster comes here)
    PagedPart<DH>& part = *reinterpret_cast<PagedPart<DH>*>(sm.slot[0]);
    decode_paged_short_copies<DH>(part, p);
    cluster_sync();
    decode_paged_short_join<DH>(part, p);
    cluster_sync();   // no CTA goes while another reads its results
  }
}

// Joins a unit's partial results, in the order of its CTAs and copies:
//   o = sum_i 2^(m_i - M) o_i / l,  l = sum_i 2^(m_i - M) l_i,  M = max m_i.
// Blocks [0, B * Hq) each write one query head's output.  The blocks after
// them, launched when weights are asked for, each write 4 * THREADS of
// the weights of one (sequence, K/V head): sum over the group's heads of
// 2^(s - M) / l, from the scores that the first kernel left.
// TWICE: a segment has twice as many rows of O, the products of P's second part last.
template <int DH, int REP, bool TWICE, int THREADS>
__global__ void __launch_bounds__(THREADS) attn_decode_paged_join(const DecodePagedParams p) {
  constexpr int kKeysPerBlock = 4 * THREADS;
  constexpr int KEYS = DecodePagedCfg<DH>::kKeys;
  const int tid = threadIdx.x;
  const int part_rows = REP == 4 ? p.G : 128;
  griddep_wait();
  if ((int)blockIdx.x < p.B * p.Hq) {
    const int bh = blockIdx.x, b = bh / p.Hq, h = bh - b * p.Hq;
    const int g = h / p.G, hg = h - g * p.G, rb = hg / 128;
    const int unit = (b * p.Hkv + g) * p.row_blocks + rb;
    const int2 ctas = __ldcg(p.unit_ctas + unit);   // (only written for a unit with keys)
    const int L = __ldcg(p.seqlens + b);
    if (L < 1 || L > paged_rows(p)) {
      // no keys: zero; a length that no sequence can have is an error
      for (int d = tid; d < DH; d += THREADS)
        p.o[(size_t)bh * DH + d] = __float2bfloat16(0.f);
      if (L != 0 && tid == 0) atomicExch(p.error_word, 1);   // ATTN_ERR_INVALID_ARG
      return;
    }
    const int n = (ctas.y - ctas.x + 1) * REP;
    const size_t segments0 = (size_t)(unit + ctas.x) * REP * part_rows;
    const size_t at0 = segments0 + (hg - 128 * rb);
    // DH threads hold a row, a column each; the block's groups of them take every
    // kGroups-th partial and are joined in turn
    constexpr int kGroups = THREADS / DH;
    const int group = tid / DH, d = tid % DH;
    // partials per round, their loads in flight together (at Dh = 256, 40 partials: 8
    // 22.7 us, 4 23.1, 16 26.0 for the whole step)
    constexpr int kG = TWICE ? 4 : 8;
    float M = -INFINITY, l = 0.f, o = 0.f;
    for (int i0 = group; i0 < n; i0 += kG * kGroups) {
      float mv[kG], lv[kG], ov[kG], rest[kG];
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        // (past the end the last one again, with the weight 0: a load under a
        // condition is not issued together with the others)
        const int i = i0 + e * kGroups;
        const int k = min(i, n - 1);
        const size_t at = at0 + (size_t)k * part_rows;
        const size_t o_at = TWICE ? segments0 + at + (size_t)(k & ~3) * part_rows : at;
        mv[e] = __ldcg(p.m_part + at);
        lv[e] = __ldcg(p.l_part + at);
        ov[e] = __ldcg(p.o_part + o_at * DH + d);
        rest[e] = TWICE ? __ldcg(p.o_part + (o_at + 4 * part_rows) * DH + d) : 0.f;
        if (i >= n) mv[e] = -INFINITY;
      }
      float Mg = M;
#pragma unroll
      for (int e = 0; e < kG; ++e) Mg = fmaxf(Mg, mv[e]);
      const float f0 = (M == -INFINITY) ? 0.f : ex2_approx(M - Mg);
      l *= f0;
      o *= f0;
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        const float f = (mv[e] == -INFINITY) ? 0.f : ex2_approx(mv[e] - Mg);
        l = fmaf(f, lv[e], l);
        o = fmaf(f, ov[e] + rest[e], o);
      }
      M = Mg;
    }
    if constexpr (kGroups > 1) {
      __shared__ float sh_o[kGroups][DH], sh_M[kGroups], sh_l[kGroups];
      sh_o[group][d] = o;
      if (d == 0) {
        sh_M[group] = M;
        sh_l[group] = l;
      }
      __syncthreads();
      if (group > 0) return;
#pragma unroll
      for (int k = 1; k < kGroups; ++k) M = fmaxf(M, sh_M[k]);
      l = o = 0.f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        const float f = (sh_M[k] == -INFINITY) ? 0.f : ex2_approx(sh_M[k] - M);
        l = fmaf(f, sh_l[k], l);
        o = fmaf(f, sh_o[k][d], o);
      }
    }
    p.o[(size_t)bh * DH + d] = __float2bfloat16(o / l);
    return;
  }
  // weights
  const int T = paged_rows(p);
  const int chunks = (T + kKeysPerBlock - 1) / kKeysPerBlock;
  const int wi = blockIdx.x - p.B * p.Hq;
  const int bg = wi / chunks, chunk = wi - bg * chunks;
  const int b = bg / p.Hkv, g = bg - b * p.Hkv;
  const PagedSeq seq = paged_seq<KEYS>(p, b);
  const int k0 = chunk * kKeysPerBlock;
  if (k0 >= seq.L) return;
  const bool any = k0 + kKeysPerBlock > seq.lo;   // some key of the chunk is visible
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (any) {
    // the heads' maxima and sums, 32 heads at a time (one warp per head)
    __shared__ float sh_m[32], sh_f[32];
    const int warp = tid / 32, lane = tid % 32;
    for (int h0 = 0; h0 < p.G; h0 += 32) {
      const int nh = min(32, p.G - h0);
      __syncthreads();
      for (int i = warp; i < nh; i += THREADS / 32) {
        const int hg = h0 + i, rb = hg / 128;
        const int unit = bg * p.row_blocks + rb;
        const int2 ctas = __ldcg(p.unit_ctas + unit);
        const int n = (ctas.y - ctas.x + 1) * REP;
        const size_t at0 = (size_t)(unit + ctas.x) * REP * part_rows + (hg - 128 * rb);
        float M = -INFINITY, l = 0.f;
        for (int e = lane; e < n; e += 32)
          M = fmaxf(M, __ldcg(p.m_part + at0 + (size_t)e * part_rows));
#pragma unroll
        for (int d = 16; d > 0; d /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        for (int e = lane; e < n; e += 32) {
          const float m = __ldcg(p.m_part + at0 + (size_t)e * part_rows);
          l += (m == -INFINITY) ? 0.f
                                : ex2_approx(m - M) * __ldcg(p.l_part + at0 + (size_t)e * part_rows);
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (lane == 0) {
          sh_m[i] = M;
          sh_f[i] = 1.0f / l;
        }
      }
      __syncthreads();
      const float* src = p.scores + ((size_t)b * p.Hq + (size_t)g * p.G + h0) * p.score_stride +
                         k0 + 4 * tid;
      // (a score row is whole tiles long: the last keys of the chunk may lie past it)
      if (k0 + 4 * tid < seq.L)
#pragma unroll 4
        for (int i = 0; i < nh; ++i) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(src + (size_t)i * p.score_stride));
          const float M = sh_m[i], f = sh_f[i];
          acc[0] = fmaf(ex2_approx(fmaf(x.x, p.scale_log2, -M)), f, acc[0]);
          acc[1] = fmaf(ex2_approx(fmaf(x.y, p.scale_log2, -M)), f, acc[1]);
          acc[2] = fmaf(ex2_approx(fmaf(x.z, p.scale_log2, -M)), f, acc[2]);
          acc[3] = fmaf(ex2_approx(fmaf(x.w, p.scale_log2, -M)), f, acc[3]);
        }
    }
  }
  float* out = p.weights + (size_t)bg * p.weights_stride;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = k0 + 4 * tid + i;
    if (t >= seq.L) break;
    const bool seen = t >= seq.lo;
    if (p.accumulate) {
      if (seen) out[t] += acc[i];
    } else {
      out[t] = seen ? acc[i] : 0.f;
    }
  }
}

template <int DH>
constexpr size_t decode_paged_smem_bytes() {
  static_assert(sizeof(PagedPart<DH>) <= 224 * 1024, "the partial results lie in the ring");
  return sizeof(DecodePagedSmem<DH>) + 1024;   // + alignment slack
}

}  // namespace chs
