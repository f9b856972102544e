// key_weights_sm103a.cuh -- the attention weight that each key of a prompt
// received (sm_103a).
//
//   w[b, g, j] (+)= sum over the query heads h of K/V head g and the voting
//                   queries i that see key j of  exp(scale q_hi . k_j - lse_hi)
//
// with lse the log-sum-exps of the forward pass.  The voting queries are the
// last `queries` of the sequence (all of them when 0).  This is the column sum
// of the probability matrix, which is recomputed tile by tile and never stored:
// 2 Dh FLOPs per visible pair on the tensor cores and one exponential, so the
// kernel is bound by those two, which run side by side.
//
// An item is 128 keys of one (sequence, K/V head) with the tiles of 128 queries
// that see any of them, head after head.  The product is taken transposed,
// S^T = K Q^T (keys as rows): a thread then owns a key, and the sum over
// queries stays in its registers -- no atomics, no shuffles, and the same bits
// every time.  With few voting queries a tile holds those of several heads (`pad`
// columns each).
//
// The log-sum-exps enter through the product too: one more step of 16 columns
// multiplies ones (in tensor memory, where K is) with -lse / scale, split into
// three bf16 parts that together hold its 24 bits.  It comes last, so only its own
// addition rounds at the size of lse / scale: 2^-24 |lse| on the exponent, what a
// subtraction in 32 bits costs as well.  Read from shared memory by the summing
// warps instead (as broadcasts, 512 bytes for four columns and warp), the
// log-sum-exps kept shared memory, which feeds the MMAs, busy for 512 cycles a
// tile.
//
// One CTA per SM: one warp loads K and Q tiles through a ring (TMA), one issues
// the tensor-core work, and two groups of four warps take turns at the tiles.
// Everything that the summing warps have to know of a tile is prepared for them
// by a warp per group, with the log-sum-exps: eight warps would each pay for
// working it out, and instructions are what this kernel runs short of (a tile
// costs a scheduler 290 of them for the sums alone, beside 512 cycles of
// exponentials).  K goes to tensor memory once per item (tcgen05.cp), so that the
// MMAs stream only Q from shared memory; three S buffers keep the tensor core
// ahead.  At the end of an item the two groups' sums are added.
//
// With enough items the CTAs walk them, heaviest first (`split` = 1).  Few and
// long items (few K/V heads, short prompts) are each shared by a cluster of
// `split` CTAs, which take equal parts of its tiles; their sums meet in the
// first one's shared memory and are added in order.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "fixed_div.h"
#include "sm103a_ptx.cuh"

namespace chs {

struct KeyWeightsParams {
  int B, Hq, Hkv, G, S;
  int causal, window, queries, accumulate;
  int items;             // key blocks * B * Hkv
  FixedDiv by_heads, by_batch;   // by Hkv, by B * Hkv
  int pad;               // columns of a tile per head: 128, or less with few voting queries
  int head_tiles;        // tiles that the group's heads take, `pad` columns each
  int split, split_log2; // CTAs per item, a power of two
  float scale_log2;
  float lse_hi, lse_lo;  // -log2(e) / scale_log2 in two parts
  const float* lse;      // [B, Hq, S]
  const int* seqlens;    // [B] or null (every sequence holds S)
  float* weights;        // [B, Hkv, stride]
  int stride;
  int* error_word;
};

template <int DH>
struct KeyWeightsCfg {
  static constexpr int kBoxes = DH / 64;
  static constexpr int kBox = 128 * 128;              // bytes: 128 rows of 64 columns
  static constexpr int kTile = kBoxes * kBox;         // ring slot: a K or Q tile
  static constexpr int kSlots = DH == 64 ? 8 : DH == 128 ? 6 : 3;
  static constexpr int kBuffers = DH == 256 ? 2 : 3;  // S
  static constexpr int kLse = 4;                      // entries per group
  static constexpr int kHand = 8;                     // hand-over buffers
  // tensor memory: S buffers | K | ones
  static constexpr uint32_t kColK = 128 * kBuffers, kColOne = kColK + DH / 2, kCols = 512;
  static_assert(kColOne + 8 <= kCols, "tensor memory");
  // warps 0-7 sums, 8 MMA, 9 K and Q, 10 and 11 entries
  static constexpr int kThreads = 384;
  static constexpr int kWarpIssuer = 8, kWarpProducer = 9, kWarpLse = 10;
  static constexpr int kLseAhead = 2;                 // entries per warp on the way
  static constexpr int kMaxSplit = 8;
  static constexpr int kLens = 256;                   // lengths kept in shared memory
};

// What the summing warps have to know of a tile.  Column c of a tile is visible
// to key k0 + t where max(0, lo + t) <= c mod pad < min(end, hi + t) and
// c < cols.
struct __align__(16) KeyWeightsEntry {
  int flags;            // of kKw...
  int lo, hi, end;
  long long out;        // the item's first key in `weights`
  int rows;             // its keys
  int cols;
};
constexpr int kKwWhole = 1;    // every column is visible to every key
constexpr int kKwNone = 2;     // no tile: an item whose keys no query of this CTA sees
constexpr int kKwLast = 4;     // this group's last tile of the item
constexpr int kKwFinish = 8;   // ... and the item's: this group writes the sums
constexpr int kKwPair = 16;    // the other group has tiles of the item too
constexpr int kKwEnd = 32;     // nothing follows
// S buffer (2 bits) and its parity, hand-over buffer (3 bits) and its parity
constexpr int kKwS = 8, kKwSPar = 10, kKwHand = 12, kKwHandPar = 15;

template <int DH>
struct KeyWeightsSmem {
  using Cfg = KeyWeightsCfg<DH>;
  uint8_t slot[Cfg::kSlots][Cfg::kTile];
  // three bf16 parts per column and five zeros: the first eight of the step's 16
  // columns (8-row core matrices, one after another)
  uint4 nlse[2][Cfg::kLse][128];
  uint4 zero[128];                           // its second eight, of every entry
  KeyWeightsEntry entry[2][Cfg::kLse];
  float hand[Cfg::kHand][128];               // one group's sums for the other
  float parts[Cfg::kMaxSplit][128];          // the cluster's sums (first CTA)
  uint64_t full[Cfg::kSlots], empty[Cfg::kSlots];
  uint64_t l_full[2][Cfg::kLse], l_empty[2][Cfg::kLse];
  uint64_t s_full[Cfg::kBuffers], s_empty[Cfg::kBuffers];
  uint64_t hand_full[Cfg::kHand], hand_empty[Cfg::kHand];
  uint64_t k_free, mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int lens[Cfg::kLens];
};

// The work of one CTA on one item: tiles [t0, t1).  Tile t holds, with pad =
// 128, queries q0 + 128 (t % n) ... of head t / n; otherwise queries q0 ... of
// heads (128 / pad) t ....
struct KeyWeightsItem {
  int b, g, k0, L, q0, q_end, n, t0, t1;
};

// `lens`: the lengths of the first KeyWeightsCfg::kLens sequences.
__device__ __forceinline__ int key_weights_len(const KeyWeightsParams& p, int b) {
  const int n = p.seqlens ? __ldcg(p.seqlens + b) : p.S;
  return n < 0 || n > p.S ? 0 : n;
}

template <int LENS>
__device__ __forceinline__ KeyWeightsItem key_weights_item(const KeyWeightsParams& p,
                                                           const int (&lens)[LENS], int item,
                                                           int rank) {
  KeyWeightsItem it;
  const int kb = p.by_batch.div(item);   // the first key blocks have the most queries: first
  const int bg = p.by_batch.mod(item);
  it.b = p.by_heads.div(bg);
  it.g = p.by_heads.mod(bg);
  it.L = it.b < LENS ? lens[it.b] : key_weights_len(p, it.b);
  it.k0 = 128 * kb;
  it.q0 = p.queries > 0 ? max(0, it.L - p.queries) : 0;
  if (p.causal) it.q0 = max(it.q0, it.k0);
  it.q_end = it.L;
  if (p.window > 0) it.q_end = (int)min((long long)it.L, (long long)it.k0 + 127 + p.window);
  it.n = it.q_end > it.q0 && it.k0 < it.L ? (it.q_end - it.q0 + 127) / 128 : 0;
  int tiles = it.n * p.G;
  if (p.pad < 128 && tiles > 0) tiles = p.head_tiles;
  // (split is a power of two)
  it.t0 = (int)((long long)tiles * rank >> p.split_log2);
  it.t1 = (int)((long long)tiles * (rank + 1) >> p.split_log2);
  return it;
}

// Item `i` of a CTA (items or more: none).  Walking CTAs go through the items
// forwards and backwards in turn, so that who had a heavy one gets a light one.
__device__ __forceinline__ int key_weights_cta_item(const KeyWeightsParams& p, int i) {
  if (p.split > 1) return i == 0 ? (int)blockIdx.x / p.split : p.items;
  const int G = gridDim.x, c = blockIdx.x;
  return i * G + ((i & 1) ? G - 1 - c : c);
}

// Walks the tiles of an item: the head and query of a tile's first column.
struct KeyWeightsTile {
  int head, query;
  __device__ __forceinline__ KeyWeightsTile(const KeyWeightsParams& p, const KeyWeightsItem& it) {
    if (p.pad == 128) {
      head = it.t0 < it.n ? 0 : it.t0 / it.n;
      query = it.q0 + 128 * (it.t0 - head * it.n);
    } else {
      head = (128 / p.pad) * it.t0;
      query = it.q0;
    }
  }
  __device__ __forceinline__ void step(const KeyWeightsParams& p, const KeyWeightsItem& it) {
    if (p.pad == 128) {
      query += 128;
      if (query >= it.q_end) {
        query = it.q0;
        ++head;
      }
    } else {
      head += 128 / p.pad;
    }
  }
};

// Position in a ring of N: index and the parity of its current use.  Whoever
// waits on a ring's barriers passes every use in turn, or can tell otherwise that
// the use before is over: the parity tells only one phase from the next.
template <int N>
struct KwRing {
  int i = 0;
  uint32_t par = 0;
  __device__ __forceinline__ void step() {
    if (++i == N) {
      i = 0;
      par ^= 1u;
    }
  }
};

// A log-sum-exp's eight columns of the extra step: -lse / scale to more than 32 bits in
// three bf16 parts, and zeros.  An infinite one is its first part alone (the others would
// be NaN): a row with lse = +inf then weighs exp(s - inf) = 0, as the definition has it.
__device__ __forceinline__ uint4 key_weights_lse_parts(float lse, float hi, float lo) {
  const float v = lse * hi;
  const float rest = fmaf(lse, hi, -v) + lse * lo;
  const float a = __bfloat162float(__float2bfloat16_rn(v));
  const float b = __bfloat162float(__float2bfloat16_rn(v - a));
  const bool whole = isinf(a);
  return make_uint4(pack_bf16x2(a, whole ? 0.f : b),
                    whole ? 0u : pack_bf16x2((v - a - b) + rest, 0.f), 0u, 0u);
}

template <int DH>
__device__ __forceinline__ void key_weights_producer(KeyWeightsSmem<DH>& sm,
                                                     const KeyWeightsParams& p,
                                                     const CUtensorMap* map_q,
                                                     const CUtensorMap* map_k, int rank, int lane,
                                                     volatile int* abort) {
  using Cfg = KeyWeightsCfg<DH>;
  KwRing<Cfg::kSlots> r;
  uint32_t loaded = 0, pars = 0;
  bool ok = true;
  auto wait_slot = [&]() -> bool {
    return __all_sync(0xffffffffu, mbar_wait(&sm.empty[r.i], r.par ^ 1u, abort));
  };
  auto mark_slot = [&] {
    loaded |= 1u << r.i;
    pars = (pars & ~(1u << r.i)) | (r.par << r.i);
    r.step();
  };
  const int heads_per_tile = 128 / p.pad;
  const int box_bytes = p.pad * 128;
  for (int i = 0; ok; ++i) {
    const int item = key_weights_cta_item(p, i);
    if (item >= p.items) break;
    const KeyWeightsItem it = key_weights_item(p, sm.lens, item, rank);
    if (it.t0 >= it.t1) continue;
    if (!(ok = wait_slot())) break;
    // (checked builds: key rows of a K/V head)
    const bool head_in = attn_check(it.b >= 0 && it.b < p.B && it.g >= 0 && it.g < p.Hkv,
                                    p.error_word);
    if (lane == 0) {
      const bool in = attn_check(it.k0 >= 0 && it.k0 < p.S, p.error_word) && head_in;
      mbar_arrive_expect_tx(&sm.full[r.i], in ? Cfg::kTile : 0);
      if (in) tma_load_4d(sm.slot[r.i], map_k, &sm.full[r.i], 0, it.k0, 0, it.b * p.Hkv + it.g);
    }
    mark_slot();
    KeyWeightsTile at(p, it);
    for (int t = it.t0; t < it.t1; ++t, at.step(p, it)) {
      if (!(ok = wait_slot())) break;
      if (lane == 0) {
        const int heads = min(heads_per_tile, p.G - at.head);
        // (checked builds: query rows of the group's heads)
        const bool in = attn_check(at.query >= 0 && at.query < p.S && at.head >= 0 && heads > 0,
                                   p.error_word) && head_in;
        mbar_arrive_expect_tx(&sm.full[r.i], in ? heads * Cfg::kBoxes * box_bytes : 0);
        if (p.pad == 128) {
          if (in)
            tma_load_4d(sm.slot[r.i], map_q, &sm.full[r.i], 0, at.query, 0,
                        it.b * p.Hq + it.g * p.G + at.head);
        } else {   // (a copy of whole rows would put a head's 64-column boxes together)
          for (int h = 0; in && h < heads; ++h)
            for (int b = 0; b < Cfg::kBoxes; ++b)
              tma_load_3d(sm.slot[r.i] + b * Cfg::kBox + h * box_bytes, map_q, &sm.full[r.i],
                          64 * b, at.query, it.b * p.Hq + it.g * p.G + at.head + h);
        }
      }
      mark_slot();
    }
  }
  // every copy this warp started has landed before the CTA may exit
  if (lane == 0)
    for (int i = 0; i < Cfg::kSlots; ++i)
      if (loaded & (1u << i)) mbar_wait_drain(&sm.full[i], (pars >> i) & 1u);
}

// The entries of one group: its tiles' descriptions and log-sum-exps (0 where
// there is no voting query: such a column is masked).  The tiles of all items are
// dealt to the groups in turn.  kLseAhead of them are on the way at any time,
// since a load takes longer than a tile.
template <int DH>
__device__ __forceinline__ void key_weights_lse(KeyWeightsSmem<DH>& sm, const KeyWeightsParams& p,
                                                int rank, int group, int lane,
                                                volatile int* abort) {
  using Cfg = KeyWeightsCfg<DH>;
  constexpr int D = Cfg::kLseAhead;
  float x[D][4];
  int flags[D], lo[D], hi[D], end[D], cols[D], rows[D];
  long long out[D];
  KwRing<Cfg::kLse> l;
  // where the walk stands: the item and this group's next tile t in it, which
  // begins at tile `part` of n of head block `head`
  int i = -1, t = 0, n = 1, head = 0, part = 0;
  uint32_t before = 0, pairs = 0;   // tiles and shared items before the item
  KeyWeightsItem it;
  it.t0 = it.t1 = 0;
  it.k0 = it.L = it.q_end = it.q0 = it.b = it.g = 0;
  const float* base = p.lse;        // the item's first head
  const int heads_per_tile = 128 / p.pad;
  int col_query[4];                 // this lane's columns: query, place from the tile's first
  long long col_at[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    col_query[k] = (32 * k + lane) % p.pad;
    col_at[k] = (long long)((32 * k + lane) / p.pad) * p.S + col_query[k];
  }
  auto fetch = [&](float (&y)[4], int& f, int& e_lo, int& e_hi, int& e_end, int& e_cols,
                   int& e_rows, long long& e_out) {
    while (t >= it.t1) {   // the next item with a tile for this group
      before += (uint32_t)(it.t1 - it.t0);
      pairs += it.t1 - it.t0 > 1 ? 1 : 0;
      do {
        const int item = key_weights_cta_item(p, ++i);
        if (item >= p.items) {
          f = kKwEnd;
          return;
        }
        it = key_weights_item(p, sm.lens, item, rank);
      } while (it.k0 >= it.L);
      t = it.t0 + (int)((before ^ (uint32_t)group) & 1u);
      n = p.pad == 128 ? it.n : 1;
      head = t < n ? 0 : n == 1 ? t : t / n;
      part = t - head * n;
      base = p.lse + ((size_t)it.b * p.Hq + it.g * p.G) * p.S;
      if (it.t0 == it.t1 && t == it.t0) {   // no query sees its keys
        f = kKwNone | kKwLast | kKwFinish;
        e_rows = it.L - it.k0;
        e_out = ((long long)it.b * p.Hkv + it.g) * p.stride + it.k0;
        return;   // (t >= t1: the next call goes on)
      }
    }
    const int query = it.q0 + 128 * part, first = head * heads_per_tile;
    const int c0 = it.k0 - query;   // (window: columns below c0 + t + window)
    e_lo = p.causal ? c0 : -(1 << 30);
    e_hi = p.window > 0 && p.window < 128 - c0 ? c0 + p.window : 128;
    e_end = min(it.q_end - query, p.pad);
    e_cols = min(heads_per_tile, p.G - first) * p.pad;   // of heads that there are
    const uint32_t tile = before + (uint32_t)(t - it.t0), use = tile / Cfg::kBuffers;
    f = (it.t1 - it.t0 > 1 ? kKwPair : 0) |
        (e_lo <= -127 && e_hi >= p.pad && e_end == p.pad && e_cols == 128 ? kKwWhole : 0) |
        ((int)(tile - use * Cfg::kBuffers) << kKwS) | ((int)(use & 1u) << kKwSPar) |
        ((int)(pairs % Cfg::kHand) << kKwHand) | ((int)(pairs / Cfg::kHand & 1u) << kKwHandPar);
    if (t + 2 >= it.t1) f |= kKwLast;
    if (t + 1 >= it.t1) {
      f |= kKwFinish;
      e_rows = it.L - it.k0;
      e_out = ((long long)it.b * p.Hkv + it.g) * p.stride + it.k0;
    }
    const float* src = base + (size_t)first * p.S + query;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      y[k] = col_query[k] < e_end && 32 * k + lane < e_cols ? __ldcg(src + col_at[k]) : 0.f;
    t += 2;
    for (part += 2; part >= n; part -= n) ++head;
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    fetch(x[d], flags[d], lo[d], hi[d], end[d], cols[d], rows[d], out[d]);
  for (;;) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.l_empty[group][l.i], l.par ^ 1u, abort))) return;
      if (!(flags[d] & (kKwNone | kKwEnd))) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          sm.nlse[group][l.i][32 * k + lane] = key_weights_lse_parts(x[d][k], p.lse_hi, p.lse_lo);
        fence_proxy_async_smem();   // (the MMA reads them)
      }
      if (lane == 0)
        sm.entry[group][l.i] =
            KeyWeightsEntry{flags[d], lo[d], hi[d], end[d], out[d], rows[d], cols[d]};
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.l_full[group][l.i]);
      l.step();
      if (flags[d] & kKwEnd) return;
      fetch(x[d], flags[d], lo[d], hi[d], end[d], cols[d], rows[d], out[d]);
    }
  }
}

template <int DH>
__device__ __forceinline__ void key_weights_issuer(KeyWeightsSmem<DH>& sm,
                                                   const KeyWeightsParams& p, uint32_t tbase,
                                                   int rank, int lane, volatile int* abort) {
  using Cfg = KeyWeightsCfg<DH>;
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
  const uint64_t desc = smem_desc_sw128(smem_u32(sm.slot[0]), 16, 1024);
  auto wait = [&](uint64_t* bar, uint32_t par) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, par, abort));
  };
  // the log-sum-exps' step: no swizzle, core matrices of 8 rows of 16 bytes
  // 128 bytes apart; the second eight columns, which meet zeros too, lie apart (the
  // first again would do but for infinite ones: 0 * inf is NaN)
  const uint64_t plain = ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
  const uint32_t zero = smem_u32(sm.zero);
  KwRing<Cfg::kSlots> r;
  KwRing<Cfg::kBuffers> s;
  KwRing<Cfg::kLse> l0, l1;   // the groups' entries
  uint32_t done = 0;    // items begun
  uint32_t group = 0;   // whose tile is next
  auto wait_entry = [&]() -> bool {
    return wait(&sm.l_full[group][group ? l1.i : l0.i], group ? l1.par : l0.par);
  };
  bool ok = true;
  for (int i = 0; ok; ++i) {
    const int item = key_weights_cta_item(p, i);
    if (item >= p.items) break;
    const KeyWeightsItem it = key_weights_item(p, sm.lens, item, rank);
    if (it.t0 >= it.t1) {
      // (an entry without a tile is passed in its turn: see KwRing's parity.  Nothing
      // else would keep its group from running several rounds of entries ahead)
      if (it.k0 >= it.L) continue;
      if (!(ok = wait_entry())) break;
      if (lane == 0) mbar_arrive(&sm.l_empty[group][group ? l1.i : l0.i]);
      (group ? l1 : l0).step();
      continue;
    }
    // K to tensor memory, once the last item's MMAs have read theirs
    if (done > 0 && !(ok = wait(&sm.k_free, (done - 1) & 1u))) break;
    ++done;
    if (!(ok = wait(&sm.full[r.i], r.par))) break;
    tc_fence_after_sync();
    const uint64_t k = desc + (uint64_t)r.i * (Cfg::kTile >> 4);
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk)
      tmem_cp_128x256b_warp(tbase + Cfg::kColK + 8 * kk,
                            k + (((kk / 4) * Cfg::kBox + (kk % 4) * 32) >> 4));
    mma_commit_warp(&sm.empty[r.i]);
    r.step();
    for (int t = it.t0; t < it.t1; ++t) {
      // (looked at together: one wait after another took 100 cycles each)
      uint64_t* const entry = &sm.l_full[group][group ? l1.i : l0.i];
      const uint32_t entry_par = group ? l1.par : l0.par;
      const bool q_here = mbar_try_wait(smem_u32(&sm.full[r.i]), r.par);
      const bool s_free = mbar_try_wait(smem_u32(&sm.s_empty[s.i]), s.par ^ 1u);
      const bool e_here = mbar_try_wait(smem_u32(entry), entry_par);
      if (!__all_sync(0xffffffffu, q_here && s_free && e_here)) {
        if (!(ok = wait(&sm.full[r.i], r.par))) break;
        if (!(ok = wait(&sm.s_empty[s.i], s.par ^ 1u))) break;
        if (!(ok = wait(entry, entry_par))) break;
      }
      tc_fence_after_sync();
      const uint64_t q = desc + (uint64_t)r.i * (Cfg::kTile >> 4);
      const uint32_t dS = tbase + 128u * s.i;
      // (a shared address of a cluster's CTA has its rank above the descriptor's bits)
      const uint32_t parts = smem_u32(sm.nlse[group][group ? l1.i : l0.i]);
      const uint64_t lse = plain | ((parts >> 4) & 0x3FFFu) | ((zero - parts) >> 4 << 16);
      if (elect_one_sync()) {
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk)
          mma_bf16_ts(dS, tbase + Cfg::kColK + 8 * kk,
                      q + (((kk / 4) * Cfg::kBox + (kk % 4) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
        mma_bf16_ts(dS, tbase + Cfg::kColOne, lse, idesc, 1u);
        mma_commit(&sm.s_full[s.i]);
        mma_commit(&sm.empty[r.i]);
      }
      __syncwarp();
      r.step();
      (group ? l1 : l0).step();
      group ^= 1u;
      s.step();
    }
    mma_commit_warp(&sm.k_free);
  }
  // nothing of this warp's may still run on the tensor core at teardown
  mma_commit_warp(&sm.mma_done);
  mbar_wait_drain(&sm.mma_done, 0);
}

// The sum of 2^(s scale_log2) over 32 columns.
__device__ __forceinline__ void key_weights_add(const uint32_t (&y)[32], float2 scale2,
                                                float2 (&sum)[2]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float2 a =
        __fmul2_rn(make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), scale2);
    sum[e & 1] = __fadd2_rn(sum[e & 1], make_float2(ex2_approx(a.x), ex2_approx(a.y)));
  }
}

// Summing warps: thread tid (0 .. 127) of a group owns key k0 + tid.
template <int DH>
__device__ __forceinline__ void key_weights_sums(KeyWeightsSmem<DH>& sm, const KeyWeightsParams& p,
                                                 uint32_t tbase, int group, int rank,
                                                 volatile int* abort) {
  using Cfg = KeyWeightsCfg<DH>;
  const int tid = threadIdx.x % 128;
  const uint32_t lane_addr = tbase + ((uint32_t)(tid & ~31) << 16);
  const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
  KwRing<Cfg::kLse> l;
  // one arrival per warp, when all of it is done with what `bar` guards
  auto release = [&](uint64_t* bar) {
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive(bar);
  };
  float total = 0.f;
  for (;; l.step()) {
    if (!mbar_wait(&sm.l_full[group][l.i], l.par, abort)) return;
    const KeyWeightsEntry& entry = sm.entry[group][l.i];
    const int4 en = *reinterpret_cast<const int4*>(&entry);   // flags, lo, hi, end
    if (en.x & kKwEnd) return;
    if (!(en.x & kKwNone)) {
      // (the tiles alternate between the groups and S is computed in order, so the
      // use of this buffer before this one is over: one parity bit is enough)
      const int sb = (en.x >> kKwS) & 3;
      if (!mbar_wait(&sm.s_full[sb], (uint32_t)(en.x >> kKwSPar) & 1u, abort)) return;
      tc_fence_after_sync();
      const uint32_t colS = lane_addr + 128u * sb;
      // a tile's sum is taken by itself and then added: the error of a long sum
      // grows with the number of tiles, not of queries
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      if (en.x & kKwWhole) {
        uint32_t y0[32], y1[32], y2[32], y3[32];
        tmem_ld_32x32b_x32(colS, y0);
        tmem_ld_32x32b_x32(colS + 32, y1);
        tmem_ld_wait(y0);
        tmem_ld_wait(y1);
        tmem_ld_32x32b_x32(colS + 64, y2);
        tmem_ld_32x32b_x32(colS + 96, y3);
        key_weights_add(y0, scale2, sum);
        key_weights_add(y1, scale2, sum);
        tmem_ld_wait(y2);
        tmem_ld_wait(y3);
        tc_fence_before_sync();
        release(&sm.s_empty[sb]);   // S is in registers
        key_weights_add(y2, scale2, sum);
        key_weights_add(y3, scale2, sum);
      } else {
        int clo = max(0, en.y + tid);
        const int chi = min(en.w, en.z + tid), cols = entry.cols;
        const uint32_t span = chi > clo ? (uint32_t)(chi - clo - 1) : 0u;
        if (chi <= clo) clo = 1 << 30;   // no column is visible
        const int in_head = p.pad - 1;   // (a power of two less one)
        // columns that some, and that all, of this warp's keys see, with one head's
        // queries in the tile: on the diagonal most 32 columns are one or the other
        const int t0 = tid & ~31;
        // (2 x 32 heads of 1024: 18.4 -> 17.6 us)
        const bool one = p.pad == 128;
        const int any_lo = one ? en.y + t0 : 0, any_hi = one ? min(en.w, en.z + t0 + 31) : 128;
        const int all_lo = one ? en.y + t0 + 31 : 128, all_hi = min(en.w, en.z + t0);
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          if (c + 32 <= any_lo || c >= any_hi) continue;
          uint32_t y[32];
          tmem_ld_32x32b_x32(colS + c, y);
          tmem_ld_wait(y);
          if (c < all_lo || c + 32 > all_hi) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float v = keep_if_le(__uint_as_float(y[e]),
                                         (uint32_t)(((c + e) & in_head) - clo), span);
              y[e] = c + e < cols ? __float_as_uint(v) : 0xff800000u;
            }
          }
          key_weights_add(y, scale2, sum);
        }
        tc_fence_before_sync();
        release(&sm.s_empty[sb]);
      }
      total += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    }
    if (en.x & kKwLast) {
      const int hb = (en.x >> kKwHand) & (Cfg::kHand - 1);
      const uint32_t hpar = (uint32_t)(en.x >> kKwHandPar) & 1u;
      if (!(en.x & kKwFinish)) {
        if (!mbar_wait(&sm.hand_empty[hb], hpar ^ 1u, abort)) return;
        sm.hand[hb][tid] = total;
        release(&sm.hand_full[hb]);
      } else {
        if (en.x & kKwPair) {
          if (!mbar_wait(&sm.hand_full[hb], hpar, abort)) return;
          total += sm.hand[hb][tid];
          release(&sm.hand_empty[hb]);
        }
        if (p.split > 1) {
          // to the cluster's first CTA
          const uint32_t mine = smem_u32(&sm.parts[rank][tid]);
          uint32_t there;
          asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"(mine));
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(total) : "memory");
        } else if (tid < entry.rows) {
          float* w = p.weights + entry.out + tid;
          *w = p.accumulate ? *w + total : total;
        }
      }
      total = 0.f;
    }
    release(&sm.l_empty[group][l.i]);
    // a tile's S was there, so its issuing warp has passed the entry
    if (!(en.x & kKwNone) && tid == 0) mbar_arrive(&sm.l_empty[group][l.i]);
  }
}

// (No early exit: the CTAs of a cluster meet at its end.)
template <int DH>
__global__ void __launch_bounds__(384, 1)
    attn_key_weights_sm103a(const __grid_constant__ CUtensorMap map_q,
                            const __grid_constant__ CUtensorMap map_k, const KeyWeightsParams p) {
  using Cfg = KeyWeightsCfg<DH>;
  using Smem = KeyWeightsSmem<DH>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~uintptr_t(1023));
  volatile int* abort = &sm.abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = p.split > 1 ? (int)blockIdx.x % p.split : 0;
  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    for (int i = 0; i < Cfg::kSlots; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2 * Cfg::kLse; ++i) {
      mbar_init(&sm.l_full[0][i], 1);    // (both groups' rings lie in a row)
      // one arrival per summing warp of a group, and one for the issuing warp: an entry
      // may be written again once both have passed it
      mbar_init(&sm.l_empty[0][i], 5);
    }
    for (int i = 0; i < Cfg::kBuffers; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_empty[i], 4);
    }
    for (int i = 0; i < Cfg::kHand; ++i) {
      mbar_init(&sm.hand_full[i], 4);
      mbar_init(&sm.hand_empty[i], 4);
    }
    mbar_init(&sm.k_free, 1);
    mbar_init(&sm.mma_done, 1);
    fence_mbarrier_init();
  }
  if (warp == Cfg::kWarpIssuer) {
    tmem_alloc(&sm.tmem_base, Cfg::kCols);
    tmem_relinquish();
  }
  for (int i = threadIdx.x; i < 128; i += Cfg::kThreads) sm.zero[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();   // (the MMA reads them)
  // (the lengths may come from the previous kernel)
  griddep_wait();
  for (int b = threadIdx.x; b < p.B; b += Cfg::kThreads) {
    if (b < Cfg::kLens) sm.lens[b] = key_weights_len(p, b);
    if (blockIdx.x == 0 && p.seqlens) {   // an impossible length is an error
      const int n = __ldcg(p.seqlens + b);
      if (n < 0 || n > p.S) atomicExch(p.error_word, 1);   // ATTN_ERR_INVALID_ARG
    }
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = sm.tmem_base;
  if (warp < 4) {   // 1, 1, 1, 0, ... in each row
    const uint32_t ones[8] = {0x3f803f80u, 0x00003f80u, 0u, 0u, 0u, 0u, 0u, 0u};
    tmem_st_32x32b_x8(tbase + ((uint32_t)(warp * 32) << 16) + Cfg::kColOne, ones);
    tmem_st_wait();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (p.split > 1) cluster_sync();   // (every CTA runs before any writes to another)
  if (warp == Cfg::kWarpProducer) {
    key_weights_producer<DH>(sm, p, &map_q, &map_k, rank, lane, abort);
  } else if (warp >= Cfg::kWarpLse) {
    key_weights_lse<DH>(sm, p, rank, warp - Cfg::kWarpLse, lane, abort);
  } else if (warp == Cfg::kWarpIssuer) {
    key_weights_issuer<DH>(sm, p, tbase, rank, lane, abort);
  } else {
    key_weights_sums<DH>(sm, p, tbase, warp / 4, rank, abort);
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == Cfg::kWarpIssuer) {
    tc_fence_after_sync();
    tmem_dealloc(tbase, Cfg::kCols);
  }
  if (threadIdx.x == 0 && sm.abort_flag) atomicExch(p.error_word, 4);   // ATTN_ERR_TIMEOUT
  if (p.split > 1) {
    // every CTA's sums are in the first one's shared memory (all waits before
    // this one are bounded, so every thread of the cluster comes here)
    cluster_sync();
    if (rank == 0 && threadIdx.x < 128) {
      const KeyWeightsItem it = key_weights_item(p, sm.lens, (int)blockIdx.x / p.split, 0);
      const int j = it.k0 + threadIdx.x;
      if (j < it.L) {
        float total = 0.f;
        for (int r = 0; r < p.split; ++r) total += sm.parts[r][threadIdx.x];
        float* w = p.weights + ((size_t)it.b * p.Hkv + it.g) * p.stride + j;
        *w = p.accumulate ? *w + total : total;
      }
    }
  }
}

template <int DH>
constexpr size_t key_weights_smem_bytes() {
  return sizeof(KeyWeightsSmem<DH>) + 1024;   // + alignment slack
}

}  // namespace chs
