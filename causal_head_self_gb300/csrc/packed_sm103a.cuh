// packed_sm103a.cuh -- packed sequences: what the attention kernels need to
// walk sequences of different lengths that lie one behind another.
//
// Sequence b holds rows cu[b] .. cu[b+1] - 1 of tensors [T, H, Dh] whose rows
// and heads lie at any strides.  Two things differ from a [B, H, S, Dh] batch:
//
//   Sequences end inside tiles.  What lies next to a sequence in memory is
//   another one's rows, and those must not reach the tensor core: a masked
//   score hides a foreign key, but a weight of 0 times an infinity in a foreign
//   V row is NaN.  So a sequence is padded to whole 128-row blocks at its
//   front, with rows that no copy reads: its last row ends a block, and only
//   its first block is short.  The tensor maps carry the row axis twice, both
//   times with the row's stride: an axis of R rows (the box's height) and one
//   of T.  A box over padded rows [t, t + R) of a sequence that starts at row a
//   behind `pad` of them is copied from
//       (t - pad, a)      where t < pad: the rows ahead of a lie before the
//                         R-row axis, and a load fills them with zeros;
//       (0, a + t - pad)  otherwise.
//   One map serves every sequence, and no row but the sequence's own is read.
//   Positions are counted with the padding: masks that compare positions do
//   not see a common shift.  Padded keys are masked; padded queries compute
//   rows that nobody stores.  (Padding at the end would need boxes that end at
//   any row, whose map starts ahead of the tensor.)
//
//   The work is known on the GPU alone.  A launch ahead of the attention
//   kernel lists the tiles, heaviest first (attn_packed_schedule); of a causal
//   forward pass over few sequences, each CTA lists its own (packed_list_own).
#pragma once

#include "sm103a_ptx.cuh"

namespace chs {

// One block of rows of a sequence.
struct __align__(16) PackedTile {
  int start;   // the sequence's first row
  int len;     // its rows
  int blk;     // which block of its padded rows
  int stat;    // its first padded row among those of all sequences
  __device__ __forceinline__ int pad() const { return -len & 127; }
};

// PackedTile::stat of sequence b, whose first row is `start`: rows of the earlier sequences, each
// rounded up to 128, are at most start + 127 b, so a sequence may start at the next multiple of
// 128 and no two meet.
__device__ __forceinline__ int packed_stat(int start, int b) {
  return (int)(((long long)start + 127ll * b + 127) / 128 * 128);
}

// Tensors, as bits of PackedRef::heads_inner.
constexpr int kPackedQ = 1, kPackedK = 2, kPackedV = 4, kPackedO = 8, kPackedDO = 16;

struct PackedRef {
  const PackedTile* tiles;   // heaviest first; null: each CTA lists its own items
  const int* num_tiles;      // [3] of one head each, then those of two and of four heads
  const int* cu;             // [B + 1], B and the most blocks of a sequence, for that
  int B, levels;
  int T;                     // rows of the packed tensors
  int heads_inner;           // tensors whose heads lie closer than their rows: map axes
                             // {Dh, head, rows, start} instead of {Dh, rows, start, head}
  int fold_max;              // short sequences: up to 1 << fold_max heads lie in one tile
};

// How many heads (1 << fold) of a sequence lie in one tile: of up to 32 rows four, of up to 64 two.
__device__ __forceinline__ int packed_fold(int len, int fold_max) {
  return len > 64 ? 0 : min(fold_max, len > 32 ? 1 : 2);
}

// Read past L1: the list was written by the launch before this one.
__device__ __forceinline__ PackedTile packed_tile(const PackedRef& p, int i) {
  const int4 e = __ldcg(reinterpret_cast<const int4*>(p.tiles + i));
  return PackedTile{e.x, e.y, e.z, e.w};
}
__device__ __forceinline__ int packed_num_tiles(const PackedRef& p) { return __ldcg(p.num_tiles); }

// Work items of tiles of one, two and four heads.
__device__ __forceinline__ int3 packed_counts(const PackedRef& p) {
  return make_int3(__ldcg(p.num_tiles), __ldcg(p.num_tiles + 1), __ldcg(p.num_tiles + 2));
}
__device__ __forceinline__ int packed_items(const int3& n, int Hq) {
  return n.x * Hq + n.y * (Hq / 2) + n.z * (Hq / 4);
}
// Item w: tile i, its first head h.  A tile's heads come one after another: those of a group
// share their K/V tiles in L2.
__device__ __forceinline__ void packed_item_of(const int3& n, int Hq, int w, int& i, int& h) {
  int fold = 0, first = 0;
  if (w >= n.x * Hq) {
    w -= n.x * Hq;
    first = n.x;
    fold = 1;
    if (w >= n.y * (Hq / 2)) {
      w -= n.y * (Hq / 2);
      first += n.y;
      fold = 2;
    }
  }
  const int per = Hq >> fold;
  i = w / per;
  h = (w - i * per) << fold;
  i += first;
}

__device__ __forceinline__ void tma_load_4d_hint(void* dst, const CUtensorMap* map, uint64_t* bar,
                                                 int c0, int c1, int c2, int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "l"(policy)
      : "memory");
}

// Padded rows [row, row + R) of the sequence that starts at row `start` behind `pad` of them,
// columns c .. c + 63 of one head; padded rows are zeros.
__device__ __forceinline__ void packed_load(void* dst, const CUtensorMap* map, uint64_t* bar, int c,
                                            int start, int pad, int row, int head, bool heads_inner,
                                            uint64_t policy) {
  const int y = min(row - pad, 0), z = start + max(row - pad, 0);
  tma_load_4d_hint(dst, map, bar, c, heads_inner ? head : y, heads_inner ? y : z,
                   heads_inner ? z : head, policy);
}

// Rows of the sequence from padded row `row` (>= pad) on, through a map with one row axis.
__device__ __forceinline__ void packed_store(const CUtensorMap* map, const void* src, int c,
                                             int start, int pad, int row, int head,
                                             bool heads_inner, uint64_t policy) {
  const int z = start + row - pad;
  tma_store_3d_hint(map, src, c, heads_inner ? head : z, heads_inner ? z : head, policy);
}

// ---------------------------------------------------------------- a CTA's own items

// With few sequences a CTA finds its own work items faster than another launch
// lists them all, and the call needs no workspace (16 short requests: 11.5 us
// with the launch, 10.2 without; on the host 22 and 11).
constexpr int kOwnSequences = 64;   // one bit each
constexpr int kOwnLevels = 1024;    // blocks of the longest sequence, at most
constexpr int kOwnItems = 32;       // per CTA, at most: one lane each

struct PackedOwn {
  int4 item[kOwnItems];   // first row, rows, block, head
  int count;
};

// Bytes of shared memory that listing takes (it may be a buffer of the kernel's).
constexpr int kOwnScratch = 8 * kOwnLevels + 4 * (kOwnLevels + 1) + 3 * 4 * kOwnSequences + 32;

// All threads of the CTA.  Items are numbered by block, the last (under a
// causal mask: the heaviest) first, then by sequence, then by head, and after
// them those of two heads and of four; item_of(k, items) is the number of this
// CTA's k-th.  For each block number the threads
// make the mask of the sequences that have it and the count of tiles from it
// on; then a lane per item finds its block by bisection and its sequence as a
// bit of the mask.
template <int BLOCK, typename ItemOf>
__device__ __forceinline__ void packed_list_own(const PackedRef& p, int Hq, void* scratch,
                                                PackedOwn& own, int* error_word, ItemOf item_of) {
  uint64_t* mask = static_cast<uint64_t*>(scratch);                    // [levels]
  int* tiles = reinterpret_cast<int*>(mask + kOwnLevels);              // [kOwnSequences] each one's
  int* start = tiles + kOwnSequences;
  int* len = start + kOwnSequences;
  unsigned* folded = reinterpret_cast<unsigned*>(len + kOwnSequences);  // [4] masks by fold
  int* from = reinterpret_cast<int*>(folded + 4);                      // [levels + 1]
  const int t = threadIdx.x;
  bool bad = false;
  if (t < kOwnSequences) {
    int a = 0, n = 0;
    if (t < p.B) {
      a = __ldcg(p.cu + t);
      n = __ldcg(p.cu + t + 1) - a;
      bad = a < 0 || n < 0 || n > p.T - a;
    }
    const int fold = bad || n == 0 ? 0 : packed_fold(n, p.fold_max);
    start[t] = a;
    len[t] = n;
    tiles[t] = bad || fold ? 0
                           : (n + 127) / 128 * 128 / BLOCK + ((n + 127) / 128 * 128 % BLOCK != 0);
    const unsigned two = __ballot_sync(0xffffffffu, fold == 1);
    const unsigned four = __ballot_sync(0xffffffffu, fold == 2);
    if (t % 32 == 0) {
      folded[t / 32] = two;
      folded[2 + t / 32] = four;
    }
  }
  if (__syncthreads_or(bad)) {
    if (t == 0) own.count = 0;
    if (t == 0 && blockIdx.x == 0) atomicExch(error_word, 1);   // ATTN_ERR_INVALID_ARG
    return;
  }
  for (int l = t; l <= p.levels; l += blockDim.x) {
    uint64_t m = 0;
    int c = 0;
#pragma unroll 4
    for (int b = 0; b < kOwnSequences; b += 4) {
      const int4 n = *reinterpret_cast<const int4*>(tiles + b);
      c += max(n.x - l, 0) + max(n.y - l, 0) + max(n.z - l, 0) + max(n.w - l, 0);
      const uint64_t bits = (n.x > l ? 1u : 0u) | (n.y > l ? 2u : 0u) | (n.z > l ? 4u : 0u) |
                            (n.w > l ? 8u : 0u);
      m |= bits << b;
    }
    if (l < p.levels) mask[l] = m;
    from[l] = c;
  }
  __syncthreads();
  if (t < 32) {
    const uint64_t two = folded[0] | (uint64_t)folded[1] << 32;
    const uint64_t four = folded[2] | (uint64_t)folded[3] << 32;
    const int3 n = make_int3(from[0], __popcll(two), __popcll(four));
    const int items = packed_items(n, Hq), w = item_of(t, items);
    const bool mine = w < items;
    if (mine) {
      int i, h, lo = 0;
      packed_item_of(n, Hq, w, i, h);
      uint64_t m = two;
      int r = i - n.x;   // the r-th sequence of the mask
      if (r >= n.y) {
        m = four;
        r -= n.y;
      } else if (r < 0) {
        int hi = p.levels;   // from[lo] > i >= from[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (from[mid] > i) lo = mid; else hi = mid;
        }
        m = mask[lo];
        r = i - from[lo + 1];
      }
      for (; r > 0; --r) m &= m - 1;
      const int b = __ffsll((long long)m) - 1;
      own.item[t] = make_int4(start[b], len[b], lo, h);
    }
    const unsigned all = __ballot_sync(0xffffffffu, mine);
    if (t == 0) own.count = __popc(all);
  }
  // the tiles' copies may overwrite the scratch
  fence_proxy_async_smem();
}

// ---------------------------------------------------------------- the list of tiles

// What a tile's time goes by (its 128-row partner blocks).
enum PackedOrder {
  kByKeys = 0,      // a block of queries: the keys it sees
  kByQueries = 1,   // a block of keys: the queries that see it
};

struct PackedSchedule {
  const int* cu;   // [B + 1]
  int B, T;
  int block;       // rows per tile: 128 or 256
  int causal, window;
  int fold_max;    // see PackedRef
  PackedTile* tiles[2];   // one list per order (block x of the grid makes list x)
  int capacity;           // tiles that a list has room for
  int order[2];
  int* num_tiles[2];   // three counts each
  int* error_word;
};

}  // namespace chs
