// packed_schedule_sm103a.cuh -- the list of a packed batch's tiles, made on the GPU.
#pragma once

#include "packed_sm103a.cuh"

namespace chs {

constexpr int kScheduleThreads = 1024;
constexpr int kScheduleBins = 2048;

// One block of threads lists the tiles of all sequences, those with the most
// work first (a counting sort by the number of 128-row blocks a tile meets, in
// kScheduleBins steps where there are more).  Offsets that are not ascending
// within [0, T] latch ATTN_ERR_INVALID_ARG and give an empty list, so the
// attention kernel does nothing.  Tiles of the same weight come in any order:
// each is computed for itself, so no result depends on it.
__global__ void __launch_bounds__(kScheduleThreads)
    attn_packed_schedule(const PackedSchedule p) {
  __shared__ int hist[kScheduleBins];
  __shared__ int warp_sum[kScheduleThreads / 32];
  __shared__ int most, bad;
  const int t = threadIdx.x, lane = t % 32, warp = t / 32;
  constexpr int kWarps = kScheduleThreads / 32;
  for (int i = t; i < kScheduleBins; i += kScheduleThreads) hist[i] = 0;
  if (t == 0) most = bad = 0;
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  const int blk_shift = p.block == 256 ? 8 : 7;
  const int order = blockIdx.x ? p.order[1] : p.order[0];
  PackedTile* tiles = blockIdx.x ? p.tiles[1] : p.tiles[0];
  int* num_tiles = blockIdx.x ? p.num_tiles[1] : p.num_tiles[0];

  // are the offsets sound, and how long is the longest sequence?
  int longest = 0;
  bool wrong = false;
  for (int b = t; b < p.B; b += kScheduleThreads) {
    const int a = p.cu[b], z = p.cu[b + 1];
    wrong |= a < 0 || z < a || z > p.T;
    longest = max(longest, z - a);
  }
  if (wrong) bad = 1;
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) atomicMax(&most, longest);
  __syncthreads();
  if (bad) {
    if (t < 3) num_tiles[t] = 0;
    if (t == 0) {
      atomicExch(p.error_word, 1);   // ATTN_ERR_INVALID_ARG
    }
    return;
  }
  // a tile's bin, the heaviest in bin 0 (rows are padded ones)
  auto padded = [](int len) { return (len + 127) / 128 * 128; };
  const int max_cost = (most + 127) / 128;
  // (the last two bins take the tiles of two and of four heads)
  const int shift = max_cost < kScheduleBins - 2 ? 0 : 33 - __clz(max_cost / kScheduleBins);
  const int fold_max = p.fold_max;
  auto bin_of = [&](int len, int blk, int fold) {
    if (fold) return kScheduleBins - 3 + fold;
    const int nb = len / 128, r0 = blk << blk_shift, r1 = min(len, r0 + p.block) - 1;
    int lo = 0, hi = nb - 1;
    if (p.causal) {
      if (order == kByKeys) {
        hi = r1 / 128;
        if (p.window > 0) lo = max(0, r0 - p.window + 1) / 128;
      } else {
        lo = r0 / 128;
        if (p.window > 0) hi = (int)min((long long)hi, ((long long)r1 + p.window - 1) / 128);
      }
    }
    return (max_cost - (hi - lo + 1)) >> shift;
  };
  // every block of every sequence once: a lane takes a short sequence, the warp a long one
  auto all_blocks = [&](auto&& take) {
    constexpr int kShort = 4;   // blocks
    for (int b0 = 32 * warp; b0 < p.B; b0 += 32 * kWarps) {
      const int b = b0 + lane;
      const int a = b < p.B ? p.cu[b] : 0, rows = b < p.B ? p.cu[b + 1] - a : 0;
      const int n = (padded(rows) + p.block - 1) >> blk_shift;
      if (n <= kShort)
        for (int i = 0; i < n; ++i) take(b, a, rows, i);
      for (unsigned m = __ballot_sync(0xffffffffu, n > kShort); m != 0; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const int a1 = __shfl_sync(0xffffffffu, a, src), rows1 = __shfl_sync(0xffffffffu, rows, src);
        const int n1 = __shfl_sync(0xffffffffu, n, src);
        for (int i = lane; i < n1; i += 32) take(b0 + src, a1, rows1, i);
      }
    }
  };
  all_blocks([&](int, int, int rows, int i) {
    atomicAdd(&hist[bin_of(padded(rows), i, packed_fold(rows, fold_max))], 1);
  });
  __syncthreads();
  // where each bin's tiles start
  static_assert(kScheduleBins == 2 * kScheduleThreads, "two bins a thread");
  const int h0 = hist[2 * t], h1 = hist[2 * t + 1];
  int run = h0 + h1;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, run, d);
    if (lane >= d) run += y;
  }
  if (lane == 31) warp_sum[warp] = run;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += y;
    }
    warp_sum[lane] = s;
  }
  __syncthreads();
  const int before = (warp > 0 ? warp_sum[warp - 1] : 0) + run - h0 - h1;
  hist[2 * t] = before;
  hist[2 * t + 1] = before + h0;
  if (t == kScheduleThreads - 1) {
    num_tiles[0] = before;
    num_tiles[1] = h0;
    num_tiles[2] = h1;
  }
  __syncthreads();
  all_blocks([&](int b, int a, int rows, int i) {
    const int at = atomicAdd(&hist[bin_of(padded(rows), i, packed_fold(rows, fold_max))], 1);
    // (checked builds: the list has room for the tile)
    if (attn_check(at >= 0 && at < p.capacity, p.error_word))
      *reinterpret_cast<int4*>(tiles + at) = make_int4(a, rows, i, packed_stat(a, b));
  });
}

}  // namespace chs
