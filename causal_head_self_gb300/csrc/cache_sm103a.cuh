// cache_sm103a.cuh -- writing to a paged key-value cache and shrinking it
// (sm_103a).  Plain copies and a selection: bound by HBM bandwidth when large,
// by launch latency when small.
#pragma once

#include <cstdint>

#include "sm103a_ptx.cuh"

namespace chs {

struct AppendParams {
  const uint4* k;        // [B, Hkv, S, Dh]
  const uint4* v;
  uint4* kpages;         // [num_pages, Hkv, page, Dh]
  uint4* vpages;
  const int* table;      // [B, cols]
  const int* seqlens;    // [B], after the append
  const int* newlens;    // [B] or null (every sequence appends S rows)
  long long rows;        // B * Hkv * S
  int Hkv, S, vecs;      // vecs: 16-byte pieces per row
  int num_pages, page, cols;
  int* error_word;
};

constexpr int kAppendThreads = 256;

// Row i < newlens[b] of the new keys and values becomes row seqlens[b] -
// newlens[b] + i of the sequence.  A thread copies a 16-byte piece of K and V
// of U rows; all its loads are issued before its stores.
template <int U>
__global__ void __launch_bounds__(kAppendThreads) attn_paged_append_sm103a(const AppendParams p) {
  griddep_wait();
  const int per_pass = kAppendThreads / p.vecs;   // rows per pass of the block
  const int vec = threadIdx.x % p.vecs, r = threadIdx.x / p.vecs;
  uint4 k[U], v[U];
  long long dst[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    dst[u] = -1;
    const long long row = ((long long)blockIdx.x * U + u) * per_pass + r;
    if (row >= p.rows) continue;
    const int i = (int)(row % p.S);
    const long long bg = row / p.S;
    const int b = (int)(bg / p.Hkv), g = (int)(bg % p.Hkv);
    const int n = __ldcg(p.seqlens + b), add = p.newlens ? __ldcg(p.newlens + b) : p.S;
    if (n == 0 && !p.newlens) continue;   // an empty slot
    if (add < 0 || add > p.S || n < add || n > p.cols * p.page) {
      if (i == 0 && g == 0 && vec == 0) atomicExch(p.error_word, 1);   // ATTN_ERR_INVALID_ARG
      continue;
    }
    if (i >= add) continue;
    const int t = n - add + i;
    const int id = __ldcg(p.table + (long long)b * p.cols + t / p.page);
    if (id < 0 || id >= p.num_pages) {
      atomicExch(p.error_word, 1);
      continue;
    }
    k[u] = __ldcg(p.k + row * p.vecs + vec);
    v[u] = __ldcg(p.v + row * p.vecs + vec);
    dst[u] = (((long long)id * p.Hkv + g) * p.page + t % p.page) * p.vecs + vec;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (dst[u] < 0) continue;
    p.kpages[dst[u]] = k[u];
    p.vpages[dst[u]] = v[u];
  }
}

struct EvictParams {
  uint4* kpages;
  uint4* vpages;
  const int* table;       // [B, cols]
  const int* table_out;   // [B, cols_out]
  const int* seqlens;     // [B]
  int* newlens;           // [B]
  const float* weights;   // [B, Hkv, stride]
  float* weights_out;     // [B, Hkv, stride_out], or weights itself
  int* keep;              // [B, Hkv, budget]
  int B, Hkv, vecs;
  int num_pages, page, cols, cols_out, stride, stride_out, budget, recent;
  int* error_word;
};

// A float as an unsigned integer in the same order; NaN comes below every
// number, and the two zeros are one.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelectThreads = 1024;

// Which rows stay.  One block per (sequence, K/V head): of the rows before the
// last `recent`, the budget - recent with the largest weights, equal ones from
// the lowest row on; and the last `recent`.  The smallest weight that stays is
// found digit by digit (11, 11 and 10 bits of the ordered integer) from
// histograms in shared memory; one more pass writes the rows' numbers and
// weights in order.  In place, row i's weight moves to a place at or before i,
// and a tile is read before anything of it is overwritten.
__global__ void __launch_bounds__(kSelectThreads, 1) attn_cache_select_sm103a(const EvictParams p) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t warp_sum[32];
  __shared__ uint32_t sh_bin, sh_left;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  griddep_wait();
  const int bg = blockIdx.x, b = bg / p.Hkv, g = bg - b * p.Hkv;
  const float* w = p.weights + (size_t)bg * p.stride;
  float* w_out = p.weights_out + (size_t)bg * p.stride_out;
  int* keep = p.keep + (size_t)bg * p.budget;
  const int n = __ldcg(p.seqlens + b);
  if (n < 0 || n > p.cols * p.page || n > p.stride) {
    for (int i = tid; i < p.budget; i += kSelectThreads) keep[i] = -1;
    if (tid == 0) atomicExch(p.error_word, 1);   // ATTN_ERR_INVALID_ARG
    if (tid == 0 && g == 0) p.newlens[b] = n;
    return;
  }
  if (n <= p.budget) {   // everything stays
    for (int i = tid; i < p.budget; i += kSelectThreads) {
      keep[i] = i < n ? i : -1;
      if (i < n && w_out != w) w_out[i] = w[i];
    }
    if (tid == 0 && g == 0) p.newlens[b] = n;
    return;
  }
  if (tid == 0 && g == 0) p.newlens[b] = p.budget;
  const int old = n - p.recent;
  uint32_t left = (uint32_t)(p.budget - p.recent);   // rows still to be chosen
  uint32_t prefix = 0, known = 0;                    // digits found so far, and their mask
  if (left > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digit = pass < 2 ? 0x7ffu : 0x3ffu;
      hist[tid] = 0;
      hist[tid + 1024] = 0;
      __syncthreads();
      constexpr int kLoads = 8;   // rows per thread and round: their loads are in flight together
      for (int i0 = 0; i0 < old; i0 += kLoads * kSelectThreads) {
        float x[kLoads];
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
          const int i = i0 + e * kSelectThreads + tid;
          x[e] = i < old ? w[i] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
          const uint32_t key = order_key(x[e]);
          const bool in = i0 + e * kSelectThreads + tid < old && (key & known) == prefix;
          const uint32_t bin = (key >> shift) & digit;
          // a warp whose rows all fall into one bin adds them at once
          const uint32_t who = __ballot_sync(0xffffffffu, in);
          if (who == 0) continue;
          const uint32_t first = __shfl_sync(0xffffffffu, bin, __ffs(who) - 1);
          if (__ballot_sync(0xffffffffu, in && bin == first) == who) {
            if (lane == 0) atomicAdd(&hist[first], (uint32_t)__popc(who));
          } else if (in) {
            atomicAdd(&hist[bin], 1u);
          }
        }
      }
      __syncthreads();
      // the bin in which the count from the top reaches `left`: thread t holds
      // bins 2047 - 2t and 2046 - 2t
      const uint32_t a = hist[2047 - 2 * tid], c = hist[2046 - 2 * tid];
      uint32_t upto = a + c;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y;
      }
      if (lane == 31) warp_sum[warp] = upto;
      __syncthreads();
      uint32_t before = lane < warp ? warp_sum[lane] : 0u;
      before = __reduce_add_sync(0xffffffffu, before);
      const uint32_t above = before + upto - (a + c);   // rows in higher bins
      if (above < left && above + a >= left) {
        sh_bin = 2047 - 2 * tid;
        sh_left = left - above;
      } else if (above + a < left && above + a + c >= left) {
        sh_bin = 2046 - 2 * tid;
        sh_left = left - above - a;
      }
      __syncthreads();
      prefix |= sh_bin << shift;
      known |= digit << shift;
      left = sh_left;
    }
  } else {
    prefix = 0xffffffffu;   // above every weight: none of the old rows stays
  }
  // rows above `prefix` stay, and the first `left` of those equal to it; a warp
  // takes 128 rows of a tile of 4096
  constexpr int kPer = 4, kTileRows = kSelectThreads * kPer;
  uint32_t base_gt = 0, base_eq = 0;
#pragma unroll 1
  for (int t0 = 0; t0 < n; t0 += kTileRows) {
    float x[kPer];
    uint32_t gt[kPer], eq[kPer], my_gt = 0, my_eq = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int t = t0 + warp * 32 * kPer + e * 32 + lane;
      x[e] = t < n ? w[t] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int t = t0 + warp * 32 * kPer + e * 32 + lane;
      const uint32_t key = order_key(x[e]);
      gt[e] = __ballot_sync(0xffffffffu, t < n && (t >= old || key > prefix));
      eq[e] = __ballot_sync(0xffffffffu, t < old && key == prefix);
      my_gt += __popc(gt[e]);
      my_eq += __popc(eq[e]);
    }
    // both counts are at most 4096: one scan for the two
    __syncthreads();   // (the tile is read, and warp_sum free)
    if (lane == 0) warp_sum[warp] = my_gt | (my_eq << 16);
    __syncthreads();
    const uint32_t all = warp_sum[lane];
    const uint32_t sum = __reduce_add_sync(0xffffffffu, all);
    const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? all : 0u);
    uint32_t g0 = base_gt + (before & 0xffffu), e0 = base_eq + (before >> 16);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int t = t0 + warp * 32 * kPer + e * 32 + lane;
      const uint32_t below = (1u << lane) - 1u;
      const uint32_t my_g = g0 + __popc(gt[e] & below), my_e = e0 + __popc(eq[e] & below);
      const bool stays = ((gt[e] >> lane) & 1u) || (((eq[e] >> lane) & 1u) && my_e < left);
      if (stays) {
        const uint32_t to = my_g + min(my_e, left);
        keep[to] = t;
        w_out[to] = x[e];
      }
      g0 += __popc(gt[e]);
      e0 += __popc(eq[e]);
    }
    base_gt += sum & 0xffffu;
    base_eq += sum >> 16;
  }
  __syncthreads();
  // rows that follow start from nothing
  for (int i = p.budget + tid; i < min(n, p.stride_out); i += kSelectThreads) w_out[i] = 0.f;
}

// 16-byte piece `vec` of row t of (b, g), or -1 for a page that is not there.
__device__ __forceinline__ long long cache_piece(const EvictParams& p, const int* table, int cols,
                                                 int b, int g, int t, int vec) {
  const int id = __ldcg(table + (long long)b * cols + t / p.page);
  if (id < 0 || id >= p.num_pages) {
    atomicExch(p.error_word, 1);   // ATTN_ERR_INVALID_ARG
    return -1;
  }
  return (((long long)id * p.Hkv + g) * p.page + t % p.page) * p.vecs + vec;
}

constexpr int kMoveThreads = 256;

// K and V rows to other pages: row i of the output is row keep[i].  A thread
// moves a 16-byte piece of K and V of U rows.
template <int U>
__global__ void __launch_bounds__(kMoveThreads) attn_cache_move_sm103a(const EvictParams p) {
  griddep_wait();
  const int per_pass = kMoveThreads / p.vecs;
  const int vec = threadIdx.x % p.vecs, r = threadIdx.x / p.vecs;
  const int blocks = (p.budget + per_pass * U - 1) / (per_pass * U);
  const int bg = blockIdx.x / blocks, blk = blockIdx.x - bg * blocks;
  const int b = bg / p.Hkv, g = bg - b * p.Hkv;
  uint4 k[U], v[U];
  int src[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = (blk * U + u) * per_pass + r;
    src[u] = i < p.budget ? __ldcg(p.keep + (size_t)bg * p.budget + i) : -1;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (src[u] < 0) continue;
    const long long at = cache_piece(p, p.table, p.cols, b, g, src[u], vec);
    if (at < 0) {
      src[u] = -1;
      continue;
    }
    k[u] = __ldcg(p.kpages + at);
    v[u] = __ldcg(p.vpages + at);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (src[u] < 0) continue;
    const int i = (blk * U + u) * per_pass + r;
    const long long at = cache_piece(p, p.table_out, p.cols_out, b, g, i, vec);
    if (at < 0) continue;
    p.kpages[at] = k[u];
    p.vpages[at] = v[u];
  }
}

// K and V rows within their own pages.  Row i comes from row keep[i] >= i, and
// keep grows, so batches of rows taken in order are safe when a batch is read
// whole before any of it is written: what it overwrites lies before the sources
// of every later batch.  A block owns a column slice of `piece` 16-byte pieces
// of K or V of one (sequence, K/V head), so nobody else touches what it moves.
template <int U>
__global__ void __launch_bounds__(kMoveThreads)
    attn_cache_move_in_place_sm103a(const EvictParams p, int piece) {
  griddep_wait();
  const int slices = p.vecs / piece;
  const int slice = blockIdx.x % slices;
  const int kv = (blockIdx.x / slices) & 1;
  const int bg = blockIdx.x / (2 * slices);
  const int b = bg / p.Hkv, g = bg - b * p.Hkv;
  uint4* pool = kv ? p.vpages : p.kpages;
  const int vec = slice * piece + threadIdx.x % piece, r = threadIdx.x / piece;
  const int per_pass = kMoveThreads / piece;
  const int* keep = p.keep + (size_t)bg * p.budget;
#pragma unroll 1
  for (int i0 = 0; i0 < p.budget; i0 += per_pass * U) {
    uint4 x[U];
    int src[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * per_pass + r;
      src[u] = i < p.budget ? __ldcg(keep + i) : -1;
      if (src[u] == i) src[u] = -1;   // it is there already
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (src[u] < 0) continue;
      const long long at = cache_piece(p, p.table, p.cols, b, g, src[u], vec);
      if (at < 0) src[u] = -1;
      else x[u] = __ldcg(pool + at);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (src[u] < 0) continue;
      const long long at =
          cache_piece(p, p.table, p.cols, b, g, i0 + u * per_pass + r, vec);
      if (at >= 0) pool[at] = x[u];
    }
  }
}

}  // namespace chs
