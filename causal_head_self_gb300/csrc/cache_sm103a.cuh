// cache_sm103a.cuh -- writing to a paged key-value cache and shrinking it
// (sm_103a).  Plain copies and a selection: bound by HBM bandwidth when large,
// by launch latency when small.
#pragma once

#include <cstdint>

#include "fixed_div.h"
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
  FixedDiv by_s, by_heads, by_page;
  int* error_word;
};

constexpr int kAppendThreads = 256;

// Row i < newlens[b] of the new keys and values becomes row seqlens[b] -
// newlens[b] + i of the sequence.  A thread copies a 16-byte piece of K and V
// of U rows.  Where a row goes takes two dependent loads (its sequence's lengths,
// then the table), so the loads of all U rows go out together, and the row's own
// bytes, whose place is known, beside the table's.
template <int U>
__global__ void __launch_bounds__(kAppendThreads) attn_paged_append_sm103a(const AppendParams p) {
  griddep_wait();
  const int per_pass = kAppendThreads / p.vecs;   // rows per pass of the block
  const int vec = threadIdx.x % p.vecs, r = threadIdx.x / p.vecs;
  const long long row0 = (long long)blockIdx.x * U * per_pass + r;
  int b[U], g[U], i[U], n[U], add[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = row0 + u * per_pass;   // (the number of rows is 32-bit)
    const int at = row < p.rows ? (int)row : 0;
    const int bg = p.by_s.div(at);
    i[u] = at - bg * p.S;
    b[u] = p.by_heads.div(bg);
    g[u] = bg - b[u] * p.Hkv;
    n[u] = p.seqlens[b[u]];
    add[u] = p.newlens ? p.newlens[b[u]] : p.S;
    if (row >= p.rows) add[u] = n[u] = 0;
  }
  uint4 k[U], v[U];
  int id[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (n[u] == 0 && !p.newlens) add[u] = 0;   // an empty slot
    if (add[u] < 0 || add[u] > p.S || n[u] < add[u] || n[u] > p.cols * p.page) {
      if (i[u] == 0 && g[u] == 0 && vec == 0) atomicExch(p.error_word, 1);   // ATTN_ERR_INVALID_ARG
      add[u] = 0;
    }
    id[u] = -1;
    if (i[u] >= add[u]) continue;
    // (checked builds: a row of k and v, an entry of the table and a row of a page)
    if (!attn_check(row0 + u * per_pass < p.rows && vec < p.vecs && b[u] >= 0 && g[u] >= 0 &&
                        g[u] < p.Hkv && i[u] >= 0 &&
                        p.by_page.div(n[u] - add[u] + i[u]) < p.cols &&
                        p.by_page.mod(n[u] - add[u] + i[u]) < p.page,
                    p.error_word))
      continue;
    const long long from = (row0 + u * per_pass) * p.vecs + vec;
    k[u] = __ldcs(p.k + from);
    v[u] = __ldcs(p.v + from);
    id[u] = p.table[(long long)b[u] * p.cols + p.by_page.div(n[u] - add[u] + i[u])];
    if (id[u] < 0 || id[u] >= p.num_pages) {
      atomicExch(p.error_word, 1);
      id[u] = -1;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (id[u] < 0) continue;
    const int row = p.by_page.mod(n[u] - add[u] + i[u]);
    const long long to = (((long long)id[u] * p.Hkv + g[u]) * p.page + row) * p.vecs + vec;
    p.kpages[to] = k[u];
    p.vpages[to] = v[u];
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
  FixedDiv by_page;
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
constexpr int kSelectBins = 8192;
constexpr int kSelectHeld = 45056;   // rows: 176 KiB beside the 32 KiB of counts

// Four consecutive rows' ordered integers, from row i (a multiple of 4) on; rows
// from `end` on are not read.
__device__ __forceinline__ uint4 order_keys(const float* w, int i, int end, bool wide) {
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (wide && i + 4 <= end) {
    x = __ldcs(reinterpret_cast<const float4*>(w + i));
  } else {
    if (i < end) x.x = w[i];
    if (i + 1 < end) x.y = w[i + 1];
    if (i + 2 < end) x.z = w[i + 2];
    if (i + 3 < end) x.w = w[i + 3];
  }
  return make_uint4(order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w));
}

// Which rows stay.  One block per (sequence, K/V head): of the rows before the
// last `recent`, the budget - recent with the largest weights, equal ones from
// the lowest row on; and the last `recent`.  The smallest weight that stays is
// found digit by digit (13, 10 and 9 bits of the ordered integer) from
// histograms in shared memory, ending as soon as a whole bin stays.  Then each
// warp numbers the rows of its part of the sequence, and the kept rows' weights
// are gathered.  In place, row i's weight comes from a row at or after i, and a
// piece of the list is read before anything of it is written.
//
// The weights are read once where a sequence fits in shared memory (HELD), with
// all loads of a thread in flight together; a block per SM is bound by the latency
// of what it does in turn, not by the bytes.  (With the weights read again for
// every digit, and a block-wide count for every 4096 rows, 16 sequences of 16384 to
// 32768 rows with 8 heads took 29 us.)
template <bool HELD>
__global__ void __launch_bounds__(kSelectThreads, 1) attn_cache_select_sm103a(const EvictParams p) {
  extern __shared__ uint4 held[];
  __shared__ __align__(16) uint32_t hist[kSelectBins];
  __shared__ uint32_t warp_sum[32];
  __shared__ uint32_t sh_bin, sh_left, sh_all;
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
  const bool wide = (reinterpret_cast<uintptr_t>(w) & 15) == 0;   // 16-byte loads
  uint32_t left = (uint32_t)(p.budget - p.recent);   // rows still to be chosen
  const bool choose = left > 0;
  uint32_t prefix = 0, known = 0;                    // digits found so far, and their mask
  // groups of four rows, kLoads of them per thread and round
  constexpr int kLoads = 8;
  const int groups = (old + 3) / 4;
  if (choose) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 19 : pass == 1 ? 9 : 0;
      const uint32_t digit = pass == 0 ? 0x1fffu : pass == 1 ? 0x3ffu : 0x1ffu;
      const int bins = (int)digit + 1, per = pass == 0 ? bins / kSelectThreads : 1;   // per thread
      for (int i = tid; i < bins; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      for (int q0 = 0; q0 < groups; q0 += kLoads * kSelectThreads) {
        uint4 key[kLoads];
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
          const int q = q0 + e * kSelectThreads + tid;
          if (q >= groups) continue;
          key[e] = HELD && pass > 0 ? held[q] : order_keys(w, 4 * q, old, wide);
        }
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
          const int q = q0 + e * kSelectThreads + tid;
          if (q >= groups) continue;
          if (HELD && pass == 0) held[q] = key[e];
          // (a run of equal bins is added at once: where many weights are equal, their
          // additions wait for one another)
          const uint32_t k4[4] = {key[e].x, key[e].y, key[e].z, key[e].w};
          uint32_t run = 0, run_bin = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (4 * q + j >= old || (k4[j] & known) != prefix) continue;
            const uint32_t bin = (k4[j] >> shift) & digit;
            if (run > 0 && bin != run_bin) {
              atomicAdd(&hist[run_bin], run);
              run = 0;
            }
            run_bin = bin;
            ++run;
          }
          if (run > 0) atomicAdd(&hist[run_bin], run);
        }
      }
      __syncthreads();
      // the bin in which the count from the top reaches `left`: thread t holds
      // `per` bins from bins - 1 - t * per down
      const int top = bins - 1 - tid * per;
      uint32_t mine = 0;
      if (pass == 0) {
        static_assert(kSelectBins == 8 * kSelectThreads, "eight bins per thread");
        const uint4* at = reinterpret_cast<const uint4*>(hist + top - 7);
        const uint4 x = at[0], y = at[1];
        mine = x.x + x.y + x.z + x.w + y.x + y.y + y.z + y.w;
      } else if (top >= 0) {
        mine = hist[top];
      }
      uint32_t upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y;
      }
      if (lane == 31) warp_sum[warp] = upto;
      __syncthreads();
      const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u);
      uint32_t above = before + upto - mine;   // rows in higher bins
      if (above < left && above + mine >= left) {
        int j = 0;
        while (above + hist[top - j] < left) above += hist[top - j++];
        sh_bin = (uint32_t)(top - j);
        sh_left = left - above;
        sh_all = hist[top - j] == left - above ? 1 : 0;
      }
      __syncthreads();
      prefix |= sh_bin << shift;
      known |= digit << shift;
      left = sh_left;
      // the whole bin stays: what is above or equal to `prefix` does, whatever the
      // digits that follow
      if (sh_all) break;
    }
  } else {
    prefix = 0xffffffffu;   // above every weight: none of the old rows stays
  }
  // Rows above `prefix` stay, and the first `left` of those equal to it.  Thread t
  // numbers rows [t * part, (t + 1) * part): it counts them, learns how many come
  // before, and goes over them again.  (part / 4 is odd: 16-byte reads of
  // neighbouring threads then fall into different banks.)
  if (choose) {
    int part = (old + 4 * kSelectThreads - 1) / (4 * kSelectThreads) * 4;
    if (part % 8 == 0) part += 4;
    const int first = min(old, tid * part), last = min(old, first + part);
    auto each = [&](auto&& take) {   // take(row, ordered integer)
      for (int t = first; t < last; t += 4) {
        const uint4 k = HELD ? held[t / 4] : order_keys(w, t, old, wide);
        take(t, k.x);
        if (t + 1 < last) take(t + 1, k.y);
        if (t + 2 < last) take(t + 2, k.z);
        if (t + 3 < last) take(t + 3, k.w);
      }
    };
    __syncthreads();   // (the ordered integers are another thread's)
    uint32_t gt = 0, eq = 0;
    each([&](int, uint32_t key) {
      gt += key > prefix ? 1u : 0u;
      eq += key == prefix ? 1u : 0u;
    });
    // (a block holds at most 2^31 rows: one scan for each of the two counts)
    const uint32_t my_gt = gt, my_eq = eq;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, gt, d), z = __shfl_up_sync(0xffffffffu, eq, d);
      if (lane >= d) {
        gt += y;
        eq += z;
      }
    }
    if (lane == 31) {
      warp_sum[warp] = gt;
      hist[warp] = eq;
    }
    __syncthreads();
    gt += __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u) - my_gt;
    eq += __reduce_add_sync(0xffffffffu, lane < warp ? hist[lane] : 0u) - my_eq;
    each([&](int t, uint32_t key) {
      if (key > prefix || (key == prefix && eq < left)) keep[gt + min(eq, left)] = t;
      gt += key > prefix ? 1u : 0u;
      eq += key == prefix ? 1u : 0u;
    });
  }
  for (int i = tid; i < p.recent; i += kSelectThreads) keep[p.budget - p.recent + i] = old + i;
  __syncthreads();
  // the kept rows' weights (the list was written by this block)
  constexpr int kMoves = 4;
  for (int i0 = 0; i0 < p.budget; i0 += kMoves * kSelectThreads) {
    int t[kMoves];
    float x[kMoves];
#pragma unroll
    for (int e = 0; e < kMoves; ++e) {
      const int i = i0 + e * kSelectThreads + tid;
      t[e] = i < p.budget ? keep[i] : -1;
    }
#pragma unroll
    for (int e = 0; e < kMoves; ++e) x[e] = t[e] >= 0 ? w[t[e]] : 0.f;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kMoves; ++e)
      if (t[e] >= 0) w_out[i0 + e * kSelectThreads + tid] = x[e];
  }
  __syncthreads();
  // rows that follow start from nothing
  for (int i = p.budget + tid; i < min(n, p.stride_out); i += kSelectThreads) w_out[i] = 0.f;
}

// The page of row t of sequence b.
__device__ __forceinline__ int cache_page(const EvictParams& p, const int* table, int cols, int b,
                                          int t) {
  // (checked builds: an entry of the table)
  if (!attn_check(b >= 0 && b < p.B && t >= 0 && p.by_page.div(t) < cols, p.error_word)) return -1;
  return __ldcg(table + (long long)b * cols + p.by_page.div(t));
}
__device__ __forceinline__ bool cache_page_ok(const EvictParams& p, int id) {
  if (id >= 0 && id < p.num_pages) return true;
  atomicExch(p.error_word, 1);   // ATTN_ERR_INVALID_ARG
  return false;
}
// A row and a piece that there are (checked builds).
__device__ __forceinline__ bool cache_row_ok(const EvictParams& p, int g, int t, int vec) {
  return attn_check(g >= 0 && g < p.Hkv && t >= 0 && p.by_page.mod(t) < p.page && vec >= 0 &&
                        vec < p.vecs,
                    p.error_word);
}
// 16-byte piece `vec` of row t of head g, in page id.
__device__ __forceinline__ long long cache_piece(const EvictParams& p, int id, int g, int t,
                                                 int vec) {
  return (((long long)id * p.Hkv + g) * p.page + p.by_page.mod(t)) * p.vecs + vec;
}

constexpr int kMoveThreads = 256;

// K and V rows to other pages: row i of the output is row keep[i].  A thread
// moves a 16-byte piece of K and V of U rows; each step's loads for all of them
// go out together (keep and the target's page, the source's page, the rows).
template <int U>
__global__ void __launch_bounds__(kMoveThreads) attn_cache_move_sm103a(const EvictParams p) {
  griddep_wait();
  const int per_pass = kMoveThreads / p.vecs;
  const int vec = threadIdx.x % p.vecs, r = threadIdx.x / p.vecs;
  const int blocks = (p.budget + per_pass * U - 1) / (per_pass * U);
  const int bg = blockIdx.x / blocks, i0 = (blockIdx.x - bg * blocks) * U * per_pass + r;
  const int b = bg / p.Hkv, g = bg - b * p.Hkv;
  int src[U], from[U], to[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = i0 + u * per_pass;
    src[u] = i < p.budget ? __ldcg(p.keep + (size_t)bg * p.budget + i) : -1;
    to[u] = i < p.cols_out * p.page ? cache_page(p, p.table_out, p.cols_out, b, i) : -1;
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    from[u] = src[u] >= 0 ? cache_page(p, p.table, p.cols, b, src[u]) : 0;
  uint4 k[U], v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (src[u] < 0) continue;
    if (!cache_page_ok(p, from[u]) || !cache_page_ok(p, to[u]) ||
        !cache_row_ok(p, g, src[u], vec)) {
      src[u] = -1;
      continue;
    }
    const long long at = cache_piece(p, from[u], g, src[u], vec);
    k[u] = __ldcs(p.kpages + at);
    v[u] = __ldcs(p.vpages + at);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (src[u] < 0) continue;
    const long long at = cache_piece(p, to[u], g, i0 + u * per_pass, vec);
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
    int src[U], from[U], to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * per_pass + r;
      src[u] = i < p.budget ? __ldcg(keep + i) : -1;
      if (src[u] == i) src[u] = -1;   // it is there already
      to[u] = i < p.cols * p.page ? cache_page(p, p.table, p.cols, b, i) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      from[u] = src[u] >= 0 ? cache_page(p, p.table, p.cols, b, src[u]) : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (src[u] < 0) continue;
      if (!cache_page_ok(p, from[u]) || !cache_page_ok(p, to[u]) ||
          !cache_row_ok(p, g, src[u], vec))
        src[u] = -1;
      else x[u] = __ldcg(pool + cache_piece(p, from[u], g, src[u], vec));
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (src[u] >= 0) pool[cache_piece(p, to[u], g, i0 + u * per_pass + r, vec)] = x[u];
  }
}

}  // namespace chs
