// tokens_sm103a.cuh -- what is done per token around attention: rotary positions (alone, or
// together with the write to the paged cache) and the plan of a serving step (pages, slots,
// positions).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "fixed_div.h"
#include "sm103a_ptx.cuh"

namespace chs {

// ---------------------------------------------------------------- rotary positions
//
// The pair (x, y) number i of a head at position p turns by the angle
// 2 pi p f_i (f_i: turns per token):
//     x' = a (x cos - y sin),  y' = a (y cos + x sin).
// f_i is a 64-bit fraction of a turn, so p f_i modulo one turn is the low half
// of an integer product: exact at any position to p 2^-64 turns, where a
// product in floating point would lose the fraction as it grows.  Its upper 32
// bits go to fp32 (2^-25 of a half turn) and to sincospif.
//
// The bound is memory: each row of q and k is read and written once.  A block
// takes a few rows; its threads first make the rows' cosines and sines (one
// pair each, kept in shared memory), then each holds eight pairs' of one row
// in registers and turns those of one head after another, two 16-byte loads
// and stores a head.  A pair is read and written by one thread, so the output
// may be the input.

// Strides in elements; row r of a call is row r % S of batch r / S.
struct RopeTensor {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;    // null: not written
  long long in_batch, in_row, in_head, out_batch, out_row, out_head;
  int copy_rest;         // out != in: the values that are not turned are copied
};

struct RopeParams {
  RopeTensor q, k;
  int Hq, Hkv;
  const int* positions;       // [rows]; a negative one leaves the row out
  const uint64_t* turns;      // [rot / 2]
  float amplitude;
  int rows, S, Dh, rot;
  int inverse;                // turn the other way
  int rows_per_block;         // a power of two, at most 8
  FixedDiv div_s;
  // with the write to the paged cache
  const __nv_bfloat16* v;
  long long v_batch, v_row, v_head;
  __nv_bfloat16 *kpages, *vpages;   // [num_pages, Hkv, page, Dh]
  const int* slots;                 // [rows] page number * page + row in it; negative: none
  int slot_end;                     // num_pages * page
  FixedDiv div_page;
  int* error_word;
};

constexpr int kRopeThreads = 256, kRopeMaxRows = 8;

// Eight pairs of a head: (lo[e], hi[e]).
struct RopePairs {
  uint4 a, b;
};

__device__ __forceinline__ float rope_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float rope_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Turn eight pairs.  Halves: pair e is (a[e], b[e]); neighbours: pairs 0-3 lie in a, 4-7 in b.
// Products and sums in fp32, each result rounded once to bf16.
template <bool INTERLEAVED>
__device__ __forceinline__ RopePairs rope_turn(const RopePairs& v, const float (&c)[8],
                                               const float (&s)[8]) {
  const uint32_t wa[4] = {v.a.x, v.a.y, v.a.z, v.a.w}, wb[4] = {v.b.x, v.b.y, v.b.z, v.b.w};
  uint32_t ra[4], rb[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (INTERLEAVED) {
      const float x0 = rope_lo(wa[e]), y0 = rope_hi(wa[e]), x1 = rope_lo(wb[e]), y1 = rope_hi(wb[e]);
      ra[e] = pack_bf16x2(x0 * c[e] - y0 * s[e], y0 * c[e] + x0 * s[e]);
      rb[e] = pack_bf16x2(x1 * c[4 + e] - y1 * s[4 + e], y1 * c[4 + e] + x1 * s[4 + e]);
    } else {
      const float x0 = rope_lo(wa[e]), x1 = rope_hi(wa[e]), y0 = rope_lo(wb[e]), y1 = rope_hi(wb[e]);
      ra[e] = pack_bf16x2(x0 * c[2 * e] - y0 * s[2 * e], x1 * c[2 * e + 1] - y1 * s[2 * e + 1]);
      rb[e] = pack_bf16x2(y0 * c[2 * e] + x0 * s[2 * e], y1 * c[2 * e + 1] + x1 * s[2 * e + 1]);
    }
  }
  return RopePairs{make_uint4(ra[0], ra[1], ra[2], ra[3]), make_uint4(rb[0], rb[1], rb[2], rb[3])};
}

template <bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads)
    attn_rope_sm103a(const RopeParams p) {
  extern __shared__ float rope_cs[];   // [rows per block][cos rot / 2 | sin rot / 2]
  const int t = threadIdx.x, half = p.rot / 2;
  griddep_wait();
  griddep_launch_dependents();
  const int row0 = blockIdx.x * p.rows_per_block;
  for (int i = t; i < p.rows_per_block * half; i += kRopeThreads) {
    const int r = i / half, j = i - r * half;
    const int pos = row0 + r < p.rows ? p.positions[row0 + r] : -1;
    const uint64_t turn = (uint64_t)(uint32_t)max(pos, 0) * p.turns[j];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    rope_cs[r * p.rot + j] = c * p.amplitude;
    rope_cs[r * p.rot + half + j] = (p.inverse ? -s : s) * p.amplitude;
  }
  __syncthreads();

  // this thread's 16 values of a head, its row, and the heads it takes
  const int chunks = p.Dh / 16, chunk = t % chunks, lanes = kRopeThreads / chunks;
  const int heads_at_once = lanes / p.rows_per_block, lane = t / chunks;
  const int r = lane / heads_at_once, row = row0 + r;
  if (row >= p.rows || p.positions[row] < 0) return;
  const bool turned = chunk < p.rot / 16;
  int at_a, at_b;   // where the two groups of eight values lie in a head
  if (!turned || INTERLEAVED) {
    at_a = 16 * chunk;
    at_b = at_a + 8;
  } else {
    at_a = 8 * chunk;
    at_b = at_a + half;
  }
  float c[8], s[8];
  if (turned) {
    const float4* c4 = reinterpret_cast<const float4*>(rope_cs + r * p.rot + 8 * chunk);
    const float4* s4 = reinterpret_cast<const float4*>(rope_cs + r * p.rot + half + 8 * chunk);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float4 x = c4[e], y = s4[e];
      c[4 * e] = x.x, c[4 * e + 1] = x.y, c[4 * e + 2] = x.z, c[4 * e + 3] = x.w;
      s[4 * e] = y.x, s[4 * e + 1] = y.y, s[4 * e + 2] = y.z, s[4 * e + 3] = y.w;
    }
  }
  const int batch = p.div_s.div(row), i = row - batch * p.S;
  // (checked builds: a row of the batch, and a head's values)
  if (!attn_check(batch >= 0 && i >= 0 && i < p.S && at_a >= 0 && at_a + 8 <= p.Dh && at_b >= 8 &&
                      at_b + 8 <= p.Dh,
                  p.error_word))
    return;
  long long page_at = -1;   // of head 0 in a pool
  long long page_head = 0;
  if (APPEND) {
    const int slot = p.slots[row];
    if (slot >= p.slot_end) {
      if (t % (kRopeThreads / p.rows_per_block) == 0) atomicCAS(p.error_word, 0, 1);
    } else if (slot >= 0) {
      const int pg = p.div_page.div(slot), page = (int)p.div_page.d;
      page_head = (long long)page * p.Dh;
      page_at = pg * (p.Hkv * page_head) + (long long)(slot - pg * page) * p.Dh;
      // (checked builds: every head's row lies inside the pools)
      if (!attn_check(page_at >= 0 && page_at + (p.Hkv - 1) * page_head + p.Dh <=
                                          (long long)p.slot_end * p.Hkv * p.Dh,
                      p.error_word))
        page_at = -1;
    }
  }
  auto load = [&](const __nv_bfloat16* x) {
    return RopePairs{*reinterpret_cast<const uint4*>(x + at_a),
                     *reinterpret_cast<const uint4*>(x + at_b)};
  };
  auto store = [&](__nv_bfloat16* x, const RopePairs& v) {
    *reinterpret_cast<uint4*>(x + at_a) = v.a;
    *reinterpret_cast<uint4*>(x + at_b) = v.b;
  };
  const int h0 = lane % heads_at_once;
  // four heads' loads in flight before the first is turned
  constexpr int kUnroll = 4;
  auto heads = [&](const RopeTensor& x, int H, bool paged) {
    const __nv_bfloat16* in = x.in + batch * x.in_batch + i * x.in_row;
    __nv_bfloat16* out = x.out + batch * x.out_batch + i * x.out_row;
    const bool to_out = x.out != nullptr && (turned || x.copy_rest);
    if (!to_out && !paged) return;
    for (int h = h0; h < H; h += kUnroll * heads_at_once) {
      RopePairs v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (h + u * heads_at_once < H) v[u] = load(in + (h + u * heads_at_once) * x.in_head);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int g = h + u * heads_at_once;
        if (g < H) {
          if (turned) v[u] = rope_turn<INTERLEAVED>(v[u], c, s);
          if (to_out) store(out + g * x.out_head, v[u]);
          if (APPEND && paged) store(p.kpages + page_at + g * page_head, v[u]);
        }
      }
    }
  };
  heads(p.q, p.Hq, false);
  heads(p.k, p.Hkv, APPEND && page_at >= 0);
  if (APPEND && page_at >= 0) {
    const __nv_bfloat16* in = p.v + batch * p.v_batch + i * p.v_row;
    for (int h = h0; h < p.Hkv; h += heads_at_once)
      store(p.vpages + page_at + h * page_head, load(in + h * p.v_head));
  }
}

// ---------------------------------------------------------------- the plan of a serving step
//
// Sequence b holds n_b rows and changes by d_b: new tokens (d_b > 0), or rows
// taken back from its end (d_b < 0; all of them: the request is finished).
// Pages that no row needs any more go onto the stack of free pages, in the
// order of the sequences and of their columns; then each page that new rows
// need comes off its top, in the same order.  The new tokens of all sequences
// are packed one behind another.  All of it is prefix sums over the sequences:
// of new tokens, of pages given back, of pages taken.
//
// One cluster does it in one launch.  Every CTA makes all the sums (B is
// small next to the launch itself), so that nothing is passed between them;
// they meet once, between the last read of what the call may write in place
// and the first write, and then write a share each.  Two accesses need no
// order: pages are read from the stack below its old top and from columns
// that shrinking sequences leave, and written above the old top and to
// columns that growing sequences gain.  Many tokens' positions and slots
// (262144 of 2048 sequences: 63 us on eight SMs, 13 so) are left to a second
// launch on every SM, which finds all it needs in the first one's results.

struct PlanParams {
  const int* delta;      // [B]
  const int* seqlens;    // [B]
  int* seqlens_out;      // [B], may be seqlens
  int* table;            // [B, cols]
  int* free_pages;       // [capacity]
  const int* num_free;   // [1]
  int* num_free_out;     // [1], may be num_free
  int* cu;               // [B + 1]
  int *positions, *slots;   // [T]
  int B, cols, page, num_pages, capacity, T;
  int fill;              // the tokens' positions and slots too
  FixedDiv div_page;
  int* error_word;
};

constexpr int kPlanThreads = 1024, kPlanMaxB = 8192, kPlanMaxCtas = 8;
constexpr size_t plan_smem_bytes(int B) { return ((size_t)4 * B + 3) * sizeof(int); }

// The last i in [0, n) with first[i] <= x, for ascending first with first[0] <= x.
__device__ __forceinline__ int plan_find(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads)
    attn_cache_plan_sm103a(const PlanParams p) {
  // per sequence: rows before; where its new tokens, pages taken and pages given back begin
  // (ends behind the last)
  extern __shared__ int plan_smem[];
  int* rows = plan_smem;
  int* tok = rows + p.B;
  int* take = tok + p.B + 1;
  int* give = take + p.B + 1;
  __shared__ long long part[3][kPlanThreads / 32];
  const int t = threadIdx.x, lane = t % 32, warp = t / 32;
  griddep_wait();
  griddep_launch_dependents();

  // a run of sequences per thread
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(t * per, p.B), b1 = min(b0 + per, p.B);
  const int room = p.cols * p.page;
  auto pages_of = [&](int n) { return p.div_page.div(n) + (p.div_page.mod(n) != 0); };
  // the change that is made: none where it, or the length, is out of range
  auto change = [&](int n, int d, bool& wrong) {
    const long long after = (long long)n + d;
    wrong = n < 0 || n > room || after < 0 || after > room;
    return wrong ? 0 : d;
  };
  long long sum[3] = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const int n = p.seqlens[b];
    bool wrong;
    const int d = change(n, p.delta[b], wrong);
    if (wrong) {
      if (blockIdx.x == 0) atomicCAS(p.error_word, 0, 1);   // ATTN_ERR_INVALID_ARG
      rows[b] = n;
      continue;
    }
    rows[b] = n;
    const int gain = pages_of(n + d) - pages_of(n);
    sum[0] += max(d, 0);
    sum[1] += max(gain, 0);
    sum[2] += max(-gain, 0);
  }
  const int top = *p.num_free;
  long long before[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long run = sum[k];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long y = __shfl_up_sync(0xffffffffu, run, d);
      if (lane >= d) run += y;
    }
    if (lane == 31) part[k][warp] = run;
    before[k] = run - sum[k];
  }
  __syncthreads();
  if (warp < 3) {
    long long run = part[warp][lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long y = __shfl_up_sync(0xffffffffu, run, d);
      if (lane >= d) run += y;
    }
    part[warp][lane] = run;
  }
  __syncthreads();
  const long long tokens = part[0][31], taken = part[1][31], given = part[2][31];
  const bool top_ok = top >= 0 && top <= p.capacity;
  const bool too_many = tokens > 0x7fffffff || !top_ok ||
                        top + given - taken > p.capacity || top + given > 0x7fffffff;
  const bool too_few = top + given < taken;
  const bool off = too_many || too_few;   // then nothing changes
  if (off && blockIdx.x == 0 && t == 0)
    atomicCAS(p.error_word, 0, too_many ? 1 : 5);   // ATTN_ERR_INVALID_ARG, ATTN_ERR_NO_MEMORY
  if (!off) {
    int at[3];
#pragma unroll
    for (int k = 0; k < 3; ++k)
      at[k] = (int)(before[k] + (warp > 0 ? part[k][warp - 1] : 0));
    for (int b = b0; b < b1; ++b) {
      bool wrong;
      const int n = rows[b], d = change(n, p.delta[b], wrong);
      const int gain = d == 0 ? 0 : pages_of(n + d) - pages_of(n);
      tok[b] = at[0];
      take[b] = at[1];
      give[b] = at[2];
      at[0] += max(d, 0);
      at[1] += max(gain, 0);
      at[2] += max(-gain, 0);
    }
    if (t == 0) {
      tok[p.B] = (int)tokens;
      take[p.B] = (int)taken;
      give[p.B] = (int)given;
    }
  }
  // every CTA has read what the writes below may change
  if (gridDim.x > 1) cluster_sync(); else __syncthreads();

  const int T0 = blockIdx.x * kPlanThreads + t, TN = gridDim.x * kPlanThreads;
  if (off) {
    for (int b = T0; b < p.B; b += TN) p.seqlens_out[b] = rows[b];
    for (int b = T0; b <= p.B; b += TN) p.cu[b] = 0;
    if (T0 == 0) *p.num_free_out = top;
    for (int i = T0; p.fill && i < p.T; i += TN) p.positions[i] = p.slots[i] = -1;
    return;
  }
  // (checked builds: column col of sequence b lies inside the table)
  auto in_table = [&](int b, int col) {
    return attn_check(b >= 0 && b < p.B && col >= 0 && col < p.cols, p.error_word);
  };
  // entry i of the stack after the pages given back were pushed
  auto stack = [&](int i) {
    if (!attn_check(i >= 0 && i < top + given, p.error_word)) return -1;
    if (i < top) return p.free_pages[i];
    const int r = i - top, b = plan_find(give, p.B, r);
    const int col = pages_of(rows[b]) - (give[b + 1] - give[b]) + (r - give[b]);
    return in_table(b, col) ? p.table[(size_t)b * p.cols + col] : -1;
  };
  auto pop = [&](int i) { return stack(top + (int)given - 1 - i); };
  for (int b = T0; b < p.B; b += TN) {
    bool wrong;
    p.seqlens_out[b] = rows[b] + change(rows[b], p.delta[b], wrong);
  }
  for (int b = T0; b <= p.B; b += TN) p.cu[b] = tok[b];
  if (T0 == 0) *p.num_free_out = top + (int)(given - taken);
  for (int i = T0; i < (int)taken; i += TN) {
    const int b = plan_find(take, p.B, i);
    const int col = pages_of(rows[b]) + (i - take[b]);
    if (in_table(b, col)) p.table[(size_t)b * p.cols + col] = pop(i);
  }
  for (int i = top + T0; i < top + (int)(given - taken); i += TN)
    if (attn_check(i < p.capacity, p.error_word)) p.free_pages[i] = stack(i);
  for (int i = T0; p.fill && i < p.T; i += TN) {
    int pos = -1, slot = -1;
    if (i < (int)tokens) {
      const int b = plan_find(tok, p.B, i), held = pages_of(rows[b]);
      pos = rows[b] + (i - tok[b]);
      const int col = p.div_page.div(pos);
      const int pg = !in_table(b, col) ? -1
                     : col < held      ? p.table[(size_t)b * p.cols + col]
                                       : pop(take[b] + col - held);
      if ((unsigned)pg < (unsigned)p.num_pages)
        slot = pg * p.page + (pos - col * p.page);
      else
        atomicCAS(p.error_word, 0, 1);
    }
    p.positions[i] = pos;
    p.slots[i] = slot;
  }
}

// The tokens' positions and slots, from the plan's results: four in a row per thread.
constexpr int kFillThreads = 256, kFillRows = 4;
__global__ void __launch_bounds__(kFillThreads)
    attn_cache_fill_sm103a(const PlanParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int tokens = min(__ldcg(p.cu + p.B), p.T);
  const int i0 = (blockIdx.x * kFillThreads + threadIdx.x) * kFillRows;
  if (i0 >= p.T) return;
  int b = 0, first = 0, next = 0;   // rows first .. next - 1 are sequence b's
  if (i0 < tokens) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (p.cu[mid] <= i0) lo = mid; else hi = mid;
    }
    b = lo;
    first = p.cu[b];
    next = p.cu[b + 1];
  }
  int pos[kFillRows], slot[kFillRows];
#pragma unroll
  for (int e = 0; e < kFillRows; ++e) {
    const int i = i0 + e;
    pos[e] = slot[e] = -1;
    if (i < tokens) {
      while (i >= next) {
        ++b;
        first = next;
        next = p.cu[b + 1];
      }
      pos[e] = p.seqlens_out[b] - (next - first) + (i - first);
      const int col = p.div_page.div(pos[e]);
      const bool in = attn_check(b < p.B && col >= 0 && col < p.cols, p.error_word);
      const int pg = in ? p.table[(size_t)b * p.cols + col] : -1;
      if ((unsigned)pg < (unsigned)p.num_pages)
        slot[e] = pg * p.page + (pos[e] - col * p.page);
      else
        atomicCAS(p.error_word, 0, 1);
    }
  }
#pragma unroll
  for (int e = 0; e < kFillRows; ++e) {
    if (i0 + e < p.T) {
      p.positions[i0 + e] = pos[e];
      p.slots[i0 + e] = slot[e];
    }
  }
}

}  // namespace chs
