// key_weights_few_sm103a.cuh -- the attention weight that each key of a prompt
// received from a few voting queries (sm_103a): attn_key_weights with `queries`
// set, or of a prompt of up to 32 rows, where the voting queries of a K/V head's
// whole group fit in one tile.
//
//   w[b, g, j] (+)= sum over heads h of the group and the last `queries` queries
//                   i >= j of  exp(scale q_hi . k_j - lse_hi)
//
// The same product as in key_weights_sm103a.cuh, S^T = K Q^T with the
// log-sum-exps as one more step, turned around in time: there a CTA keeps 128
// keys and walks the queries; here it keeps the group's queries (`pad` rows per
// head, up to 256 in all) and their log-sum-exps in shared memory and walks the
// keys, 128 at a time.  A block of keys is then one wide tile: one K tile is
// loaded, one S computed, one sum taken, and nothing is handed over.  (Walking
// queries, a block of keys cost two tiles with a K, Q and log-sum-exp set of
// their own: 61 us for 4 x 8 heads of 16384 to 32768 keys and 64 queries, against
// 15 us of memory traffic.)  Now 43 us: the exponentials alone are 1024 cycles per SM
// for 128 keys and 256 queries, 22 us in all, and a step of MMAs and waits, 382 cycles
// to issue per 128 columns, feeds them; without the sums 36 us are left.
//
// Split: as in the paged decode, the blocks of all (sequence, K/V head) units
// form a line, a unit's first place standing for the cost of its start, and each
// CTA (one per SM) takes an equal part.  Blocks alternate between two groups of
// four summing warps, each with an S buffer of its own, which is filled and freed by
// halves of 128 columns: one half's next block is computed while the other half is
// summed (by whole buffers 46 us instead of
// 43; with four groups of summing warps 49).
//
// Rows that pad the tile, and those past the end of a head's queries, become copies of the
// head's last voting query (its first head's, past the last head), which every key of the
// sequence is visible to, with a log-sum-exp of 3e38: their terms are 0 whenever that
// query's own are a number.  (Rows of zeros would meet an infinite key as 0 * inf = NaN,
// and -inf would make NaN of an infinite score.)  Only blocks that reach into the voting
// queries themselves are masked.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "key_weights_sm103a.cuh"
#include "sm103a_ptx.cuh"

namespace chs {

template <int DH>
struct KeyFewCfg {
  static constexpr int kBoxes = DH / 64;
  static constexpr int kCols = DH == 256 ? 128 : 256;   // voting rows, at most
  static constexpr int kQBox = kCols * 128;             // bytes: kCols rows of 64 columns
  static constexpr int kKBox = 128 * 128;
  static constexpr int kKTile = kBoxes * kKBox;
  static constexpr int kSlots = DH == 64 ? 8 : DH == 128 ? 4 : 2;   // K tiles
  // warps 0-3 and 4-7 sums, 8 MMA, 9 K and Q, 10 log-sum-exps
  static constexpr int kThreads = 352;
  static constexpr int kWarpIssuer = 8, kWarpProducer = 9, kWarpLse = 10;
};

template <int DH>
struct KeyFewSmem {
  using Cfg = KeyFewCfg<DH>;
  uint8_t q[Cfg::kBoxes * Cfg::kQBox];
  uint8_t k[Cfg::kSlots][Cfg::kKTile];
  // the log-sum-exps' step, [two blocks of 8 columns][rows]: parts and zeros | ones
  uint4 nlse[2][Cfg::kCols];
  uint4 ones[2][128];
  uint64_t full[Cfg::kSlots], empty[Cfg::kSlots];
  uint64_t q_loaded, q_ready, q_free;
  uint64_t s_full[2][2], s_empty[2][2], mma_done;   // [buffer][half]
  uint32_t tmem_base;
  int abort_flag;
};

struct KeyFewParams {
  int B, Hq, Hkv, G, S;
  int causal, queries, accumulate;
  int pad, cols;         // rows per head; rows of the tile (a multiple of 32)
  int ctas;
  float scale_log2;
  float lse_hi, lse_lo;  // -log2(e) / scale_log2 in two parts
  const float* lse;      // [B, Hq, S]
  const int* seqlens;    // [B] or null (every sequence holds S)
  float* weights;        // [B, Hkv, stride]
  int stride;
  int* error_word;
};

// Blocks [block, block + count) of unit (b, g) of L keys; its voting queries are
// q0 .. L - 1.
struct KeyFewSegment {
  int b, g, L, q0, block, count;
};

// The segments of one CTA in order; every warp walks them for itself.
struct KeyFewWalk {
  int cur, end;
  int b, g, at;   // next: unit, and place in it (0: before its blocks)
  int L;

  static __device__ __forceinline__ int len(const KeyFewParams& p, int b) {
    const int n = p.seqlens ? __ldcg(p.seqlens + b) : p.S;
    return n < 0 || n > p.S ? 0 : n;
  }
  static __device__ __forceinline__ int places(int n) { return n > 0 ? (n + 127) / 128 + 1 : 0; }

  __device__ __forceinline__ void init(const KeyFewParams& p, int cta) {   // one whole warp
    const int lane = threadIdx.x % 32;
    int total = 0;
    for (int bb = lane; bb < p.B; bb += 32) total += places(len(p, bb)) * p.Hkv;
    total = __reduce_add_sync(0xffffffffu, total);
    const int share = max(1, (total + p.ctas - 1) / p.ctas);
    cur = (int)min((long long)total, (long long)cta * share);
    end = min(total, cur + share);
    b = g = at = L = 0;
    if (cur >= end) return;
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int n = b0 + lane < p.B ? len(p, b0 + lane) : 0;
      const int mine = places(n) * p.Hkv;
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
        L = __shfl_sync(0xffffffffu, n, from);
        const int offset = cur - before - __shfl_sync(0xffffffffu, upto - mine, from);
        g = offset / places(L);
        at = offset - g * places(L);
        return;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }

  __device__ __forceinline__ bool next(const KeyFewParams& p, KeyFewSegment& s) {
    while (cur < end) {
      if (g == p.Hkv) {
        g = 0;
        do {
          L = len(p, ++b);
        } while (L == 0);
      }
      const int take = min(places(L) - at, end - cur);
      s.b = b;
      s.g = g;
      s.L = L;
      s.q0 = max(0, L - p.queries);
      s.block = max(at - 1, 0);
      s.count = at == 0 ? take - 1 : take;
      cur += take;
      at += take;
      if (at == places(L)) {
        at = 0;
        ++g;
      }
      if (s.count > 0) return true;
    }
    return false;
  }
};

template <int DH>
__global__ void __launch_bounds__(KeyFewCfg<DH>::kThreads, 1)
    attn_key_weights_few_sm103a(const __grid_constant__ CUtensorMap map_q,
                                const __grid_constant__ CUtensorMap map_k, const KeyFewParams p) {
  using Cfg = KeyFewCfg<DH>;
  using Smem = KeyFewSmem<DH>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~uintptr_t(1023));
  volatile int* abort = &sm.abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    for (int i = 0; i < Cfg::kSlots; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.q_loaded, 1);
    mbar_init(&sm.q_ready, 1);
    mbar_init(&sm.q_free, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.s_full[i / 2][i % 2], 1);
      mbar_init(&sm.s_empty[i / 2][i % 2], 4);   // one arrival per warp of a group
    }
    mbar_init(&sm.mma_done, 1);
    fence_mbarrier_init();
  }
  if (warp == Cfg::kWarpIssuer) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  // ones in the first three columns of A, zeros in the others and in B's second
  // eight (the first eight come with each unit)
  for (int i = threadIdx.x; i < 128; i += Cfg::kThreads) {
    sm.ones[0][i] = make_uint4(0x3f803f80u, 0x00003f80u, 0u, 0u);
    sm.ones[1][i] = make_uint4(0u, 0u, 0u, 0u);
  }
  for (int i = threadIdx.x; i < Cfg::kCols; i += Cfg::kThreads)
    sm.nlse[1][i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = sm.tmem_base;
  // the lengths, q, k and lse may come from the previous kernel
  griddep_wait();
  if (blockIdx.x == 0 && p.seqlens)
    for (int b = threadIdx.x; b < p.B; b += Cfg::kThreads) {   // an impossible length is an error
      const int n = __ldcg(p.seqlens + b);
      if (n < 0 || n > p.S) atomicExch(p.error_word, 1);   // ATTN_ERR_INVALID_ARG
    }
  __syncwarp();
  KeyFewWalk walk;
  walk.init(p, blockIdx.x);
  KeyFewSegment s;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t par) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, par, abort));
  };

  if (warp == Cfg::kWarpProducer) {
    KwRing<Cfg::kSlots> r;
    uint32_t loaded = 0, pars = 0, nseg = 0;
    while (ok && walk.next(p, s)) {
      // the group's voting queries, once the last unit's MMAs have read theirs
      if (nseg > 0 && !(ok = wait(&sm.q_free, (nseg - 1) & 1u))) break;
      ++nseg;
      // (checked builds: rows of a K/V head and its query heads)
      const bool head_in = attn_check(s.b >= 0 && s.b < p.B && s.g >= 0 && s.g < p.Hkv,
                                      p.error_word);
      const bool q_in = attn_check(s.q0 >= 0 && s.q0 < p.S, p.error_word) && head_in;
      if (lane == 0)
        mbar_arrive_expect_tx(&sm.q_loaded, q_in ? p.G * Cfg::kBoxes * p.pad * 128 : 0);
      __syncwarp();
      for (int i = lane; q_in && i < p.G * Cfg::kBoxes; i += 32) {
        const int h = i / Cfg::kBoxes, x = i - h * Cfg::kBoxes;
        tma_load_3d(sm.q + x * Cfg::kQBox + h * p.pad * 128, &map_q, &sm.q_loaded, 64 * x, s.q0,
                    s.b * p.Hq + s.g * p.G + h);
      }
      for (int j = 0; j < s.count; ++j) {
        if (!(ok = wait(&sm.empty[r.i], r.par ^ 1u))) break;
        if (lane == 0) {
          const bool in =
              attn_check(s.block >= 0 && 128 * (s.block + j) < p.S, p.error_word) && head_in;
          mbar_arrive_expect_tx(&sm.full[r.i], in ? Cfg::kKTile : 0);
          if (in)
            tma_load_4d(sm.k[r.i], &map_k, &sm.full[r.i], 0, 128 * (s.block + j), 0,
                        s.b * p.Hkv + s.g);
        }
        loaded |= 1u << r.i;
        pars = (pars & ~(1u << r.i)) | (r.par << r.i);
        r.step();
      }
    }
    // every copy this warp started has landed before the CTA may exit
    if (lane == 0) {
      if (nseg > 0) mbar_wait_drain(&sm.q_loaded, (nseg - 1) & 1u);
      for (int i = 0; i < Cfg::kSlots; ++i)
        if (loaded & (1u << i)) mbar_wait_drain(&sm.full[i], (pars >> i) & 1u);
    }
  } else if (warp == Cfg::kWarpLse) {
    uint32_t nseg = 0;
    const int pad_log2 = 31 - __clz(p.pad);   // (a power of two)
    while (ok && walk.next(p, s)) {
      const int n = s.L - s.q0;   // voting queries
      const float* lse = p.lse + ((size_t)s.b * p.Hq + (size_t)s.g * p.G) * p.S + s.q0;
      float x[Cfg::kCols / 32];
#pragma unroll
      for (int k = 0; k < Cfg::kCols / 32; ++k) {
        const int col = 32 * k + lane, h = col >> pad_log2, i = col - h * p.pad;
        x[k] = h < p.G && i < n ? __ldcg(lse + (size_t)h * p.S + i) : 0.f;
      }
      if (nseg > 0 && !(ok = wait(&sm.q_free, (nseg - 1) & 1u))) break;
#pragma unroll
      for (int k = 0; k < Cfg::kCols / 32; ++k)
        sm.nlse[0][32 * k + lane] = key_weights_lse_parts(x[k], p.lse_hi, p.lse_lo);
      if (!(ok = wait(&sm.q_loaded, nseg & 1u))) break;
      ++nseg;
      if (n < p.pad || p.G * p.pad < p.cols) {   // there are rows without a query
#pragma unroll 1
        for (int col = lane; col < p.cols; col += 32) {
          const int h = col >> pad_log2;
          if (h < p.G && col - h * p.pad < n) continue;
          sm.nlse[0][col] = make_uint4(0x0000ff7fu, 0u, 0u, 0u);   // the lowest bf16 number
          const int from = (h < p.G ? h * p.pad : 0) + n - 1;
#pragma unroll 1
          for (int box = 0; box < Cfg::kBoxes; ++box) {
            uint8_t* q = sm.q + box * Cfg::kQBox;
            uint4 y[8];   // (a row's 16-byte pieces are swizzled by its number)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              y[e] = *reinterpret_cast<const uint4*>(q + from * 128 + ((e ^ from) & 7) * 16);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(q + col * 128 + ((e ^ col) & 7) * 16) = y[e];
          }
        }
      }
      fence_proxy_async_smem();   // (the MMA reads them)
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_ready);
    }
  } else if (warp == Cfg::kWarpIssuer) {
    const int halves = p.cols > 128 ? 2 : 1;
    const uint64_t dk = smem_desc_sw128(smem_u32(sm.k[0]), 16, 1024);
    const uint64_t dq = smem_desc_sw128(smem_u32(sm.q), 16, 1024);
    // no swizzle: core matrices of 8 rows of 16 bytes 128 bytes apart, the second
    // eight columns behind the first
    constexpr uint64_t kPlain = ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
    const uint64_t d1 = kPlain | ((smem_u32(sm.ones) >> 4) & 0x3FFFu) | (uint64_t)(2048 >> 4) << 16;
    const uint64_t dl =
        kPlain | ((smem_u32(sm.nlse) >> 4) & 0x3FFFu) | (uint64_t)(Cfg::kCols * 16 >> 4) << 16;
    KwRing<Cfg::kSlots> r;
    KwRing<2> b;   // S buffers
    uint32_t nseg = 0;
    while (ok && walk.next(p, s)) {
      // (q_loaded: what the copies wrote; q_ready: what the other warp did)
      if (!(ok = wait(&sm.q_loaded, nseg & 1u)) || !(ok = wait(&sm.q_ready, nseg & 1u))) break;
      ++nseg;
      for (int j = 0; j < s.count; ++j) {
        if (!(ok = wait(&sm.full[r.i], r.par))) break;
        const uint64_t k = dk + (uint64_t)r.i * (Cfg::kKTile >> 4);
        for (int h = 0; h < halves; ++h) {
          if (!(ok = wait(&sm.s_empty[b.i][h], b.par ^ 1u))) break;
          tc_fence_after_sync();
          const uint32_t dS = tbase + 256u * b.i + 128u * h;
          const uint32_t idesc = idesc_bf16_f32(128, 0, false, false) |
                                 (uint32_t)(min(128, p.cols - 128 * h) >> 3) << 17;
          const uint64_t qh = dq + (uint64_t)h * (128 * 128 >> 4), lh = dl + (uint64_t)h * 128;
          if (elect_one_sync()) {
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk)
              mma_bf16_ss(dS, k + (((kk / 4) * Cfg::kKBox + (kk % 4) * 32) >> 4),
                          qh + (((kk / 4) * Cfg::kQBox + (kk % 4) * 32) >> 4), idesc,
                          kk > 0 ? 1u : 0u);
            mma_bf16_ss(dS, d1, lh, idesc, 1u);
            mma_commit(&sm.s_full[b.i][h]);
            if (h + 1 == halves) {
              mma_commit(&sm.empty[r.i]);
              if (j + 1 == s.count) mma_commit(&sm.q_free);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        __syncwarp();
        r.step();
        b.step();
      }
    }
    // nothing of this warp's may still run on the tensor core at teardown
    mma_commit_warp(&sm.mma_done);
    mbar_wait_drain(&sm.mma_done, 0);
  } else {
    const int group = warp / 4, tid = threadIdx.x % 128;
    const uint32_t colS = tbase + ((uint32_t)(tid & ~31) << 16) + 256u * group;
    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
    const uint32_t in_head = (uint32_t)p.pad - 1u;   // (a power of two less one)
    uint32_t count = 0, par = 0;
    const int halves = p.cols > 128 ? 2 : 1;
    auto release = [&](int h) {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.s_empty[group][h]);
    };
    while (ok && walk.next(p, s)) {
      for (int j = 0; j < s.count; ++j, ++count) {
        if ((count & 1u) != (uint32_t)group) continue;
        const int key0 = 128 * (s.block + j), key = key0 + tid;
        const bool masked = p.causal && key0 + 127 > s.q0;   // it reaches into the voting queries
        const uint32_t hidden = (uint32_t)max(0, key - s.q0);   // of a head's columns, the first
        // columns are summed by 128 at most, and those sums added: the error of a long
        // sum grows with their number
        float total = 0.f;
#pragma unroll 1
        for (int h = 0; h < halves; ++h) {
          if (!(ok = mbar_wait(&sm.s_full[group][h], par, abort))) break;
          tc_fence_after_sync();
          const uint32_t col = colS + 128u * h;
          const int cols = min(128, p.cols - 128 * h);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          if (cols == 128 && !masked) {
            uint32_t y0[32], y1[32], y2[32], y3[32];
            tmem_ld_32x32b_x32(col, y0);
            tmem_ld_32x32b_x32(col + 32, y1);
            tmem_ld_wait(y0);
            tmem_ld_wait(y1);
            tmem_ld_32x32b_x32(col + 64, y2);
            tmem_ld_32x32b_x32(col + 96, y3);
            key_weights_add(y0, scale2, sum);
            key_weights_add(y1, scale2, sum);
            tmem_ld_wait(y2);
            tmem_ld_wait(y3);
            release(h);   // S is in registers
            key_weights_add(y2, scale2, sum);
            key_weights_add(y3, scale2, sum);
          } else {
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) {
              uint32_t y[32];
              tmem_ld_32x32b_x32(col + c, y);
              tmem_ld_wait(y);
              if (masked) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (((uint32_t)(128 * h + c + e) & in_head) < hidden) y[e] = 0xff800000u;
              }
              key_weights_add(y, scale2, sum);
            }
            release(h);
          }
          total += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        }
        if (!ok) break;
        par ^= 1u;
        if (key < s.L) {
          float* w = p.weights + ((size_t)s.b * p.Hkv + s.g) * p.stride + key;
          *w = p.accumulate ? *w + total : total;
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == Cfg::kWarpIssuer) {
    tc_fence_after_sync();
    tmem_dealloc(tbase, 512);
  }
  if (threadIdx.x == 0 && sm.abort_flag) atomicExch(p.error_word, 4);   // ATTN_ERR_TIMEOUT
}

template <int DH>
constexpr size_t key_few_smem_bytes() {
  return sizeof(KeyFewSmem<DH>) + 1024;   // + alignment slack
}

}  // namespace chs
