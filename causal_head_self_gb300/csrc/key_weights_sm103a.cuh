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
// A CTA takes 128 keys of one (sequence, K/V head) and walks the tiles of 128
// queries that see any of them, head after head.  The product is taken
// transposed, S^T = K Q^T (keys as rows): a thread then owns a key, and the sum
// over queries stays in its registers -- no atomics, no shuffles, and the same
// bits every time.  The queries' -lse / ln 2 are laid out in shared memory, one
// tile after another, and read as broadcasts.
//
// Two CTAs share an SM (one at Dh = 256), so that one's exponentials run beside
// the other's products.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "sm103a_ptx.cuh"

namespace chs {

struct KeyWeightsParams {
  int B, Hq, Hkv, G, S;
  int causal, window, queries, accumulate;
  int key_blocks;
  float scale_log2;
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
  static constexpr int kTile = kBoxes * kBox;
  static constexpr int kStages = DH == 64 ? 4 : 2;    // Q tiles
  static constexpr int kCtasPerSm = DH == 256 ? 1 : 2;
  static constexpr uint32_t kCols = 256;              // S0, S1
  static constexpr int kThreads = 192;                // warps 0-3 sums, 4 loads, 5 MMA
  static constexpr int kLse = 4;                      // tiles of log-sum-exps held
};

template <int DH>
struct KeyWeightsSmem {
  using Cfg = KeyWeightsCfg<DH>;
  uint8_t k[Cfg::kTile];
  uint8_t q[Cfg::kStages][Cfg::kTile];
  float nlse[Cfg::kLse][128];
  uint64_t k_full, q_full[Cfg::kStages], q_empty[Cfg::kStages];
  uint64_t l_full[Cfg::kLse], l_empty[Cfg::kLse];
  uint64_t s_full[2], s_empty[2], mma_done;
  uint32_t tmem_base;
  int abort_flag;
};

// The tiles of one CTA: query rows [q0 + 128 i, ...) below q_end, i < n, for
// each head of the group.
struct KeyWeightsItem {
  int b, g, kb, L, q0, q_end, n;
};

__device__ __forceinline__ KeyWeightsItem key_weights_item(const KeyWeightsParams& p, int item) {
  KeyWeightsItem it;
  const int per = p.B * p.Hkv;
  it.kb = item / per;   // the first key blocks have the most queries: they come first
  const int bg = item - it.kb * per;
  it.b = bg / p.Hkv;
  it.g = bg - it.b * p.Hkv;
  it.L = p.seqlens ? __ldcg(p.seqlens + it.b) : p.S;
  if (it.L < 0 || it.L > p.S) it.L = 0;
  const int k0 = 128 * it.kb;
  it.q0 = p.queries > 0 ? max(0, it.L - p.queries) : 0;
  if (p.causal) it.q0 = max(it.q0, k0);
  it.q_end = it.L;
  if (p.window > 0) it.q_end = (int)min((long long)it.L, (long long)k0 + 127 + p.window);
  it.n = it.q_end > it.q0 ? (it.q_end - it.q0 + 127) / 128 : 0;
  return it;
}

__device__ __forceinline__ void mbar_wait_drain_kw(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) return;
  }
}

template <int DH>
__global__ void __launch_bounds__(192, KeyWeightsCfg<DH>::kCtasPerSm)
    attn_key_weights_sm103a(const __grid_constant__ CUtensorMap map_q,
                            const __grid_constant__ CUtensorMap map_k, const KeyWeightsParams p) {
  using Cfg = KeyWeightsCfg<DH>;
  using Smem = KeyWeightsSmem<DH>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~uintptr_t(1023));
  volatile int* abort = &sm.abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  griddep_wait();
  const KeyWeightsItem it = key_weights_item(p, blockIdx.x);
  const int k0 = 128 * it.kb;
  if (k0 >= it.L) {
    // (an empty sequence has no keys; an impossible length is an error)
    if (it.L == 0 && it.kb == 0 && threadIdx.x == 0 && p.seqlens && __ldcg(p.seqlens + it.b) != 0)
      atomicExch(p.error_word, 1);   // ATTN_ERR_INVALID_ARG
    return;
  }
  const int tiles = it.n * p.G;
  if (tiles == 0) {   // no voting query sees these keys
    const int j = k0 + threadIdx.x;
    if (!p.accumulate && threadIdx.x < 128 && j < it.L)
      p.weights[((size_t)it.b * p.Hkv + it.g) * p.stride + j] = 0.f;
    return;
  }
  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    mbar_init(&sm.k_full, 1);
    for (int i = 0; i < Cfg::kStages; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
    }
    for (int i = 0; i < Cfg::kLse; ++i) {
      mbar_init(&sm.l_full[i], 32);
      mbar_init(&sm.l_empty[i], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_empty[i], 128);
    }
    mbar_init(&sm.mma_done, 1);
    fence_mbarrier_init();
  }
  if (warp == 5) {
    tmem_alloc(&sm.tmem_base, Cfg::kCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = sm.tmem_base;

  if (warp == 4) {
    // loads: K once, then per tile Q (one lane) and the log-sum-exps (the warp,
    // fetched a tile ahead)
    const int bg = it.b * p.Hkv + it.g;
    if (lane == 0) {
      mbar_arrive_expect_tx(&sm.k_full, Cfg::kTile);
      for (int x = 0; x < Cfg::kBoxes; ++x)
        tma_load_3d(sm.k + x * Cfg::kBox, &map_k, &sm.k_full, 64 * x, k0, bg);
    }
    uint32_t q_loads = 0;
    bool ok = true;
    float l[4];
    auto fetch = [&](int h, int qt) {
      const float* src = p.lse + ((size_t)it.b * p.Hq + it.g * p.G + h) * p.S;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = it.q0 + 128 * qt + 32 * e + lane;
        l[e] = i < it.q_end ? __ldcg(src + i) : 0.f;
      }
    };
    fetch(0, 0);
    int t = 0;
    for (int h = 0; ok && h < p.G; ++h)
      for (int qt = 0; qt < it.n; ++qt, ++t) {
        const int st = t % Cfg::kStages, ls = t % Cfg::kLse;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_empty[st],
                                                     ((t / Cfg::kStages) & 1) ^ 1u, abort))))
          break;
        if (lane == 0) {
          // (checked builds: a query row of the prompt)
          const bool in = attn_check(it.q0 + 128 * qt < p.S, p.error_word);
          mbar_arrive_expect_tx(&sm.q_full[st], in ? Cfg::kTile : 0);
          for (int x = 0; in && x < Cfg::kBoxes; ++x)
            tma_load_3d(sm.q[st] + x * Cfg::kBox, &map_q, &sm.q_full[st], 64 * x,
                        it.q0 + 128 * qt, it.b * p.Hq + it.g * p.G + h);
        }
        ++q_loads;
        if (!(ok = __all_sync(0xffffffffu,
                              mbar_wait(&sm.l_empty[ls], ((t / Cfg::kLse) & 1) ^ 1u, abort))))
          break;
#pragma unroll
        for (int e = 0; e < 4; ++e) sm.nlse[ls][32 * e + lane] = l[e] * -1.4426950408889634f;
        mbar_arrive(&sm.l_full[ls]);
        if (qt + 1 < it.n) fetch(h, qt + 1);
        else if (h + 1 < p.G) fetch(h + 1, 0);
      }
    // every copy this warp started has landed before the CTA may exit
    if (lane == 0) {
      mbar_wait_drain_kw(&sm.k_full, 0);
      for (uint32_t i = 0; i < (uint32_t)Cfg::kStages; ++i)
        if (q_loads > i) {
          const uint32_t last = (q_loads - 1 - i) / Cfg::kStages;   // last use of stage i
          mbar_wait_drain_kw(&sm.q_full[i], last & 1u);
        }
    }
  } else if (warp == 5) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
    const uint64_t dk = smem_desc_sw128(0, 16, 1024) | (smem_u32(sm.k) >> 4);
    const uint64_t dq = smem_desc_sw128(0, 16, 1024) | (smem_u32(sm.q[0]) >> 4);
    bool ok = __all_sync(0xffffffffu, mbar_wait(&sm.k_full, 0, abort));
    for (int t = 0; ok && t < tiles; ++t) {
      const int st = t % Cfg::kStages;
      if (!(ok = __all_sync(0xffffffffu,
                            mbar_wait(&sm.q_full[st], (t / Cfg::kStages) & 1, abort))))
        break;
      if (!(ok = __all_sync(0xffffffffu,
                            mbar_wait(&sm.s_empty[t & 1], ((t >> 1) & 1) ^ 1u, abort))))
        break;
      tc_fence_after_sync();
      const uint32_t dS = tbase + 128u * (t & 1);
      const uint64_t b = dq + (uint64_t)st * (Cfg::kTile >> 4);
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk) {
        const uint32_t off = ((kk / 4) * Cfg::kBox + (kk % 4) * 32) >> 4;
        mma_bf16_ss_warp(dS, dk + off, b + off, idesc, kk > 0 ? 1u : 0u);
      }
      mma_commit_warp(&sm.s_full[t & 1]);
      mma_commit_warp(&sm.q_empty[st]);
    }
    // nothing of this warp's may still run on the tensor core at teardown
    mma_commit_warp(&sm.mma_done);
    mbar_wait_drain_kw(&sm.mma_done, 0);
  } else {
    const int j = k0 + threadIdx.x;   // this thread's key
    const uint32_t lane_addr = tbase + ((uint32_t)(warp * 32) << 16);
    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
    float total = 0.f;
    bool ok = true;
    int t = 0;
    for (int h = 0; ok && h < p.G; ++h)
      for (int qt = 0; qt < it.n; ++qt, ++t) {
        const int ls = t % Cfg::kLse;
        if (!(ok = mbar_wait(&sm.l_full[ls], (t / Cfg::kLse) & 1, abort))) break;
        if (!(ok = mbar_wait(&sm.s_full[t & 1], (t >> 1) & 1, abort))) break;
        tc_fence_after_sync();
        const uint32_t colS = lane_addr + 128u * (t & 1);
        // visible columns [clo, chi) of this key: queries at or after it, inside
        // the window, below the end
        const int q0 = it.q0 + 128 * qt;
        int clo = p.causal ? max(0, j - q0) : 0;
        int chi = it.q_end - q0;
        if (p.window > 0) chi = (int)min((long long)chi, (long long)j + p.window - q0);
        chi = min(chi, 128);
        const bool full = __all_sync(0xffffffffu, clo == 0 && chi == 128);
        const uint32_t span = chi > clo ? (uint32_t)(chi - clo - 1) : 0u;
        if (chi <= clo) clo = 1 << 30;   // no column is visible
        // a tile's sum is taken by itself and then added: the error of a long
        // sum grows with the number of tiles, not of queries
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float4* nl = reinterpret_cast<const float4*>(sm.nlse[ls]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t y[32];
          tmem_ld_32x32b_x32(colS + 32 * c, y);
          tmem_ld_wait(y);
          if (c == 3) {   // S is in registers: its buffer is free
            tc_fence_before_sync();
            mbar_arrive(&sm.s_empty[t & 1]);
          }
          if (!full) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              y[e] = __float_as_uint(
                  keep_if_le(__uint_as_float(y[e]), (uint32_t)(32 * c + e - clo), span));
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 n4 = nl[8 * c + e];
            const float2 a = __ffma2_rn(make_float2(__uint_as_float(y[4 * e]),
                                                    __uint_as_float(y[4 * e + 1])),
                                        scale2, make_float2(n4.x, n4.y));
            const float2 b = __ffma2_rn(make_float2(__uint_as_float(y[4 * e + 2]),
                                                    __uint_as_float(y[4 * e + 3])),
                                        scale2, make_float2(n4.z, n4.w));
            sum[0] = __fadd2_rn(sum[0], make_float2(ex2_approx(a.x), ex2_approx(a.y)));
            sum[1] = __fadd2_rn(sum[1], make_float2(ex2_approx(b.x), ex2_approx(b.y)));
          }
        }
        mbar_arrive(&sm.l_empty[ls]);
        total += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
    if (ok && j < it.L) {
      float* w = p.weights + ((size_t)it.b * p.Hkv + it.g) * p.stride + j;
      *w = p.accumulate ? *w + total : total;
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after_sync();
    tmem_dealloc(tbase, Cfg::kCols);
  }
  if (threadIdx.x == 0 && sm.abort_flag) atomicExch(p.error_word, 4);   // ATTN_ERR_TIMEOUT
}

template <int DH>
constexpr size_t key_weights_smem_bytes() {
  return sizeof(KeyWeightsSmem<DH>) + 1024;   // + alignment slack
}

}  // namespace chs
