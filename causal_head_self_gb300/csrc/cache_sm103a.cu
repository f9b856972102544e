// cache_sm103a.cu -- host launchers of the paged cache's kernels: append, key
// weights of a prompt, eviction.
#include <algorithm>

#include "cache_sm103a.cuh"
#include "key_weights_few_sm103a.cuh"
#include "key_weights_sm103a.cuh"
#include "launch.h"

namespace chs {

cudaError_t launch_paged_append(const void* k, const void* v, void* kpages, void* vpages,
                                const int* table, const int* seqlens, const int* newlens, int B,
                                int Hkv, int S, const PagedCache& cache, int Dh,
                                const DeviceInfo& dev, cudaStream_t stream) {
  AppendParams prm;
  prm.k = static_cast<const uint4*>(k);
  prm.v = static_cast<const uint4*>(v);
  prm.kpages = static_cast<uint4*>(kpages);
  prm.vpages = static_cast<uint4*>(vpages);
  prm.table = table;
  prm.seqlens = seqlens;
  prm.newlens = newlens;
  prm.rows = (long long)B * Hkv * S;
  prm.Hkv = Hkv;
  prm.S = S;
  prm.vecs = Dh / 8;
  prm.num_pages = cache.num_pages;
  prm.page = cache.page;
  prm.cols = cache.cols;
  prm.by_s = make_fixed_div((uint32_t)S);
  prm.by_heads = make_fixed_div((uint32_t)Hkv);
  prm.by_page = make_fixed_div((uint32_t)cache.page);
  prm.error_word = dev.error_word;
  const int per_pass = kAppendThreads / prm.vecs;
  constexpr int U = 4;
  const long long blocks1 = (prm.rows + per_pass - 1) / per_pass;
  if (blocks1 <= 8LL * dev.num_sms)
    return launch_pdl(attn_paged_append_sm103a<1>, dim3((unsigned)blocks1), dim3(kAppendThreads), 0,
                      stream, prm);
  return launch_pdl(attn_paged_append_sm103a<U>, dim3((unsigned)((blocks1 + U - 1) / U)),
                    dim3(kAppendThreads), 0, stream, prm);
}

template <int DH>
static cudaError_t launch_key_weights_dh(const CUtensorMap& mq, const CUtensorMap& mk,
                                         const KeyWeightsParams& prm, const DeviceInfo& dev,
                                         cudaStream_t stream) {
  constexpr size_t smem = key_weights_smem_bytes<DH>();
  static_assert(smem <= 232448, "shared memory budget of one sm_103a CTA");
  static std::atomic<int> configured[kMaxDevices];
  cudaError_t e = configure_once(configured, dev.device, [] {
    return cudaFuncSetAttribute(attn_key_weights_sm103a<DH>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  const dim3 block(KeyWeightsCfg<DH>::kThreads);
  if (prm.split == 1)
    return launch_pdl(attn_key_weights_sm103a<DH>,
                      dim3(prm.items < dev.num_sms ? prm.items : dev.num_sms), block, smem, stream,
                      mq, mk, prm);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(prm.items * prm.split);
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = prm.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, attn_key_weights_sm103a<DH>, mq, mk, prm);
}

template <int DH>
static cudaError_t launch_key_few_dh(const CUtensorMap& mq, const CUtensorMap& mk,
                                     const KeyFewParams& prm, const DeviceInfo& dev,
                                     cudaStream_t stream) {
  constexpr size_t smem = key_few_smem_bytes<DH>();
  static_assert(smem <= 232448, "shared memory budget of one sm_103a CTA");
  static std::atomic<int> configured[kMaxDevices];
  cudaError_t e = configure_once(configured, dev.device, [] {
    return cudaFuncSetAttribute(attn_key_weights_few_sm103a<DH>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_key_weights_few_sm103a<DH>, dim3(prm.ctas),
                    dim3(KeyFewCfg<DH>::kThreads), smem, stream, mq, mk, prm);
}

cudaError_t launch_key_weights(const void* q, const void* k, const float* lse, const int* seqlens,
                               float* weights, int stride, int B, int Hq, int Hkv, int S, int Dh,
                               int causal, int window, int queries, int accumulate,
                               float scale_log2, const DeviceInfo& dev, cudaStream_t stream) {
  const int G = Hq / Hkv;
  // Every row votes: one form, however it is asked for; short prompts take the one for few
  // voting queries, others the general one.  GPU time in us, general -> few, at 8, 17, 32,
  // 33 and 64 rows: 64 prompts, 32 heads on 8: 14.3 -> 10.4, 14.4 -> 13.5, 14.4 -> 9.6,
  // 16.8 -> 17.2, 15.7 -> 16.5; 32 heads on 32: 18.1 -> 17.8, 18.1 -> 17.8, 18.1 -> 16.4,
  // 18.8 -> 19.8, 18.8 -> 22.9; 300 prompts, 8 heads on one: 13.0 -> 10.6, 13.0 -> 14.2,
  // 13.1 -> 10.4, 16.2 -> 14.9, 14.9 -> 15.9.
  if (queries == 0 || queries >= S) queries = S <= 32 ? S : 0;
  // rows per head in a tile: with up to 64 voting queries it holds several heads'
  int pad = 128;
  if (queries > 0)
    while (pad > 16 && pad / 2 >= queries) pad /= 2;
  const double per_lse = -1.4426950408889634 / (double)scale_log2;   // -log2(e) / scale_log2
  const int most = Dh == 256 ? KeyFewCfg<256>::kCols : KeyFewCfg<128>::kCols;
  // The whole group's voting queries in one tile (and no window, which would leave
  // most blocks of keys without any): the queries stay, the keys pass by.
  if (queries > 0 && queries <= 128 && window == 0 && (long long)G * pad <= most) {
    CUtensorMap mq, mk;
    if (!encode_bf16_map(&mq, q, Dh, S, (long long)B * Hq, pad) ||
        !encode_bf16_rows_map(&mk, k, Dh, S, (long long)B * Hkv, 128))
      return cudaErrorInvalidValue;
    KeyFewParams prm;
    prm.B = B;
    prm.Hq = Hq;
    prm.Hkv = Hkv;
    prm.G = G;
    prm.S = S;
    prm.causal = causal;
    prm.queries = queries;
    prm.accumulate = accumulate;
    prm.pad = pad;
    prm.cols = (G * pad + 31) / 32 * 32;
    const long long places = ((long long)(S + 127) / 128 + 1) * B * Hkv;
    prm.ctas = places < dev.num_sms ? (int)places : dev.num_sms;
    prm.scale_log2 = scale_log2;
    prm.lse_hi = (float)per_lse;
    prm.lse_lo = (float)(per_lse - (double)prm.lse_hi);
    prm.lse = lse;
    prm.seqlens = seqlens;
    prm.weights = weights;
    prm.stride = stride;
    prm.error_word = dev.error_word;
    return Dh == 256   ? launch_key_few_dh<256>(mq, mk, prm, dev, stream)
           : Dh == 128 ? launch_key_few_dh<128>(mq, mk, prm, dev, stream)
                       : launch_key_few_dh<64>(mq, mk, prm, dev, stream);
  }
  CUtensorMap mq, mk;
  if (!(pad == 128 ? encode_bf16_rows_map(&mq, q, Dh, S, (long long)B * Hq, 128)
                   : encode_bf16_map(&mq, q, Dh, S, (long long)B * Hq, pad)) ||
      !encode_bf16_rows_map(&mk, k, Dh, S, (long long)B * Hkv, 128))
    return cudaErrorInvalidValue;
  KeyWeightsParams prm;
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.G = G;
  prm.S = S;
  prm.causal = causal;
  prm.window = window;
  prm.queries = queries;
  prm.accumulate = accumulate;
  prm.items = (S + 127) / 128 * B * Hkv;
  prm.pad = pad;
  prm.head_tiles = (G - 1) / (128 / pad) + 1;   // (heads: their columns may pass 32 bits)
  prm.by_heads = make_fixed_div((uint32_t)Hkv);
  prm.by_batch = make_fixed_div((uint32_t)(B * Hkv));
  // a cluster per item where that fills the SMs no more than once, and leaves
  // each CTA a tile (of the longest sequence's first keys: those have the most)
  long long voting = queries ? queries : S;
  if (window > 0) voting = std::min(voting, (long long)window + 127);
  const long long tiles = pad < 128 ? prm.head_tiles : G * ((voting + 127) / 128);
  prm.split = 1;
  prm.split_log2 = 0;
  while (prm.split < 8 && 2LL * prm.split * prm.items <= dev.num_sms && 2LL * prm.split <= tiles) {
    prm.split *= 2;
    ++prm.split_log2;
  }
  prm.scale_log2 = scale_log2;
  prm.lse_hi = (float)per_lse;
  prm.lse_lo = (float)(per_lse - (double)prm.lse_hi);
  prm.lse = lse;
  prm.seqlens = seqlens;
  prm.weights = weights;
  prm.stride = stride;
  prm.error_word = dev.error_word;
  return Dh == 256   ? launch_key_weights_dh<256>(mq, mk, prm, dev, stream)
         : Dh == 128 ? launch_key_weights_dh<128>(mq, mk, prm, dev, stream)
                     : launch_key_weights_dh<64>(mq, mk, prm, dev, stream);
}

cudaError_t launch_cache_evict(void* kpages, void* vpages, const int* table, const int* table_out,
                               int cols_out, const int* seqlens, int* newlens,
                               const float* weights, int stride, float* weights_out,
                               int stride_out, int* keep, int B, int Hkv, const PagedCache& cache,
                               int Dh, int budget, int recent, const DeviceInfo& dev,
                               cudaStream_t stream) {
  EvictParams prm;
  prm.kpages = static_cast<uint4*>(kpages);
  prm.vpages = static_cast<uint4*>(vpages);
  prm.table = table;
  prm.table_out = table_out;
  prm.seqlens = seqlens;
  prm.newlens = newlens;
  prm.weights = weights;
  prm.weights_out = weights_out;
  prm.keep = keep;
  prm.B = B;
  prm.Hkv = Hkv;
  prm.vecs = Dh / 8;
  prm.num_pages = cache.num_pages;
  prm.page = cache.page;
  prm.cols = cache.cols;
  prm.cols_out = cols_out;
  prm.stride = stride;
  prm.stride_out = stride_out;
  prm.budget = budget;
  prm.recent = recent;
  prm.error_word = dev.error_word;
  prm.by_page = make_fixed_div((uint32_t)cache.page);
  const long long rows = (long long)cache.cols * cache.page;
  cudaError_t e;
  if (rows <= kSelectHeld) {
    static std::atomic<int> configured[kMaxDevices];
    e = configure_once(configured, dev.device, [] {
      return cudaFuncSetAttribute(attn_cache_select_sm103a<true>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectHeld * 4);
    });
    if (e != cudaSuccess) return e;
    e = launch_pdl(attn_cache_select_sm103a<true>, dim3(B * Hkv), dim3(kSelectThreads),
                   (size_t)(rows + 3) / 4 * 16, stream, prm);
  } else {
    e = launch_pdl(attn_cache_select_sm103a<false>, dim3(B * Hkv), dim3(kSelectThreads), 0, stream,
                   prm);
  }
  if (e != cudaSuccess) return e;
  if (table_out == table) {
    constexpr int U = 4;
    // column slices of 64 bytes at least, as few as give every SM two blocks
    int piece = prm.vecs;
    while (piece > 4 && 2LL * B * Hkv * (prm.vecs / piece) < 2LL * dev.num_sms) piece /= 2;
    return launch_pdl(attn_cache_move_in_place_sm103a<U>,
                      dim3((unsigned)(2 * B * Hkv * (prm.vecs / piece))), dim3(kMoveThreads), 0,
                      stream, prm, piece);
  }
  constexpr int U = 2;   // (1: as fast; 4: 97 us instead of 93 for 537 MB; 8: 130)
  const int per_pass = kMoveThreads / prm.vecs;
  const int blocks = (budget + per_pass * U - 1) / (per_pass * U);
  return launch_pdl(attn_cache_move_sm103a<U>, dim3((unsigned)B * Hkv * blocks), dim3(kMoveThreads),
                    0, stream, prm);
}

}  // namespace chs
