// decode_paged_sm103a.cu -- host launcher of the paged decode kernels.
#include "decode_paged_sm103a.cuh"
#include "launch.h"

namespace chs {

namespace {

constexpr int kCopiesMaxGroup = 32;   // head groups up to this run with REP = 4
constexpr int kShortCtas = 8;         // of a cluster, at most

int tile_keys(int Dh) { return Dh == 256 ? DecodePagedCfg<256>::kKeys : DecodePagedCfg<128>::kKeys; }

// o_part | m_part | l_part | unit_ctas | scores, each 256-byte aligned
struct Layout {
  size_t m_off, l_off, units_off, scores_off, total;
};

int score_stride(const PagedCache& c) { return (c.cols * c.page + 127) / 128 * 128; }

template <int DH>
cudaError_t allow_short(int device) {
  static std::atomic<int> configured[kMaxDevices];
  return configure_once(configured, device, [] {
    return cudaFuncSetAttribute(attn_decode_paged_sm103a<DH, 4, true>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)decode_paged_smem_bytes<DH>());
  });
}

struct ShortLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  ShortLaunch(int ctas, int split, size_t smem, cudaStream_t stream) {
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(DecodePagedCfg<128>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

// How many clusters of `split` CTAs run at once (every head size takes a whole SM per
// CTA).
int clusters_at_once(int split, const DeviceInfo& dev) {
  static std::atomic<int> known[kMaxDevices][kShortCtas + 1];
  const bool tracked = dev.device >= 0 && dev.device < kMaxDevices;
  int n = tracked ? known[dev.device][split].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  ShortLaunch l(split * dev.num_sms, split, decode_paged_smem_bytes<128>(), nullptr);
  l.cfg.numAttrs = 1;
  if (allow_short<128>(dev.device) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, attn_decode_paged_sm103a<128, 4, true>, &l.cfg) !=
          cudaSuccess)
    return 0;
  if (tracked) known[dev.device][split].store(n, std::memory_order_relaxed);
  return n;
}

// Tiles of a unit, at most.
long long most_tiles(const PagedCache& c, int Dh, int window) {
  const int keys = tile_keys(Dh);
  const long long rows = (long long)c.cols * c.page, tiles = (rows + keys - 1) / keys;
  const long long seen = window > 0 ? ((long long)window + keys - 2) / keys + 1 : tiles;
  return tiles < seen ? tiles : seen;
}

// The CTAs per unit (a cluster) of a call that runs in the short form, or 0.  All
// clusters run at once, and no CTA gets more than kShortTiles tiles: up to there the
// short form was no slower at equal or at ragged lengths, with all head layouts that
// were tried but 32 query heads on one K/V head.  GPU time, line of tiles -> short
// form (32 query heads, 8 K/V heads of 128): 4 x 1024 keys 11.4 -> 8.9 us, 16 x 1024
// 16.8 -> 13.2 (ragged 15.1 -> 13.1), 1 x 8192 13.6 -> 12.5; 8 query heads on one of
// 256, 16 sequences with a window of 4096: 22.7 -> 20.5.  With 16 tiles per CTA
// 1 x 16384 keys 16.6 -> 18.2.
constexpr int kShortTiles = 12;

int short_split(int B, int Hq, int Hkv, const PagedCache& c, int Dh, int window,
                const DeviceInfo& dev) {
  if (Hq / Hkv > kCopiesMaxGroup) return 0;
  const long long units = (long long)B * Hkv, tiles = most_tiles(c, Dh, window);
  if (units > dev.num_sms || tiles > kShortCtas * kShortTiles) return 0;
  int split = tiles < kShortCtas ? (int)tiles : kShortCtas;
  while (split > 1 && units > clusters_at_once(split, dev)) --split;
  return tiles <= (long long)kShortTiles * split ? split : 0;
}

Layout layout(int B, int Hq, int Hkv, const PagedCache& c, int Dh, bool scores, bool one_launch,
              int num_sms) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const int G = Hq / Hkv;
  const size_t units = (size_t)B * Hkv * ((G + 127) / 128);
  // (the short form keeps its partial results in shared memory)
  const size_t rows =
      one_launch ? 0 : (units + num_sms) * (G <= kCopiesMaxGroup ? 4 * (size_t)G : 128);
  Layout w;
  w.m_off = up(rows * (G <= kPagedTwoParts ? 2 : 1) * Dh * sizeof(float));
  w.l_off = w.m_off + up(rows * sizeof(float));
  w.units_off = w.l_off + up(rows * sizeof(float));
  w.scores_off = w.units_off + (rows > 0 ? up(units * sizeof(int2)) : 0);
  w.total = w.scores_off + (scores ? (size_t)B * Hq * score_stride(c) * sizeof(float) : 0);
  return w;
}

template <int DH>
cudaError_t launch_short(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                         const DecodePagedParams& prm, const DeviceInfo& dev, cudaStream_t stream) {
  const cudaError_t e = allow_short<DH>(dev.device);
  if (e != cudaSuccess) return e;
  const ShortLaunch l(prm.ctas, prm.split, decode_paged_smem_bytes<DH>(), stream);
  return cudaLaunchKernelEx(&l.cfg, attn_decode_paged_sm103a<DH, 4, true>, mq, mk, mv, prm);
}

template <int DH, int REP, bool TWICE, int THREADS>
cudaError_t launch_join(const DecodePagedParams& prm, cudaStream_t stream) {
  unsigned blocks = (unsigned)prm.B * prm.Hq;
  if (prm.weights)
    blocks += (unsigned)prm.B * prm.Hkv *
              ((prm.cols * prm.page + 4 * THREADS - 1) / (4 * THREADS));
  return launch_pdl(attn_decode_paged_join<DH, REP, TWICE, THREADS>, dim3(blocks), dim3(THREADS), 0,
                    stream, prm);
}

template <int DH, int REP>
cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                   const DecodePagedParams& prm, const DeviceInfo& dev, cudaStream_t stream) {
  constexpr size_t smem = decode_paged_smem_bytes<DH>();
  static_assert(smem <= 232448, "shared memory budget of one sm_103a CTA");
  static std::atomic<int> configured[kMaxDevices];
  cudaError_t e = configure_once(configured, dev.device, [] {
    return cudaFuncSetAttribute(attn_decode_paged_sm103a<DH, REP, false>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_decode_paged_sm103a<DH, REP, false>, dim3(prm.ctas),
                 dim3(DecodePagedCfg<DH>::kThreads), smem, stream, mq, mk, mv, prm);
  if (e != cudaSuccess) return e;
  // Many partial results in few units take more threads, as long as each SM has a
  // block at most: 8 heads on 1, 16384 keys 44 -> 32 us for the step; 2 x 32 heads on 8,
  // 8192 keys 19.8 -> 15.5.  Few do not: 4 x 32 heads on 8 with weights, 16384 to 32768
  // keys (20 partial results) 69 -> 72 us.  (Weights have no say: the output's bits do
  // not depend on whether they are asked for.)
  const int partials = REP * (prm.ctas / (prm.B * prm.Hkv * prm.row_blocks) + 1);
  const bool wide = partials > 32 && prm.B * prm.Hq <= dev.num_sms;
  if (REP == 4 && prm.G <= kPagedTwoParts)
    return wide ? launch_join<DH, REP, REP == 4, 1024>(prm, stream)
                : launch_join<DH, REP, REP == 4, 256>(prm, stream);
  return wide ? launch_join<DH, REP, false, 1024>(prm, stream)
              : launch_join<DH, REP, false, 256>(prm, stream);
}

template <int DH>
cudaError_t launch_rep(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                       const DecodePagedParams& prm, const DeviceInfo& dev, cudaStream_t stream) {
  if (prm.split > 0) return launch_short<DH>(mq, mk, mv, prm, dev, stream);
  return prm.G <= kCopiesMaxGroup ? launch<DH, 4>(mq, mk, mv, prm, dev, stream)
                                  : launch<DH, 1>(mq, mk, mv, prm, dev, stream);
}

}  // namespace

int paged_box_rows(int page, int Dh) {
  int a = page, b = tile_keys(Dh);
  while (b) {
    const int r = a % b;
    a = b;
    b = r;
  }
  return a;
}

size_t decode_paged_workspace_bytes(int B, int Hq, int Hkv, const PagedCache& cache, int Dh,
                                    int window, bool scores, const DeviceInfo& dev) {
  const bool one_launch = short_split(B, Hq, Hkv, cache, Dh, window, dev) > 0;
  return layout(B, Hq, Hkv, cache, Dh, scores, one_launch, dev.num_sms).total;
}

cudaError_t launch_decode_paged(const void* q, const void* kpages, const void* vpages,
                                const int* table, const int* seqlens, void* o, float* weights,
                                int weights_stride, int accumulate, void* workspace, int B, int Hq,
                                int Hkv, const PagedCache& cache, int Dh, int window,
                                float scale_log2, const DeviceInfo& dev, cudaStream_t stream) {
  const int G = Hq / Hkv;
  const int box = paged_box_rows(cache.page, Dh);
  const long long pages = (long long)cache.num_pages * Hkv;
  CUtensorMap mq, mk, mv;
  // rows per load: the kernel's rows, or half of the 32 that hold the heads twice
  const int q_rows = G <= kPagedTwoParts ? kPagedTwoParts : G <= kCopiesMaxGroup ? 32 : 128;
  if (!encode_bf16_map(&mq, q, Dh, G, (long long)B * Hkv, q_rows) ||
      !encode_bf16_map(&mk, kpages, Dh, cache.page, pages, box) ||
      !encode_bf16_map(&mv, vpages, Dh, cache.page, pages, box))
    return cudaErrorInvalidValue;
  DecodePagedParams prm;
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.G = G;
  prm.window = window;
  prm.num_pages = cache.num_pages;
  prm.page = cache.page;
  prm.cols = cache.cols;
  prm.box_rows = box;
  prm.row_blocks = (G + 127) / 128;
  prm.split = short_split(B, Hq, Hkv, cache, Dh, window, dev);
  const long long places = (most_tiles(cache, Dh, window) + 1) * B * Hkv * prm.row_blocks;
  prm.ctas = prm.split > 0 ? B * Hkv * prm.split : places < dev.num_sms ? (int)places : dev.num_sms;
  prm.score_stride = score_stride(cache);
  prm.scale_log2 = scale_log2;
  prm.accumulate = accumulate;
  prm.seqlens = seqlens;
  prm.table = table;
  const Layout w = layout(B, Hq, Hkv, cache, Dh, weights != nullptr, prm.split > 0, dev.num_sms);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  prm.o_part = reinterpret_cast<float*>(ws);
  prm.m_part = reinterpret_cast<float*>(ws + w.m_off);
  prm.l_part = reinterpret_cast<float*>(ws + w.l_off);
  prm.unit_ctas = reinterpret_cast<int2*>(ws + w.units_off);
  prm.scores = weights ? reinterpret_cast<float*>(ws + w.scores_off) : nullptr;
  prm.weights = weights;
  prm.weights_stride = weights_stride;
  prm.o = static_cast<__nv_bfloat16*>(o);
  prm.error_word = dev.error_word;
  prm.fault = dev.fault;
  return Dh == 256   ? launch_rep<256>(mq, mk, mv, prm, dev, stream)
         : Dh == 128 ? launch_rep<128>(mq, mk, mv, prm, dev, stream)
                     : launch_rep<64>(mq, mk, mv, prm, dev, stream);
}

}  // namespace chs
