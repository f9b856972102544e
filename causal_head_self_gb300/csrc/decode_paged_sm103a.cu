// decode_paged_sm103a.cu -- host launcher of the paged decode kernels.
#include "decode_paged_sm103a.cuh"
#include "launch.h"

namespace chs {

namespace {

constexpr int kCopiesMaxGroup = 32;   // head groups up to this run with REP = 4

int tile_keys(int Dh) { return Dh == 256 ? DecodePagedCfg<256>::kKeys : DecodePagedCfg<128>::kKeys; }

// o_part | m_part | l_part | unit_ctas | scores, each 256-byte aligned
struct Layout {
  size_t m_off, l_off, units_off, scores_off, total;
};

int score_stride(const PagedCache& c) { return (c.cols * c.page + 127) / 128 * 128; }

Layout layout(int B, int Hq, int Hkv, const PagedCache& c, int Dh, bool scores, int num_sms) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const int G = Hq / Hkv;
  const size_t units = (size_t)B * Hkv * ((G + 127) / 128);
  const size_t rows = (units + num_sms) * (G <= kCopiesMaxGroup ? 4 * (size_t)G : 128);
  Layout w;
  w.m_off = up(rows * Dh * sizeof(float));
  w.l_off = w.m_off + up(rows * sizeof(float));
  w.units_off = w.l_off + up(rows * sizeof(float));
  w.scores_off = w.units_off + up(units * sizeof(int2));
  w.total = w.scores_off + (scores ? (size_t)B * Hq * score_stride(c) * sizeof(float) : 0);
  return w;
}

template <int DH, int REP>
cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                   const DecodePagedParams& prm, int device, cudaStream_t stream) {
  constexpr size_t smem = decode_paged_smem_bytes<DH>();
  static_assert(smem <= 232448, "shared memory budget of one sm_103a CTA");
  static std::atomic<int> configured[kMaxDevices];
  cudaError_t e = configure_once(configured, device, [] {
    return cudaFuncSetAttribute(attn_decode_paged_sm103a<DH, REP>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_decode_paged_sm103a<DH, REP>, dim3(prm.ctas),
                 dim3(DecodePagedCfg<DH>::kThreads), smem, stream, mq, mk, mv, prm);
  if (e != cudaSuccess) return e;
  unsigned blocks = (unsigned)prm.B * prm.Hq;
  if (prm.weights)
    blocks += (unsigned)prm.B * prm.Hkv *
              ((prm.cols * prm.page + kPagedWeightKeys - 1) / kPagedWeightKeys);
  return launch_pdl(attn_decode_paged_join<DH, REP>, dim3(blocks), dim3(kPagedJoinThreads), 0,
                    stream, prm);
}

template <int DH>
cudaError_t launch_rep(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                       const DecodePagedParams& prm, int device, cudaStream_t stream) {
  return prm.G <= kCopiesMaxGroup ? launch<DH, 4>(mq, mk, mv, prm, device, stream)
                                  : launch<DH, 1>(mq, mk, mv, prm, device, stream);
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
                                    bool scores, int num_sms) {
  return layout(B, Hq, Hkv, cache, Dh, scores, num_sms).total;
}

cudaError_t launch_decode_paged(const void* q, const void* kpages, const void* vpages,
                                const int* table, const int* seqlens, void* o, float* weights,
                                int weights_stride, int accumulate, void* workspace, int B, int Hq,
                                int Hkv, const PagedCache& cache, int Dh, int window,
                                float scale_log2, const DeviceInfo& dev, cudaStream_t stream) {
  const int G = Hq / Hkv, keys = tile_keys(Dh);
  const int box = paged_box_rows(cache.page, Dh);
  const long long pages = (long long)cache.num_pages * Hkv;
  CUtensorMap mq, mk, mv;
  if (!encode_bf16_map(&mq, q, Dh, G, (long long)B * Hkv, G <= kCopiesMaxGroup ? 32 : 128) ||
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
  const long long rows = (long long)cache.cols * cache.page;
  long long tiles = (rows + keys - 1) / keys;   // at most, per unit
  if (window > 0 && tiles > ((long long)window + keys - 2) / keys + 1)
    tiles = ((long long)window + keys - 2) / keys + 1;
  const long long places = (tiles + 1) * B * Hkv * prm.row_blocks;
  prm.ctas = places < dev.num_sms ? (int)places : dev.num_sms;
  prm.score_stride = score_stride(cache);
  prm.scale_log2 = scale_log2;
  prm.accumulate = accumulate;
  prm.seqlens = seqlens;
  prm.table = table;
  const Layout w = layout(B, Hq, Hkv, cache, Dh, weights != nullptr, dev.num_sms);
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
  return Dh == 256   ? launch_rep<256>(mq, mk, mv, prm, dev.device, stream)
         : Dh == 128 ? launch_rep<128>(mq, mk, mv, prm, dev.device, stream)
                     : launch_rep<64>(mq, mk, mv, prm, dev.device, stream);
}

}  // namespace chs
