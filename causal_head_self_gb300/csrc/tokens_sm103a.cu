// tokens_sm103a.cu -- launchers of the rotary positions and of the serving step's plan.
#include "launch.h"
#include "tokens_sm103a.cuh"

namespace chs {

static RopeTensor rope_tensor(const RopeRows& in, const RopeRows* out) {
  RopeTensor x{};
  x.in = static_cast<const __nv_bfloat16*>(in.data);
  x.in_batch = in.batch;
  x.in_row = in.row;
  x.in_head = in.head;
  if (out) {
    x.out = static_cast<__nv_bfloat16*>(const_cast<void*>(out->data));
    x.out_batch = out->batch;
    x.out_row = out->row;
    x.out_head = out->head;
    x.copy_rest = out->data != in.data;
  }
  return x;
}

cudaError_t launch_rope(const RopeShape& s, const RopeRows& q, const RopeRows* q_out,
                        const RopeRows& k, const RopeRows* k_out, const RopeAppend* append,
                        const DeviceInfo& dev, cudaStream_t stream) {
  RopeParams p{};
  p.q = rope_tensor(q, q_out);
  p.k = rope_tensor(k, k_out);
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  p.positions = s.positions;
  p.turns = reinterpret_cast<const uint64_t*>(s.turns);
  p.amplitude = s.amplitude;
  p.rows = s.B * s.S;
  p.S = s.S;
  p.Dh = s.Dh;
  p.rot = s.rot;
  p.inverse = s.inverse;
  p.div_s = make_fixed_div((uint32_t)s.S);
  p.error_word = dev.error_word;
  // several rows a block share the launch of its threads, as long as the blocks fill the SMs
  int per = kRopeMaxRows;
  while (per > 1 && p.rows / per < 4 * dev.num_sms) per /= 2;
  p.rows_per_block = per;
  const dim3 grid((unsigned)((p.rows + per - 1) / per)), block(kRopeThreads);
  const size_t smem = (size_t)per * s.rot * sizeof(float);
  if (!append)
    return launch_pdl(s.interleaved ? attn_rope_sm103a<true, false> : attn_rope_sm103a<false, false>,
                      grid, block, smem, stream, p);
  p.v = static_cast<const __nv_bfloat16*>(append->v.data);
  p.v_batch = append->v.batch;
  p.v_row = append->v.row;
  p.v_head = append->v.head;
  p.kpages = static_cast<__nv_bfloat16*>(append->kpages);
  p.vpages = static_cast<__nv_bfloat16*>(append->vpages);
  p.slots = append->slots;
  p.slot_end = append->num_pages * append->page;
  p.div_page = make_fixed_div((uint32_t)append->page);
  return launch_pdl(s.interleaved ? attn_rope_sm103a<true, true> : attn_rope_sm103a<false, true>,
                    grid, block, smem, stream, p);
}

// Tokens that the plan's own cluster fills in: beyond, it takes longer than another launch.
constexpr int kPlanFillRows = 16384;

int cache_plan_max_sequences() { return kPlanMaxB; }

cudaError_t launch_cache_plan(const CachePlan& c, const DeviceInfo& dev, cudaStream_t stream) {
  PlanParams p{};
  p.delta = c.delta;
  p.seqlens = c.seqlens;
  p.seqlens_out = c.seqlens_out;
  p.table = c.table;
  p.free_pages = c.free_pages;
  p.num_free = c.num_free;
  p.num_free_out = c.num_free_out;
  p.cu = c.cu;
  p.positions = c.positions;
  p.slots = c.slots;
  p.B = c.B;
  p.cols = c.cols;
  p.page = c.page;
  p.num_pages = c.num_pages;
  p.capacity = c.capacity;
  p.T = c.T;
  p.div_page = make_fixed_div((uint32_t)c.page);
  p.error_word = dev.error_word;
  static std::atomic<int> configured[kMaxDevices];
  cudaError_t e = configure_once(configured, dev.device, [] {
    return cudaFuncSetAttribute(attn_cache_plan_sm103a, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)plan_smem_bytes(kPlanMaxB));
  });
  if (e != cudaSuccess) return e;
  // one CTA where its threads write no more than four entries each, else a cluster; more
  // tokens than that are a second launch's
  p.fill = c.T <= kPlanFillRows;
  int ctas = 1;
  while (ctas < kPlanMaxCtas && (p.fill ? c.T : 0) + c.B > 4ll * kPlanThreads * ctas) ctas *= 2;
  if (!p.fill) ctas = kPlanMaxCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = plan_smem_bytes(c.B);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, attn_cache_plan_sm103a, p);
  if (e != cudaSuccess || p.fill) return e;
  constexpr int per = kFillThreads * kFillRows;
  return launch_pdl(attn_cache_fill_sm103a, dim3((unsigned)((c.T + (long long)per - 1) / per)),
                    dim3(kFillThreads), 0, stream, p);
}

}  // namespace chs
