// packed_sm103a.cu -- attention over packed sequences, forward: the list of tiles, then the
// prefill kernels over it.
#include "launch.h"
#include "packed_schedule_sm103a.cuh"
#include "prefill_k64_sm103a.cuh"
#include "prefill_sm103a.cuh"

namespace chs {

cudaError_t launch_packed_schedule(const PackedShape& s, int block, int fold_max, int lists, const int* order,
                                   void* const* tiles, int* const* counts, const DeviceInfo& dev,
                                   cudaStream_t stream) {
  PackedSchedule p{};
  p.cu = s.cu;
  p.B = s.B;
  p.T = s.T;
  p.block = block;
  p.causal = s.causal;
  p.window = s.window;
  p.fold_max = fold_max;
  for (int i = 0; i < lists; ++i) {
    p.tiles[i] = static_cast<PackedTile*>(tiles[i]);
    p.order[i] = order[i];
    p.num_tiles[i] = counts[i];
  }
  p.capacity = (int)packed_max_tiles(s.B, s.T);
  p.error_word = dev.error_word;
  return launch_pdl(attn_packed_schedule, dim3(lists), dim3(kScheduleThreads), 0, stream, p);
}

namespace {

struct FwdMaps {
  CUtensorMap q, k, v, o;
  int heads_inner = 0;
};

// Box heights: q_rows, kv_rows, 32 output rows (one softmax warp's).
bool fwd_maps(FwdMaps* m, const PackedShape& s, const PackedRows& q, const PackedRows& k,
              const PackedRows& v, const PackedRows& o, int q_rows, int kv_rows) {
  bool hq, hk, hv, ho;
  if (!encode_packed_map(&m->q, q, s.Dh, s.T, q_rows, true, &hq) ||
      !encode_packed_map(&m->k, k, s.Dh, s.T, kv_rows, true, &hk) ||
      !encode_packed_map(&m->v, v, s.Dh, s.T, kv_rows, true, &hv) ||
      !encode_packed_map(&m->o, o, s.Dh, s.T, 32, false, &ho))
    return false;
  m->heads_inner = (hq ? kPackedQ : 0) | (hk ? kPackedK : 0) | (hv ? kPackedV : 0) |
                   (ho ? kPackedO : 0);
  return true;
}

template <int DH>
cudaError_t launch_wide(const PackedShape& s, const PackedRows& q, const PackedRows& k,
                        const PackedRows& v, const PackedRows& o, float* lse, const PackedRef& ref,
                        float scale_log2, const DeviceInfo& dev, cudaStream_t stream) {
  constexpr size_t smem = prefill_smem_bytes<DH, true>();
  static_assert(smem <= 232448, "shared memory budget of one sm_103a CTA");
  FwdMaps m;
  if (!fwd_maps(&m, s, q, k, v, o, 128, 128)) return cudaErrorInvalidValue;
  // the register split needs the full launch registers, as in the batch form
  static std::atomic<int> configured[kMaxDevices];
  cudaError_t e = configure_once(configured, dev.device, [] {
    cudaFuncAttributes fa;
    cudaError_t r = cudaFuncGetAttributes(&fa, attn_prefill_sm103a<DH, true>);
    if (r != cudaSuccess) return r;
    if (fa.numRegs < PrefillCfg<DH>::kRegsLaunch) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(attn_prefill_sm103a<DH, true>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  PrefillParams p{};
  p.B = 1;
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  p.causal = s.causal;
  p.window = s.window;
  p.scale_log2 = scale_log2;
  p.lse = lse;
  p.error_word = dev.error_word;
  p.fault = dev.fault;
  p.div_hq = make_fixed_div((uint32_t)s.Hq);
  p.div_group = make_fixed_div((uint32_t)(s.Hq / s.Hkv));
  p.pk = ref;
  p.pk.heads_inner = m.heads_inner;
  p.o = static_cast<__nv_bfloat16*>(const_cast<void*>(o.data));
  p.o_row = o.row;
  p.o_head = o.head;
  const long long most = ((long long)s.T / 256 + s.B) * s.Hq;
  const int grid = most < dev.num_sms ? (int)most : dev.num_sms;
  return launch_pdl(attn_prefill_sm103a<DH, true>, dim3(grid), dim3(PrefillCfg<DH>::kThreads),
                    smem, stream, m.q, m.k, m.v, m.o, p);
}

template <int DH>
cudaError_t launch_k64(const PackedShape& s, const PackedRows& q, const PackedRows& k,
                       const PackedRows& v, const PackedRows& o, float* lse, const PackedRef& ref,
                       float scale_log2, const DeviceInfo& dev, cudaStream_t stream) {
  using Cfg = PrefillK64Cfg<DH>;
  constexpr size_t smem = prefill_k64_smem_bytes<DH, true>();
  const int q_rows = ref.fold_max ? 32 : 128;
  FwdMaps m;
  if (!fwd_maps(&m, s, q, k, v, o, q_rows, Cfg::kKeys)) return cudaErrorInvalidValue;
  static std::atomic<int> configured[kMaxDevices];
  cudaError_t e = configure_once(configured, dev.device, [] {
    return cudaFuncSetAttribute(attn_prefill_k64_sm103a<DH, true>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  PrefillK64Params p{};
  p.B = 1;
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  p.causal = s.causal;
  p.window = s.window;
  p.scale_log2 = scale_log2;
  p.group = s.Hq / s.Hkv;
  p.o = static_cast<__nv_bfloat16*>(const_cast<void*>(o.data));
  p.o_row = o.row;
  p.o_head = o.head;
  p.o_wide = (reinterpret_cast<uintptr_t>(o.data) & 31) == 0 && o.row % 16 == 0 && o.head % 16 == 0;
  p.lse = lse;
  p.error_word = dev.error_word;
  p.fault = dev.fault;
  p.pk = ref;
  p.pk.heads_inner = m.heads_inner;
  p.q_rows = q_rows;
  const long long most = packed_max_tiles(s.B, s.T) * s.Hq;
  const int cap = Cfg::kCtasPerSm * dev.num_sms;
  const int grid = most < cap ? (int)most : cap;
  return launch_pdl(attn_prefill_k64_sm103a<DH, true>, dim3(grid), dim3(Cfg::kThreads), smem,
                    stream, m.q, m.k, m.v, m.o, p);
}

// Head sizes 64 and 128: the 64-key kernel up to this many rows per sequence on average.  Its
// items are half as long, two CTAs share an SM, and it reads K and V twice as often: longer
// sequences, and more K/V heads, are for the ping-pong kernel's 256-row items.  In us, 64-key
// against ping-pong, 32 query heads, 15000 to 16384 rows in all:
//   Dh 64,  32 K/V heads: 74 : 81 (768 rows each), 124 : 123 (1024), 158 : 148 (1536);
//           16: 229 : 246 (3000), 318 : 315 (4096);  8: 286 : 315 (4096), 536 : 575 (8192),
//           2233 : 2180 (16384);  1: 534 : 575 (8192), 2054 : 2180 (16384);
//   Dh 128, 32: 129 : 114 (768; of two sequences of 1024, whose K and V stay in L2, the 64-key
//           kernel is 7 % faster);  16: 169 : 188 (1024), 209 : 184 (1536);  8: 188 : 204 (1536),
//           238 : 252 (2048), 302 : 282 (3000);  1: 177 : 198 (1536), 227 : 222 (2048).
constexpr long long kL2KeyBytes = 96ll << 20;   // K and V that L2 keeps beside the rest

bool takes_k64(const PackedShape& s) {
  if (s.Dh == 256) return true;
  const int group = s.Hq / s.Hkv;
  long long rows;
  if (s.Dh == 64)
    rows = group >= 4 ? 12288 : group >= 2 ? 3500 : 900;
  else if (group >= 2)
    rows = group >= 4 ? 2048 : 1280;
  else
    rows = 4ll * s.T * s.Hkv * s.Dh <= kL2KeyBytes ? 1536 : 512;
  return s.T <= rows * s.B;
}

// Does each CTA list its own items?  Few sequences, no more than a lane's item each per CTA, and
// a causal mask (under which the last blocks are the heaviest).
bool lists_own(const PackedShape& s, const DeviceInfo& dev) {
  const bool k64 = takes_k64(s);
  const int block = k64 ? 128 : 256;
  const int ctas = (k64 && s.Dh <= 128 ? 2 : 1) * dev.num_sms;
  const long long items = ((long long)s.T / block + s.B) * s.Hq;
  return s.causal && s.B <= kOwnSequences && s.T / block + 1 <= kOwnLevels &&
         items <= (long long)ctas * kOwnItems;
}

}  // namespace

// The workspace: the tile counts (256 bytes), then the list.
size_t fwd_packed_workspace_bytes(const PackedShape& s, const DeviceInfo& dev) {
  if (lists_own(s, dev)) return 0;
  return 256 + ((size_t)packed_max_tiles(s.B, s.T) * sizeof(PackedTile) + 255) / 256 * 256;
}

cudaError_t launch_fwd_packed(const PackedShape& s, const PackedRows& q, const PackedRows& k,
                              const PackedRows& v, const PackedRows& o, float* lse,
                              void* workspace, float scale_log2, const DeviceInfo& dev,
                              cudaStream_t stream) {
  const bool k64 = takes_k64(s);
  const int block = k64 ? 128 : 256;
  const int fold_max = takes_k64(s) ? packed_fold_max(s, kFoldMeanRows) : 0;
  PackedRef ref{nullptr, nullptr, s.cu, s.B, s.T / block + 1, s.T, 0, fold_max};
  if (!lists_own(s, dev)) {
    int* count = static_cast<int*>(workspace);
    void* tiles = static_cast<char*>(workspace) + 256;
    const int order = kByKeys;
    const cudaError_t e = launch_packed_schedule(s, block, fold_max, 1, &order, &tiles, &count, dev, stream);
    if (e != cudaSuccess) return e;
    ref.tiles = static_cast<PackedTile*>(tiles);
    ref.num_tiles = count;
  }
  if (s.Dh == 256) return launch_k64<256>(s, q, k, v, o, lse, ref, scale_log2, dev, stream);
  if (k64)
    return s.Dh == 128 ? launch_k64<128>(s, q, k, v, o, lse, ref, scale_log2, dev, stream)
                       : launch_k64<64>(s, q, k, v, o, lse, ref, scale_log2, dev, stream);
  return s.Dh == 128 ? launch_wide<128>(s, q, k, v, o, lse, ref, scale_log2, dev, stream)
                     : launch_wide<64>(s, q, k, v, o, lse, ref, scale_log2, dev, stream);
}

}  // namespace chs
