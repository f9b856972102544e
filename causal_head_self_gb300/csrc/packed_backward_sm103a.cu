// packed_backward_sm103a.cu -- attention over packed sequences, backward: the lists of tiles,
// D and lse2 per row, then the passes of the batch form over the lists.
#include "backward256_sm103a.cuh"
#include "backward_sm103a.cuh"
#include "launch.h"

namespace chs {

namespace {

// Rows of the statistics: each sequence's from a multiple of 128 on (packed_schedule_sm103a.cuh).
long long stat_rows(int B, int T) { return ((long long)T + 127ll * B + 127) / 128 * 128; }

size_t list_bytes(int B, int T) {
  return ((size_t)packed_max_tiles(B, T) * sizeof(PackedTile) + 255) / 256 * 256;
}

struct BwdMaps {
  CUtensorMap q, k, v, dout;
  int heads_inner = 0;
};

bool bwd_maps(BwdMaps* m, const PackedShape& s, const PackedRows& q, const PackedRows& k,
              const PackedRows& v, const PackedRows& dout, int q_rows, int kv_rows) {
  bool hq, hk, hv, hd;
  if (!encode_packed_map(&m->q, q, s.Dh, s.T, q_rows, true, &hq) ||
      !encode_packed_map(&m->k, k, s.Dh, s.T, kv_rows, true, &hk) ||
      !encode_packed_map(&m->v, v, s.Dh, s.T, kv_rows, true, &hv) ||
      !encode_packed_map(&m->dout, dout, s.Dh, s.T, q_rows, true, &hd))
    return false;
  m->heads_inner = (hq ? kPackedQ : 0) | (hk ? kPackedK : 0) | (hv ? kPackedV : 0) |
                   (hd ? kPackedDO : 0);
  return true;
}

template <int DH>
cudaError_t launch_prep(const PackedShape& s, const PackedRows& q, const PackedRows& k,
                        const PackedRows& v, const PackedRows& o, const PackedRows& dout,
                        const float* lse, const BwdParams& p, cudaStream_t stream) {
  auto bf = [](const PackedRows& x) { return static_cast<const __nv_bfloat16*>(x.data); };
  BwdPrepPacked a{bf(q),  bf(k),  bf(v),  bf(o),  bf(dout), q.row,    q.head,    k.row, k.head,
                  v.row,  v.head, o.row,  o.head, dout.row, dout.head};
  a.lse = lse;
  a.lse2 = const_cast<float*>(p.lse2);
  a.delta = const_cast<float*>(p.delta);
  a.pk = p.pk;
  a.Hq = s.Hq;
  a.group = p.group;
  a.causal = s.causal;
  a.window = s.window;
  a.S_pad = p.S_pad;
  a.scale_log2 = p.scale_log2;
  a.error_word = p.error_word;
  a.cu = s.cu;
  a.B = s.B;
  const long long blocks = packed_max_tiles(s.B, s.T) * s.Hq;
  const long long few = s.causal && s.window > 0 && s.window <= kPrepKeys
                            ? blocks
                            : (long long)s.B * ((s.Hq + kFewHeads - 1) / kFewHeads);
  const cudaError_t e =
      launch_pdl(attn_bwd_prep_few<DH>, dim3((unsigned)few), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_bwd_prep_packed<DH>, dim3((unsigned)blocks), dim3(256), 0, stream, a);
}

template <int DH, int PK>
cudaError_t launch_passes(const PackedShape& s, const BwdMaps& m, const BwdParams& pk,
                          const BwdParams& pq, const DeviceInfo& dev, cudaStream_t stream) {
  constexpr size_t smem_kv = bwd_dkdv_smem_bytes<DH>(), smem_q = bwd_dq_smem_bytes<DH>();
  static std::atomic<int> configured[kMaxDevices];
  cudaError_t e = configure_once(configured, dev.device, [] {
    cudaError_t r = cudaFuncSetAttribute(attn_bwd_dkdv<DH, PK>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_kv);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(attn_bwd_dq<DH, PK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_q);
  });
  if (e != cudaSuccess) return e;
  const long long most = packed_max_tiles(s.B, s.T);
  const int grid_kv = (int)(most * s.Hkv < dev.num_sms ? most * s.Hkv : dev.num_sms);
  e = launch_pdl(attn_bwd_dkdv<DH, PK>, dim3(grid_kv), dim3(BwdCfg<DH>::kThreads), smem_kv,
                 stream, m.q, m.k, m.v, m.dout, pk);
  if (e != cudaSuccess) return e;
  const int grid_q = (int)(most * s.Hq < dev.num_sms ? most * s.Hq : dev.num_sms);
  return launch_pdl(attn_bwd_dq<DH, PK>, dim3(grid_q), dim3(BwdCfg<DH>::kThreads), smem_q,
                    stream, m.q, m.k, m.v, m.dout, pq);
}

cudaError_t launch_passes256(const PackedShape& s, const BwdMaps& small_q, const BwdMaps& small_k,
                             const BwdParams& pk, const BwdParams& pq, const DeviceInfo& dev,
                             cudaStream_t stream) {
  using Cfg = Bwd256Cfg;
  constexpr size_t smem_dv = bwd256_kv_smem_bytes<false>(), smem_dk = bwd256_kv_smem_bytes<true>(),
                   smem_dq = bwd256_dq_smem_bytes();
  static std::atomic<int> configured[kMaxDevices];
  cudaError_t e = configure_once(configured, dev.device, [] {
    cudaError_t r = cudaFuncSetAttribute(attn_bwd256_kv<false, 1>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_dv);
    if (r != cudaSuccess) return r;
    r = cudaFuncSetAttribute(attn_bwd256_kv<true, 1>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_dk);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(attn_bwd256_dq<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_dq);
  });
  if (e != cudaSuccess) return e;
  const long long most = packed_max_tiles(s.B, s.T);
  const int grid_kv = (int)(most * s.Hkv < dev.num_sms ? most * s.Hkv : dev.num_sms);
  e = launch_pdl(attn_bwd256_kv<false, 1>, dim3(grid_kv), dim3(Cfg::kThreads), smem_dv, stream,
                 small_q.q, small_q.k, small_q.v, small_q.dout, pk);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_bwd256_kv<true, 1>, dim3(grid_kv), dim3(Cfg::kThreads), smem_dk, stream,
                 small_q.q, small_q.k, small_q.v, small_q.dout, pk);
  if (e != cudaSuccess) return e;
  const int grid_q = (int)(most * s.Hq < dev.num_sms ? most * s.Hq : dev.num_sms);
  return launch_pdl(attn_bwd256_dq<1>, dim3(grid_q), dim3(Cfg::kThreads), smem_dq, stream,
                    small_k.q, small_k.k, small_k.v, small_k.dout, pq);
}

}  // namespace

// The workspace: the tile counts (256 bytes), two lists, lse2 and D.
size_t bwd_packed_workspace_bytes(int B, int Hq, int T) {
  return 256 + 2 * list_bytes(B, T) + 2 * (size_t)Hq * stat_rows(B, T) * sizeof(float);
}

cudaError_t launch_bwd_packed(const PackedShape& s, const PackedRows& q, const PackedRows& k,
                              const PackedRows& v, const PackedRows& o, const PackedRows& dout,
                              const float* lse, const PackedRows& dq, const PackedRows& dk,
                              const PackedRows& dv, void* workspace, float scale,
                              const DeviceInfo& dev, cudaStream_t stream) {
  char* ws = static_cast<char*>(workspace);
  int* counts[2] = {reinterpret_cast<int*>(ws), reinterpret_cast<int*>(ws) + 4};
  void* lists[2] = {ws + 256, ws + 256 + list_bytes(s.B, s.T)};
  const int order[2] = {kByQueries, kByKeys};
  // two or four heads of short sequences in one block of queries, as in the forward pass (head
  // size 256 streams blocks of 64 queries, which a short sequence does not waste)
  const int fold_max = s.Dh == 256 ? 0 : packed_fold_max(s, kFoldMeanRowsBackward);
  // the maps first: nothing is launched where one cannot be made
  BwdMaps m, m2;
  if (s.Dh == 256 ? !bwd_maps(&m, s, q, k, v, dout, 64, 128) ||
                        !bwd_maps(&m2, s, q, k, v, dout, 128, 64)
                  : !bwd_maps(&m, s, q, k, v, dout, fold_max ? 32 : 128, 128))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_packed_schedule(s, 128, fold_max, 2, order, lists, counts, dev, stream);
  if (e != cudaSuccess) return e;
  BwdParams p{};
  p.B = 1;
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  p.causal = s.causal;
  p.window = s.window;
  p.scale = scale;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.S_pad = (int)stat_rows(s.B, s.T);
  p.group = s.Hq / s.Hkv;
  // a window this short leaves every query few keys
  constexpr int kShortWindow = 256;
  p.two_parts = s.window > 0 && s.window <= kShortWindow;
  float* stats = reinterpret_cast<float*>(ws + 256 + 2 * list_bytes(s.B, s.T));
  p.lse2 = stats;
  p.delta = stats + (size_t)s.Hq * p.S_pad;
  auto bf = [](const PackedRows& x) { return static_cast<__nv_bfloat16*>(const_cast<void*>(x.data)); };
  p.dq = bf(dq);
  p.dk = bf(dk);
  p.dv = bf(dv);
  p.dq_row = dq.row;
  p.dq_head = dq.head;
  p.dk_row = dk.row;
  p.dk_head = dk.head;
  p.dv_row = dv.row;
  p.dv_head = dv.head;
  p.wide = 1;
  for (const PackedRows* x : {&dq, &dk, &dv})
    if ((reinterpret_cast<uintptr_t>(x->data) & 31) != 0 || x->row % 16 != 0 || x->head % 16 != 0)
      p.wide = 0;
  p.error_word = dev.error_word;
  p.fault = dev.fault;
  BwdParams pk = p, pq = p;
  pk.pk = PackedRef{static_cast<PackedTile*>(lists[0]), counts[0], s.cu, s.B, 0, s.T, m.heads_inner, fold_max};
  pq.pk = PackedRef{static_cast<PackedTile*>(lists[1]), counts[1], s.cu, s.B, 0, s.T, m.heads_inner, fold_max};
  e = s.Dh == 256   ? launch_prep<256>(s, q, k, v, o, dout, lse, pq, stream)
      : s.Dh == 128 ? launch_prep<128>(s, q, k, v, o, dout, lse, pq, stream)
                    : launch_prep<64>(s, q, k, v, o, dout, lse, pq, stream);
  if (e != cudaSuccess) return e;
  if (s.Dh == 256) return launch_passes256(s, m, m2, pk, pq, dev, stream);
  if (fold_max)
    return s.Dh == 128 ? launch_passes<128, 2>(s, m, pk, pq, dev, stream)
                       : launch_passes<64, 2>(s, m, pk, pq, dev, stream);
  return s.Dh == 128 ? launch_passes<128, 1>(s, m, pk, pq, dev, stream)
                     : launch_passes<64, 1>(s, m, pk, pq, dev, stream);
}

}  // namespace chs
