// launch.h -- internal interface between the C-ABI layer and the kernel
// translation units.  Not part of the public ABI (see include/attn.h).
#pragma once

#include <atomic>
#include <utility>

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime_api.h>

namespace chs {

// Kernel attributes (shared-memory size, carveout) are set once per device:
// `flags` is a per-kernel array of kMaxDevices entries.
constexpr int kMaxDevices = 64;
template <typename F>
inline cudaError_t configure_once(std::atomic<int>* flags, int device, F&& set) {
  const bool tracked = device >= 0 && device < kMaxDevices;
  if (tracked && flags[device].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = set();
  if (e == cudaSuccess && tracked) flags[device].store(1, std::memory_order_release);
  return e;
}

// Launch `kernel` on `stream` as a programmatic dependent of the kernel
// before it: its CTAs may be scheduled while that kernel finishes, and each
// waits (griddep_wait) for it to complete before touching global memory.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

struct DeviceInfo {
  int device;
  int num_sms;
  int* error_word;   // device address of this device's latched error word
  int fault;         // test hook passed to the kernels (attn_debug_inject_fault)
};

// Encode a 3-D tensor map over a [outer, stride_rows, Dh] bf16 tensor of
// which the first `rows` rows per outer index are visible: dims {Dh, rows,
// outer}, 128-byte swizzle, box {64, box_rows, 1}.  Rows at or past `rows`
// are never read; a box reaching past them is zero-filled
// (stride_rows = 0 means stride_rows = rows).
bool encode_bf16_map(CUtensorMap* map, const void* base, int Dh, int rows, long long outer,
                     int box_rows, int stride_rows = 0);

// The same tensor as a 4-D map, dims {64, rows, Dh / 64, outer}, box {64,
// box_rows, Dh / 64, 1}: one copy brings whole rows, laid out in shared memory as
// the 64-column boxes of the 3-D map one after another.
bool encode_bf16_rows_map(CUtensorMap* map, const void* base, int Dh, int rows, long long outer,
                          int box_rows);

// Queries: Sq rows per (b, h), at positions start_pos .. start_pos + Sq - 1.
// K, V: Tkv rows per (b, K/V head) in memory, of which the first
// start_pos + Sq are visible (a plain prefill: Tkv = Sq, start_pos = 0).
// lse (optional, [B, Hq, Sq] fp32) receives each row's log-sum-exp.
cudaError_t launch_prefill(const void* q, const void* k, const void* v, void* o, float* lse,
                           int B, int Hq, int Hkv, int Sq, int Tkv, int start_pos, int Dh,
                           int causal, int window, float scale_log2, const DeviceInfo& dev,
                           cudaStream_t stream);

struct DecodePlan {
  int chunk;          // keys per split
  int nsplit;         // splits per (b, query head)
  int heads_per_cta;  // query heads of a GQA group handled by one CTA
};

DecodePlan plan_decode(int B, int Hq, int Hkv, int Tmax, int Dh, int num_sms);

// Bytes of split partials (o, max, sum) a decode call with this plan needs.
size_t decode_partials_bytes(int B, int Hq, int Dh, const DecodePlan& plan);

// Completion counters (one int per CTA group) a decode call needs.  They
// must be zero before the call, and every call leaves them zero again, so a
// buffer that only ever holds counters stays valid across calls and shapes.
size_t decode_counter_count(int B, int Hq, int Hkv, const DecodePlan& plan);

// ring = 1: the Tmax cache rows of a head hold position t at row t % Tmax
// (the last Tmax positions of an unbounded sequence).
cudaError_t launch_decode(const void* q, const void* kc, const void* vc, const int* seqlens,
                          void* o, int B, int Hq, int Hkv, int Tmax, int Dh, int window,
                          int ring, float scale_log2, const DecodePlan& plan, int* counters,
                          void* partials, const DeviceInfo& dev, cudaStream_t stream);

// Tensor-core decode for query-head groups (Hq / Hkv >= kDecodeTcMinGroup):
// splits of whole 128-key tiles, one CTA per (split, b, K/V head, 128 heads),
// then a combine kernel.  Linear caches, and rings (ring = 1: position t at
// row t % Tmax, window <= Tmax, window <= 0 meaning Tmax).  Measured against
// the CUDA-core kernel on the same inputs (back-to-back launches): groups of
// 4 run at 6.8 TB/s instead of 6.3 (Dh 128), 5.6 instead of 3.8 (Dh 64) and
// 6.0 instead of 5.7 (Dh 256), groups of 2 at 6.7 instead of 6.6; with one
// query head per K/V head the CUDA-core kernel is as fast (Dh 128) or faster
// (Dh 64: 6.3 against 5.1 TB/s), so it keeps that case.
constexpr int kDecodeTcMinGroup = 2;
DecodePlan plan_decode_tc(int B, int Hq, int Hkv, int Tmax, int num_sms);
cudaError_t launch_decode_tc(const void* q, const void* kc, const void* vc, const int* seqlens,
                             void* o, int B, int Hq, int Hkv, int Tmax, int Dh, int window,
                             int ring, float scale_log2, const DecodePlan& plan, void* partials,
                             const DeviceInfo& dev, cudaStream_t stream);

// Backward pass (Dh 64 or 128): dq [B, Hq, S, Dh], dk and dv [B, Hkv, S, Dh]
// from q, k, v, the forward output o, its log-sum-exps lse [B, Hq, S] and
// dout; workspace holds bwd_workspace_bytes(B, Hq, S) bytes (16-byte aligned).
size_t bwd_workspace_bytes(int B, int Hq, int S);
cudaError_t launch_bwd(const void* q, const void* k, const void* v, const void* o,
                       const void* dout, const float* lse, void* dq, void* dk, void* dv,
                       float* workspace, int B, int Hq, int Hkv, int S, int Dh, int causal,
                       int window, float scale, const DeviceInfo& dev, cudaStream_t stream);

// ---------------------------------------------------------------- packed sequences
// Rows of heads [T, H, Dh] bf16 at any strides, in elements (include/attn.h).
struct PackedRows {
  const void* data;
  long long row, head;
  int H;
};

// A map over such a tensor with boxes of box_rows x 64, with the row axis once or (padded, for
// loads that begin with padding) twice: packed_sm103a.cuh.  *heads_inner says in which order
// its axes lie.
bool encode_packed_map(CUtensorMap* map, const PackedRows& x, int Dh, int T, int box_rows,
                       bool padded, bool* heads_inner);

struct PackedShape {
  int B, Hq, Hkv, T, Dh;
  int causal, window;
  const int* cu;   // [B + 1] first rows of the sequences, and the last one's end
};

// Two or four query heads of a K/V head go into one tile of a short sequence (as 1 << the
// result), where sequences have up to mean_rows rows on average: Q then comes in copies of 32
// rows.  The forward pass loses nothing by it (sequences of 100 to 256 rows: the same time);
// the backward's kernels take 13 % longer over 128 sequences of 128 and win at 64 rows (a fifth
// of the time) and below.
constexpr int kFoldMeanRows = 256, kFoldMeanRowsBackward = 96;
inline int packed_fold_max(const PackedShape& s, int mean_rows) {
  const int group = s.Hq / s.Hkv;
  if (s.T > (long long)mean_rows * s.B) return 0;
  return group % 4 == 0 ? 2 : group % 2 == 0 ? 1 : 0;
}

// Device memory that the calls need: the lists of tiles, and the backward's row statistics.
size_t fwd_packed_workspace_bytes(const PackedShape& s, const DeviceInfo& dev);
size_t bwd_packed_workspace_bytes(int B, int Hq, int T);
// Most 128-row tiles that B sequences of T rows in all can have.
inline long long packed_max_tiles(int B, int T) { return (long long)T / 128 + B; }

cudaError_t launch_fwd_packed(const PackedShape& s, const PackedRows& q, const PackedRows& k,
                              const PackedRows& v, const PackedRows& o, float* lse,
                              void* workspace, float scale_log2, const DeviceInfo& dev,
                              cudaStream_t stream);
cudaError_t launch_bwd_packed(const PackedShape& s, const PackedRows& q, const PackedRows& k,
                              const PackedRows& v, const PackedRows& o, const PackedRows& dout,
                              const float* lse, const PackedRows& dq, const PackedRows& dk,
                              const PackedRows& dv, void* workspace, float scale,
                              const DeviceInfo& dev, cudaStream_t stream);
// Lists of tiles of `block` rows, heaviest first: list[i] for order[i] (PackedOrder); tiles and
// counts (three each) lie in device memory.
cudaError_t launch_packed_schedule(const PackedShape& s, int block, int fold_max, int lists, const int* order,
                                   void* const* tiles, int* const* counts, const DeviceInfo& dev,
                                   cudaStream_t stream);

// ---------------------------------------------------------------- tokens
// [B, S, H, Dh] bf16 at any strides, in elements.
struct RopeRows {
  const void* data;
  long long batch, row, head;
};

struct RopeShape {
  int B, S, Hq, Hkv, Dh, rot;
  const int* positions;              // [B * S]
  const unsigned long long* turns;   // [rot / 2], 2^-64 turns per token
  float amplitude;
  int interleaved, inverse;
};

struct RopeAppend {
  RopeRows v;
  void *kpages, *vpages;
  const int* slots;   // [B * S]
  int num_pages, page;
};

// q_out and k_out may be the inputs, or null (k_out with append: k goes to the cache alone).
cudaError_t launch_rope(const RopeShape& s, const RopeRows& q, const RopeRows* q_out,
                        const RopeRows& k, const RopeRows* k_out, const RopeAppend* append,
                        const DeviceInfo& dev, cudaStream_t stream);

// The pages, slots and positions of a step (include/attn.h).
struct CachePlan {
  const int *delta, *seqlens;
  int *seqlens_out, *table, *free_pages;
  const int* num_free;
  int *num_free_out, *cu, *positions, *slots;
  int B, cols, page, num_pages, capacity, T;
};
int cache_plan_max_sequences();
cudaError_t launch_cache_plan(const CachePlan& c, const DeviceInfo& dev, cudaStream_t stream);

// ---------------------------------------------------------------- paged cache
// K and V pools [num_pages, Hkv, page, Dh]; row t of sequence b in page
// table[b, t / page] at row t % page (include/attn.h).
struct PagedCache {
  int num_pages, page, cols;   // cols: table columns
};

// Rows per TMA box: the largest that divides both a page and a key tile.
int paged_box_rows(int page, int Dh);

// Device memory that a paged decode call needs: partial results, and with
// `scores` the raw score of every (query head, key).
size_t decode_paged_workspace_bytes(int B, int Hq, int Hkv, const PagedCache& cache, int Dh,
                                    int window, bool scores, const DeviceInfo& dev);

// One decode step over a paged cache; weights (optional, [B, Hkv,
// weights_stride] fp32) receive each key's weight summed over its head group.
cudaError_t launch_decode_paged(const void* q, const void* kpages, const void* vpages,
                                const int* table, const int* seqlens, void* o, float* weights,
                                int weights_stride, int accumulate, void* workspace, int B, int Hq,
                                int Hkv, const PagedCache& cache, int Dh, int window,
                                float scale_log2, const DeviceInfo& dev, cudaStream_t stream);

// Rows of k, v [B, Hkv, S, Dh] to the cache; newlens null: all S rows.
cudaError_t launch_paged_append(const void* k, const void* v, void* kpages, void* vpages,
                                const int* table, const int* seqlens, const int* newlens, int B,
                                int Hkv, int S, const PagedCache& cache, int Dh,
                                const DeviceInfo& dev, cudaStream_t stream);

// The weights that a prompt's keys received: [B, Hkv, stride] fp32.
cudaError_t launch_key_weights(const void* q, const void* k, const float* lse, const int* seqlens,
                               float* weights, int stride, int B, int Hq, int Hkv, int S, int Dh,
                               int causal, int window, int queries, int accumulate,
                               float scale_log2, const DeviceInfo& dev, cudaStream_t stream);

// Keeps `budget` rows of each (sequence, K/V head); table_out == table: in place.
cudaError_t launch_cache_evict(void* kpages, void* vpages, const int* table, const int* table_out,
                               int cols_out, const int* seqlens, int* newlens,
                               const float* weights, int stride, float* weights_out,
                               int stride_out, int* keep, int B, int Hkv, const PagedCache& cache,
                               int Dh, int budget, int recent, const DeviceInfo& dev,
                               cudaStream_t stream);

}  // namespace chs
