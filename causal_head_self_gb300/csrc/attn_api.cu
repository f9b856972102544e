// attn_api.cu -- the C ABI declared in include/attn.h: argument checks,
// per-device state (SM count, latched error word, decode workspace), tensor
// maps, and the kernel launches.  No torch types cross this boundary.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <atomic>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "launch.h"

namespace {

constexpr int kMaxDevices = 64;

// Latched device-side status of the kernels (one per device: every device
// that loads this library holds its own copy of the symbol).
__device__ int g_attn_error_word;

struct DeviceState {
  bool ready = false;
  chs::DeviceInfo info{};
  // decode workspace: split partials, and completion counters kept in a
  // buffer of their own (always zero between calls)
  void* partials = nullptr;
  size_t partials_bytes = 0;
  int* counters = nullptr;
  size_t counters_n = 0;
  // backward workspace: per-row log-sum-exp (log2 units) and D = dO . o
  void* bwd_ws = nullptr;
  size_t bwd_ws_bytes = 0;
};

// Grow a device buffer (never inside a stream capture); zero it if asked.
int grow_buffer(void** buf, size_t* have, size_t need, bool zero, cudaStream_t stream) {
  if (*have >= need) return ATTN_OK;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone)
    return ATTN_ERR_NO_MEMORY;   // cudaMalloc cannot run inside a capture
  if (*buf) cudaFree(*buf);      // cudaFree waits for work still using it
  *buf = nullptr;
  *have = 0;
  if (cudaMalloc(buf, need) != cudaSuccess) {
    *buf = nullptr;
    cudaGetLastError();
    return ATTN_ERR_NO_MEMORY;
  }
  if (zero && cudaMemset(*buf, 0, need) != cudaSuccess) {
    cudaFree(*buf);
    *buf = nullptr;
    return ATTN_ERR_CUDA;
  }
  *have = need;
  return ATTN_OK;
}

std::mutex g_mutex;
DeviceState g_devices[kMaxDevices];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

bool load_encode_fn() {
  if (g_encode) return true;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult qres;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &qres) != cudaSuccess ||
      qres != cudaDriverEntryPointSuccess || fn == nullptr)
    return false;
  g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  return true;
}

// Per-device set-up on first use, with that device current.
int device_state(DeviceState** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return ATTN_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mutex);
  DeviceState& st = g_devices[dev];
  if (!st.ready) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return ATTN_ERR_CUDA;
    void* word = nullptr;
    if (cudaGetSymbolAddress(&word, g_attn_error_word) != cudaSuccess) return ATTN_ERR_CUDA;
    if (!load_encode_fn()) return ATTN_ERR_CUDA;
    st.info.device = dev;
    st.info.num_sms = sms;
    st.info.error_word = static_cast<int*>(word);
    st.info.fault = 0;
    st.ready = true;
  }
  *out = &st;
  return ATTN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// scale == 0 -> 1/sqrt(Dh); returns false for a negative or non-finite scale
bool resolve_scale(float scale, int Dh, float* scale_log2) {
  if (!std::isfinite(scale) || scale < 0.f) return false;
  const double s = scale == 0.f ? 1.0 / std::sqrt((double)Dh) : (double)scale;
  *scale_log2 = (float)(s * 1.4426950408889634);   // log2(e)
  return true;
}

}  // namespace

namespace chs {

// A tensor map is a pure function of these arguments, so a call that repeats
// an earlier one (the usual case: the same buffers every step) takes the map
// from a small per-thread cache instead of encoding it again.
namespace {
struct MapKey {
  const void* base;
  long long outer;
  int Dh, rows, box_rows, stride_rows;   // stride_rows 0: the 4-D form (whole rows)
  long long row = 0, head = 0;           // packed rows: their strides (0: the other forms)
  bool operator==(const MapKey& o) const {
    return base == o.base && outer == o.outer && Dh == o.Dh && rows == o.rows &&
           box_rows == o.box_rows && stride_rows == o.stride_rows && row == o.row &&
           head == o.head;
  }
};
struct MapCache {
  static constexpr int kEntries = 64;
  MapKey key[kEntries];
  alignas(64) CUtensorMap map[kEntries];
  int used = 0, next = 0;
};
thread_local MapCache t_maps;

bool cached_map(CUtensorMap* map, const MapKey& key, int rank, const cuuint64_t* dims,
                const cuuint64_t* strides, const cuuint32_t* box) {
  MapCache& c = t_maps;
  for (int i = 0; i < c.used; ++i) {
    if (c.key[i] == key) {
      *map = c.map[i];
      return true;
    }
  }
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  if (g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
               const_cast<void*>(key.base), dims, strides, box, elem,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  const int slot = c.next;
  c.key[slot] = key;
  c.map[slot] = *map;
  c.next = (slot + 1) % MapCache::kEntries;
  if (c.used < MapCache::kEntries) ++c.used;
  return true;
}
}  // namespace

bool encode_bf16_map(CUtensorMap* map, const void* base, int Dh, int rows, long long outer,
                     int box_rows, int stride_rows) {
  if (stride_rows == 0) stride_rows = rows;
  if (rows < 1 || stride_rows < rows) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)Dh, (cuuint64_t)rows, (cuuint64_t)outer};
  const cuuint64_t strides[2] = {(cuuint64_t)Dh * 2, (cuuint64_t)Dh * 2 * (cuuint64_t)stride_rows};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  return cached_map(map, MapKey{base, outer, Dh, rows, box_rows, stride_rows}, 3, dims, strides,
                    box);
}

bool encode_bf16_rows_map(CUtensorMap* map, const void* base, int Dh, int rows, long long outer,
                          int box_rows) {
  if (rows < 1) return false;
  const cuuint64_t row = (cuuint64_t)Dh * 2;
  const cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)Dh / 64, (cuuint64_t)outer};
  const cuuint64_t strides[3] = {row, 128, row * (cuuint64_t)rows};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, (cuuint32_t)Dh / 64, 1};
  return cached_map(map, MapKey{base, outer, Dh, rows, box_rows, 0}, 4, dims, strides, box);
}

bool encode_packed_map(CUtensorMap* map, const PackedRows& x, int Dh, int T, int box_rows,
                       bool padded, bool* heads_inner) {
  // strides of an axis with one entry do not matter: any that the map takes
  const long long head = x.H > 1 ? x.head : T > 1 ? x.row : Dh;
  const long long row = T > 1 ? x.row : head;
  // the axes in the order of their strides
  *heads_inner = x.H > 1 && head < row;
  const cuuint64_t R = (cuuint64_t)row * 2, H = (cuuint64_t)head * 2;
  const cuuint64_t rows = (cuuint64_t)T, heads = (cuuint64_t)x.H, height = (cuuint64_t)box_rows;
  const cuuint32_t b = (cuuint32_t)box_rows;
  const MapKey key{x.data, x.H, Dh, T, box_rows, padded ? -1 : -2, row, head};
  const cuuint64_t d = (cuuint64_t)Dh;
  if (padded) {
    // the row axis twice (packed_sm103a.cuh)
    const cuuint64_t dims_in[4] = {d, heads, height, rows}, dims[4] = {d, height, rows, heads};
    const cuuint64_t strides_in[3] = {H, R, R}, strides[3] = {R, R, H};
    const cuuint32_t box_in[4] = {64, 1, b, 1}, box[4] = {64, b, 1, 1};
    return *heads_inner ? cached_map(map, key, 4, dims_in, strides_in, box_in)
                        : cached_map(map, key, 4, dims, strides, box);
  }
  const cuuint64_t dims_in[3] = {d, heads, rows}, dims[3] = {d, rows, heads};
  const cuuint64_t strides_in[2] = {H, R}, strides[2] = {R, H};
  const cuuint32_t box_in[3] = {64, 1, b}, box[3] = {64, b, 1};
  return *heads_inner ? cached_map(map, key, 3, dims_in, strides_in, box_in)
                      : cached_map(map, key, 3, dims, strides, box);
}

}  // namespace chs

extern "C" {

int attn_version(void) { return (1 << 16) | 0; }

const char* attn_error_string(int code) {
  switch (code) {
    case ATTN_OK: return "ATTN_OK";
    case ATTN_ERR_INVALID_ARG: return "ATTN_ERR_INVALID_ARG";
    case ATTN_ERR_UNSUPPORTED: return "ATTN_ERR_UNSUPPORTED";
    case ATTN_ERR_CUDA: return "ATTN_ERR_CUDA";
    case ATTN_ERR_TIMEOUT: return "ATTN_ERR_TIMEOUT";
    case ATTN_ERR_NO_MEMORY: return "ATTN_ERR_NO_MEMORY";
    case ATTN_ERR_SCRATCH_LIMIT: return "ATTN_ERR_SCRATCH_LIMIT";
    case ATTN_ERR_CHECK: return "ATTN_ERR_CHECK";
    default: return "ATTN_ERR_UNKNOWN";
  }
}

// The test hook's current fault (attn_debug_inject_fault); 0 in normal use.
static std::atomic<int> g_fault{0};

static chs::DeviceInfo launch_info(const DeviceState* st) {
  chs::DeviceInfo d = st->info;
  d.fault = g_fault.load(std::memory_order_relaxed);
  return d;
}

int attn_debug_inject_fault(int kind) {
  if (kind < 0 || kind > 4) return ATTN_ERR_INVALID_ARG;
  g_fault.store(kind, std::memory_order_relaxed);
  return ATTN_OK;
}

// Shared by attn_fwd and attn_fwd_chunk: queries at positions
// start_pos .. start_pos + Sq - 1 against the first start_pos + Sq of Tkv
// key/value rows per head.
static int fwd_common(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                      int Hq, int Hkv, int Sq, int Tkv, int start_pos, int Dh, int causal,
                      int window, float scale, cudaStream_t stream) {
  if (B < 0 || Sq < 0 || Tkv < 0 || start_pos < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0)
    return ATTN_ERR_INVALID_ARG;
  if ((long long)start_pos + Sq > Tkv) return ATTN_ERR_INVALID_ARG;
  if (Dh != 64 && Dh != 128 && Dh != 256) return ATTN_ERR_UNSUPPORTED;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (window < 0) window = 0;
  if (window > 0 && !causal) return ATTN_ERR_INVALID_ARG;
  float scale_log2 = 0.f;
  if (!resolve_scale(scale, Dh, &scale_log2)) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || Sq == 0) return ATTN_OK;
  if (!q || !k || !v || !o) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
  const size_t qo_bytes = (size_t)B * Hq * Sq * Dh * 2, kv_bytes = (size_t)B * Hkv * Tkv * Dh * 2;
  if ((long long)B * Hq * ((Sq + 127) / 128) > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  if (overlaps(o, qo_bytes, q, qo_bytes) || overlaps(o, qo_bytes, k, kv_bytes) ||
      overlaps(o, qo_bytes, v, kv_bytes))
    return ATTN_ERR_INVALID_ARG;
  if (lse != nullptr) {
    const size_t lse_bytes = (size_t)B * Hq * Sq * 4;
    if ((reinterpret_cast<uintptr_t>(lse) & 3) != 0 || overlaps(lse, lse_bytes, o, qo_bytes) ||
        overlaps(lse, lse_bytes, q, qo_bytes) || overlaps(lse, lse_bytes, k, kv_bytes) ||
        overlaps(lse, lse_bytes, v, kv_bytes))
      return ATTN_ERR_INVALID_ARG;
  }
  DeviceState* st = nullptr;
  int rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  cudaError_t e = chs::launch_prefill(q, k, v, o, lse, B, Hq, Hkv, Sq, Tkv, start_pos, Dh, causal,
                                      window, scale_log2, launch_info(st), stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_fwd(const void* q, const void* k, const void* v, void* o, int B, int Hq, int Hkv, int S,
             int Dh, int causal, int window, float scale, cudaStream_t stream) {
  return fwd_common(q, k, v, o, nullptr, B, Hq, Hkv, S, S, 0, Dh, causal, window, scale, stream);
}

int attn_fwd_lse(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                 int Hkv, int S, int Dh, int causal, int window, float scale,
                 cudaStream_t stream) {
  if (lse == nullptr && B > 0 && S > 0) return ATTN_ERR_INVALID_ARG;
  return fwd_common(q, k, v, o, lse, B, Hq, Hkv, S, S, 0, Dh, causal, window, scale, stream);
}

int attn_fwd_chunk(const void* q, const void* kcache, const void* vcache, void* o, int B, int Hq,
                   int Hkv, int Sq, int Tmax, int start_pos, int Dh, int causal, int window,
                   float scale, cudaStream_t stream) {
  if (Tmax < 1) return ATTN_ERR_INVALID_ARG;
  return fwd_common(q, kcache, vcache, o, nullptr, B, Hq, Hkv, Sq, Tmax, start_pos, Dh, causal,
                    window, scale, stream);
}

// Argument and aliasing checks of every decode entry point (attn_decode,
// attn_decode_ring, attn_decode_noalloc), so that all three return the same
// errors for the same arguments.  On ATTN_OK, *window and *scale_log2 hold
// the resolved window (0: none) and softmax scale times log2(e); *empty is
// set when B == 0 (nothing to launch).
static int decode_check_args(const void* q, const void* kcache, const void* vcache,
                             const int* seqlens, const void* o, int B, int Hq, int Hkv, int Tmax,
                             int Dh, int* window, int ring, float scale, float* scale_log2,
                             bool* empty) {
  *empty = false;
  if (B < 0 || Tmax < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (Dh != 64 && Dh != 128 && Dh != 256) return ATTN_ERR_UNSUPPORTED;
  if (*window < 0) *window = 0;
  if (ring && *window > Tmax) return ATTN_ERR_INVALID_ARG;   // the ring holds Tmax positions
  if (!resolve_scale(scale, Dh, scale_log2)) return ATTN_ERR_INVALID_ARG;
  if (B == 0) {
    *empty = true;
    return ATTN_OK;
  }
  if (!q || !kcache || !vcache || !seqlens || !o) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kcache) || !aligned16(vcache) || !aligned16(o) ||
      (reinterpret_cast<uintptr_t>(seqlens) & 3u))
    return ATTN_ERR_INVALID_ARG;
  const size_t qo_bytes = (size_t)B * Hq * Dh * 2;
  const size_t kv_bytes = (size_t)B * Hkv * Tmax * Dh * 2;
  if (overlaps(o, qo_bytes, q, qo_bytes) || overlaps(o, qo_bytes, kcache, kv_bytes) ||
      overlaps(o, qo_bytes, vcache, kv_bytes) || overlaps(o, qo_bytes, seqlens, (size_t)B * 4))
    return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Hkv * (Hq / Hkv) > 65535LL * 65535LL) return ATTN_ERR_INVALID_ARG;
  if (B > 65535) return ATTN_ERR_INVALID_ARG;   // grid.z
  return ATTN_OK;
}

// Shared by attn_decode (ring = 0) and attn_decode_ring (ring = 1).
static int decode_common(const void* q, const void* kcache, const void* vcache, const int* seqlens,
                         void* o, int B, int Hq, int Hkv, int Tmax, int Dh, int window, int ring,
                         float scale, cudaStream_t stream) {
  float scale_log2 = 0.f;
  bool empty = false;
  int rc = decode_check_args(q, kcache, vcache, seqlens, o, B, Hq, Hkv, Tmax, Dh, &window, ring,
                             scale, &scale_log2, &empty);
  if (rc != ATTN_OK || empty) return rc;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  if (Hq / Hkv >= chs::kDecodeTcMinGroup) {
    // two or more query heads per cached byte: the tensor-core path (a contraction)
    const chs::DecodePlan plan = chs::plan_decode_tc(B, Hq, Hkv, Tmax, st->info.num_sms);
    if ((long long)B * Hkv * ((Hq / Hkv + 127) / 128) > 65535) return ATTN_ERR_INVALID_ARG;
    void* partials = nullptr;
    {
      std::lock_guard<std::mutex> lock(g_mutex);
      rc = grow_buffer(&st->partials, &st->partials_bytes,
                       chs::decode_partials_bytes(B, Hq, Dh, plan), false, stream);
      if (rc != ATTN_OK) return rc;
      partials = st->partials;
    }
    cudaError_t e = chs::launch_decode_tc(q, kcache, vcache, seqlens, o, B, Hq, Hkv, Tmax, Dh,
                                          window, ring, scale_log2, plan, partials,
                                          launch_info(st), stream);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
  }
  const chs::DecodePlan plan = chs::plan_decode(B, Hq, Hkv, Tmax, Dh, st->info.num_sms);
  if ((long long)Hkv * ((Hq / Hkv) / plan.heads_per_cta) > 65535) return ATTN_ERR_INVALID_ARG;
  const size_t need_partials = chs::decode_partials_bytes(B, Hq, Dh, plan);
  const size_t need_counters = chs::decode_counter_count(B, Hq, Hkv, plan);
  void* partials = nullptr;
  int* counters = nullptr;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    rc = grow_buffer(&st->partials, &st->partials_bytes, need_partials, false, stream);
    if (rc != ATTN_OK) return rc;
    size_t counter_bytes = st->counters_n * sizeof(int);
    void* cbuf = st->counters;
    rc = grow_buffer(&cbuf, &counter_bytes, need_counters * sizeof(int), true, stream);
    st->counters = static_cast<int*>(cbuf);
    st->counters_n = counter_bytes / sizeof(int);
    if (rc != ATTN_OK) return rc;
    partials = st->partials;
    counters = st->counters;
  }
  cudaError_t e = chs::launch_decode(q, kcache, vcache, seqlens, o, B, Hq, Hkv, Tmax, Dh, window,
                                     ring, scale_log2, plan, counters, partials, launch_info(st),
                                     stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
             const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int S, int Dh,
             int causal, int window, float scale, cudaStream_t stream) {
  if (B < 0 || S < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (Dh != 64 && Dh != 128 && Dh != 256) return ATTN_ERR_UNSUPPORTED;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (window < 0) window = 0;
  if (window > 0 && !causal) return ATTN_ERR_INVALID_ARG;
  float scale_log2 = 0.f;
  if (!resolve_scale(scale, Dh, &scale_log2)) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || S == 0) return ATTN_OK;
  const void* in[] = {q, k, v, o, dout};
  void* out[] = {dq, dk, dv};
  for (const void* x : in)
    if (!x || !aligned16(x)) return ATTN_ERR_INVALID_ARG;
  for (const void* x : out)
    if (!x || !aligned16(x)) return ATTN_ERR_INVALID_ARG;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Hq * ((S + 127) / 128) > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  const size_t qb = (size_t)B * Hq * S * Dh * 2, kb = (size_t)B * Hkv * S * Dh * 2;
  const size_t in_bytes[] = {qb, kb, kb, qb, qb};
  const size_t out_bytes[] = {qb, kb, kb};
  for (int a = 0; a < 3; ++a) {
    for (int b = 0; b < 5; ++b)
      if (overlaps(out[a], out_bytes[a], in[b], in_bytes[b])) return ATTN_ERR_INVALID_ARG;
    if (overlaps(out[a], out_bytes[a], lse, (size_t)B * Hq * S * 4)) return ATTN_ERR_INVALID_ARG;
    for (int b = a + 1; b < 3; ++b)
      if (overlaps(out[a], out_bytes[a], out[b], out_bytes[b])) return ATTN_ERR_INVALID_ARG;
  }
  DeviceState* st = nullptr;
  int rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  void* ws = nullptr;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    rc = grow_buffer(&st->bwd_ws, &st->bwd_ws_bytes, chs::bwd_workspace_bytes(B, Hq, S), false,
                     stream);
    if (rc != ATTN_OK) return rc;
    ws = st->bwd_ws;
  }
  const float sc = scale == 0.f ? (float)(1.0 / std::sqrt((double)Dh)) : scale;
  cudaError_t e = chs::launch_bwd(q, k, v, o, dout, lse, dq, dk, dv, static_cast<float*>(ws), B,
                                  Hq, Hkv, S, Dh, causal, window, sc, launch_info(st), stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_decode(const void* q, const void* kcache, const void* vcache, const int* seqlens, void* o,
                int B, int Hq, int Hkv, int Tmax, int Dh, int window, float scale,
                cudaStream_t stream) {
  return decode_common(q, kcache, vcache, seqlens, o, B, Hq, Hkv, Tmax, Dh, window, 0, scale,
                       stream);
}

int attn_decode_ring(const void* q, const void* kcache, const void* vcache, const int* seqlens,
                     void* o, int B, int Hq, int Hkv, int C, int Dh, int window, float scale,
                     cudaStream_t stream) {
  return decode_common(q, kcache, vcache, seqlens, o, B, Hq, Hkv, C, Dh, window, 1, scale, stream);
}

int attn_status(cudaStream_t stream) {
  DeviceState* st = nullptr;
  int rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ATTN_ERR_CUDA;
  int word = 0;
  if (cudaMemcpyAsync(&word, st->info.error_word, sizeof(int), cudaMemcpyDeviceToHost, stream) !=
          cudaSuccess ||
      cudaMemsetAsync(st->info.error_word, 0, sizeof(int), stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return ATTN_ERR_CUDA;
  return word;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// attn_decode_noalloc: the decode step for callers that must not allocate
// device memory.  Its split partials and completion counters live in one
// file-scope device array instead of the library's cudaMalloc'd workspace.
namespace {

constexpr size_t kNoAllocScratchBytes = size_t(16) << 20;   // 16 MiB per device

// Held by every device that loads this library, until the process exits.
// In host code this name is only a stand-in: the device address comes from
// cudaGetSymbolAddress, taken once per device below.
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

unsigned char* g_noalloc_ptr[kMaxDevices] = {};

}  // namespace

extern "C" int attn_decode_noalloc(const void* q, const void* kcache, const void* vcache,
                                   const int* seqlens, void* o, int B, int Hq, int Hkv, int Tmax,
                                   int Dh, int window, float scale, cudaStream_t stream) {
  float scale_log2 = 0.f;
  bool empty = false;
  int rc = decode_check_args(q, kcache, vcache, seqlens, o, B, Hq, Hkv, Tmax, Dh, &window, 0,
                             scale, &scale_log2, &empty);
  if (rc != ATTN_OK || empty) return rc;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  // the fixed array's address, looked up once per device with that device current
  auto scratch_ptr = [&](unsigned char** out) -> int {
    std::lock_guard<std::mutex> lock(g_mutex);
    const int dev = st->info.device;
    if (!g_noalloc_ptr[dev]) {
      void* ptr = nullptr;
      if (cudaGetSymbolAddress(&ptr, g_noalloc_scratch) != cudaSuccess || ptr == nullptr)
        return ATTN_ERR_CUDA;
      g_noalloc_ptr[dev] = static_cast<unsigned char*>(ptr);
    }
    *out = g_noalloc_ptr[dev];
    return ATTN_OK;
  };
  unsigned char* scratch = nullptr;
  if (Hq / Hkv >= chs::kDecodeTcMinGroup) {
    // query-head groups: the tensor-core path, as in attn_decode; its
    // split partials are the scratch's only content (it keeps no counters)
    const chs::DecodePlan plan = chs::plan_decode_tc(B, Hq, Hkv, Tmax, st->info.num_sms);
    if ((long long)B * Hkv * ((Hq / Hkv + 127) / 128) > 65535) return ATTN_ERR_INVALID_ARG;
    if (chs::decode_partials_bytes(B, Hq, Dh, plan) > kNoAllocScratchBytes)
      return ATTN_ERR_SCRATCH_LIMIT;
    if ((rc = scratch_ptr(&scratch)) != ATTN_OK) return rc;
    cudaError_t e = chs::launch_decode_tc(q, kcache, vcache, seqlens, o, B, Hq, Hkv, Tmax, Dh,
                                          window, 0, scale_log2, plan, scratch,
                                          launch_info(st), stream);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
  }
  const chs::DecodePlan plan = chs::plan_decode(B, Hq, Hkv, Tmax, Dh, st->info.num_sms);
  if ((long long)Hkv * ((Hq / Hkv) / plan.heads_per_cta) > 65535) return ATTN_ERR_INVALID_ARG;
  // scratch layout: counters (256-byte aligned) | split partials
  const size_t n_counters = chs::decode_counter_count(B, Hq, Hkv, plan);
  const size_t counter_bytes = (n_counters * sizeof(int) + 255) / 256 * 256;
  const size_t partial_bytes = chs::decode_partials_bytes(B, Hq, Dh, plan);
  if (counter_bytes + partial_bytes > kNoAllocScratchBytes) return ATTN_ERR_SCRATCH_LIMIT;
  if ((rc = scratch_ptr(&scratch)) != ATTN_OK) return rc;
  int* counters = reinterpret_cast<int*>(scratch);
  // the array keeps the previous call's contents: the counters must start at zero
  if (cudaMemsetAsync(counters, 0, n_counters * sizeof(int), stream) != cudaSuccess)
    return ATTN_ERR_CUDA;
  cudaError_t e = chs::launch_decode(q, kcache, vcache, seqlens, o, B, Hq, Hkv, Tmax, Dh, window,
                                     0, scale_log2, plan, counters, scratch + counter_bytes,
                                     launch_info(st), stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// The paged cache: append, decode, key weights, eviction.
namespace {

// Rows of a sequence, or of a list of them, at most: positions are 32-bit, and the kernels
// count a few thousand past the end.
constexpr int kMostRows = 0x7fffffff - 16384;

// Shape checks that every paged entry point shares.
int paged_check(int B, int Hkv, const chs::PagedCache& c, int Dh) {
  if (B < 0 || Hkv < 1 || c.num_pages < 1 || c.cols < 1 || c.page < 1) return ATTN_ERR_INVALID_ARG;
  if (Dh != 64 && Dh != 128 && Dh != 256) return ATTN_ERR_UNSUPPORTED;
  if (c.page % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  if ((long long)c.cols * c.page > kMostRows) return ATTN_ERR_INVALID_ARG;
  // a pool's (page, head) pairs are 32-bit
  if ((long long)c.num_pages * Hkv > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

struct Span {
  const void* p;
  size_t bytes;
};

// Pointers that a kernel reads or writes: none null, aligned to `align`.
bool usable(const void* p, uintptr_t align) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0;
}

// Does `out` overlap any of the others?
template <size_t N>
bool overlaps_any(const Span& out, const Span (&others)[N]) {
  for (const Span& s : others)
    if (s.p && overlaps(out.p, out.bytes, s.p, s.bytes)) return true;
  return false;
}

size_t pool_bytes(int Hkv, const chs::PagedCache& c, int Dh) {
  return (size_t)c.num_pages * Hkv * c.page * Dh * 2;
}

}  // namespace

extern "C" int attn_paged_append(const void* k, const void* v, void* kpages, void* vpages,
                                 const int* table, const int* seqlens, const int* newlens, int B,
                                 int Hkv, int S, int num_pages, int page, int cols, int Dh,
                                 cudaStream_t stream) {
  const chs::PagedCache cache{num_pages, page, cols};
  int rc = paged_check(B, Hkv, cache, Dh);
  if (rc != ATTN_OK) return rc;
  if (S < 0) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || S == 0) return ATTN_OK;
  if (!usable(k, 16) || !usable(v, 16) || !usable(kpages, 16) || !usable(vpages, 16) ||
      !usable(table, 4) || !usable(seqlens, 4) || (newlens && !usable(newlens, 4)))
    return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Hkv * S > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  const size_t in = (size_t)B * Hkv * S * Dh * 2, pool = pool_bytes(Hkv, cache, Dh);
  const Span rest[] = {{k, in}, {v, in}, {table, (size_t)B * cols * 4}, {seqlens, (size_t)B * 4},
                       {newlens, (size_t)B * 4}};
  if (overlaps_any({kpages, pool}, rest) || overlaps_any({vpages, pool}, rest) ||
      overlaps(kpages, pool, vpages, pool))
    return ATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st)) != ATTN_OK) return rc;
  const cudaError_t e = chs::launch_paged_append(k, v, kpages, vpages, table, seqlens, newlens, B,
                                                 Hkv, S, cache, Dh, launch_info(st), stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// The size rules of a paged decode call, shared with its workspace query.
static int decode_paged_check(int B, int Hq, int Hkv, const chs::PagedCache& cache, int Dh) {
  const int rc = paged_check(B, Hkv, cache, Dh);
  if (rc != ATTN_OK) return rc;
  if (Hq < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  // the line of tiles (64 keys at least, and a place per unit) and the grids are 32-bit
  const long long rows = (long long)cache.cols * cache.page;
  const long long units = (long long)B * Hkv * ((Hq / Hkv + 127) / 128);
  if (units > (1 << 24) || units * ((rows + 63) / 64 + 1) > 0x7fffffffLL - 1024)
    return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Hq + (long long)B * Hkv * ((rows + 511) / 512) > 0x7fffffffLL)
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

extern "C" int attn_decode_paged_workspace(int B, int Hq, int Hkv, int page, int cols, int Dh,
                                           int with_weights, size_t* bytes) {
  const chs::PagedCache cache{1, page, cols};
  int rc = decode_paged_check(B, Hq, Hkv, cache, Dh);
  if (rc != ATTN_OK) return rc;
  if (!bytes) return ATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st)) != ATTN_OK) return rc;
  // (a call with a window needs no more than one without)
  *bytes = chs::decode_paged_workspace_bytes(B, Hq, Hkv, cache, Dh, 0, with_weights != 0,
                                             launch_info(st));
  return ATTN_OK;
}

extern "C" int attn_decode_paged(const void* q, const void* kpages, const void* vpages,
                                 const int* table, const int* seqlens, void* o, float* weights,
                                 int weights_stride, int accumulate, void* workspace,
                                 size_t workspace_bytes, int B, int Hq, int Hkv, int num_pages,
                                 int page, int cols, int Dh, int window, float scale,
                                 cudaStream_t stream) {
  const chs::PagedCache cache{num_pages, page, cols};
  int rc = decode_paged_check(B, Hq, Hkv, cache, Dh);
  if (rc != ATTN_OK) return rc;
  if (window < 0) window = 0;
  if (weights && weights_stride < cols * page) return ATTN_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return ATTN_ERR_INVALID_ARG;
  float scale_log2 = 0.f;
  if (!resolve_scale(scale, Dh, &scale_log2)) return ATTN_ERR_INVALID_ARG;
  if (B == 0) return ATTN_OK;
  if (!usable(q, 16) || !usable(kpages, 16) || !usable(vpages, 16) || !usable(o, 16) ||
      !usable(table, 4) || !usable(seqlens, 4) || (weights && !usable(weights, 4)) ||
      (workspace_bytes > 0 && !usable(workspace, 256)))
    return ATTN_ERR_INVALID_ARG;
  const size_t qo = (size_t)B * Hq * Dh * 2, pool = pool_bytes(Hkv, cache, Dh);
  const size_t wb = weights ? (size_t)B * Hkv * weights_stride * 4 : 0;
  const Span in[] = {{q, qo}, {kpages, pool}, {vpages, pool}, {table, (size_t)B * cols * 4},
                     {seqlens, (size_t)B * 4}};
  if (overlaps_any({o, qo}, in) || overlaps_any({workspace, workspace_bytes}, in) ||
      overlaps(o, qo, workspace, workspace_bytes))
    return ATTN_ERR_INVALID_ARG;
  if (weights && (overlaps_any({weights, wb}, in) || overlaps(weights, wb, o, qo) ||
                  overlaps(weights, wb, workspace, workspace_bytes)))
    return ATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st)) != ATTN_OK) return rc;
  const chs::DeviceInfo dev = launch_info(st);
  if (workspace_bytes < chs::decode_paged_workspace_bytes(B, Hq, Hkv, cache, Dh, window,
                                                          weights != nullptr, dev))
    return ATTN_ERR_SCRATCH_LIMIT;
  const cudaError_t e = chs::launch_decode_paged(
      q, kpages, vpages, table, seqlens, o, weights, weights_stride, accumulate, workspace, B, Hq,
      Hkv, cache, Dh, window, scale_log2, dev, stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" int attn_key_weights(const void* q, const void* k, const float* lse, const int* seqlens,
                                float* weights, int weights_stride, int B, int Hq, int Hkv, int S,
                                int Dh, int queries, int causal, int window, int accumulate,
                                float scale, cudaStream_t stream) {
  if (B < 0 || S < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (Dh != 64 && Dh != 128 && Dh != 256) return ATTN_ERR_UNSUPPORTED;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return ATTN_ERR_INVALID_ARG;
  if (window < 0) window = 0;
  if (window > 0 && !causal) return ATTN_ERR_INVALID_ARG;
  if (queries < 0) queries = 0;
  if (weights_stride < S) return ATTN_ERR_INVALID_ARG;
  float scale_log2 = 0.f;
  if (!resolve_scale(scale, Dh, &scale_log2)) return ATTN_ERR_INVALID_ARG;
  if (scale_log2 < 1e-18f) return ATTN_ERR_INVALID_ARG;   // lse / scale has to stay finite
  if (B == 0 || S == 0) return ATTN_OK;
  if (!usable(q, 16) || !usable(k, 16) || !usable(lse, 4) || !usable(weights, 4) ||
      (seqlens && !usable(seqlens, 4)))
    return ATTN_ERR_INVALID_ARG;
  const long long key_blocks = ((long long)S + 127) / 128;
  if ((key_blocks + 1) * B * Hkv > 0x7fffffffLL - 1024 || (long long)S > 0x7fffffffLL - 1024 ||
      key_blocks * (Hq / Hkv) > 0x7fffffffLL || (long long)B * Hq > 0x7fffffffLL)
    return ATTN_ERR_INVALID_ARG;
  const size_t qb = (size_t)B * Hq * S * Dh * 2, kb = (size_t)B * Hkv * S * Dh * 2;
  const Span in[] = {{q, qb}, {k, kb}, {lse, (size_t)B * Hq * S * 4}, {seqlens, (size_t)B * 4}};
  if (overlaps_any({weights, (size_t)B * Hkv * weights_stride * 4}, in)) return ATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  const int rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  const cudaError_t e = chs::launch_key_weights(q, k, lse, seqlens, weights, weights_stride, B, Hq,
                                                Hkv, S, Dh, causal, window, queries, accumulate,
                                                scale_log2, launch_info(st), stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" int attn_cache_evict(void* kpages, void* vpages, float* weights, int weights_stride,
                                const int* table, const int* seqlens, int budget, int recent,
                                const int* table_out, int cols_out, float* weights_out,
                                int weights_out_stride, int* newlens, int* keep, int B, int Hkv,
                                int num_pages, int page, int cols, int Dh, cudaStream_t stream) {
  const chs::PagedCache cache{num_pages, page, cols};
  int rc = paged_check(B, Hkv, cache, Dh);
  if (rc != ATTN_OK) return rc;
  if (table_out == nullptr) {
    table_out = table;
    cols_out = cols;
  }
  if (weights_out == nullptr) {
    weights_out = weights;
    weights_out_stride = weights_stride;
  }
  if (budget < 1 || recent < 0 || recent > budget) return ATTN_ERR_INVALID_ARG;
  // the kernels step through `keep` in 32 bits, up to a block's rows past its end
  if (budget > kMostRows) return ATTN_ERR_INVALID_ARG;
  const long long rows = (long long)cols * page;
  const long long most = budget < rows ? budget : rows;   // rows that a sequence may end with
  if (weights_stride < rows || weights_out_stride < most || cols_out < 1 ||
      (long long)cols_out * page > kMostRows || (long long)cols_out * page < most)
    return ATTN_ERR_INVALID_ARG;
  if (table_out == table && cols_out != cols) return ATTN_ERR_INVALID_ARG;
  if (weights_out == weights && weights_out_stride != weights_stride) return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Hkv > 0xffffffLL ||
      (long long)B * Hkv * (((long long)budget + 15) / 16 + 1) > 0x7fffffffLL)
    return ATTN_ERR_INVALID_ARG;
  if (B == 0) return ATTN_OK;
  if (!usable(kpages, 16) || !usable(vpages, 16) || !usable(weights, 4) || !usable(table, 4) ||
      !usable(seqlens, 4) || !usable(table_out, 4) || !usable(weights_out, 4) ||
      !usable(newlens, 4) || !usable(keep, 4))
    return ATTN_ERR_INVALID_ARG;
  const size_t pool = pool_bytes(Hkv, cache, Dh), lens = (size_t)B * 4;
  const size_t wb = (size_t)B * Hkv * weights_stride * 4;
  const size_t wob = (size_t)B * Hkv * weights_out_stride * 4;
  const size_t kb = (size_t)B * Hkv * budget * 4;
  const Span in[] = {{table, (size_t)B * cols * 4}, {table_out, (size_t)B * cols_out * 4},
                     {seqlens, lens}};
  const Span out[] = {{kpages, pool}, {vpages, pool}, {newlens, lens}, {keep, kb},
                      {weights_out, wob}};
  for (size_t i = 0; i < 5; ++i) {
    if (overlaps_any(out[i], in)) return ATTN_ERR_INVALID_ARG;
    for (size_t j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return ATTN_ERR_INVALID_ARG;
    // the weights: read, and written only where they are weights_out too
    if (!(i == 4 && weights_out == weights) && overlaps(out[i].p, out[i].bytes, weights, wb))
      return ATTN_ERR_INVALID_ARG;
  }
  DeviceState* st = nullptr;
  if ((rc = device_state(&st)) != ATTN_OK) return rc;
  const cudaError_t e = chs::launch_cache_evict(
      kpages, vpages, table, table_out, cols_out, seqlens, newlens, weights, weights_stride,
      weights_out, weights_out_stride, keep, B, Hkv, cache, Dh, budget, recent, launch_info(st),
      stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// Packed sequences and tokens: attention over sequences of different lengths, rotary
// positions, the plan of a serving step.
namespace {

// A tensor of B x S rows of H heads, as a call got it.
struct Rows {
  const attn_rows_t* t;
  int B, S, H, Dh;
  long long batch() const { return B > 1 ? t->batch_stride : 0; }
  long long row() const { return S > 1 ? t->row_stride : 0; }
  long long head() const { return H > 1 ? t->head_stride : 0; }
  // elements from the first to behind the last
  long long extent() const {
    return (B - 1) * batch() + (S - 1) * row() + (H - 1) * head() + Dh;
  }
  size_t bytes() const { return (size_t)extent() * 2; }
  bool empty() const { return B == 0 || S == 0 || H == 0; }
};

// A map's strides are of 40 bits, in bytes; no tensor on a GPU reaches 2^46 elements.
constexpr long long kMostStride = 1ll << 38, kMostExtent = 1ll << 46;

// Aligned, with strides that are whole 16 bytes and (of axes with more than one entry) at
// least `least`.
bool rows_usable(const Rows& x, long long least) {
  if (x.empty()) return true;
  if (!x.t || !x.t->data || !aligned16(x.t->data)) return false;
  const long long stride[] = {x.t->batch_stride, x.t->row_stride, x.t->head_stride};
  const int n[] = {x.B, x.S, x.H};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (stride[i] % 8 != 0 || stride[i] < least || stride[i] > kMostStride ||
                     (stride[i] > 0 && n[i] - 1 > kMostExtent / stride[i])))
      return false;
  return true;
}

// No two elements at one place: each axis steps over everything of the axes below it.
bool rows_distinct(const Rows& x) {
  if (x.empty()) return true;
  long long stride[] = {x.batch(), x.row(), x.head()};
  long long n[] = {x.B, x.S, x.H};
  long long extent = x.Dh;
  for (int pass = 0; pass < 3; ++pass) {
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && (at < 0 || stride[i] < stride[at])) at = i;
    if (at < 0) break;
    if (stride[at] < extent) return false;
    extent += (n[at] - 1) * stride[at];
    n[at] = 1;
  }
  return true;
}

bool rows_same(const Rows& a, const Rows& b) {
  return a.t->data == b.t->data && a.batch() == b.batch() && a.row() == b.row() &&
         a.head() == b.head();
}

// How far x reaches from each multiple of `step` that it starts at, if its strides of at least
// `step` are multiples of it; else more than `step`.
long long reach(const Rows& x, long long step) {
  long long n = x.Dh;
  const long long stride[] = {x.batch(), x.row(), x.head()};
  const int count[] = {x.B, x.S, x.H};
  for (int i = 0; i < 3; ++i) {
    if (stride[i] < step)
      n += (count[i] - 1) * stride[i];
    else if (stride[i] % step != 0)
      return step + 1;
  }
  return n;
}

// May the two share an element?  Parts of one wider tensor (a projection's output, split into
// queries, keys and values along its heads, or along an axis around or inside them) lie between
// one another: at one of the strides, each within its own part of every step.
bool rows_overlap(const Rows& a, const Rows& b) {
  if (a.empty() || b.empty()) return false;
  if (!overlaps(a.t->data, a.bytes(), b.t->data, b.bytes())) return false;
  const long long between = (long long)(reinterpret_cast<uintptr_t>(b.t->data) -
                                        reinterpret_cast<uintptr_t>(a.t->data)) / 2;
  for (const Rows* x : {&a, &b}) {
    for (const long long step : {x->batch(), x->row(), x->head()}) {
      if (step <= 0) continue;
      const long long wa = reach(a, step), wb = reach(b, step);
      const long long d = (between % step + step) % step;   // b's place in a's step
      if (wa <= step && wb <= step && d >= wa && d + wb <= step) return false;
    }
  }
  return true;
}

bool rows_overlap(const Rows& a, const void* p, size_t bytes) {
  return !a.empty() && p != nullptr && bytes > 0 && overlaps(a.t->data, a.bytes(), p, bytes);
}

chs::PackedRows packed_rows(const Rows& x) {
  return chs::PackedRows{x.t->data, x.t->row_stride, x.t->head_stride, x.H};
}
chs::RopeRows rope_rows(const Rows& x) {
  if (x.empty() || !x.t) return chs::RopeRows{};
  return chs::RopeRows{x.t->data, x.batch(), x.row(), x.head()};
}

// The size rules of the packed calls, shared with their workspace queries.
int packed_check(int B, int Hq, int T) {
  if (B < 0 || T < 0 || Hq < 1) return ATTN_ERR_INVALID_ARG;
  // rows of the statistics, tiles and work items are 32-bit
  if ((long long)T + 127ll * B > kMostRows) return ATTN_ERR_INVALID_ARG;
  if (chs::packed_max_tiles(B, T) * Hq > kMostRows) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

int packed_shape(chs::PackedShape* s, float* scale_log2, const int* cu, int B, int Hq, int Hkv,
                 int T, int Dh, int causal, int window, float scale) {
  if (Hkv < 1 || Hq < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (Dh != 64 && Dh != 128 && Dh != 256) return ATTN_ERR_UNSUPPORTED;
  const int rc = packed_check(B, Hq, T);
  if (rc != ATTN_OK) return rc;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (window < 0) window = 0;
  if (window > 0 && !causal) return ATTN_ERR_INVALID_ARG;
  if (window > T) window = T;   // (the same, and sums of positions and windows stay in 32 bits)
  if (!resolve_scale(scale, Dh, scale_log2)) return ATTN_ERR_INVALID_ARG;
  *s = chs::PackedShape{B, Hq, Hkv, T, Dh, causal, window, cu};
  return ATTN_OK;
}

}  // namespace

extern "C" int attn_fwd_packed_workspace(int B, int Hq, int T, int Dh, int causal,
                                         size_t* bytes) {
  chs::PackedShape s;
  float scale_log2;
  int rc = packed_shape(&s, &scale_log2, nullptr, B, Hq, Hq, T, Dh, causal, 0, 0.f);
  if (rc != ATTN_OK) return rc;
  if (!bytes) return ATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st)) != ATTN_OK) return rc;
  const chs::DeviceInfo dev = launch_info(st);
  // a call's kernel, and with it the need for a list, goes by its K/V heads too: the most that
  // any number of them takes
  size_t most = 0;
  for (long long g = 1; g * g <= Hq; ++g) {
    if (Hq % g != 0) continue;
    for (const int kv : {(int)g, Hq / (int)g}) {
      s.Hkv = kv;
      most = std::max(most, chs::fwd_packed_workspace_bytes(s, dev));
    }
  }
  *bytes = most;
  return ATTN_OK;
}

extern "C" int attn_bwd_packed_workspace(int B, int Hq, int T, size_t* bytes) {
  const int rc = packed_check(B, Hq, T);
  if (rc != ATTN_OK) return rc;
  if (!bytes) return ATTN_ERR_INVALID_ARG;
  *bytes = chs::bwd_packed_workspace_bytes(B, Hq, T);
  return ATTN_OK;
}

extern "C" int attn_fwd_packed(const attn_rows_t* q, const attn_rows_t* k, const attn_rows_t* v,
                               const attn_rows_t* o, float* lse, const int* cu_seqlens,
                               void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv,
                               int T, int Dh, int causal, int window, float scale,
                               cudaStream_t stream) {
  chs::PackedShape s;
  float scale_log2 = 0.f;
  int rc = packed_shape(&s, &scale_log2, cu_seqlens, B, Hq, Hkv, T, Dh, causal, window, scale);
  if (rc != ATTN_OK) return rc;
  if (B == 0 || T == 0) return ATTN_OK;
  const Rows Q{q, 1, T, Hq, Dh}, K{k, 1, T, Hkv, Dh}, V{v, 1, T, Hkv, Dh}, O{o, 1, T, Hq, Dh};
  for (const Rows* x : {&Q, &K, &V, &O})
    if (!rows_usable(*x, Dh)) return ATTN_ERR_INVALID_ARG;
  if (!rows_distinct(O)) return ATTN_ERR_INVALID_ARG;
  if (!usable(cu_seqlens, 4) || (lse && !usable(lse, 4)) ||
      (workspace_bytes > 0 && !usable(workspace, 256)))
    return ATTN_ERR_INVALID_ARG;
  const size_t lb = lse ? (size_t)Hq * T * 4 : 0, cb = ((size_t)B + 1) * 4;
  for (const Rows* x : {&Q, &K, &V}) {
    if (rows_overlap(O, *x) || rows_overlap(*x, lse, lb) ||
        rows_overlap(*x, workspace, workspace_bytes))
      return ATTN_ERR_INVALID_ARG;
  }
  if (rows_overlap(O, lse, lb) || rows_overlap(O, cu_seqlens, cb) ||
      rows_overlap(O, workspace, workspace_bytes) ||
      (workspace_bytes > 0 && overlaps(workspace, workspace_bytes, cu_seqlens, cb)) ||
      (lse && (overlaps(lse, lb, cu_seqlens, cb) || (workspace_bytes > 0 && overlaps(lse, lb, workspace, workspace_bytes)))))
    return ATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st)) != ATTN_OK) return rc;
  const chs::DeviceInfo dev = launch_info(st);
  if (workspace_bytes < chs::fwd_packed_workspace_bytes(s, dev)) return ATTN_ERR_SCRATCH_LIMIT;
  const cudaError_t e = chs::launch_fwd_packed(s, packed_rows(Q), packed_rows(K), packed_rows(V),
                                               packed_rows(O), lse, workspace, scale_log2,
                                               dev, stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" int attn_bwd_packed(const attn_rows_t* q, const attn_rows_t* k, const attn_rows_t* v,
                               const attn_rows_t* o, const attn_rows_t* dout, const float* lse,
                               const attn_rows_t* dq, const attn_rows_t* dk, const attn_rows_t* dv,
                               const int* cu_seqlens, void* workspace, size_t workspace_bytes,
                               int B, int Hq, int Hkv, int T, int Dh, int causal, int window,
                               float scale, cudaStream_t stream) {
  chs::PackedShape s;
  float scale_log2 = 0.f;
  int rc = packed_shape(&s, &scale_log2, cu_seqlens, B, Hq, Hkv, T, Dh, causal, window, scale);
  if (rc != ATTN_OK) return rc;
  if (B == 0 || T == 0) return ATTN_OK;
  const Rows in[] = {{q, 1, T, Hq, Dh}, {k, 1, T, Hkv, Dh}, {v, 1, T, Hkv, Dh}, {o, 1, T, Hq, Dh},
                     {dout, 1, T, Hq, Dh}};
  const Rows out[] = {{dq, 1, T, Hq, Dh}, {dk, 1, T, Hkv, Dh}, {dv, 1, T, Hkv, Dh}};
  for (const Rows& x : in)
    if (!rows_usable(x, Dh)) return ATTN_ERR_INVALID_ARG;
  for (const Rows& x : out)
    if (!rows_usable(x, Dh) || !rows_distinct(x)) return ATTN_ERR_INVALID_ARG;
  if (!usable(cu_seqlens, 4) || !usable(lse, 4) || !usable(workspace, 256))
    return ATTN_ERR_INVALID_ARG;
  const size_t lb = (size_t)Hq * T * 4, cb = ((size_t)B + 1) * 4;
  for (const Rows& x : in)
    if (rows_overlap(x, workspace, workspace_bytes)) return ATTN_ERR_INVALID_ARG;
  for (int a = 0; a < 3; ++a) {
    for (const Rows& x : in)
      if (rows_overlap(out[a], x)) return ATTN_ERR_INVALID_ARG;
    for (int b = a + 1; b < 3; ++b)
      if (rows_overlap(out[a], out[b])) return ATTN_ERR_INVALID_ARG;
    if (rows_overlap(out[a], lse, lb) || rows_overlap(out[a], cu_seqlens, cb) ||
        rows_overlap(out[a], workspace, workspace_bytes))
      return ATTN_ERR_INVALID_ARG;
  }
  if (overlaps(workspace, workspace_bytes, cu_seqlens, cb) ||
      overlaps(workspace, workspace_bytes, lse, lb))
    return ATTN_ERR_INVALID_ARG;
  if (workspace_bytes < chs::bwd_packed_workspace_bytes(B, Hq, T)) return ATTN_ERR_SCRATCH_LIMIT;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st)) != ATTN_OK) return rc;
  const float sc = scale == 0.f ? (float)(1.0 / std::sqrt((double)Dh)) : scale;
  const cudaError_t e = chs::launch_bwd_packed(
      s, packed_rows(in[0]), packed_rows(in[1]), packed_rows(in[2]), packed_rows(in[3]),
      packed_rows(in[4]), lse, packed_rows(out[0]), packed_rows(out[1]), packed_rows(out[2]),
      workspace, sc, launch_info(st), stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" int attn_rope_frequencies(unsigned long long* turns, float* amplitude, int rotary_dim,
                                     double base, int scaling, double factor, double low,
                                     double high, double original_len) {
  if (!turns || !amplitude || rotary_dim < 16 || rotary_dim > 256 || rotary_dim % 16 != 0)
    return ATTN_ERR_INVALID_ARG;
  if (scaling < ATTN_ROPE_NONE || scaling > ATTN_ROPE_YARN) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(base) || base < 1.0) return ATTN_ERR_INVALID_ARG;
  if (scaling != ATTN_ROPE_NONE && (!std::isfinite(factor) || factor < 1.0))
    return ATTN_ERR_INVALID_ARG;
  const bool blend = scaling == ATTN_ROPE_TURNS || scaling == ATTN_ROPE_YARN;
  if (blend && (!std::isfinite(low) || !std::isfinite(high) || !(high > low) ||
                !std::isfinite(original_len) || !(original_len > 0.0)))
    return ATTN_ERR_INVALID_ARG;
  if (scaling == ATTN_ROPE_BASE) base *= std::pow(factor, rotary_dim / (rotary_dim - 2.0));
  for (int i = 0; i < rotary_dim / 2; ++i) {
    // at most 1 / (2 pi)
    double f = std::pow(base, -2.0 * i / rotary_dim) / 6.283185307179586476925;
    if (scaling == ATTN_ROPE_LINEAR) f /= factor;
    if (blend) {
      const double keep = std::fmin(1.0, std::fmax(0.0, (original_len * f - low) / (high - low)));
      f *= keep + (1.0 - keep) / factor;
    }
    turns[i] = (unsigned long long)std::rint(std::ldexp(f, 64));
  }
  *amplitude = scaling == ATTN_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return ATTN_OK;
}

namespace {

// Shared by attn_rope and attn_rope_append.
int rope_common(const attn_rows_t* q, const attn_rows_t* q_out, int Hq, const attn_rows_t* k,
                const attn_rows_t* k_out, int Hkv, const attn_rows_t* v, const int* positions,
                const unsigned long long* turns, float amplitude, void* kpages, void* vpages,
                const int* slots, int num_pages, int page, bool append, int B, int S, int Dh,
                int rot, int interleaved, int inverse, cudaStream_t stream) {
  if (B < 0 || S < 0 || Hq < 0 || Hkv < 0 || Hq + Hkv < 1) return ATTN_ERR_INVALID_ARG;
  if (Dh != 64 && Dh != 128 && Dh != 256) return ATTN_ERR_UNSUPPORTED;
  if (rot < 0 || rot > Dh || rot % 16 != 0) return ATTN_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1) ||
      !std::isfinite(amplitude))
    return ATTN_ERR_INVALID_ARG;
  if ((long long)B * S > kMostRows || Hq > (1 << 24) || Hkv > (1 << 24))
    return ATTN_ERR_INVALID_ARG;
  if (append) {
    const int rc = paged_check(B, Hkv, chs::PagedCache{num_pages, page, 1}, Dh);
    if (rc != ATTN_OK) return rc;
    if ((long long)num_pages * page > kMostRows) return ATTN_ERR_INVALID_ARG;   // slots are 32-bit
  }
  if (B == 0 || S == 0) return ATTN_OK;
  const int n = B * S;
  const Rows Q{q, B, S, Hq, Dh}, QO{q_out, B, S, Hq, Dh}, K{k, B, S, Hkv, Dh},
      KO{k_out, B, S, k_out || !append ? Hkv : 0, Dh}, V{v, B, S, append ? Hkv : 0, Dh};
  for (const Rows* x : {&Q, &K, &V})
    if (!rows_usable(*x, 0)) return ATTN_ERR_INVALID_ARG;
  for (const Rows* x : {&QO, &KO})
    if (!rows_usable(*x, Dh) || !rows_distinct(*x)) return ATTN_ERR_INVALID_ARG;
  if (!usable(positions, 4) || (rot > 0 && !usable(turns, 8))) return ATTN_ERR_INVALID_ARG;
  if (append && (!usable(kpages, 16) || !usable(vpages, 16) || !usable(slots, 4)))
    return ATTN_ERR_INVALID_ARG;
  const size_t lens = (size_t)n * 4, tb = (size_t)rot / 2 * 8;
  const size_t pool = append ? pool_bytes(Hkv, chs::PagedCache{num_pages, page, 1}, Dh) : 0;
  // an output is its own input, or apart from every tensor
  if ((!QO.empty() && !rows_same(Q, QO) && rows_overlap(QO, Q)) || rows_overlap(QO, K) ||
      rows_overlap(QO, V) || rows_overlap(QO, KO) || rows_overlap(KO, Q) || rows_overlap(KO, V) ||
      (!KO.empty() && !rows_same(K, KO) && rows_overlap(KO, K)))
    return ATTN_ERR_INVALID_ARG;
  for (const Rows* x : {&QO, &KO})
    if (rows_overlap(*x, positions, lens) || rows_overlap(*x, turns, tb) ||
        rows_overlap(*x, slots, append ? lens : 0))
      return ATTN_ERR_INVALID_ARG;
  if (append) {
    for (const void* x : {kpages, vpages}) {
      for (const Rows* y : {&Q, &QO, &K, &KO, &V})
        if (rows_overlap(*y, x, pool)) return ATTN_ERR_INVALID_ARG;
      if (overlaps(x, pool, positions, lens) || overlaps(x, pool, slots, lens) ||
          (tb > 0 && overlaps(x, pool, turns, tb)))
        return ATTN_ERR_INVALID_ARG;
    }
    if (overlaps(kpages, pool, vpages, pool)) return ATTN_ERR_INVALID_ARG;
  }
  DeviceState* st = nullptr;
  const int rc = device_state(&st);
  if (rc != ATTN_OK) return rc;
  const chs::RopeShape s{B, S, Hq, Hkv, Dh, rot, positions, turns, amplitude, interleaved, inverse};
  const chs::RopeRows qi = rope_rows(Q), qo = rope_rows(QO), ki = rope_rows(K), ko = rope_rows(KO);
  const chs::RopeAppend a{rope_rows(V), kpages, vpages, slots, num_pages, page};
  const cudaError_t e = chs::launch_rope(s, qi, QO.empty() ? nullptr : &qo, ki,
                                         KO.empty() ? nullptr : &ko, append ? &a : nullptr,
                                         launch_info(st), stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" int attn_rope(const attn_rows_t* q, const attn_rows_t* q_out, int Hq,
                         const attn_rows_t* k, const attn_rows_t* k_out, int Hkv,
                         const int* positions, const unsigned long long* turns, float amplitude,
                         int B, int S, int Dh, int rotary_dim, int interleaved, int inverse,
                         cudaStream_t stream) {
  return rope_common(q, q_out, Hq, k, k_out, Hkv, nullptr, positions, turns, amplitude, nullptr,
                     nullptr, nullptr, 0, 0, false, B, S, Dh, rotary_dim, interleaved, inverse,
                     stream);
}

extern "C" int attn_rope_append(const attn_rows_t* q, const attn_rows_t* q_out, int Hq,
                                const attn_rows_t* k, const attn_rows_t* k_out,
                                const attn_rows_t* v, int Hkv, const int* positions,
                                const unsigned long long* turns, float amplitude, void* kpages,
                                void* vpages, const int* slots, int num_pages, int page, int B,
                                int S, int Dh, int rotary_dim, int interleaved,
                                cudaStream_t stream) {
  return rope_common(q, q_out, Hq, k, k_out, Hkv, v, positions, turns, amplitude, kpages, vpages,
                     slots, num_pages, page, true, B, S, Dh, rotary_dim, interleaved, 0, stream);
}

extern "C" int attn_cache_plan(const int* delta, const int* seqlens, int* seqlens_out, int* table,
                               int* free_pages, const int* num_free, int* num_free_out,
                               int* cu_seqlens, int* positions, int* slots, int B, int cols,
                               int page, int num_pages, int capacity, int T,
                               cudaStream_t stream) {
  int rc = paged_check(B, 1, chs::PagedCache{num_pages, page, cols}, 64);
  if (rc != ATTN_OK) return rc;
  if (T < 0 || T > kMostRows || capacity < 1 || capacity > kMostRows) return ATTN_ERR_INVALID_ARG;
  if ((long long)num_pages * page > kMostRows) return ATTN_ERR_INVALID_ARG;   // slots are 32-bit
  if (B > chs::cache_plan_max_sequences()) return ATTN_ERR_UNSUPPORTED;
  // (of no sequences: no lengths and no table)
  if ((B > 0 && (!usable(delta, 4) || !usable(seqlens, 4) || !usable(seqlens_out, 4) ||
                 !usable(table, 4))) ||
      !usable(free_pages, 4) || !usable(num_free, 4) || !usable(num_free_out, 4) ||
      !usable(cu_seqlens, 4) || (T > 0 && (!usable(positions, 4) || !usable(slots, 4))))
    return ATTN_ERR_INVALID_ARG;
  const size_t lens = (size_t)B * 4, rows = (size_t)T * 4;
  const Span in[] = {{B > 0 ? delta : nullptr, lens}, {B > 0 ? seqlens : nullptr, lens},
                     {num_free, 4}};
  const Span out[] = {{B > 0 ? seqlens_out : nullptr, lens}, {num_free_out, 4},
                      {B > 0 ? table : nullptr, (size_t)B * cols * 4},
                      {free_pages, (size_t)capacity * 4}, {cu_seqlens, lens + 4},
                      {T > 0 ? positions : nullptr, rows}, {T > 0 ? slots : nullptr, rows}};
  for (int i = 0; i < 7; ++i) {
    if (!out[i].p) continue;
    for (int j = 0; j < 3; ++j) {
      const bool in_place = (i == 0 && j == 1 && seqlens_out == seqlens) ||
                            (i == 1 && j == 2 && num_free_out == num_free);
      if (!in_place && overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
        return ATTN_ERR_INVALID_ARG;
    }
    for (int j = 0; j < i; ++j)
      if (out[j].p && overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
        return ATTN_ERR_INVALID_ARG;
  }
  DeviceState* st = nullptr;
  if ((rc = device_state(&st)) != ATTN_OK) return rc;
  const cudaError_t e = chs::launch_cache_plan(
      chs::CachePlan{delta, seqlens, seqlens_out, table, free_pages, num_free, num_free_out,
                     cu_seqlens, positions, slots, B, cols, page, num_pages, capacity, T},
      launch_info(st), stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
