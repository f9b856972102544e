// backward_sm103a.cuh -- backward pass of causal self-attention on the
// 5th-generation tensor cores (sm_103a), Dh = 64 or 128.
//
// Given q, k, v, the forward output o, its row log-sum-exps and the upstream
// gradient dO, the gradients follow from the chain rule through
// o_i = sum_j p_ij v_j, p_i = softmax(s_i) and s_ij = scale q_i . k_j, with
// the softmax derivative dp_i/dz_j = p_i (delta_ij - p_j) of "Механизм
// внимания", section "Почему делить на корень из d_h":
//     dV = P^T dO,   dP = dO V^T,   dS = P o (dP - D),  D_i = dO_i . o_i,
//     dK = scale dS^T Q,   dQ = scale dS K.
// (D_i = sum_j p_ij dp_ij, the contraction of that Jacobian, because
// o_i = sum_j p_ij v_j.)  As section "Эффективные реализации" of the same
// page describes for FlashAttention, the weights P are recomputed block by
// block from the saved log-sum-exp, never stored.
//
// Three kernels, all deterministic (no atomics anywhere):
//   attn_bwd_prep      D_i and the log-sum-exp in units of log2, per row;
//   attn_bwd_dkdv      one CTA per 128-key block of one K/V head: K and V
//                      stay in shared memory while the query blocks of every
//                      query head of the group stream past; S^T = K Q^T and
//                      dP^T = V dO^T land in tensor memory, the softmax
//                      warps turn them into P^T and dS^T (bf16, written over
//                      them), and dV += P^T dO, dK += dS^T Q accumulate in
//                      tensor memory (M = 128 keys);
//   attn_bwd_dq        one CTA per 128-row query block: Q and dO stay, the
//                      key blocks stream past; S = Q K^T and dP = dO V^T
//                      (two dP buffers, so the next block's S and dP run
//                      while dS is formed), dS as above, dQ += dS K
//                      (M = 128 queries).
// dQ is computed by its own pass (recomputing S and dP) instead of being
// reduced across key blocks with atomics: 7 MMAs per block pair instead of 5,
// in exchange for a deterministic result.
//
// Roles: the first 4 kWG warps run the element-wise work and the epilogues,
// kWG warpgroups on kWG column ranges of the same 128 rows (a warp of each has
// 32 tensor-memory lanes; a thread of the dQ pass one of them, of the dK/dV
// pass 16 columns of four), so each does a share of every step's
// exponentials and the shares run side by side (kWG = 2: two halves); the
// next warp's lane 0 issues every TMA copy, the last warp every MMA (one
// elected lane).  Every wait is bounded.
//
// PK = 1 is the same over packed sequences (packed_sm103a.cuh): an item's
// rows, keys and place come from the lists of tiles (one heaviest first for
// each pass) instead of the launch's shape; rows are counted with the
// sequence's padding in front, for lse2 and D too.  Padded queries have
// lse2 = +inf and so weigh nothing; padded keys are masked.  PK = 2, for
// sequences that are short on average, is that with folded tiles: two or four
// query heads of a short sequence in one block of queries.  In a batch of
// short sequences few keys share a query's weight, each term of a gradient's
// sum is large, and so is what the terms' rounding to bf16 leaves: twice the
// final rounding's error in squares.  P and dS of a sequence's first two query
// blocks (where most of the gradients' size lies in long sequences too) enter
// the products as two bf16 parts, hi + lo, 2^-16 of each: two more products for
// those blocks, and under a short window for all.  (dQ of 24 documents of 16 to
// 2048 rows: 1.5 times the error of a single rounding of the result before,
// 1.25 times with it.)  D of queries that see few keys: attn_bwd_prep_few.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>

#include "packed_sm103a.cuh"
#include "sm103a_ptx.cuh"

namespace chs {

struct BwdParams {
  int B, Hq, Hkv, S;
  int causal, window;     // as in the forward (window > 0 only with causal)
  float scale_log2;       // scale * log2(e)
  float scale;            // applied to dK and dQ
  int S_pad;              // S rounded up to 128: row stride of lse2 and delta
  int nblk;               // ceil(S / 128)
  int group;              // Hq / Hkv
  int num_items;
  const float* lse2;      // [B * Hq, S_pad] log2 of sum_j 2^(s_ij log2 e); +inf past S
  const float* delta;     // [B * Hq, S_pad] D_i = dO_i . o_i; 0 past S
  __nv_bfloat16* dq;      // [B, Hq, S, DH]
  __nv_bfloat16* dk;      // [B, Hkv, S, DH]
  __nv_bfloat16* dv;      // [B, Hkv, S, DH]
  int* error_word;
  int fault;              // test hook: 4 = the dK/dV pass never loads its first K/V block
  // PK: the pass's tiles of 128 rows; S, nblk and num_items are then each
  // item's own; strides in elements between rows and heads of dq, dk and dv
  PackedRef pk;
  int wide;               // PK: rows of dq, dk and dv are 32-byte aligned
  int two_parts;          // PK: P and dS in two parts in every block (few keys per query)
  long long dq_row, dq_head, dk_row, dk_head, dv_row, dv_head;
};

// The rows that an item belongs to: a (batch, head)'s, or a packed sequence's.
struct BwdSeq {
  int S;       // rows (PK: with the padding)
  int nblk;    // ceil(S / 128)
  int start;   // PK: first row
  int pad;     // PK: rows of padding ahead of it
  int stat;    // PK: first row of its lse2 and D
  // PK: 1 << fold heads of a short sequence lie one below another in a block of queries (as in
  // prefill_k64_sm103a.cuh), rows() rows each: the last of the padded block, which keys are
  // counted by
  int fold;
  __device__ __forceinline__ int rows() const { return 128 >> fold; }
  // padded row of row t of a block of queries, and its head among the block's
  __device__ __forceinline__ int row_of(int block, int t) const {
    return 128 * block + 128 - rows() + (t & (rows() - 1));
  }
  __device__ __forceinline__ int head_of(int t) const { return t >> (7 - fold); }
};

// PK: the pass's tiles (of one, two and four heads).  An item of the dK/dV pass is a tile's K/V
// head, one of the dQ pass a folded tile's heads.
template <int PK>
__device__ __forceinline__ int3 bwd_counts(const BwdParams& p) {
  if constexpr (PK == 2) return packed_counts(p.pk);
  return make_int3(PK ? packed_num_tiles(p.pk) : 0, 0, 0);
}
template <int PK>
__device__ __forceinline__ int bwd_num_kv_items(const BwdParams& p, const int3& n) {
  return PK ? (n.x + n.y + n.z) * p.Hkv : p.num_items;
}
template <int PK>
__device__ __forceinline__ int bwd_num_q_items(const BwdParams& p, const int3& n) {
  return PK == 2 ? packed_items(n, p.Hq) : PK ? n.x * p.Hq : p.num_items;
}
// Item w of the dQ pass: tile i, its (first) head h.
template <int PK>
__device__ __forceinline__ void bwd_q_item_at(const BwdParams& p, const int3& n, int w, int& i,
                                              int& h) {
  if constexpr (PK == 2) {
    packed_item_of(n, p.Hq, w, i, h);
  } else {
    i = w / p.Hq;
    h = w - i * p.Hq;
  }
}

template <int PK>
__device__ __forceinline__ BwdSeq bwd_seq_of(const BwdParams& p, const PackedTile& e) {
  if constexpr (PK)
    return BwdSeq{e.len + e.pad(), (e.len + 127) / 128, e.start, e.pad(), e.stat,
                  PK == 2 ? packed_fold(e.len, p.pk.fold_max) : 0};
  return BwdSeq{p.S, p.nblk, 0, 0, 0, 0};
}

// Rows [row, row + R), columns c .. c + 63 of a head: of `bh` in a batch, of
// head bh of the packed sequence.
template <int PK>
__device__ __forceinline__ void bwd_load(void* dst, const CUtensorMap* map, uint64_t* bar, int c,
                                         int row, int bh, const BwdParams& p, const BwdSeq& q,
                                         int tensor, uint64_t policy) {
  if constexpr (PK)
    packed_load(dst, map, bar, c, q.start, q.pad, row, bh, p.pk.heads_inner & tensor, policy);
  else
    tma_load_3d_hint(dst, map, bar, c, row, bh, policy);
}
// (the resident blocks, loaded once per item)
template <int PK>
__device__ __forceinline__ void bwd_load_once(void* dst, const CUtensorMap* map, uint64_t* bar,
                                              int c, int row, int bh, const BwdParams& p,
                                              const BwdSeq& q, int tensor) {
  if constexpr (PK)
    packed_load(dst, map, bar, c, q.start, q.pad, row, bh, p.pk.heads_inner & tensor,
                policy_evict_first());
  else
    tma_load_3d(dst, map, bar, c, row, bh);
}

// A block of queries (Q or dO), columns c .. c + 63: of head bh, or (PK) of the heads from bh on
// that it is folded of.
template <int PK>
__device__ __forceinline__ void bwd_load_queries(uint8_t* dst, const CUtensorMap* map,
                                                 uint64_t* bar, int c, int block, int bh,
                                                 const BwdParams& p, const BwdSeq& q, int tensor,
                                                 uint64_t policy) {
  if constexpr (PK) {
    // (copies of 32 rows where tiles may be folded)
    for (int r = 0; r < 128; r += PK == 2 ? 32 : 128)
      packed_load(dst + r * 128, map, bar, c, q.start, q.pad, q.row_of(block, r), bh + q.head_of(r),
                  p.pk.heads_inner & tensor, policy);
  } else {
    tma_load_3d_hint(dst, map, bar, c, 128 * block, bh, policy);
  }
}

// (checked builds: a packed sequence lies inside the packed tensors)
template <int PK>
__device__ __forceinline__ bool bwd_inside(const BwdParams& p, const BwdSeq& q) {
  return !PK || (q.start >= 0 && q.start <= p.pk.T - (q.S - q.pad));
}

// Is row i one whose gradient is stored?
template <int PK>
__device__ __forceinline__ bool bwd_real(const BwdSeq& q, int i) {
  return PK ? i >= q.pad : i < q.S;
}

// Where row i of a gradient lies.
template <int PK>
__device__ __forceinline__ size_t bwd_row(const BwdSeq& q, int bh, int i, int DH, long long row,
                                          long long head) {
  if constexpr (PK) return (size_t)((q.start + (long long)(i - q.pad)) * row + bh * head);
  return ((size_t)bh * q.S + i) * DH;
}

template <int DH>
struct BwdCfg {
  static constexpr int kBox = 128 * 64 * 2;         // one 128-row x 64-column box
  static constexpr int kTile = (DH / 64) * kBox;    // a 128 x DH tile
  // warps 0 .. 4 kWG - 1: element-wise work (warp w: tensor-memory lanes
  // 32 (w % 4) .., columns kCols (w / 4) .. + kCols - 1 of S and dP); then one
  // TMA warp and one MMA warp
  static constexpr int kWG = 2;                 // element-wise warpgroups
  static constexpr int kCols = 128 / kWG;       // columns of S / dP per warpgroup
  static constexpr int kChunks = kCols / 32;    // 32-column tensor-memory loads per row
  static constexpr int kEW = 128 * kWG;         // element-wise threads
  static constexpr int kThreads = 32 * (4 * kWG + 2);
  static constexpr int kWarpProducer = 4 * kWG, kWarpIssuer = 4 * kWG + 1;
  static constexpr uint32_t kColS = 0, kColDP = 128, kColA0 = 256, kColA1 = 384;
  // the dQ pass has one accumulator (dQ at kColA0): its second dP buffer
  // takes the columns of the dK/dV pass's second accumulator
  static constexpr uint32_t kColDP1 = kColA1;
  static_assert(kColA0 + DH <= kColDP1, "dQ accumulator and the second dP buffer");
  // the dK/dV pass at Dh 64: its accumulators side by side leave room for a second S buffer, and
  // shared memory for a third stage of queries
  static constexpr int kBufsS = DH == 64 ? 2 : 1, kStagesQ = DH == 64 ? 3 : 2;
  static constexpr uint32_t kColAcc1 = kColA0 + DH, kColS1 = 384;
  static_assert(kBufsS == 1 || kColAcc1 + DH <= kColS1, "two S buffers");
};

// Where the bf16 pairs of columns 16 kk .. 16 kk + 15 of a 128-column S or dP
// buffer are written (P over S, dS over dP): each warpgroup's pairs go to the
// first half of its own kCols columns, so that one warpgroup's stores never
// land on columns another warpgroup has still to load.
__host__ __device__ constexpr uint32_t bwd_packed_col(int kk) {
  constexpr int cols = BwdCfg<64>::kCols;
  return (uint32_t)(cols * (16 * kk / cols) + (16 * kk % cols) / 2);
}

// PK: the low parts of columns 16 kk .. (see above) lie behind their high
// parts, in the other half of each warpgroup's columns.
__host__ __device__ constexpr uint32_t bwd_low_col(int kk) {
  return bwd_packed_col(kk) + BwdCfg<64>::kCols / 2;
}

// PK: do P and dS of these query blocks (of 128 rows) enter the products in two parts?
constexpr int kBwdExactBlocks = 2;
template <int PK>
__device__ __forceinline__ bool bwd_two_parts(const BwdParams& p, int qb) {
  return PK && (qb < kBwdExactBlocks || p.two_parts);
}

// What bf16 leaves of (a, b), whose rounded pair is `hi`, as a pair.
__device__ __forceinline__ uint32_t bwd_low_pair(float a, float b, uint32_t hi) {
  return pack_bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}

// D_i = sum_d dO[i, d] o[i, d] (fp32 products of the bf16 values) and
// lse2_i = lse_i * log2(e) for every row of [B * Hq, S_pad]; rows past S get
// D = 0 and lse2 = +inf (their weights exp2(x - lse2) are then 0).  DH / 8
// lanes per row, 16 bytes of o and of dO each; a block covers kPrepRowSets
// row sets, all of whose loads are issued before the first is used.
constexpr int kPrepRowSets = 4;
template <int DH>
constexpr int bwd_prep_rows_per_block() { return kPrepRowSets * 256 / (DH / 8); }

template <int DH>
__global__ void __launch_bounds__(256)
    attn_bwd_prep(const __nv_bfloat16* __restrict__ o, const __nv_bfloat16* __restrict__ dout,
                  const float* __restrict__ lse, float* __restrict__ lse2,
                  float* __restrict__ delta, long long rows, int S, int S_pad) {
  constexpr int kLanes = DH / 8;                // 16 or 8 lanes per row
  constexpr int kRowsPerSet = 256 / kLanes;
  // o, dO and lse may come from the previous kernel in the stream
  griddep_wait();
  griddep_launch_dependents();
  const int sub = threadIdx.x % kLanes;
  long long r[kPrepRowSets];
  bool valid[kPrepRowSets];
  uint4 a[kPrepRowSets], b[kPrepRowSets];
#pragma unroll
  for (int k = 0; k < kPrepRowSets; ++k) {
    r[k] = (long long)blockIdx.x * bwd_prep_rows_per_block<DH>() + k * kRowsPerSet +
           threadIdx.x / kLanes;
    const long long bh = r[k] / S_pad;
    const int i = (int)(r[k] - bh * S_pad);
    valid[k] = r[k] < rows && i < S;
    a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
    if (valid[k]) {
      const size_t base = ((size_t)bh * S + i) * DH + 8 * sub;
      a[k] = *reinterpret_cast<const uint4*>(o + base);
      b[k] = *reinterpret_cast<const uint4*>(dout + base);
    }
  }
#pragma unroll
  for (int k = 0; k < kPrepRowSets; ++k) {
    const uint32_t wa[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
    const uint32_t wb[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
    float acc = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc = fmaf(__uint_as_float(wa[e] << 16), __uint_as_float(wb[e] << 16), acc);
      acc = fmaf(__uint_as_float(wa[e] & 0xffff0000u), __uint_as_float(wb[e] & 0xffff0000u), acc);
    }
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
    if (sub == 0 && r[k] < rows) {
      const long long bh = r[k] / S_pad;
      const int i = (int)(r[k] - bh * S_pad);
      delta[r[k]] = valid[k] ? acc : 0.f;
      lse2[r[k]] = valid[k] ? lse[(size_t)bh * S + i] * 1.4426950408889634f
                            : __int_as_float(0x7f800000);
    }
  }
}

// The same over packed sequences: one block per listed tile of 128 rows and
// query head, tensors at their strides, lse [Hq, T].
//
// D = dO . o is only as exact as o, which the forward pass rounded to bf16.
// Where a query sees few keys o is large, and D's error then outweighs all
// others (gradients of sequences of a dozen rows: twice the error of a single
// rounding of the result, with it 1.1 times).  So D of a query whose keys lie
// within 32 rows (kPrepKeys: the first rows of a sequence, and all rows under a
// window of up to 32) comes from its definition instead, D = sum_j p_ij dP_ij:
// one warp per 16 rows makes S and dP of the keys about them with mma.sync (a
// 16 x 8 tile; a tcgen05 tile is 128 rows), each thread's 16-byte loads giving
// the same eight values of both operands, in whatever order the product runs.
// That is a launch of its own (it wants registers, the other rows' launch
// wants threads), beside which the other rows' runs.
struct BwdPrepPacked {
  const __nv_bfloat16 *q, *k, *v, *o, *dout;
  long long q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head, do_row, do_head;
  const float* lse;
  float *lse2, *delta;
  PackedRef pk;
  const int* cu;
  int B, Hq, group, causal, window;
  long long S_pad;
  float scale_log2;
  int* error_word;
};

constexpr int kPrepKeys = 32;

// (checked builds: `rows` statistics from `at` on lie inside the workspace)
__device__ __forceinline__ bool bwd_prep_inside(const BwdPrepPacked& p, size_t at, int rows) {
  return attn_check(at + rows <= (size_t)p.Hq * p.S_pad, p.error_word);
}

// Is D of the sequence's row i made from P and dP?
__device__ __forceinline__ bool bwd_prep_exact(const BwdPrepPacked& p, int len, int i) {
  if (!p.causal) return i >= 0 && len <= kPrepKeys;
  return i >= 0 && (i < kPrepKeys || (p.window > 0 && p.window <= kPrepKeys));
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D of rows i0 .. i0 + 15 (a warp's) from keys j0 .. j1 - 1, 16 at a time: half a row of 128
// values of each operand is on its way before the first product.
template <int DH>
__device__ __forceinline__ void bwd_prep_rows(const BwdPrepPacked& p, const PackedTile& e, int h,
                                              int i0, int j0, int j1, int lane) {
  const int g = lane / 4, c = lane % 4;   // rows i0 + g and i0 + g + 8; columns 2 c, 2 c + 1
  const int hk = h / p.group;
  // (checked builds: a sequence and a head of the packed tensors)
  if (!attn_check(e.start >= 0 && e.len <= p.pk.T - e.start && h >= 0 && h < p.Hq, p.error_word))
    return;
  auto row = [&](const __nv_bfloat16* x, long long rs, long long hs, int head, int i, int at) {
    if (i < 0 || i >= e.len) return make_uint4(0u, 0u, 0u, 0u);
    return *reinterpret_cast<const uint4*>(x + (e.start + (long long)i) * rs + head * hs + at);
  };
  bool exact[2];
  float l2[2], sum[2] = {0.f, 0.f}, mass[2] = {0.f, 0.f};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int i = i0 + g + 8 * half;
    exact[half] = i < e.len && bwd_prep_exact(p, e.len, i);
    l2[half] = exact[half] ? p.lse[(size_t)h * p.pk.T + e.start + i] * 1.4426950408889634f : 0.f;
  }
#pragma unroll 1
  for (; j0 < j1; j0 += 16) {
    if (j0 + 15 < 0 || j0 >= e.len) continue;
    float s[2][4], d[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[n][x] = d[n][x] = 0.f;
#pragma unroll 1
    for (int at = 8 * c; at < DH; at += 64) {
      uint4 q[2][2], dy[2][2], k[2][2], v[2][2];   // [32 values][rows g and g + 8, or key tile]
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          q[x][n] = row(p.q, p.q_row, p.q_head, h, i0 + g + 8 * n, at + 32 * x);
          dy[x][n] = row(p.dout, p.do_row, p.do_head, h, i0 + g + 8 * n, at + 32 * x);
          k[x][n] = row(p.k, p.k_row, p.k_head, hk, j0 + 8 * n + g, at + 32 * x);
          v[x][n] = row(p.v, p.v_row, p.v_head, hk, j0 + 8 * n + g, at + 32 * x);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          mma_16816(s[n], q[x][0].x, q[x][1].x, q[x][0].y, q[x][1].y, k[x][n].x, k[x][n].y);
          mma_16816(s[n], q[x][0].z, q[x][1].z, q[x][0].w, q[x][1].w, k[x][n].z, k[x][n].w);
          mma_16816(d[n], dy[x][0].x, dy[x][1].x, dy[x][0].y, dy[x][1].y, v[x][n].x, v[x][n].y);
          mma_16816(d[n], dy[x][0].z, dy[x][1].z, dy[x][0].w, dy[x][1].w, v[x][n].z, v[x][n].w);
        }
      }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int i = i0 + g + 8 * half, j = j0 + 8 * n + 2 * c + x;
          const bool seen = j >= 0 && j < e.len && (!p.causal || j <= i) &&
                            (p.window == 0 || i - j < p.window);
          const float w = ex2_approx(fmaf(s[n][2 * half + x], p.scale_log2, -l2[half]));
          sum[half] += seen ? w * d[n][2 * half + x] : 0.f;
          mass[half] += seen ? w : 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float x = sum[half], y = mass[half];
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    y += __shfl_xor_sync(0xffffffffu, y, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    y += __shfl_xor_sync(0xffffffffu, y, 2);
    // (the weights' sum is 1 but for lse's rounding, which the passes' weights have too: divided
    // by it, the row's dS sum to 0)
    const size_t at = (size_t)h * p.S_pad + (e.stat + e.pad() + i0 + g + 8 * half);
    if (exact[half] && c == 0 && bwd_prep_inside(p, at, 1)) p.delta[at] = x / y;
  }
}

// The rows whose D comes from P and dP, 16 a warp: under a short window a tile's, one tile and
// head a block; else the sequence's first ones, one sequence and four heads a block.
constexpr int kFewHeads = 4;
template <int DH>
__global__ void __launch_bounds__(256, 2) attn_bwd_prep_few(const BwdPrepPacked p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int3 n = packed_counts(p.pk);
  if (n.x + n.y + n.z == 0) return;   // (nothing to do, or offsets that are not sound)
  if (p.causal && p.window > 0 && p.window <= kPrepKeys) {
    const int tile = blockIdx.x / p.Hq, h = blockIdx.x - tile * p.Hq;
    if (tile >= n.x + n.y + n.z) return;
    const PackedTile e = packed_tile(p.pk, tile);
    const int i0 = 128 * e.blk - e.pad() + 16 * warp;
    if (i0 > -16) bwd_prep_rows<DH>(p, e, h, i0, i0 - kPrepKeys, i0 + 16, lane);
    return;
  }
  const int blocks = (p.Hq + kFewHeads - 1) / kFewHeads;
  const int b = blockIdx.x / blocks, h = kFewHeads * (blockIdx.x - b * blocks) + warp / 2;
  const int start = p.cu[b], len = p.cu[b + 1] - start, i0 = 16 * (warp % 2);
  if (h >= p.Hq || i0 >= len || (!p.causal && len > kPrepKeys)) return;
  const PackedTile e{start, len, 0, packed_stat(start, b)};
  bwd_prep_rows<DH>(p, e, h, i0, 0, p.causal ? i0 + 16 : kPrepKeys, lane);
}

template <int DH>
__device__ __forceinline__ void bwd_prep_tile(const BwdPrepPacked& p) {
  constexpr int kLanes = DH / 8;
  constexpr int kRowsPerSet = 256 / kLanes;
  constexpr int kSets = 128 / kRowsPerSet;
  const int tile = blockIdx.x / p.Hq, h = blockIdx.x - tile * p.Hq;
  // (the list has room for every block's tile: its entry and the counts come at once)
  const PackedTile e = packed_tile(p.pk, tile);
  const int3 n = packed_counts(p.pk);
  if (tile >= n.x + n.y + n.z) return;
  const int sub = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  const __nv_bfloat16* po = p.o + h * p.o_head + 8 * sub;
  const __nv_bfloat16* pd = p.dout + h * p.do_head + 8 * sub;
  const size_t to = (size_t)h * p.S_pad + (e.stat + 128 * e.blk);
  const int first = 128 * e.blk - e.pad();   // the block's first row, counted from the sequence's
  // (checked builds: the block's rows are the sequence's, and that lies in the packed tensors)
  if (!attn_check(e.start >= 0 && e.len <= p.pk.T - e.start && first + 128 <= e.len, p.error_word) ||
      !bwd_prep_inside(p, to, 128))
    return;
  constexpr int kBatch = kSets < kPrepRowSets ? kSets : kPrepRowSets;
#pragma unroll 1
  for (int s = 0; s < kSets; s += kBatch) {
    uint4 a[kBatch], b[kBatch];
    float l[kBatch];
    bool valid[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = first + (s + k) * kRowsPerSet + r0;
      valid[k] = i >= 0;
      a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
      l[k] = __int_as_float(0x7f800000);
      if (valid[k]) {
        if (sub == 0) l[k] = p.lse[(size_t)h * p.pk.T + e.start + i];
        a[k] = *reinterpret_cast<const uint4*>(po + (e.start + (long long)i) * p.o_row);
        b[k] = *reinterpret_cast<const uint4*>(pd + (e.start + (long long)i) * p.do_row);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const uint32_t wa[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
      const uint32_t wb[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
      float acc = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        acc = fmaf(__uint_as_float(wa[x] << 16), __uint_as_float(wb[x] << 16), acc);
        acc = fmaf(__uint_as_float(wa[x] & 0xffff0000u), __uint_as_float(wb[x] & 0xffff0000u), acc);
      }
#pragma unroll
      for (int m = kLanes / 2; m > 0; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
      const int r = (s + k) * kRowsPerSet + r0, i = first + r;
      if (sub == 0) {
        if (!bwd_prep_exact(p, e.len, i)) p.delta[to + r] = valid[k] ? acc : 0.f;
        p.lse2[to + r] = l[k] * 1.4426950408889634f;
      }
    }
  }
}

template <int DH>
__global__ void __launch_bounds__(256) attn_bwd_prep_packed(const BwdPrepPacked p) {
  // beside the launch of the other rows, which started once the lists and the inputs were
  // complete and whose results this one does not read; it ends after that one, so that the
  // passes see the results of both
  griddep_launch_dependents();
  bwd_prep_tile<DH>(p);
  griddep_wait();
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// x if off <= span (unsigned), else 0 (a predicated select; see keep_if_le)
__device__ __forceinline__ float zero_unless_le(float x, uint32_t off, uint32_t span) {
  float d;
  asm("{\n .reg .pred p;\n setp.le.u32 p, %1, %2;\n selp.f32 %0, %3, 0f00000000, p;\n}"
      : "=f"(d) : "r"(off), "r"(span), "f"(x));
  return d;
}

__device__ __forceinline__ void bwd_wait_drain(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) return;
  }
}

// Heaviest-first snake order over the CTAs (as in the forward kernels).
__device__ __forceinline__ int bwd_item(int k, int c, int G) {
  return k * G + ((k & 1) ? (G - 1 - c) : c);
}

// Query blocks [lo, hi] that see some key of key block kb (128-row blocks).
__device__ __forceinline__ void bwd_qblocks_of(const BwdParams& p, const BwdSeq& q, int kb,
                                               int& lo, int& hi) {
  if (!p.causal) {
    lo = 0;
    hi = q.nblk - 1;
    return;
  }
  lo = kb;   // query i sees key j only if j <= i
  hi = q.nblk - 1;
  if (p.window > 0) hi = min(hi, (128 * kb + 127 + p.window - 1) / 128);   // i - j < W
}

// Key blocks [lo, hi] that query block qb sees.
__device__ __forceinline__ void bwd_kblocks_of(const BwdParams& p, const BwdSeq& q, int qb,
                                               int& lo, int& hi) {
  if (!p.causal) {
    lo = 0;
    hi = q.nblk - 1;
    return;
  }
  hi = qb;
  lo = p.window > 0 ? max(0, 128 * qb - p.window + 1) / 128 : 0;
}

// Does some (query, key) pair of query block qb x key block kb fall outside
// the mask (or past S)?
__device__ __forceinline__ bool bwd_needs_mask(const BwdParams& p, const BwdSeq& q, int qb, int kb) {
  if (128 * kb + 127 >= q.S || 128 * qb + 127 >= q.S || 128 * kb < q.pad) return true;
  if (!p.causal) return false;
  if (128 * kb + 127 > 128 * qb) return true;                                  // j > i somewhere
  if (p.window > 0 && 128 * qb + 127 - 128 * kb >= p.window) return true;      // i - j >= W somewhere
  return false;
}

// ============================================================ dK, dV pass

template <int DH>
struct __align__(1024) BwdKvSmem {
  using Cfg = BwdCfg<DH>;
  uint8_t k[Cfg::kTile];           // this item's key block (stays)
  uint8_t v[Cfg::kTile];           // this item's value block (stays)
  uint8_t q[Cfg::kStagesQ][Cfg::kTile];    // query blocks
  uint8_t dO[Cfg::kStagesQ][Cfg::kTile];   // their output gradients
  float lse2[Cfg::kStagesQ][128];          // their log-sum-exps (log2 units)
  float dlt[Cfg::kStagesQ][128];           // their D_i
  uint64_t kv_full, kv_empty;
  uint64_t q_full[Cfg::kStagesQ], q_empty[Cfg::kStagesQ];
  uint64_t s_full[Cfg::kBufsS], p_full[Cfg::kBufsS];
  uint64_t dp_full, ds_full, acc_final, mma_done;
  uint32_t tmem_base;
  int abort_flag;
};

// Item w of the dK/dV pass: key block kb (heaviest, i.e. earliest, first
// under a causal mask) of K/V head bkv = b * Hkv + g.
struct BwdKvItem {
  int kb, bkv, b, g, lo, hi;   // PK: b = 0, bkv = g
  BwdSeq seq;
};

// PK: the tile of the CTA's k-th item, if there is one.  Each role reads it an item ahead (a
// read of L2 takes a few hundred ns, and an item of a short sequence no more than a few us).
template <int PK, bool Q>
__device__ __forceinline__ PackedTile bwd_tile_ahead(const BwdParams& p, int k, int num_items,
                                                     const int3& n) {
  if constexpr (PK) {
    const int w = bwd_item(k, blockIdx.x, gridDim.x);
    if (w < num_items) {
      int i = w / p.Hkv, h;
      if (Q) bwd_q_item_at<PK>(p, n, w, i, h);
      return packed_tile(p.pk, i);
    }
  }
  return PackedTile{};
}

// (without lo and hi; PK: of tile e)
template <int PK>
__device__ __forceinline__ BwdKvItem bwd_kv_place_of(const BwdParams& p, int w,
                                                     const PackedTile& e) {
  BwdKvItem r;
  if constexpr (PK) {
    r.kb = e.blk;
    r.b = 0;
    r.g = r.bkv = w - w / p.Hkv * p.Hkv;
    r.seq = bwd_seq_of<PK>(p, e);
    return r;
  }
  const int per = p.B * p.Hkv;
  r.kb = w / per;
  r.bkv = w - r.kb * per;
  r.b = r.bkv / p.Hkv;
  r.g = r.bkv - r.b * p.Hkv;
  r.seq = bwd_seq_of<PK>(p, PackedTile{});
  return r;
}

template <int PK>
__device__ __forceinline__ BwdKvItem bwd_kv_item_of(const BwdParams& p, int w,
                                                    const PackedTile& e) {
  BwdKvItem r = bwd_kv_place_of<PK>(p, w, e);
  bwd_qblocks_of(p, r.seq, r.kb, r.lo, r.hi);
  return r;
}

template <int DH, int PK>
__device__ __forceinline__ void bwd_dkdv_producer(BwdKvSmem<DH>& sm, const BwdParams& p,
                                                  const CUtensorMap* map_q,
                                                  const CUtensorMap* map_k,
                                                  const CUtensorMap* map_v,
                                                  const CUtensorMap* map_do, volatile int* abort) {
  using Cfg = BwdCfg<DH>;
  constexpr int kBoxes = DH / 64;
  const uint64_t keep = policy_evict_last();   // query blocks are re-read by other key blocks
  uint32_t u = 0, loaded = 0, par = 0;
  int items = 0;
  bool ok = true;
  const int3 counts = bwd_counts<PK>(p);
  const int num_items = bwd_num_kv_items<PK>(p, counts);
  PackedTile next = bwd_tile_ahead<PK, false>(p, 0, num_items, counts);
  for (int it = 0; ok; ++it) {
    const int w = bwd_item(it, blockIdx.x, gridDim.x);
    if (w >= num_items) break;
    const BwdKvItem I = bwd_kv_item_of<PK>(p, w, next);
    next = bwd_tile_ahead<PK, false>(p, it + 1, num_items, counts);
    if (items > 0 && !(ok = mbar_wait(&sm.kv_empty, (uint32_t)(items - 1) & 1u, abort))) break;
    // (checked builds: a key block of the sequence, of a K/V head of the batch)
    const bool kv_in_range = attn_check(I.kb >= 0 && 128 * I.kb < I.seq.S && I.bkv >= 0 &&
                                            I.bkv < p.B * p.Hkv && bwd_inside<PK>(p, I.seq),
                                        p.error_word);
    mbar_arrive_expect_tx(&sm.kv_full, kv_in_range ? 2u * Cfg::kTile : 0u);
    if (kv_in_range && (p.fault != 4 || it != 0)) {   // (the test hook withholds one K/V block)
      for (int hf = 0; hf < kBoxes; ++hf) {
        bwd_load_once<PK>(sm.k + hf * Cfg::kBox, map_k, &sm.kv_full, 64 * hf, 128 * I.kb,
                               I.bkv, p, I.seq, kPackedK);
        bwd_load_once<PK>(sm.v + hf * Cfg::kBox, map_v, &sm.kv_full, 64 * hf, 128 * I.kb,
                               I.bkv, p, I.seq, kPackedV);
      }
    }
    ++items;
    const int rows = I.seq.rows(), heads = 1 << I.seq.fold;   // (128 and 1 but for folded tiles)
    for (int hh = 0; ok && hh < p.group; hh += heads) {
      const int bh = I.b * p.Hq + I.g * p.group + hh;
      for (int qb = I.lo; qb <= I.hi; ++qb, ++u) {
        const int st = (int)(u % (uint32_t)Cfg::kStagesQ);
        const uint32_t ph = (u / (uint32_t)Cfg::kStagesQ) & 1u;
        if (!(ok = mbar_wait(&sm.q_empty[st], ph ^ 1u, abort))) break;
        const size_t row0 = (size_t)bh * p.S_pad + (I.seq.stat + 128 * qb);
        // (checked builds: a query block of the sequence, of a query head of
        // the batch, whose per-row statistics lie inside the workspace)
        const bool in_range = attn_check(qb >= 0 && 128 * qb < I.seq.S && bh >= 0 &&
                                             bh + heads <= p.B * p.Hq &&
                                             row0 + (size_t)(heads - 1) * p.S_pad + 128 <=
                                                 (size_t)p.B * p.Hq * p.S_pad,
                                         p.error_word);
        mbar_arrive_expect_tx(&sm.q_full[st], in_range ? 2u * Cfg::kTile + 2u * 512u : 0u);
        for (int hf = 0; in_range && hf < kBoxes; ++hf) {
          bwd_load_queries<PK>(sm.q[st] + hf * Cfg::kBox, map_q, &sm.q_full[st], 64 * hf, qb, bh,
                               p, I.seq, kPackedQ, keep);
          bwd_load_queries<PK>(sm.dO[st] + hf * Cfg::kBox, map_do, &sm.q_full[st], 64 * hf, qb, bh,
                               p, I.seq, kPackedDO, keep);
        }
        for (int x = 0; in_range && x < heads; ++x) {
          const size_t at = row0 + (size_t)x * p.S_pad + (128 - rows);
          bulk_load(sm.lse2[st] + x * rows, p.lse2 + at, 4 * rows, &sm.q_full[st], keep);
          bulk_load(sm.dlt[st] + x * rows, p.delta + at, 4 * rows, &sm.q_full[st], keep);
        }
        loaded |= 1u << st;
        par = (par & ~(1u << st)) | (ph << st);
      }
    }
  }
  // every copy this thread started has landed before the CTA may exit
  if (items > 0) bwd_wait_drain(&sm.kv_full, (uint32_t)(items - 1) & 1u);
  for (int i = 0; i < Cfg::kStagesQ; ++i)
    if (loaded & (1u << i)) bwd_wait_drain(&sm.q_full[i], (par >> i) & 1u);
}

// MMA issue order per item of N steps (one step = one query block of one
// query head): S(0), dP(0), then per step n: dV(n) once P(n) is written,
// S(n+1) (its columns held P(n), which dV(n), issued before it, reads),
// dK(n) once dS(n) is written, dP(n+1) (its columns held dS(n)).  The
// element-wise work of step n+1 therefore overlaps dK(n) and dP(n+1).
// With two S buffers (Dh 64) S(n+1) goes first: its columns held P(n-1), and
// the scores of the next step are there when the element-wise warps are.
template <int DH, int PK>
__device__ __forceinline__ void bwd_dkdv_issuer(BwdKvSmem<DH>& sm, const BwdParams& p,
                                                volatile int* abort) {
  using Cfg = BwdCfg<DH>;
  constexpr uint32_t idesc_ss = idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t idesc_acc = idesc_bf16_f32(128, DH, false, true);
  constexpr uint64_t kKmajor = smem_desc_sw128(0, 16, 1024);
  constexpr uint64_t kMnMajor = smem_desc_sw128(0, Cfg::kBox, 1024);
  const uint64_t dk_ = kKmajor | (smem_u32(sm.k) >> 4);
  const uint64_t dv_ = kKmajor | (smem_u32(sm.v) >> 4);
  const uint64_t dq_k = kKmajor | (smem_u32(sm.q[0]) >> 4);
  const uint64_t ddo_k = kKmajor | (smem_u32(sm.dO[0]) >> 4);
  const uint64_t dq_mn = kMnMajor | (smem_u32(sm.q[0]) >> 4);
  const uint64_t ddo_mn = kMnMajor | (smem_u32(sm.dO[0]) >> 4);
  constexpr uint64_t kStage = Cfg::kTile >> 4;   // q[1] - q[0] (and dO) in descriptor units
  constexpr bool kTwoS = Cfg::kBufsS == 2;
  auto stage = [](uint32_t x) { return x % (uint32_t)Cfg::kStagesQ; };
  auto stage_ph = [](uint32_t x) { return (x / (uint32_t)Cfg::kStagesQ) & 1u; };
  auto buf = [](uint32_t x) { return kTwoS ? x & 1u : 0u; };             // of S and P
  auto buf_ph = [](uint32_t x) { return (kTwoS ? x >> 1 : x) & 1u; };
  auto col_s = [&](uint32_t x) { return buf(x) ? Cfg::kColS1 : Cfg::kColS; };
  // D (128 x 128) = A (128 x DH) B^T, both K-major (DH contiguous)
  auto mma_nt = [&](uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk) {
      const uint32_t off = ((kk / 4) * Cfg::kBox + (kk % 4) * 32) >> 4;
      mma_bf16_ss_warp(d, a + off, b + off, idesc_ss, kk > 0 ? 1u : 0u);
    }
  };
  // D (128 x DH) (+)= A (tensor memory, 128 x 128 bf16 pairs at bwd_packed_col) B,
  // B MN-major (DH contiguous)
  auto mma_acc = [&](uint32_t d, uint32_t a, uint64_t b, bool first, bool two) {
#pragma unroll
    for (int kk = 0; kk < 128 / 16; ++kk)
      mma_bf16_ts_warp(d, a + bwd_packed_col(kk), b + kk * (2048 >> 4), idesc_acc,
                       (!first || kk > 0) ? 1u : 0u);
    if (PK && two) {
#pragma unroll
      for (int kk = 0; kk < 128 / 16; ++kk)
        mma_bf16_ts_warp(d, a + bwd_low_col(kk), b + kk * (2048 >> 4), idesc_acc, 1u);
    }
  };
  auto wait_all = [&](uint64_t* bar, uint32_t ph) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, ph, abort));
  };
  uint32_t u = 0;
  int items = 0;
  bool ok = true;
  const int3 counts = bwd_counts<PK>(p);
  const int num_items = bwd_num_kv_items<PK>(p, counts);
  PackedTile next = bwd_tile_ahead<PK, false>(p, 0, num_items, counts);
  for (int it = 0; ok; ++it) {
    const int w = bwd_item(it, blockIdx.x, gridDim.x);
    if (w >= num_items) break;
    const BwdKvItem I = bwd_kv_item_of<PK>(p, w, next);
    next = bwd_tile_ahead<PK, false>(p, it + 1, num_items, counts);
    const int N = (PK ? p.group >> I.seq.fold : p.group) * (I.hi - I.lo + 1);
    if (!(ok = wait_all(&sm.kv_full, (uint32_t)items & 1u))) break;
    ++items;
    // S of step x
    auto scores = [&](uint32_t x) -> bool {
      if (!wait_all(&sm.q_full[stage(x)], stage_ph(x))) return false;
      tc_fence_after_sync();
      mma_nt(col_s(x), dk_, dq_k + stage(x) * kStage);                   // S^T = K Q^T
      mma_commit_warp(&sm.s_full[buf(x)]);
      return true;
    };
    if (!(ok = scores(u))) break;
    mma_nt(Cfg::kColDP, dv_, ddo_k + stage(u) * kStage);
    mma_commit_warp(&sm.dp_full);
    if (N == 1) mma_commit_warp(&sm.kv_empty);
    int qb = I.lo;   // step n's query block (of one head after another)
    for (int n = 0; n < N; ++n, ++u) {
      const uint64_t st = stage(u), st1 = stage(u + 1);
      const bool two = bwd_two_parts<PK>(p, qb);
      if (PK) qb = qb == I.hi ? I.lo : qb + 1;
      if (kTwoS && n + 1 < N && !(ok = scores(u + 1))) break;
      if (!(ok = wait_all(&sm.p_full[buf(u)], buf_ph(u)))) break;
      tc_fence_after_sync();
      mma_acc(Cfg::kColA0, col_s(u), ddo_mn + st * kStage, n == 0, two);     // dV += P^T dO
      if (!kTwoS && n + 1 < N && !(ok = scores(u + 1))) break;
      if (!(ok = wait_all(&sm.ds_full, u & 1u))) break;
      tc_fence_after_sync();
      mma_acc(Cfg::kColAcc1, Cfg::kColDP, dq_mn + st * kStage, n == 0, two); // dK += dS^T Q
      mma_commit_warp(&sm.q_empty[st]);
      if (n + 1 < N) {
        mma_nt(Cfg::kColDP, dv_, ddo_k + st1 * kStage);                 // dP^T(n+1) = V dO^T
        mma_commit_warp(&sm.dp_full);
        if (n + 2 == N) mma_commit_warp(&sm.kv_empty);
      }
    }
    if (ok) mma_commit_warp(&sm.acc_final);
  }
  mma_commit_warp(&sm.mma_done);
  bwd_wait_drain(&sm.mma_done, 0);
}

// The same with two 32-byte stores, dst 32-byte aligned.  A row is a thread's, so each store
// instruction touches 32 rows: half as many of them, of whole sectors.
__device__ __forceinline__ void bwd_store32_wide(__nv_bfloat16* dst, const uint32_t (&r)[32],
                                                 float mul) {
  const uint64_t policy = policy_evict_first();
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w[e] = pack_bf16x2(__uint_as_float(r[16 * q + 2 * e]) * mul,
                         __uint_as_float(r[16 * q + 2 * e + 1]) * mul);
    st_global_v8_hint(dst + 16 * q, w, policy);
  }
}

// Store 32 fp32 accumulator columns (times `mul`) as bf16 to dst (16-byte aligned).
__device__ __forceinline__ void bwd_store32(__nv_bfloat16* dst, const uint32_t (&r)[32], float mul) {
  uint4* d = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_bf16x2(__uint_as_float(r[8 * q + 2 * e]) * mul,
                         __uint_as_float(r[8 * q + 2 * e + 1]) * mul);
    d[q] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Element-wise work of the dK/dV pass (warps 0-7; warpgroup wg owns query
// columns kCols wg .. kCols (wg + 1) - 1, each warp 32 key rows, which are its
// tensor-memory lanes).  A thread has 16 columns of four rows: with a row each
// it would need lse2 and D of every column, and reading them took the shared
// memory's whole bandwidth for twice as long as the exponentials take (128
// lanes x 128 columns x 2 values a step).  Per step: P^T = exp2(S^T * scale*log2e - lse2[query])
// (0 where masked), written as bf16 pairs (see bwd_packed_col) and kept in
// fp32 registers; then dS^T = P^T o (dP^T - D[query]), as bf16 pairs over dP^T.
// Per item: the first half of the warpgroups write dV, the second scale * dK.
template <int DH, int PK>
__device__ __forceinline__ void bwd_dkdv_softmax(BwdKvSmem<DH>& sm, const BwdParams& p,
                                                 uint32_t tbase, volatile int* abort, int warp,
                                                 int lane) {
  using Cfg = BwdCfg<DH>;
  const int wg = warp / 4;
  const int t = (warp % 4) * 32 + lane;
  const uint32_t lane_addr = tbase + ((uint32_t)((warp % 4) * 32) << 16);
  constexpr bool kTwoS = Cfg::kBufsS == 2;
  static_assert(Cfg::kCols == 64, "two halves of 16 lanes x 64 columns per warp");
  const int c2 = 2 * (lane % 4);   // this thread's first column of every eight
  const uint32_t colDP = lane_addr + Cfg::kColDP + Cfg::kCols * wg;
  const float2 neg_sl2 = make_float2(-p.scale_log2, -p.scale_log2);
  uint32_t u = 0;
  int items = 0;
  bool ok = true;
  const int3 counts = bwd_counts<PK>(p);
  const int num_items = bwd_num_kv_items<PK>(p, counts);
  PackedTile next = bwd_tile_ahead<PK, false>(p, 0, num_items, counts);
  for (int it = 0; ok; ++it) {
    const int w = bwd_item(it, blockIdx.x, gridDim.x);
    if (w >= num_items) break;
    const BwdKvItem I = bwd_kv_item_of<PK>(p, w, next);
    next = bwd_tile_ahead<PK, false>(p, it + 1, num_items, counts);
    const int j = 128 * I.kb + t;   // the key that this thread stores
    const int j0 = 128 * I.kb + 32 * (warp % 4) + lane / 4;   // those it computes: j0 + 0, 8, 16, 24
    const int heads = 1 << I.seq.fold;
    for (int hh = 0; ok && hh < p.group; hh += heads) {
      for (int qb = I.lo; qb <= I.hi; ++qb, ++u) {
        const int st = (int)(u % (uint32_t)Cfg::kStagesQ);
        // this step's S buffer, its phase, and this warpgroup's scores in it
        const uint32_t b = kTwoS ? u & 1u : 0u, ph = (kTwoS ? u >> 1 : u) & 1u;
        const uint32_t colS = lane_addr + (b ? Cfg::kColS1 : Cfg::kColS) + Cfg::kCols * wg;
        // the stage's lse2 / D (bulk copies counted on q_full)
        if (!(ok = mbar_wait(&sm.q_full[st], (u / (uint32_t)Cfg::kStagesQ) & 1u, abort))) break;
        // (read ahead of the wait for the scores)
        const uint32_t at_l = smem_u32(sm.lse2[st] + Cfg::kCols * wg + c2);
        const uint32_t at_d = smem_u32(sm.dlt[st] + Cfg::kCols * wg + c2);
        float2 l[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) l[k] = ld_shared_f2(at_l + 32 * k);
        if (!(ok = mbar_wait(&sm.s_full[b], ph, abort))) break;
        tc_fence_after_sync();

        uint32_t x[2][32];
#pragma unroll
        for (int h = 0; h < 2; ++h) tmem_ld_16x256b_x8(colS + (h << 20), x[h]);
#pragma unroll
        for (int h = 0; h < 2; ++h) tmem_ld_wait(x[h]);
        float pf[2][32];   // P^T (fp32)
        // (the mask in a loop of its own: a branch at every pair would keep the exponentials of
        // one pair from overlapping the next one's.  A second loop with the mask in it, as in the
        // dQ pass, is 2 % slower over 8192 rows and as much faster over sequences of 300)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 xs =
                __ffma2_rn(make_float2(__uint_as_float(x[h][e]), __uint_as_float(x[h][e + 1])),
                           neg_sl2, l[e / 4]);
            pf[h][e] = ex2_approx(-xs.x);   // (the sign is the instruction's)
            pf[h][e + 1] = ex2_approx(-xs.y);
          }
        }
        if (bwd_needs_mask(p, I.seq, qb, I.kb)) {
          int i0 = 128 * qb + Cfg::kCols * wg, most = Cfg::kCols - 1, column = -1;
          if (PK == 2 && I.seq.fold) {   // columns count within a head
            i0 = 128 - I.seq.rows();
            column = most = I.seq.rows() - 1;
          }
          most = min(most, I.seq.S - 1 - i0);                                // i < S
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            // visible query columns of key row + 8 h: [clo, chi] of this warpgroup's (query
            // i = 128 qb + kCols wg + c)
            const int j = j0 + 8 * h;
            int clo = 0, chi = most;
            if (p.causal) clo = j - i0;                                      // i >= j
            if (p.window > 0) chi = min(chi, j - i0 + p.window - 1);         // i - j < W
            const uint32_t span = chi >= clo ? (uint32_t)(chi - clo) : 0u;
            if (chi < clo) clo = 1 << 30;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              int at = 8 * (e / 2) + c2 + e % 2;
              if (PK == 2) at &= column;
              float& y = pf[h / 2][4 * (e / 2) + 2 * (h % 2) + e % 2];
              y = zero_unless_le(y, (uint32_t)(at - clo), span);
            }
          }
        }
        const bool two = bwd_two_parts<PK>(p, qb);
        // pf as bf16 pairs over the columns it came from, its low parts behind them
        auto write = [&](uint32_t col) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w16[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w16[e] = pack_bf16x2(pf[h][2 * e], pf[h][2 * e + 1]);
            tmem_st_16x128b_x8(col + (h << 20), w16);
          }
          if (PK && two) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w16[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float a = pf[h][2 * e], b = pf[h][2 * e + 1];
                w16[e] = bwd_low_pair(a, b, pack_bf16x2(a, b));
              }
              tmem_st_16x128b_x8(col + (h << 20) + Cfg::kCols / 2, w16);
            }
          }
        };
        write(colS);   // (every score of this thread's is in registers)
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&sm.p_full[b]);

        float2 d[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = ld_shared_f2(at_d + 32 * k);
        if (!(ok = mbar_wait(&sm.dp_full, u & 1u, abort))) break;
        tc_fence_after_sync();
#pragma unroll
        for (int h = 0; h < 2; ++h) tmem_ld_16x256b_x8(colDP + (h << 20), x[h]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tmem_ld_wait(x[h]);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 dd = __fadd2_rn(
                make_float2(__uint_as_float(x[h][e]), __uint_as_float(x[h][e + 1])),
                make_float2(-d[e / 4].x, -d[e / 4].y));
            const float2 ds = __fmul2_rn(make_float2(pf[h][e], pf[h][e + 1]), dd);
            pf[h][e] = ds.x;   // (the weights are not needed any more)
            pf[h][e + 1] = ds.y;
          }
        }
        write(colDP);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&sm.ds_full);
      }
    }
    if (!ok) break;

    // ---- epilogue: dV and scale * dK of key j
    if (!(ok = mbar_wait(&sm.acc_final, (uint32_t)items & 1u, abort))) break;
    ++items;
    tc_fence_after_sync();
    const bool store = bwd_real<PK>(I.seq, j);
    constexpr int kHalf = Cfg::kWG / 2;              // warpgroups per accumulator
    const bool is_dv = wg < kHalf;
    __nv_bfloat16* dst = is_dv ? p.dv + bwd_row<PK>(I.seq, I.bkv, j, DH, p.dv_row, p.dv_head)
                               : p.dk + bwd_row<PK>(I.seq, I.bkv, j, DH, p.dk_row, p.dk_head);
    const uint32_t colA = lane_addr + (is_dv ? Cfg::kColA0 : Cfg::kColAcc1);
    const float mul = is_dv ? 1.0f : p.scale;
#pragma unroll 1
    for (int c = wg % kHalf; c < DH / 32; c += kHalf) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(colA + 32 * c, r);
      tmem_ld_wait(r);
      if (store) {
        if (PK && p.wide)
          bwd_store32_wide(dst + 32 * c, r, mul);
        else
          bwd_store32(dst + 32 * c, r, mul);
      }
    }
    // the next item's first dV / dK overwrite the accumulators only after
    // this thread's next arrive on p_full / ds_full, which follows these loads
  }
}

template <int DH, int PK = 0>
__global__ void __launch_bounds__(BwdCfg<DH>::kThreads, 1)
    attn_bwd_dkdv(const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ CUtensorMap map_do, const BwdParams p) {
  using Cfg = BwdCfg<DH>;
  using Smem = BwdKvSmem<DH>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~uintptr_t(1023));
  volatile int* abort = &sm.abort_flag;
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (warp == Cfg::kWarpProducer && lane == 0) {
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
    prefetch_tensormap(&map_do);
  }
  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    mbar_init(&sm.kv_full, 1);
    mbar_init(&sm.kv_empty, 1);
    for (int i = 0; i < Cfg::kStagesQ; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
    }
    for (int i = 0; i < Cfg::kBufsS; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], Cfg::kEW);
    }
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.ds_full, Cfg::kEW);
    mbar_init(&sm.acc_final, 1);
    mbar_init(&sm.mma_done, 1);
    fence_mbarrier_init();
  }
  if (warp == Cfg::kWarpProducer) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  // launched as a programmatic dependent of the prep kernel: its D and lse2
  // (and the inputs) are read only after it has completed; then the dQ pass,
  // which needs no output of this one, may be scheduled on SMs this grid frees
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const uint32_t tbase = sm.tmem_base;
  // compile-time tensor-memory columns: the allocation must start at column 0
  if (tbase != 0 && threadIdx.x == 0) sm.abort_flag = 1;
  if (tbase == 0) {
    if (warp == Cfg::kWarpProducer) {
      if (lane == 0) bwd_dkdv_producer<DH, PK>(sm, p, &map_q, &map_k, &map_v, &map_do, abort);
    } else if (warp == Cfg::kWarpIssuer) {
      bwd_dkdv_issuer<DH, PK>(sm, p, abort);
    } else {
      bwd_dkdv_softmax<DH, PK>(sm, p, tbase, abort, warp, lane);
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == Cfg::kWarpProducer) {
    tc_fence_after_sync();
    tmem_dealloc(tbase, 512);
  }
  if (threadIdx.x == 0 && sm.abort_flag) atomicExch(p.error_word, 4);   // ATTN_ERR_TIMEOUT
}

// ============================================================ dQ pass

template <int DH>
struct __align__(1024) BwdQSmem {
  using Cfg = BwdCfg<DH>;
  static constexpr int kStagesK = 3, kStagesV = 2;
  uint8_t q[Cfg::kTile];           // this item's query block (stays)
  uint8_t dO[Cfg::kTile];          // and its output gradient
  uint8_t k[kStagesK][Cfg::kTile];   // key blocks: read by S(n) and dQ(n)
  uint8_t v[kStagesV][Cfg::kTile];   // value blocks: read by dP(n) only
  uint64_t q_full, q_empty;
  uint64_t k_full[kStagesK], k_empty[kStagesK];
  uint64_t v_full[kStagesV], v_empty[kStagesV];
  uint64_t s_full, s_free, acc_final, mma_done;
  uint64_t dp_full[2], ds_full[2];   // per dP / dS buffer
  uint32_t tmem_base;
  int abort_flag;
};

// Item w of the dQ pass: query block qb (heaviest, i.e. last, first under a
// causal mask) of query head bh = b * Hq + h.
struct BwdQItem {
  int qb, bh, bkv, lo, hi;   // PK: bh and bkv are the heads alone
  BwdSeq seq;
};

// (without lo and hi; PK: of tile e)
template <int PK>
__device__ __forceinline__ BwdQItem bwd_q_place_of(const BwdParams& p, int w, const PackedTile& e,
                                                   const int3& n) {
  BwdQItem r;
  if constexpr (PK) {
    int i;
    bwd_q_item_at<PK>(p, n, w, i, r.bh);
    r.qb = e.blk;
    r.bkv = r.bh / p.group;
    r.seq = bwd_seq_of<PK>(p, e);
    return r;
  }
  const int per = p.B * p.Hq;
  const int blk = w / per;
  r.qb = p.nblk - 1 - blk;
  r.bh = w - blk * per;
  const int b = r.bh / p.Hq;
  r.bkv = b * p.Hkv + (r.bh - b * p.Hq) / p.group;   // g(h) = floor(h / (H/G))
  r.seq = bwd_seq_of<PK>(p, PackedTile{});
  return r;
}

template <int PK>
__device__ __forceinline__ BwdQItem bwd_q_item_of(const BwdParams& p, int w, const PackedTile& e,
                                                  const int3& n) {
  BwdQItem r = bwd_q_place_of<PK>(p, w, e, n);
  bwd_kblocks_of(p, r.seq, r.qb, r.lo, r.hi);
  return r;
}

template <int DH, int PK>
__device__ __forceinline__ void bwd_dq_producer(BwdQSmem<DH>& sm, const BwdParams& p,
                                                const CUtensorMap* map_q, const CUtensorMap* map_k,
                                                const CUtensorMap* map_v,
                                                const CUtensorMap* map_do, volatile int* abort) {
  using Cfg = BwdCfg<DH>;
  using Smem = BwdQSmem<DH>;
  constexpr int kBoxes = DH / 64;
  const uint64_t keep = policy_evict_last();   // key blocks are re-read by other query blocks
  uint32_t u = 0, k_loaded = 0, k_par = 0, v_loaded = 0, v_par = 0;
  uint32_t ks = 0, kph = 0;   // K stage and its phase for block u (u % 3, (u / 3) & 1)
  int items = 0;
  bool ok = true;
  const int3 counts = bwd_counts<PK>(p);
  const int num_items = bwd_num_q_items<PK>(p, counts);
  PackedTile next = bwd_tile_ahead<PK, true>(p, 0, num_items, counts);
  for (int it = 0; ok; ++it) {
    const int w = bwd_item(it, blockIdx.x, gridDim.x);
    if (w >= num_items) break;
    const BwdQItem I = bwd_q_item_of<PK>(p, w, next, counts);
    next = bwd_tile_ahead<PK, true>(p, it + 1, num_items, counts);
    if (items > 0 && !(ok = mbar_wait(&sm.q_empty, (uint32_t)(items - 1) & 1u, abort))) break;
    // (checked builds: a query block of the sequence, of a query head of the batch)
    const bool q_in_range = attn_check(I.qb >= 0 && 128 * I.qb < I.seq.S && I.bh >= 0 &&
                                           I.bh < p.B * p.Hq && bwd_inside<PK>(p, I.seq),
                                       p.error_word);
    mbar_arrive_expect_tx(&sm.q_full, q_in_range ? 2u * Cfg::kTile : 0u);
    for (int hf = 0; q_in_range && hf < kBoxes; ++hf) {
      if constexpr (PK) {
        bwd_load_queries<PK>(sm.q + hf * Cfg::kBox, map_q, &sm.q_full, 64 * hf, I.qb, I.bh, p,
                             I.seq, kPackedQ, policy_evict_first());
        bwd_load_queries<PK>(sm.dO + hf * Cfg::kBox, map_do, &sm.q_full, 64 * hf, I.qb, I.bh, p,
                             I.seq, kPackedDO, policy_evict_first());
      } else {
        tma_load_3d(sm.q + hf * Cfg::kBox, map_q, &sm.q_full, 64 * hf, 128 * I.qb, I.bh);
        tma_load_3d(sm.dO + hf * Cfg::kBox, map_do, &sm.q_full, 64 * hf, 128 * I.qb, I.bh);
      }
    }
    ++items;
    for (int kb = I.lo; kb <= I.hi; ++kb, ++u) {
      // (checked builds: a key block of the sequence, of a K/V head of the batch)
      const bool in_range = attn_check(kb >= 0 && 128 * kb < I.seq.S && I.bkv >= 0 &&
                                           I.bkv < p.B * p.Hkv,
                                       p.error_word);
      const uint32_t bytes = in_range ? (uint32_t)Cfg::kTile : 0u;
      if (!(ok = mbar_wait(&sm.k_empty[ks], kph ^ 1u, abort))) break;
      mbar_arrive_expect_tx(&sm.k_full[ks], bytes);
      for (int hf = 0; in_range && hf < kBoxes; ++hf)
        bwd_load<PK>(sm.k[ks] + hf * Cfg::kBox, map_k, &sm.k_full[ks], 64 * hf, 128 * kb,
                          I.bkv, p, I.seq, kPackedK, keep);
      k_loaded |= 1u << ks;
      k_par = (k_par & ~(1u << ks)) | (kph << ks);
      if (++ks == Smem::kStagesK) { ks = 0; kph ^= 1u; }
      const uint32_t vs = u & 1u, vph = (u >> 1) & 1u;
      if (!(ok = mbar_wait(&sm.v_empty[vs], vph ^ 1u, abort))) break;
      mbar_arrive_expect_tx(&sm.v_full[vs], bytes);
      for (int hf = 0; in_range && hf < kBoxes; ++hf)
        bwd_load<PK>(sm.v[vs] + hf * Cfg::kBox, map_v, &sm.v_full[vs], 64 * hf, 128 * kb,
                          I.bkv, p, I.seq, kPackedV, keep);
      v_loaded |= 1u << vs;
      v_par = (v_par & ~(1u << vs)) | (vph << vs);
    }
  }
  if (items > 0) bwd_wait_drain(&sm.q_full, (uint32_t)(items - 1) & 1u);
  for (int i = 0; i < Smem::kStagesK; ++i)
    if (k_loaded & (1u << i)) bwd_wait_drain(&sm.k_full[i], (k_par >> i) & 1u);
  for (int i = 0; i < Smem::kStagesV; ++i)
    if (v_loaded & (1u << i)) bwd_wait_drain(&sm.v_full[i], (v_par >> i) & 1u);
}

// MMA issue order per item of N key blocks: S(0), dP(0), then per block n:
// S(n+1) once the element-wise warps have read S(n), dP(n+1) into the other
// of two dP buffers, then dQ(n) once dS(n) is written over dP(n).  With two
// buffers the next block's S and dP run on the tensor core while the
// element-wise warps turn dP(n) into dS(n), and dQ(n) is the only MMA that
// waits for them; dP(n+2) reuses dP(n)'s columns after dQ(n), issued before
// it, has read dS(n) there.  A value block is released when its dP is done,
// a key block only after dQ: three key stages let block n+2's keys load
// while blocks n and n+1 are in use.
template <int DH, int PK>
__device__ __forceinline__ void bwd_dq_issuer(BwdQSmem<DH>& sm, const BwdParams& p,
                                              volatile int* abort) {
  using Cfg = BwdCfg<DH>;
  using Smem = BwdQSmem<DH>;
  constexpr uint32_t idesc_ss = idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t idesc_acc = idesc_bf16_f32(128, DH, false, true);
  constexpr uint64_t kKmajor = smem_desc_sw128(0, 16, 1024);
  constexpr uint64_t kMnMajor = smem_desc_sw128(0, Cfg::kBox, 1024);
  const uint64_t dq_ = kKmajor | (smem_u32(sm.q) >> 4);
  const uint64_t ddo_ = kKmajor | (smem_u32(sm.dO) >> 4);
  const uint64_t dk_k = kKmajor | (smem_u32(sm.k[0]) >> 4);
  const uint64_t dv_k = kKmajor | (smem_u32(sm.v[0]) >> 4);
  const uint64_t dk_mn = kMnMajor | (smem_u32(sm.k[0]) >> 4);
  constexpr uint64_t kStage = Cfg::kTile >> 4;
  auto mma_nt = [&](uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk) {
      const uint32_t off = ((kk / 4) * Cfg::kBox + (kk % 4) * 32) >> 4;
      mma_bf16_ss_warp(d, a + off, b + off, idesc_ss, kk > 0 ? 1u : 0u);
    }
  };
  auto wait_all = [&](uint64_t* bar, uint32_t ph) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, ph, abort));
  };
  uint32_t u = 0;
  int items = 0;
  bool ok = true;
  const int3 counts = bwd_counts<PK>(p);
  const int num_items = bwd_num_q_items<PK>(p, counts);
  PackedTile next = bwd_tile_ahead<PK, true>(p, 0, num_items, counts);
  for (int it = 0; ok; ++it) {
    const int w = bwd_item(it, blockIdx.x, gridDim.x);
    if (w >= num_items) break;
    const BwdQItem I = bwd_q_item_of<PK>(p, w, next, counts);
    next = bwd_tile_ahead<PK, true>(p, it + 1, num_items, counts);
    const int N = I.hi - I.lo + 1;
    if (!(ok = wait_all(&sm.q_full, (uint32_t)items & 1u))) break;
    ++items;
    // block u (counted across items) uses K stage u % 3, V stage u & 1 and
    // dP buffer u & 1
    auto col_dp = [](uint32_t b) { return b ? Cfg::kColDP1 : Cfg::kColDP; };
    auto kst = [](uint32_t x) { return x % (uint32_t)Smem::kStagesK; };
    auto kph = [](uint32_t x) { return (x / (uint32_t)Smem::kStagesK) & 1u; };
    if (!(ok = wait_all(&sm.k_full[kst(u)], kph(u)))) break;
    tc_fence_after_sync();
    mma_nt(Cfg::kColS, dq_, dk_k + kst(u) * kStage);
    mma_commit_warp(&sm.s_full);
    if (!(ok = wait_all(&sm.v_full[u & 1u], (u >> 1) & 1u))) break;
    tc_fence_after_sync();
    mma_nt(col_dp(u & 1u), ddo_, dv_k + (u & 1u) * kStage);
    mma_commit_warp(&sm.dp_full[u & 1u]);
    mma_commit_warp(&sm.v_empty[u & 1u]);
    if (N == 1) mma_commit_warp(&sm.q_empty);
    for (int n = 0; n < N; ++n, ++u) {
      const uint32_t st = u & 1u, st1 = (u + 1) & 1u;
      if (n + 1 < N) {
        if (!(ok = wait_all(&sm.s_free, u & 1u))) break;
        if (!(ok = wait_all(&sm.k_full[kst(u + 1)], kph(u + 1)))) break;
        tc_fence_after_sync();
        mma_nt(Cfg::kColS, dq_, dk_k + kst(u + 1) * kStage);             // S(n+1) = Q K^T
        mma_commit_warp(&sm.s_full);
        if (!(ok = wait_all(&sm.v_full[st1], ((u + 1) >> 1) & 1u))) break;
        tc_fence_after_sync();
        mma_nt(col_dp(st1), ddo_, dv_k + st1 * kStage);                  // dP(n+1) = dO V^T
        mma_commit_warp(&sm.dp_full[st1]);
        mma_commit_warp(&sm.v_empty[st1]);
        if (n + 2 == N) mma_commit_warp(&sm.q_empty);
      }
      if (!(ok = wait_all(&sm.ds_full[st], (u >> 1) & 1u))) break;
      tc_fence_after_sync();
#pragma unroll
      for (int kk = 0; kk < 128 / 16; ++kk)                              // dQ += dS K
        mma_bf16_ts_warp(Cfg::kColA0, col_dp(st) + bwd_packed_col(kk),
                         dk_mn + kst(u) * kStage + kk * (2048 >> 4),
                         idesc_acc, (n > 0 || kk > 0) ? 1u : 0u);
      if (PK && bwd_two_parts<PK>(p, I.qb)) {
#pragma unroll
        for (int kk = 0; kk < 128 / 16; ++kk)
          mma_bf16_ts_warp(Cfg::kColA0, col_dp(st) + bwd_low_col(kk),
                           dk_mn + kst(u) * kStage + kk * (2048 >> 4), idesc_acc, 1u);
      }
      mma_commit_warp(&sm.k_empty[kst(u)]);
    }
    if (ok) mma_commit_warp(&sm.acc_final);
  }
  mma_commit_warp(&sm.mma_done);
  bwd_wait_drain(&sm.mma_done, 0);
}

// PK: lse2 and D of row t of the CTA's k-th item, whose tile is e.
template <int PK>
__device__ __forceinline__ float2 bwd_stats_ahead(const BwdParams& p, int k, int num_items,
                                                  const PackedTile& e, int t, const int3& n) {
  const int w = bwd_item(k, blockIdx.x, gridDim.x);
  if (w >= num_items) return make_float2(0.f, 0.f);
  const BwdSeq q = bwd_seq_of<PK>(p, e);
  int i, h;
  bwd_q_item_at<PK>(p, n, w, i, h);
  const size_t at = (size_t)(h + q.head_of(t)) * p.S_pad + (q.stat + q.row_of(e.blk, t));
  return make_float2(p.lse2[at], p.delta[at]);
}

// Element-wise work of the dQ pass (warps 0-7; thread t of warpgroup wg owns
// query row 128 qb + t and key columns kCols wg .. kCols (wg + 1) - 1):
// P = exp2(S * scale*log2e - lse2_i) (0 where masked), kept in fp32
// registers; dS = P o (dP - D_i) as bf16 pairs over dP (see bwd_packed_col).
// Per item: scale * dQ out, the 32-column chunks dealt to the warpgroups.
template <int DH, int PK>
__device__ __forceinline__ void bwd_dq_softmax(BwdQSmem<DH>& sm, const BwdParams& p,
                                               uint32_t tbase, volatile int* abort, int warp,
                                               int lane) {
  using Cfg = BwdCfg<DH>;
  const int wg = warp / 4;
  const int t = (warp % 4) * 32 + lane;
  const uint32_t lane_addr = tbase + ((uint32_t)((warp % 4) * 32) << 16);
  const uint32_t colS = lane_addr + Cfg::kColS + Cfg::kCols * wg;
  const uint32_t colDP0 = lane_addr + Cfg::kColDP + Cfg::kCols * wg;    // dP buffer 0
  const uint32_t colDP1 = lane_addr + Cfg::kColDP1 + Cfg::kCols * wg;   // dP buffer 1
  const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
  uint32_t u = 0;
  int items = 0;
  bool ok = true;
  const int3 counts = bwd_counts<PK>(p);
  const int num_items = bwd_num_q_items<PK>(p, counts);
  float2 ahead = make_float2(0.f, 0.f);
  PackedTile next = bwd_tile_ahead<PK, true>(p, 0, num_items, counts);
  for (int it = 0; ok; ++it) {
    const int w = bwd_item(it, blockIdx.x, gridDim.x);
    if (w >= num_items) break;
    const BwdQItem I = bwd_q_item_of<PK>(p, w, next, counts);
    next = bwd_tile_ahead<PK, true>(p, it + 1, num_items, counts);
    // this thread's query, and its head
    const int i = PK ? I.seq.row_of(I.qb, t) : 128 * I.qb + t;
    const int bh = PK ? I.bh + I.seq.head_of(t) : I.bh;
    float L, Di;
    if (PK && it > 0) {
      L = ahead.x;
      Di = ahead.y;
    } else {
      L = p.lse2[(size_t)bh * p.S_pad + (I.seq.stat + i)];
      Di = p.delta[(size_t)bh * p.S_pad + (I.seq.stat + i)];
    }
    const float2 negL = make_float2(-L, -L), negD = make_float2(-Di, -Di);
    for (int kb = I.lo; kb <= I.hi; ++kb, ++u) {
      if (!(ok = mbar_wait(&sm.s_full, u & 1u, abort))) break;
      tc_fence_after_sync();
      // visible keys of query i: [klo, khi], as columns [clo, chi] of this warpgroup's
      const bool msk = bwd_needs_mask(p, I.seq, I.qb, kb);
      const int j0 = 128 * kb + Cfg::kCols * wg;
      int khi = I.seq.S - 1;
      if (p.causal) khi = min(khi, i);
      int klo = p.window > 0 ? i - p.window + 1 : 0;
      if (PK) klo = max(klo, I.seq.pad);
      int clo = klo - j0;
      const int chi = khi - j0;
      const uint32_t span = chi >= clo ? (uint32_t)(chi - clo) : 0u;
      if (chi < clo) clo = 1 << 30;

      uint32_t x[Cfg::kChunks][32];
#pragma unroll
      for (int c = 0; c < Cfg::kChunks; ++c) tmem_ld_32x32b_x32(colS + 32 * c, x[c]);
#pragma unroll
      for (int c = 0; c < Cfg::kChunks; ++c) tmem_ld_wait(x[c]);
      // S is in registers: the next S may overwrite it
      tc_fence_before_sync();
      mbar_arrive(&sm.s_free);
      float pf[Cfg::kCols];
      // (a branch around the loop, not at every pair; a masked block's loop masks as it goes:
      // 50 sequences of 300 rows 2 % faster than with the mask in a loop of its own)
      auto weights = [&](auto masked) {
#pragma unroll
        for (int e = 0; e < Cfg::kCols / 2; ++e) {
          const int col = 2 * e, c = col / 32, k = col % 32;
          const float2 xs = __ffma2_rn(
              make_float2(__uint_as_float(x[c][k]), __uint_as_float(x[c][k + 1])), sl2, negL);
          pf[col] = ex2_approx(xs.x);
          pf[col + 1] = ex2_approx(xs.y);
          if constexpr (masked) {
            pf[col] = zero_unless_le(pf[col], (uint32_t)(col - clo), span);
            pf[col + 1] = zero_unless_le(pf[col + 1], (uint32_t)(col + 1 - clo), span);
          }
        }
      };
      if (msk)
        weights(std::true_type{});
      else
        weights(std::false_type{});

      const uint32_t b = u & 1u;   // this block's dP buffer
      const uint32_t colDP = b ? colDP1 : colDP0;
      if (!(ok = mbar_wait(&sm.dp_full[b], (u >> 1) & 1u, abort))) break;
      tc_fence_after_sync();
#pragma unroll
      for (int c = 0; c < Cfg::kChunks; ++c) {
        uint32_t y[32];
        tmem_ld_32x32b_x32(colDP + 32 * c, y);
        tmem_ld_wait(y);
        uint32_t w16[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int col = 32 * c + 2 * e;
          const float2 dd = __fadd2_rn(
              make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), negD);
          const float2 ds = __fmul2_rn(make_float2(pf[col], pf[col + 1]), dd);
          w16[e] = pack_bf16x2(ds.x, ds.y);
          if (PK) {
            pf[col] = ds.x;
            pf[col + 1] = ds.y;
          }
        }
        tmem_st_32x32b_x16(colDP + 16 * c, w16);
      }
      if (PK && bwd_two_parts<PK>(p, I.qb)) {   // (as in the dK/dV pass)
#pragma unroll
        for (int c = 0; c < Cfg::kChunks; ++c) {
          uint32_t w16[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float x0 = pf[32 * c + 2 * e], x1 = pf[32 * c + 2 * e + 1];
            w16[e] = bwd_low_pair(x0, x1, pack_bf16x2(x0, x1));
          }
          tmem_st_32x32b_x16(colDP + Cfg::kCols / 2 + 16 * c, w16);
        }
      }
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(&sm.ds_full[b]);
    }
    if (!ok) break;

    // PK: the next item's statistics, an epilogue ahead
    if constexpr (PK) ahead = bwd_stats_ahead<PK>(p, it + 1, num_items, next, t, counts);

    // ---- epilogue: scale * dQ of query i, this warpgroup's chunks of the columns
    if (!(ok = mbar_wait(&sm.acc_final, (uint32_t)items & 1u, abort))) break;
    ++items;
    tc_fence_after_sync();
    const bool store = bwd_real<PK>(I.seq, i);
    const size_t row = bwd_row<PK>(I.seq, bh, i, DH, p.dq_row, p.dq_head);
#pragma unroll 1
    for (int c = wg; c < DH / 32; c += Cfg::kWG) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(lane_addr + Cfg::kColA0 + 32 * c, r);
      tmem_ld_wait(r);
      if (store) {
        if (PK && p.wide)
          bwd_store32_wide(p.dq + row + 32 * c, r, p.scale);
        else
          bwd_store32(p.dq + row + 32 * c, r, p.scale);
      }
    }
  }
}

template <int DH, int PK = 0>
__global__ void __launch_bounds__(BwdCfg<DH>::kThreads, 1)
    attn_bwd_dq(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v,
                const __grid_constant__ CUtensorMap map_do, const BwdParams p) {
  using Cfg = BwdCfg<DH>;
  using Smem = BwdQSmem<DH>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~uintptr_t(1023));
  volatile int* abort = &sm.abort_flag;
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (warp == Cfg::kWarpProducer && lane == 0) {
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
    prefetch_tensormap(&map_do);
  }
  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int i = 0; i < Smem::kStagesK; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < Smem::kStagesV; ++i) {
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 1);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.s_free, Cfg::kEW);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.dp_full[i], 1);
      mbar_init(&sm.ds_full[i], Cfg::kEW);
    }
    mbar_init(&sm.acc_final, 1);
    mbar_init(&sm.mma_done, 1);
    fence_mbarrier_init();
  }
  if (warp == Cfg::kWarpProducer) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = sm.tmem_base;
  if (tbase != 0 && threadIdx.x == 0) sm.abort_flag = 1;
  if (tbase == 0) {
    if (warp == Cfg::kWarpProducer) {
      if (lane == 0) bwd_dq_producer<DH, PK>(sm, p, &map_q, &map_k, &map_v, &map_do, abort);
    } else if (warp == Cfg::kWarpIssuer) {
      bwd_dq_issuer<DH, PK>(sm, p, abort);
    } else {
      bwd_dq_softmax<DH, PK>(sm, p, tbase, abort, warp, lane);
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == Cfg::kWarpProducer) {
    tc_fence_after_sync();
    tmem_dealloc(tbase, 512);
  }
  if (threadIdx.x == 0 && sm.abort_flag) atomicExch(p.error_word, 4);   // ATTN_ERR_TIMEOUT
  // Launched as a programmatic dependent of the dK/dV pass, this grid may run
  // beside that pass's last CTAs (it reads nothing the pass writes: only the
  // inputs and the prep kernel's D and lse2, complete before any dK/dV CTA
  // let this grid be scheduled).  It does not finish before the dK/dV pass
  // has, so that the next kernel in the stream sees dK and dV as well.
  if (threadIdx.x == 0) griddep_wait();
}

template <int DH>
constexpr size_t bwd_dkdv_smem_bytes() { return sizeof(BwdKvSmem<DH>) + 1024; }
template <int DH>
constexpr size_t bwd_dq_smem_bytes() { return sizeof(BwdQSmem<DH>) + 1024; }

}  // namespace chs
