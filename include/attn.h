/*
 * attn.h -- C ABI of the GB300 (sm_103a) scaled dot-product causal
 * multi-head self-attention library (libattn_sm103a.so).
 *
 * The operation is the one defined in "Механизм внимания"
 * (llm-arch-research.openidealab.com/textbook/attention), section
 * "Scaled dot-product attention":
 *
 *     O = softmax(Q K^T * scale + M) V        per (batch b, query head h)
 *
 * with M in {0, -inf} the mask of sections "Маскирование" (causal: key j is
 * visible to query i only if j <= i) and "Скользящее окно" (sliding window),
 * and query head h reading K/V head g(h) = floor(h / (Hq / Hkv)) as in
 * section "Виды по числу голов K/V: MHA, GQA, MQA" (Hkv == Hq is MHA,
 * Hkv == 1 is MQA).
 *
 * Conventions shared by every entry point:
 *   - Tensors are bf16, contiguous, row-major, in the layout [B, H, S, Dh]
 *     ("多头注意力机制" (blog.euler0525.cn), section "Multi-head Attention":
 *     heads moved ahead of the sequence axis).  All tensor pointers are
 *     DEVICE pointers, 16-byte aligned.  The caller owns every tensor.
 *   - Dh must be 64, 128 or 256 (the Gemma head size) for every entry
 *     point (ATTN_ERR_UNSUPPORTED otherwise).
 *   - Hq % Hkv == 0 is required (ATTN_ERR_INVALID_ARG otherwise).
 *   - scale == 0 selects 1/sqrt(Dh), the textbook's choice (divide by the
 *     square root of the HEAD size, not the model width); a positive scale is
 *     used as given; a negative or non-finite scale is ATTN_ERR_INVALID_ARG.
 *   - window <= 0 means no window.  window = W > 0 keeps key j visible to the
 *     query at position i only if i - W < j <= i: W keys including the
 *     query's own (the i - j < W form the textbook quotes from HuggingFace;
 *     the page's own rule 0 <= i - j <= W equals window W + 1 here).
 *   - Argument errors are returned before anything is launched.  Kernels run
 *     asynchronously on `stream`; a launch failure returns ATTN_ERR_CUDA.
 *     Errors found on the device (a bounded wait that gave up, an invalid
 *     sequence length) are latched in a per-device error word that
 *     attn_status() reads.  After a non-OK status the output is undefined.
 *   - The same inputs give bit-identical outputs (no atomics in any
 *     reduction; the decode split plan depends only on the arguments and
 *     the device's SM count).
 *   - Workspaces (the decode split partials and completion counters, the
 *     backward pass's per-row statistics) belong to the library, one set
 *     per device, grown under a lock and never shrunk.  They are shared by
 *     every stream of the device: calls that use them (attn_decode,
 *     attn_decode_ring, attn_bwd) may be issued from several host threads,
 *     but must not run concurrently on different streams of one device.
 *     attn_decode_noalloc uses a fixed array of its own instead, under the
 *     same rule (see there).  Growing a workspace is refused inside a
 *     stream capture (ATTN_ERR_NO_MEMORY): make one call outside the
 *     capture first.
 */
#ifndef CAUSAL_HEAD_SELF_ATTN_H_
#define CAUSAL_HEAD_SELF_ATTN_H_

#include <stddef.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1,  /* bad shape, pointer, alignment, aliasing, scale or window */
  ATTN_ERR_UNSUPPORTED = 2,  /* a head size the entry point does not take */
  ATTN_ERR_CUDA = 3,         /* a CUDA runtime or launch error */
  ATTN_ERR_TIMEOUT = 4,      /* a kernel's bounded wait gave up (reported by attn_status) */
  ATTN_ERR_NO_MEMORY = 5,    /* a library workspace could not be allocated */
  ATTN_ERR_SCRATCH_LIMIT = 6, /* attn_decode_noalloc: the call needs more than its fixed scratch */
  ATTN_ERR_CHECK = 7          /* checked builds only (ATTN_CHECK): a kernel's own range check of a
                                 copy it was about to issue failed; the copy was skipped */
} attn_status_t;

/*
 * attn_fwd -- prefill / full-sequence attention.
 *   q  [B, Hq,  S, Dh]   queries          (device, bf16, read)
 *   k  [B, Hkv, S, Dh]   keys             (device, bf16, read)
 *   v  [B, Hkv, S, Dh]   values           (device, bf16, read)
 *   o  [B, Hq,  S, Dh]   output           (device, bf16, written; must not
 *                                           overlap q, k or v)
 *   causal   1: causal mask; 0: every key visible (window must then be <= 0)
 *   window, scale: see the conventions above.
 * B == 0 or S == 0 is a no-op returning ATTN_OK.
 * Work: 4*Dh FLOPs per visible (query, key) pair per query head; wholly
 * masked tiles (128 query rows by 128 keys, or by 64 keys at Dh 256 and at
 * Dh 128 up to 1536 keys per head) are never computed.
 */
int attn_fwd(const void* q, const void* k, const void* v, void* o, int B, int Hq, int Hkv,
             int S, int Dh, int causal, int window, float scale, cudaStream_t stream);

/*
 * attn_fwd_lse -- attn_fwd that also writes each query row's log-sum-exp,
 *   lse  [B, Hq, S]  (device, fp32, written; 4-byte aligned, must not
 *                     overlap the other tensors)
 *   lse[b, h, i] = log sum_j exp(s_ij) over the visible keys j, natural log,
 *   with s_ij = scale * q_i . k_j the scaled score (the softmax
 *   normaliser of "Механизм внимания", section "Scaled dot-product
 *   attention", in log form).  attn_bwd recomputes the weights from it.
 * o is bit-identical to attn_fwd's.  lse == NULL is ATTN_ERR_INVALID_ARG
 * (unless B == 0 or S == 0, a no-op).
 */
int attn_fwd_lse(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                 int Hkv, int S, int Dh, int causal, int window, float scale,
                 cudaStream_t stream);

/*
 * attn_bwd -- backward pass of attn_fwd: the gradients of a loss L with
 * respect to q, k and v, given dout = dL/do.  The chain rule through the
 * definition, with the softmax derivative dp_i/dz_j = p_i (delta_ij - p_j)
 * of "Механизм внимания", section "Почему делить на корень из d_h"; the
 * weights are recomputed block by block from lse (section "Эффективные
 * реализации": FlashAttention recomputes them in the backward pass):
 *     dV = P^T dO,  dS = P o (dO V^T - D),  D_i = dO_i . o_i,
 *     dQ = scale dS K,  dK = scale dS^T Q.
 *   q, k, v, causal, window, scale  exactly as passed to attn_fwd_lse
 *   o     [B, Hq,  S, Dh]  attn_fwd_lse's output       (device, bf16, read)
 *   dout  [B, Hq,  S, Dh]  dL/do                       (device, bf16, read)
 *   lse   [B, Hq,  S]      attn_fwd_lse's lse          (device, fp32, read)
 *   dq    [B, Hq,  S, Dh]  dL/dq                       (device, bf16, written)
 *   dk    [B, Hkv, S, Dh]  dL/dk, summed over the query heads of each group
 *   dv    [B, Hkv, S, Dh]  dL/dv, likewise             (device, bf16, written)
 * dq, dk and dv must not overlap each other or any input.  Dh must be 64,
 * 128 or 256 (ATTN_ERR_UNSUPPORTED otherwise).  The result is deterministic
 * (no atomics): at Dh 64 and 128 one pass computes dK and dV per key block, a
 * second dQ per query block; at Dh 256, where a 256-column accumulator fills
 * half of tensor memory, dV, dK and dQ each take a pass of their own.
 * Per-row intermediates live in a library-owned device workspace
 * (8 bytes per query row, allocated on first use and grown on demand,
 * ATTN_ERR_NO_MEMORY if that fails); backward calls that overlap on the GPU
 * race on it.  B == 0 or S == 0 is a no-op.
 * Work: 10*Dh FLOPs per visible (query, key) pair per query head (S
 * recomputed, dP, dV, dQ, dK: 2*Dh each), 2.5 x attn_fwd's; the kernels
 * execute 14*Dh (S and dP are computed in both passes; at Dh 256, 16*Dh:
 * S in all three passes, dP in two).
 */
int attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
             const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int S, int Dh,
             int causal, int window, float scale, cudaStream_t stream);

/*
 * attn_fwd_chunk -- prefill of one chunk against a KV cache ("Механизм
 * внимания", section "Prefill и decode": a long prompt may be fed in chunks;
 * the chunk's keys and values are written into the cache first, then its
 * queries attend to everything cached before them and to the chunk).
 *   q       [B, Hq, Sq, Dh]     the chunk's queries        (device, bf16, read)
 *   kcache  [B, Hkv, Tmax, Dh]  cached keys                (device, bf16, read)
 *   vcache  [B, Hkv, Tmax, Dh]  cached values              (device, bf16, read)
 *   o       [B, Hq, Sq, Dh]     output                     (device, bf16, written;
 *                                                           must not overlap the others)
 *   start_pos  position of the chunk's first token; the chunk's own keys
 *              are cache rows start_pos .. start_pos + Sq - 1, and only rows
 *              [0, start_pos + Sq) are read (0 <= start_pos, start_pos + Sq <= Tmax).
 * Query row r sits at position start_pos + r and, with causal = 1, sees keys
 * 0 .. start_pos + r (the window, if any, as in attn_fwd); with causal = 0
 * every key 0 .. start_pos + Sq - 1.  start_pos = 0 and Tmax = Sq is exactly
 * attn_fwd (the same kernel and bits).  Errors and the empty case (B == 0 or
 * Sq == 0) as in attn_fwd.
 */
int attn_fwd_chunk(const void* q, const void* kcache, const void* vcache, void* o, int B, int Hq,
                   int Hkv, int Sq, int Tmax, int start_pos, int Dh, int causal, int window,
                   float scale, cudaStream_t stream);

/*
 * attn_decode -- one KV-cache decode step ("Механизм внимания", section
 * "Prefill и decode": the new token's key and value are appended to the
 * cache first, then its query meets every cached key, its own included).
 *   q        [B, Hq, 1, Dh]     the new tokens' queries   (device, bf16, read)
 *   kcache   [B, Hkv, Tmax, Dh] cached keys               (device, bf16, read)
 *   vcache   [B, Hkv, Tmax, Dh] cached values             (device, bf16, read)
 *   seqlens  [B]                keys held per sequence, 1 <= seqlens[b] <= Tmax
 *                               (device, int32, read).  Only rows
 *                               [0, seqlens[b]) of a cache are read.
 *   o        [B, Hq, 1, Dh]     output (device, bf16, written)
 * The query of sequence b sits at position seqlens[b] - 1 and sees keys
 * [max(0, seqlens[b] - window), seqlens[b]) (all of them when window <= 0).
 * A seqlens entry outside [1, Tmax] zeroes that sequence's output and latches
 * ATTN_ERR_INVALID_ARG for attn_status().
 * With Hq / Hkv >= 2 (GQA and MQA) the step runs on the tensor cores (the
 * group's query heads packed as the rows of one contraction with each key
 * tile) followed by a small combine kernel (a programmatic dependent launch
 * on the same stream); with one query head per K/V head (MHA) on the CUDA
 * cores, whose last CTA per head merges the splits.
 * The split-KV partials live in a library-owned device workspace, allocated
 * on first use per device and grown on demand (cudaMalloc): make the first
 * call with the largest shape outside any CUDA graph capture.  Calls on one
 * device share that workspace, so decode calls that overlap on the GPU
 * (different streams, no ordering) race.
 * B == 0 is a no-op returning ATTN_OK.
 */
int attn_decode(const void* q, const void* kcache, const void* vcache, const int* seqlens,
                void* o, int B, int Hq, int Hkv, int Tmax, int Dh, int window, float scale,
                cudaStream_t stream);

/*
 * attn_decode_ring -- the decode step over a rolling-buffer cache
 * ("Механизм внимания", section "Скользящее окно": with a window the cache
 * need only hold the last W positions, and a ring buffer does that).
 *   kcache, vcache [B, Hkv, C, Dh]: position t of sequence b is at row t % C
 *                  (the last min(seqlens[b], C) positions are held).
 *   seqlens [B]    tokens of sequence b so far, own token included (>= 1,
 *                  any size below 2^31 - C); the query sits at position
 *                  seqlens[b] - 1.
 *   window         W <= C: keys [seqlens[b] - W, seqlens[b]) are visible;
 *                  window <= 0 means W = C (every held position).
 *                  window > C is ATTN_ERR_INVALID_ARG.
 * Other arguments, the workspace and the errors as in attn_decode.  While a
 * sequence has not wrapped (seqlens[b] <= C) and window <= 0 the result is
 * bit-identical to attn_decode on the same buffers.
 */
int attn_decode_ring(const void* q, const void* kcache, const void* vcache, const int* seqlens,
                     void* o, int B, int Hq, int Hkv, int C, int Dh, int window, float scale,
                     cudaStream_t stream);

/*
 * attn_decode_noalloc -- the same decode step as attn_decode (same arguments,
 * same result up to rounding, same errors), for callers that must not
 * allocate device memory.  The pages describe no such call; it exists for
 * this library's users.  A serving runtime that reserves nearly all device
 * memory up front for its own KV-cache pool, or a process that runs under a
 * fixed device-memory budget, cannot let a library allocate behind its back:
 * an allocation there can fail, and cudaMalloc / cudaFree also stall on the
 * device.  attn_decode allocates its workspace on first use; this entry point
 * calls no cudaMalloc, cudaFree or other allocating routine.
 *   - Its scratch (split partials and completion counters) is one fixed
 *     16 MiB device array inside this library.  Every GPU that loads the
 *     library holds it until the process exits.
 *   - It runs the kernels attn_decode runs for the same arguments (the
 *     tensor-core path for Hq / Hkv >= 2 at every head size, the CUDA-core
 *     path otherwise), with the same split plan, so the results are the
 *     same bits.
 *   - On the CUDA-core path a call needs 4*B*Hq bytes of counters (one per
 *     query head, rounded up to 256 bytes) plus
 *     B*Hq*nsplit*(Dh+2)*4 bytes of partials (each part rounded up to 256),
 *     where nsplit is the split count attn_decode would use; on the
 *     tensor-core path only the partials.  A call that needs more than
 *     16 MiB returns ATTN_ERR_SCRATCH_LIMIT before anything runs.  (The
 *     B=16, Hq=32, Hkv=8, Tmax=32768, Dh=128 decode step needs about 4.3 MB.)
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress); make that first call before any stream capture.
 *   - Every call shares the one array, which keeps the previous call's
 *     contents; each call clears the counters it uses (cudaMemsetAsync on
 *     `stream`).  Calls that overlap on the GPU (on different streams with no
 *     ordering between them) race on the array and give wrong results.
 */
int attn_decode_noalloc(const void* q, const void* kcache, const void* vcache,
                        const int* seqlens, void* o, int B, int Hq, int Hkv, int Tmax, int Dh,
                        int window, float scale, cudaStream_t stream);

/*
 * The paged key-value cache.  A serving runtime that holds many sequences of
 * different and growing lengths keeps their keys and values in pages of one
 * pool instead of a [B, Hkv, Tmax, Dh] block per sequence:
 *   kpages, vpages [num_pages, Hkv, page, Dh]  the pools (device, bf16)
 *   table          [B, cols]  page numbers (device, int32): row t of sequence
 *                  b is row t % page of page table[b * cols + t / page]
 *   seqlens        [B]        keys held per sequence (device, int32)
 * `page` is a multiple of 8 (ATTN_ERR_UNSUPPORTED otherwise).  A linear cache
 * [B, Hkv, Tmax, Dh] is the special case of num_pages = B, page = Tmax,
 * cols = 1, table = 0 .. B - 1.  In every call below:
 *   - A length of 0 is a sequence without keys (an empty slot of a padded
 *     batch): nothing of it is read or written but a zero output.  A length
 *     outside [0, cols * page] latches ATTN_ERR_INVALID_ARG for attn_status().
 *   - Only table entries of rows that the call uses are read; the others may
 *     hold anything.  An entry outside [0, num_pages) that is used latches
 *     ATTN_ERR_INVALID_ARG (nothing outside the pools is touched).  Sequences
 *     may share pages that the call only reads; a page that it writes must
 *     belong to one sequence and appear there once (the contents are
 *     undefined otherwise).
 *   - Rows outside a sequence's visible keys are never used, whatever they
 *     hold (infinities and NaN included), and rows that the call does not
 *     write keep their bits.
 *   - The library keeps no workspace for these calls: they may run at the
 *     same time on several streams and in several captured graphs, each with
 *     its own workspace where one is asked for.
 */

/*
 * attn_paged_append -- write new keys and values to the cache.
 *   k, v     [B, Hkv, S, Dh]  new rows (device, bf16, read)
 *   seqlens  [B]  keys held AFTER the append
 *   newlens  [B]  rows of k and v that are real, the first newlens[b] of S
 *                 (device, int32, or NULL: all S), 0 <= newlens[b] <=
 *                 min(S, seqlens[b]); another value latches
 *                 ATTN_ERR_INVALID_ARG and appends nothing to the sequence
 * Row i becomes row seqlens[b] - newlens[b] + i of sequence b.  With S = 1 the
 * call is a decode step's append (seqlens as attn_decode_paged takes them).
 * With NULL a length below S latches the error too, except 0 (an empty slot).
 */
int attn_paged_append(const void* k, const void* v, void* kpages, void* vpages, const int* table,
                      const int* seqlens, const int* newlens, int B, int Hkv, int S, int num_pages,
                      int page, int cols, int Dh, cudaStream_t stream);

/*
 * attn_decode_paged -- attn_decode over a paged cache: one query per sequence,
 * at position seqlens[b] - 1, against keys [max(0, seqlens[b] - window),
 * seqlens[b]) (all of them when window <= 0).
 *   q, o     [B, Hq, 1, Dh]  queries, output (device, bf16; o is all zero
 *                            for a length of 0)
 *   weights  [B, Hkv, weights_stride] (device, fp32) or NULL: the softmax
 *            weight of each key, summed over the query heads of its K/V head,
 *            is added to weights[b, g, t] (accumulate = 1) or stored there
 *            (accumulate = 0, which also stores 0 for keys before the
 *            window), for t < seqlens[b]; entries from seqlens[b] on are left
 *            as they are.  weights_stride >= cols * page.
 *   workspace  device, 256-byte aligned, of at least the bytes that
 *            attn_decode_paged_workspace gives for the same shapes
 *            (ATTN_ERR_SCRATCH_LIMIT otherwise).  Its contents need not be
 *            kept between calls; calls that may overlap on the GPU need one
 *            each.
 * Any Hq / Hkv runs on the tensor cores.  The same inputs give the same bits.
 * Where the softmax weights meet V they are held to 2^-14 of each (two bf16
 * parts) with up to 16 query heads per K/V head, and rounded to bf16 (2^-8, as
 * in attn_fwd and attn_decode) with more.  Their sum, and `weights`, are of
 * fp32 ones.
 * An infinity in a visible V row can make that column of the output NaN (a key
 * may also meet weights of exactly 0 in the tensor-core product).
 */
int attn_decode_paged(const void* q, const void* kpages, const void* vpages, const int* table,
                      const int* seqlens, void* o, float* weights, int weights_stride,
                      int accumulate, void* workspace, size_t workspace_bytes, int B, int Hq,
                      int Hkv, int num_pages, int page, int cols, int Dh, int window, float scale,
                      cudaStream_t stream);

/* The workspace of an attn_decode_paged call on the current device, in bytes:
 * partial results, and with weights the step's scores (4 bytes for each query
 * head and row that the table has room for).  0 for a small table without
 * weights: the workspace may be NULL then. */
int attn_decode_paged_workspace(int B, int Hq, int Hkv, int page, int cols, int Dh,
                                int with_weights, size_t* bytes);

/*
 * attn_key_weights -- the attention weight that the keys of a prompt received:
 *   weights[b, g, j] (+)= sum over query heads h of K/V head g and voting
 *                         queries i that see key j of exp(s_hij - lse[b, h, i])
 * with s the scaled scores of attn_fwd_lse and lse its log-sum-exps, so that
 * each term is a softmax weight.  Nothing of size S x S is stored.
 *   q, k     [B, Hq | Hkv, S, Dh]   as attn_fwd_lse took them (device, bf16)
 *   lse      [B, Hq, S]             (device, fp32); only voting rows are read
 *   seqlens  [B] or NULL            real rows of a padded prompt, in [0, S]
 *                                   (device, int32; NULL: all S)
 *   weights  [B, Hkv, weights_stride]  (device, fp32), weights_stride >= S;
 *            entries [0, seqlens[b]) are written, the others left alone
 *   queries  the last `queries` rows of each sequence vote (0 or more than
 *            there are: every row)
 *   causal, window, scale  as in attn_fwd_lse (a scale below 1e-18 is
 *            ATTN_ERR_INVALID_ARG here);  accumulate as above
 * (With causal = 0 a padded prompt's lse has to be that of its real rows.)
 * Infinities and NaN in q, k and lse give what the formula gives, to the keys
 * that see them alone: a voting row with lse = +inf weighs nothing.
 */
int attn_key_weights(const void* q, const void* k, const float* lse, const int* seqlens,
                     float* weights, int weights_stride, int B, int Hq, int Hkv, int S, int Dh,
                     int queries, int causal, int window, int accumulate, float scale,
                     cudaStream_t stream);

/*
 * attn_cache_evict -- shrink each sequence of a paged cache to at most
 * `budget` keys.  A sequence of n > budget keys keeps, for each K/V head on
 * its own, the last `recent` rows and, of the rows before them, the
 * budget - recent with the largest weights (equal weights: the lower row; NaN
 * counts below every number).  The kept rows keep their order and become rows
 * 0 .. budget - 1; keys were rotated by position before they were cached, if
 * at all, so attention does not see the move.  Shorter sequences keep all.
 *   weights      [B, Hkv, weights_stride]  accumulated weights (device, fp32);
 *                weights_stride >= cols * page
 *   seqlens      [B]  read
 *   table_out    [B, cols_out]  pages that receive the kept rows; they must not
 *                be among the pages in use by the sequences' rows.  NULL (or
 *                table itself): in place.
 *   weights_out  [B, Hkv, weights_out_stride]  receives the kept rows' weights,
 *                and zeros in entries [newlens[b], seqlens[b]), so that rows
 *                appended later start from nothing.  NULL (or weights itself):
 *                in place.
 *   newlens      [B]  written: min(seqlens[b], budget).  Not seqlens itself.
 *   keep         [B, Hkv, budget]  written: the former row of each kept row,
 *                ascending, then -1
 * 1 <= budget <= 2^31 - 16385, 0 <= recent <= budget, and cols_out * page and
 * weights_out_stride hold min(budget, cols * page) rows
 * (ATTN_ERR_INVALID_ARG otherwise).  A length outside its range leaves the
 * sequence alone.
 */
int attn_cache_evict(void* kpages, void* vpages, float* weights, int weights_stride,
                     const int* table, const int* seqlens, int budget, int recent,
                     const int* table_out, int cols_out, float* weights_out,
                     int weights_out_stride, int* newlens, int* keep, int B, int Hkv, int num_pages,
                     int page, int cols, int Dh, cudaStream_t stream);

/*
 * Packed sequences.  A batch of sequences of different lengths lies one behind
 * another, without padding: tokens are rows of [T, H, Dh], and sequence b holds
 * rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (device, int32, [B + 1],
 * ascending within [0, T]; a length of 0 is an empty place).  Rows of no
 * sequence (ahead of the first, behind the last) are neither used, whatever
 * they hold, nor written.  Tensors come at any strides of whole 16 bytes, so
 * that a projection's output [T, Hq + 2 Hkv, Dh] is taken as it lies, and
 * heads-first tensors [H, T, Dh] too:
 */
typedef struct {
  void* data;             /* device, bf16, 16-byte aligned (inputs are only read) */
  /* elements (multiples of 8) between batches, rows and heads; an axis of one
     entry has any.  The packed calls have no batch axis.  The Dh values of a
     head lie side by side. */
  long long batch_stride, row_stride, head_stride;
} attn_rows_t;
/*
 * In the packed calls below:
 *   - Strides are at least Dh.  The elements of an output are distinct, and
 *     apart from every other tensor's (ATTN_ERR_INVALID_ARG otherwise);
 *     tensors between one another (slices of one wider tensor along its heads,
 *     or along an axis around or inside them) are apart.
 *   - Offsets that are not ascending within [0, T] latch ATTN_ERR_INVALID_ARG
 *     for attn_status(), and nothing is written.
 *   - workspace: device, 256-byte aligned, of at least the bytes that the
 *     query gives (ATTN_ERR_SCRATCH_LIMIT otherwise).  Its contents need not be
 *     kept; calls that may overlap on the GPU need one each.  The library keeps
 *     none, so the calls may run on several streams at the same time and in
 *     several captured graphs.
 *   - No sequence's result depends on another's rows, infinities and NaN
 *     included.  Within a sequence an infinity or NaN in a row (of K and V, in
 *     the backward pass of any tensor) can reach the rows of its 128-row block
 *     that the mask hides it from, as in attn_fwd and attn_bwd.
 *   - The same inputs give the same bits.
 *   - Which kernels run goes by T / B, the rows per sequence with the rows of
 *     no sequence and the empty places counted.  It costs time where a few long
 *     sequences stand among many empty places, or short ones in a long buffer.
 *   - B == 0 or T == 0 is a no-op.
 */

/*
 * attn_fwd_packed -- attn_fwd of every sequence: row i of a sequence sees its
 * own rows j <= i (causal = 1; i - j < window where a window is given) or all
 * of them (causal = 0).
 *   q, o  [T, Hq, Dh],  k, v  [T, Hkv, Dh]
 *   lse   [Hq, T]  (device, fp32, written) or NULL: as in attn_fwd_lse
 * Where the softmax weights meet V they are rounded to bf16 (2^-8 of each, as
 * in attn_fwd); their sum, and lse, are of fp32 ones.
 * Work is listed on the GPU, so the call reads no lengths on the host.
 */
int attn_fwd_packed(const attn_rows_t* q, const attn_rows_t* k, const attn_rows_t* v,
                    const attn_rows_t* o, float* lse, const int* cu_seqlens, void* workspace,
                    size_t workspace_bytes, int B, int Hq, int Hkv, int T, int Dh, int causal,
                    int window, float scale, cudaStream_t stream);

/* The workspace of an attn_fwd_packed call on the current device, in bytes, with any number of
 * K/V heads: a list of blocks; 0 for causal calls of few sequences, whose workspace may be
 * NULL. */
int attn_fwd_packed_workspace(int B, int Hq, int T, int Dh, int causal, size_t* bytes);

/*
 * attn_bwd_packed -- attn_bwd of every sequence: dq [T, Hq, Dh], dk and dv
 * [T, Hkv, Dh] (summed over the query heads of each group) from q, k, v, the
 * o and lse that attn_fwd_packed gave for them, and dout = dL/do.
 * P and dS enter their products rounded to bf16 (2^-8 of each, as in attn_bwd),
 * but in two bf16 parts (2^-16) for the queries of a sequence's first two
 * 128-row blocks, of which the first is the short one, and for all under a
 * window of up to 256.
 * D_i is dO_i . o_i with o as it was rounded, but for queries whose keys all
 * lie within 32 rows (causal: a sequence's first 32 rows, and all under a
 * window of up to 32; else all of a sequence of up to 32) it is
 * sum_j p_ij dP_ij / sum_j p_ij, and o is not used.  So o and lse that were
 * joined from several sets of keys, of which k and v are one, do not give that
 * set's part of the gradient here (in attn_bwd they do).
 */
int attn_bwd_packed(const attn_rows_t* q, const attn_rows_t* k, const attn_rows_t* v,
                    const attn_rows_t* o, const attn_rows_t* dout, const float* lse,
                    const attn_rows_t* dq, const attn_rows_t* dk, const attn_rows_t* dv,
                    const int* cu_seqlens, void* workspace, size_t workspace_bytes, int B, int Hq,
                    int Hkv, int T, int Dh, int causal, int window, float scale,
                    cudaStream_t stream);

/* The workspace of an attn_bwd_packed call, in bytes. */
int attn_bwd_packed_workspace(int B, int Hq, int T, size_t* bytes);

/*
 * attn_rope -- rotary positions.  Of each head of q and k the first rotary_dim
 * values (a multiple of 16, at most Dh; 0: none) are turned in pairs: at
 * position p, pair i by the angle 2 pi p turns[i] / 2^64,
 *     (x, y) -> amplitude (x cos - y sin, y cos + x sin).
 *   interleaved = 0: pair i is values i and i + rotary_dim / 2;
 *   interleaved = 1: values 2 i and 2 i + 1.
 *   q, q_out  [B, S, Hq, Dh], k, k_out  [B, S, Hkv, Dh], each at its own
 *         strides: packed tokens with B = 1, heads-first batches
 *         [B, H, S, Dh] as they lie.  An output is its input or apart from
 *         every tensor.  Inputs may have strides of 0.  Hq or Hkv may be 0.
 *   positions  [B, S]  (device, int32); a negative one leaves the row out:
 *         nothing of it is written
 *   turns  [rotary_dim / 2]  (device, 64-bit, 8-byte aligned): turns per token
 *         in units of 2^-64, as attn_rope_frequencies makes them.  p turns[i]
 *         is reduced to one turn exactly, whatever the position.
 *   inverse = 1: the other way, as a gradient goes back (with the same
 *         amplitude)
 * The turned values are computed in fp32 and rounded once.
 */
int attn_rope(const attn_rows_t* q, const attn_rows_t* q_out, int Hq, const attn_rows_t* k,
              const attn_rows_t* k_out, int Hkv, const int* positions,
              const unsigned long long* turns, float amplitude, int B, int S, int Dh,
              int rotary_dim, int interleaved, int inverse, cudaStream_t stream);

/*
 * attn_rope_append -- attn_rope, and the write to a paged cache in the same
 * pass: the turned k and v [B, S, Hkv, Dh] of row r go to row slots[r] % page
 * of page slots[r] / page of the pools (see above; any page size that is a
 * multiple of 8).
 *   slots  [B, S]  (device, int32): attn_cache_plan gives them; a negative one
 *         writes nothing to the cache, one of num_pages * page or more latches
 *         ATTN_ERR_INVALID_ARG and writes nothing there either.  Two rows have
 *         one slot in no call.
 *   k_out  NULL: the turned keys go to the cache alone
 * A row with a negative position is left out altogether.
 */
int attn_rope_append(const attn_rows_t* q, const attn_rows_t* q_out, int Hq, const attn_rows_t* k,
                     const attn_rows_t* k_out, const attn_rows_t* v, int Hkv, const int* positions,
                     const unsigned long long* turns, float amplitude, void* kpages, void* vpages,
                     const int* slots, int num_pages, int page, int B, int S, int Dh,
                     int rotary_dim, int interleaved, cudaStream_t stream);

/*
 * attn_rope_frequencies -- turns per token of each pair, and the amplitude:
 * f_i = base^(-2 i / rotary_dim) / (2 pi), for longer contexts scaled by
 *   ATTN_ROPE_LINEAR  f_i / factor (positions pressed together);
 *   ATTN_ROPE_BASE    base * factor^(rotary_dim / (rotary_dim - 2)) for base;
 *   ATTN_ROPE_TURNS   by the turns r = original_len f_i that a pair makes over
 *                     the context it was trained on: f_i from r = high on,
 *                     f_i / factor up to r = low, linear in r between them;
 *   ATTN_ROPE_YARN    the same, with amplitude 0.1 ln(factor) + 1.
 * (The blend is linear in r, as YaRN was published.  A model whose own code
 * blends linearly in the pair's number i, between two rounded numbers, has
 * other frequencies: give attn_rope those, made on the host.)
 * A host call: turns [rotary_dim / 2] and amplitude are host memory.
 */
enum { ATTN_ROPE_NONE = 0, ATTN_ROPE_LINEAR, ATTN_ROPE_BASE, ATTN_ROPE_TURNS, ATTN_ROPE_YARN };
int attn_rope_frequencies(unsigned long long* turns, float* amplitude, int rotary_dim, double base,
                          int scaling, double factor, double low, double high,
                          double original_len);

/*
 * attn_cache_plan -- the pages, slots and positions of a serving step, made on
 * the GPU from the lengths alone (no length is read on the host).  Sequence b
 * of a paged cache holds seqlens[b] rows and changes by delta[b]: so many new
 * tokens, or (negative) rows taken back from its end.
 *   1. Pages that no row needs any more go onto the stack of free pages, by
 *      sequence, then by column.
 *   2. Pages that new rows need come off its top, in the same order, into the
 *      table.
 *   3. The new tokens of all sequences, packed in their order, get their
 *      position and their slot (page number * page + row in the page).
 *   delta, seqlens     [B]           (device, int32, read)
 *   seqlens_out        [B]           written: seqlens + delta; may be seqlens
 *   table              [B, cols]     columns that a sequence gains are written
 *   free_pages         [capacity]    the stack; its first *num_free entries are
 *                                    free pages, entries that it gains are written
 *   num_free, num_free_out  [1]      its height before and after; may be the same
 *   cu_seqlens         [B + 1]       written: first packed row of each
 *                                    sequence's new tokens, then their number
 *   positions, slots   [T]           written: for each packed row, then -1 (of
 *                                    more than T new tokens, the first T's)
 * (all device, int32).  All or nothing: where the stack would pass capacity
 * (ATTN_ERR_INVALID_ARG) or free pages do not suffice (ATTN_ERR_NO_MEMORY, both
 * latched for attn_status()), lengths, table and stack stay as they were,
 * cu_seqlens is all 0 and the rest -1.  A
 * length outside [0, cols * page], before or after, latches
 * ATTN_ERR_INVALID_ARG and leaves that sequence as it is.  A used page number
 * outside [0, num_pages) latches it too and gives slots of -1.
 * A page that is given back belongs to one sequence.  Attention of the new
 * tokens is attn_fwd_packed's where their sequences held nothing before, and
 * attn_decode_paged's of one token per sequence; several tokens of a sequence
 * that holds rows already are planned and written, but no call attends from
 * them to the pages.  Up to 8192 sequences
 * (ATTN_ERR_UNSUPPORTED).  B == 0 is a step of no tokens: cu_seqlens[0] is 0,
 * positions and slots are -1.
 */
int attn_cache_plan(const int* delta, const int* seqlens, int* seqlens_out, int* table,
                    int* free_pages, const int* num_free, int* num_free_out, int* cu_seqlens,
                    int* positions, int* slots, int B, int cols, int page, int num_pages,
                    int capacity, int T, cudaStream_t stream);

/*
 * attn_status -- synchronise `stream`, then return (and clear) the current
 * device's latched error word: ATTN_OK, ATTN_ERR_TIMEOUT, ATTN_ERR_INVALID_ARG,
 * or ATTN_ERR_CUDA if the synchronisation itself failed (or a prefill kernel
 * found its dynamic shared memory not 1024-byte aligned and wrote nothing).
 */
int attn_status(cudaStream_t stream);

/*
 * attn_debug_inject_fault -- test hook for the failure path; the pages
 * describe no such call.  Every later attn_fwd / attn_decode /
 * attn_decode_noalloc / attn_bwd launch (attn_fwd_packed as attn_fwd,
 * attn_bwd_packed as attn_bwd) in this process runs with the given fault until
 * it is reset with kind 0:
 *   0  none (the default)
 *   1  attn_fwd: the producer never loads the first K tile of each CTA's
 *      first work item, so the MMA issuers' bounded waits run out
 *   2  attn_decode (CUDA-core path, Hq == Hkv): the producer never loads the
 *      first key block of each CTA
 *   3  attn_decode (tensor-core path, Hq / Hkv >= 2): the producer never loads
 *      the first K tile of each CTA
 *   4  attn_bwd: the dK/dV pass's producer never loads the K/V block of each
 *      CTA's first work item
 * A faulted launch ends by itself after its waits give up (about 2 s): no
 * GPU fault, trap or hang.  attn_status() then returns ATTN_ERR_TIMEOUT and
 * clears it; the outputs of that launch are undefined, and the next launch
 * without a fault is correct (the decode completion counters are left at
 * zero).  Returns ATTN_OK, or ATTN_ERR_INVALID_ARG for an unknown kind.
 * Not for production use: the setting is process-wide and unsynchronised
 * with launches already queued.
 */
int attn_debug_inject_fault(int kind);

/* attn_error_string -- a static, human-readable name for a status code. */
const char* attn_error_string(int code);

/* attn_version -- library ABI version, (major << 16) | minor. */
int attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CAUSAL_HEAD_SELF_ATTN_H_ */
