/*
 * sigattn.h -- C ABI of the B200 (sm_100a) sigmoid-attention library.
 *
 * The library computes bidirectional sigmoid attention over ragged, padded
 * batches ("Better Models, Faster Training: Sigmoid Attention for single-cell
 * Foundation Models", sec. 2A):
 *
 *     O = sigma(Q K^T / sqrt(d) + b) V,   sigma(x) = 1/(1+e^-x),   b = -ln(n_b)
 *
 * and its gradient with respect to Q, K and V (sec. 2B: sigma' = sigma(1-sigma);
 * sec. 2C: one kernel for dQ and one for dK/dV, activations recomputed, no
 * atomics). n_b is the valid length of sequence b; tokens at positions >= n_b
 * are padding and are ignored on both the query and the key side (sec. 2C,
 * native padding support): P_ij = 0 unless i < n_b and j < n_b.
 *
 * Conventions shared by every call
 *  - Tensors Q, K, V, dO, O, dQ, dK, dV are bf16, contiguous [B][H][Lmax][d]
 *    (d fastest), in device memory, 16-byte aligned. d must be 64 or 128.
 *  - lengths is int32 [B] in device memory; each n_b must lie in [0, Lmax].
 *    A value outside that range is treated as 0 (all outputs of sequence b
 *    are zero) and raises SIGATTN_ERR_INVALID_ARG in the workspace's sticky
 *    error word (read it with sigattn_read_error).
 *  - Outputs are fully written: rows i >= n_b of O, dQ, dK and dV are exact
 *    zeros. Values in padded rows of the inputs never change an output, but
 *    must be finite: a padded value v enters a valid result only as 0 * v
 *    inside the tensor-core sums (the discarded results of padded rows
 *    themselves may use it).
 *  - The scale is 1/sqrt(d) and the bias -ln(n_b) is computed in-kernel; the
 *    bias has no gradient. There is no causal mask.
 *  - Arithmetic: bf16 operands, fp32 accumulation, P (and dS) rounded to bf16
 *    before the second matrix product, outputs rounded to nearest bf16. sigma
 *    takes one hardware exp2 per score: with u = e^-|x|, sigma(x) = u r(u)
 *    for x < 0 and r(u) for x >= 0, where r is a polynomial for 1/(1+u) of
 *    relative error <= 8e-4 (about 1e-7 for the tail weights near 1/n that
 *    the bias -ln n makes typical); see sigattn_eval_sigmoid.
 *  - workspace: caller-owned device memory of at least
 *    sigattn_workspace_size(B, H, Lmax, d) bytes, 16-byte aligned. Each call
 *    writes its work list there; calls that may run concurrently (different
 *    streams) need different workspaces. Word 0 is a sticky error status, so
 *    zero the workspace once after allocating it (cudaMemset); the library
 *    keeps it consistent afterwards.
 *  - stream: a cudaStream_t (NULL = legacy default stream). Calls only
 *    enqueue work: they neither allocate nor synchronise, so a sequence of
 *    calls can be captured into a CUDA graph and replayed (make one call on
 *    the device outside the capture first: it sets up per-device kernel
 *    attributes).
 *  - Return value: a sigattn_status. Argument errors are reported before
 *    anything is enqueued. A kernel-side timeout (a bounded wait that gave up)
 *    is recorded in the workspace and surfaces through sigattn_read_error.
 *  - Outputs must not overlap the inputs or each other: the kernels read
 *    input tiles while other tiles of the outputs are being written.
 *  - Ownership: the library keeps no pointer after a call returns.
 */
#ifndef SIGATTN_H_
#define SIGATTN_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SIGATTN_API __attribute__((visibility("default")))
#else
#define SIGATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SIGATTN_OK = 0,
  SIGATTN_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size, bad length */
  SIGATTN_ERR_UNSUPPORTED = 2, /* d not in {64, 128}, or a size beyond the limits */
  SIGATTN_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed */
  SIGATTN_ERR_TIMEOUT = 4      /* a kernel's bounded wait expired (sticky, in the workspace) */
} sigattn_status;

/* Work-list kinds (used by the plan helpers). */
enum { SIGATTN_KIND_FWD = 0, SIGATTN_KIND_DQ = 1, SIGATTN_KIND_DKDV = 2 };

/* Limits: 1 <= B <= SIGATTN_MAX_BATCH, 1 <= H, 1 <= Lmax <= SIGATTN_MAX_LEN. */
#define SIGATTN_MAX_BATCH 4096
#define SIGATTN_MAX_LEN (1 << 20)

/* Library version, e.g. 100 for 0.1.0. */
SIGATTN_API int sigattn_version(void);

/* Human-readable name of a status code (static string). */
SIGATTN_API const char* sigattn_status_str(int status);

/* Rows of one work item for a kind: 256 (forward), 128 (dQ), 128 (dK/dV).
 * Returns -1 for an unknown kind. */
SIGATTN_API int sigattn_block_rows(int kind);

/* Bytes of workspace needed for any of the three calls with these sizes
 * (a 256-byte header plus one 16-byte entry per possible work item).
 * Returns 0 if the sizes are out of range. */
SIGATTN_API size_t sigattn_workspace_size(int B, int H, int Lmax, int d);

/* Forward pass (sec. 2A): o = sigma(q k^T / sqrt(d) - ln n) v.
 * q, k, v: inputs; o: output. All [B][H][Lmax][d] bf16 on the device. */
SIGATTN_API int sigattn_fwd(const void* q, const void* k, const void* v, void* o, const int32_t* lengths, int B, int H,
                int Lmax, int d, void* workspace, size_t workspace_bytes, void* stream);

/* Backward pass, query side (sec. 2B/2C): dq = (1/sqrt(d)) * dS k with
 * dS = (dout v^T) * P * (1 - P). dout is the gradient of the loss w.r.t. o. */
SIGATTN_API int sigattn_bwd_dq(const void* q, const void* k, const void* v, const void* dout, void* dq,
                   const int32_t* lengths, int B, int H, int Lmax, int d, void* workspace,
                   size_t workspace_bytes, void* stream);

/* Backward pass, key/value side (sec. 2B/2C): dk = (1/sqrt(d)) * dS^T q and
 * dv = P^T dout. */
SIGATTN_API int sigattn_bwd_dkdv(const void* q, const void* k, const void* v, const void* dout, void* dk, void* dv,
                     const int32_t* lengths, int B, int H, int Lmax, int d, void* workspace,
                     size_t workspace_bytes, void* stream);

/* The whole backward pass in one call: dq as sigattn_bwd_dq, dk and dv as
 * sigattn_bwd_dkdv, with identical results (the same kernels, each with one
 * owner per output block and a fixed summation order). The two gradients
 * depend only on q, k, v and dout (sec. 2B/2C: no row statistics of the
 * forward pass are needed), so one plan launch builds both work lists and
 * the dK/dV kernel takes each SM as soon as the dQ kernel's CTA on it has
 * finished, instead of after the last of them: the end of the dQ kernel,
 * where fewer work items than SMs remain, overlaps the start of the dK/dV
 * kernel. The call's last kernel completes only after both have, so later
 * work in the stream sees all three outputs.
 *  - workspace: at least sigattn_bwd_workspace_size(B, H, Lmax, d) bytes
 *    (two work lists); 16-byte aligned and zeroed once, as for every call.
 *    Errors of both kernels go to its sticky error word.
 *  - dq, dk, dv must not overlap each other or the inputs.
 * Returns 0 from sigattn_bwd_workspace_size if the sizes are out of range. */
SIGATTN_API size_t sigattn_bwd_workspace_size(int B, int H, int Lmax, int d);
SIGATTN_API int sigattn_bwd(const void* q, const void* k, const void* v, const void* dout, void* dq, void* dk,
                            void* dv, const int32_t* lengths, int B, int H, int Lmax, int d, void* workspace,
                            size_t workspace_bytes, void* stream);
/* The same for the packed layout (arguments as sigattn_bwd_dq_varlen; the
 * workspace is sigattn_bwd_workspace_size(B, H, max_seqlen, d) bytes). */
SIGATTN_API int sigattn_bwd_varlen(const void* q, const void* k, const void* v, const void* dout, void* dq, void* dk,
                                   void* dv, const int32_t* cu_seqlens, int B, int H, int max_seqlen, int total,
                                   int d, void* workspace, size_t workspace_bytes, void* stream);

/* Key ranges: the padded-layout calls restricted to the keys at positions
 * [key_begin, key_begin + key_count) of every sequence, for attention whose
 * keys are split over several calls or GPUs (sequence sharding). Because each
 * weight sigma(q.k/sqrt(d) - ln n) stands on its own, with no normalisation
 * over the keys (sec. 2A), O = sigma(S + b) V is the plain sum over key ranges
 * of each range's contribution, and so is dQ = scale dS K (sec. 2B/2C); dK and
 * dV of a key depend on that key and on all queries only. The bias still uses
 * each sequence's full length n_b.
 *  - q, dout: [B][H][Lmax][d] bf16, all query rows. k, v: [B][H][key_count][d]
 *    bf16 holding keys key_begin .. key_begin + key_count - 1 of every
 *    sequence; a key at position key_begin + j is valid if it is < n_b.
 *  - 0 <= key_begin, 1 <= key_count, key_begin + key_count <= Lmax; the
 *    workspace is sigattn_workspace_size(B, H, Lmax, d) as usual.
 *  - sigattn_fwd_partial writes o_partial [B][H][Lmax][d] fp32 (16-byte
 *    aligned): for valid rows i the sum over the range's valid keys j of
 *    P_ij V_j, not rounded; rows i >= n_b, and every row of a sequence with no
 *    valid key in the range, are 0. Summing the partials of ranges that tile
 *    [0, Lmax) gives O in fp32.
 *  - sigattn_bwd_dq_partial writes dq_partial [B][H][Lmax][d] fp32 likewise:
 *    the range's share of dQ, scale included.
 *  - sigattn_bwd_dkdv_range writes dk, dv [B][H][key_count][d] bf16: the rows
 *    of dK and dV for the range's keys (zero for keys >= n_b). With
 *    key_begin a multiple of 128 they are the same bits as the matching rows
 *    of sigattn_bwd_dkdv.
 *  - Everything else as for sigattn_fwd / sigattn_bwd_dq / sigattn_bwd_dkdv. */
SIGATTN_API int sigattn_fwd_partial(const void* q, const void* k, const void* v, float* o_partial,
                                    const int32_t* lengths, int B, int H, int Lmax, int d, int key_begin,
                                    int key_count, void* workspace, size_t workspace_bytes, void* stream);
SIGATTN_API int sigattn_bwd_dq_partial(const void* q, const void* k, const void* v, const void* dout,
                                       float* dq_partial, const int32_t* lengths, int B, int H, int Lmax, int d,
                                       int key_begin, int key_count, void* workspace, size_t workspace_bytes,
                                       void* stream);
SIGATTN_API int sigattn_bwd_dkdv_range(const void* q, const void* k, const void* v, const void* dout, void* dk,
                                       void* dv, const int32_t* lengths, int B, int H, int Lmax, int d, int key_begin,
                                       int key_count, void* workspace, size_t workspace_bytes, void* stream);

/* The softmax counterpart of sigattn_fwd, for comparisons on equal terms
 * (Better Models, Faster Training, sec. 4A compares the sigmoid kernel with
 * softmax attention's FlashAttention-2 on padded batches): the same plan,
 * scheduler, data movement and MMAs, with the sigmoid replaced by a softmax
 * over each sequence's valid keys,
 *     O_i = sum_{j<n} exp(S_ij) V_j / sum_{j<n} exp(S_ij),  S = Q K^T / sqrt(d),
 * computed online (running row maximum, lazily rescaled O and row sums).
 * Forward only, d = 64 only (SIGATTN_ERR_UNSUPPORTED otherwise), padded
 * layout; arguments, outputs (rows >= n_b zero) and workspace as sigattn_fwd.
 * No log-sum-exp is returned. */
SIGATTN_API int sigattn_softmax_fwd(const void* q, const void* k, const void* v, void* o, const int32_t* lengths,
                                    int B, int H, int Lmax, int d, void* workspace, size_t workspace_bytes,
                                    void* stream);

/* Round `count` fp32 values to bf16 (nearest even), x -> y, both device
 * pointers, 16-byte aligned; count a multiple of 8. The last step after the
 * fp32 partial sums of key ranges were added (e.g. by an all-reduce). */
SIGATTN_API int sigattn_cast_bf16(const float* x, void* y, long long count, void* stream);

/* Packed ("varlen") layout: the same three operations on sequences stored
 * back to back instead of padded to Lmax, so padding costs neither FLOPs nor
 * HBM bytes. Sequence b's tokens are rows cu_seqlens[b] .. cu_seqlens[b+1]-1
 * of every tensor; n_b = cu_seqlens[b+1] - cu_seqlens[b].
 *  - Tensors are bf16, contiguous [total][H][d] (d fastest, then heads, then
 *    tokens), in device memory, 16-byte aligned; d is 64 or 128.
 *  - cu_seqlens is int32 [B+1] in device memory, nondecreasing, with
 *    0 <= cu_seqlens[b] and cu_seqlens[B] <= total. max_seqlen >= every n_b
 *    plays the part of Lmax (work-list size, limits). A sequence whose bounds
 *    break these rules gets no work: its rows are left untouched and
 *    SIGATTN_ERR_INVALID_ARG is raised in the workspace's sticky error word.
 *  - Only rows that belong to a sequence are written; rows outside every
 *    [cu_seqlens[b], cu_seqlens[b+1]) are never touched. Results equal those of
 *    the padded calls on the same sequences. The last row block of a sequence
 *    reads up to 255 rows past its end (the next sequence, or rows after
 *    cu_seqlens[B]); those enter a result of the sequence only as 0 * value
 *    and must be finite, as padded rows must be in the padded layout.
 *  - 1 <= total <= INT32_MAX - 4096; workspace: sigattn_workspace_size(B, H,
 *    max_seqlen, d) bytes. Everything else as for the padded calls. */
SIGATTN_API int sigattn_fwd_varlen(const void* q, const void* k, const void* v, void* o, const int32_t* cu_seqlens,
                                   int B, int H, int max_seqlen, int total, int d, void* workspace,
                                   size_t workspace_bytes, void* stream);
SIGATTN_API int sigattn_bwd_dq_varlen(const void* q, const void* k, const void* v, const void* dout, void* dq,
                                      const int32_t* cu_seqlens, int B, int H, int max_seqlen, int total, int d,
                                      void* workspace, size_t workspace_bytes, void* stream);
SIGATTN_API int sigattn_bwd_dkdv_varlen(const void* q, const void* k, const void* v, const void* dout, void* dk,
                                        void* dv, const int32_t* cu_seqlens, int B, int H, int max_seqlen, int total,
                                        int d, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Serving from a paged cache: the keys and values of earlier tokens stay in
 * fixed-size pages, and each call attends with a chunk of new tokens (a whole
 * prompt, part of one, or a single token per sequence; any mixture in one
 * batch). A step is: sigattn_paged_reserve (pages and slots for the new
 * tokens), sigattn_paged_write (rotate and store them), sigattn_fwd_paged
 * (attend), and when a request ends or tokens are taken back
 * sigattn_paged_release. All bookkeeping stays on the device, so a step can be
 * captured into a CUDA graph and replayed.
 *
 * Conventions of the paged calls
 *  - k_cache, v_cache: [num_pages][Hkv][page_size][d] bf16, contiguous, 16-byte
 *    aligned; d is 64 or 128, page_size 16, 32, 64, 128 or 256. Slot s is row
 *    s % page_size of page s / page_size; num_pages * page_size and num_pages
 *    * Hkv may not exceed INT32_MAX.
 *  - block_table: int32 [B][max_pages]; entry k of row b is the page that holds
 *    tokens [k * page_size, (k + 1) * page_size) of sequence b. Entries past
 *    a sequence's pages are not read. max_pages * page_size <=
 *    SIGATTN_MAX_PAGED_LEN.
 *  - Hq query heads share Hkv key/value heads: Hq = G * Hkv, and query head h
 *    reads key/value head h / G; G <= 128.
 *  - cu_seqlens: int32 [B+1] as in the packed layout: the new tokens of
 *    sequence b are rows cu_seqlens[b] .. cu_seqlens[b+1]-1. kv_lens: int32
 *    [B], the tokens of sequence b in the cache, its new ones included.
 *  - q, k, v, q_out are rows of [heads][d] bf16 with a stride between tokens
 *    (in elements, a multiple of 8, >= heads * d), so that they may be slices
 *    of one fused projection; 16-byte aligned.
 *  - workspace: 16-byte aligned, zeroed once, with the sticky error word of
 *    every call; sigattn_paged_workspace_size bytes for sigattn_fwd_paged and
 *    256 bytes for the others. Calls that may run concurrently need
 *    different workspaces. The calls leave their own counters there at zero;
 *    after SIGATTN_ERR_TIMEOUT zero the workspace again (sigattn_read_error
 *    does that for its header).
 *  - 1 <= B <= SIGATTN_MAX_BATCH. Values found to be bad on the device raise
 *    SIGATTN_ERR_INVALID_ARG in the sticky error word, as stated at each call;
 *    nothing out of bounds is ever read or written. */
#define SIGATTN_MAX_PAGED_LEN (1 << 24)

/* Take pages for new tokens: sequence b has cached_lens[b] tokens and gets
 * new_lens[b] more. Its first ceil(cached / page_size) table entries are in
 * use; the further pages that cached + new tokens need are popped from the
 * stack free_pages[0 .. *free_count), top first, in batch order (sequence 0's
 * first page is the top), and written to its row of block_table.
 * Written besides (int32, on the device):
 *  - cu_seqlens [B+1]: exclusive prefix sums of new_lens;
 *  - kv_lens [B]: cached + new (may be the same array as cached_lens);
 *  - slots [rows]: each new token's slot, in cu_seqlens order; rows at or past
 *    cu_seqlens[B] get -1 (which sigattn_paged_write skips), so a captured
 *    step may carry a padded number of rows;
 *  - positions [rows] (optional, NULL to omit): each new token's position in
 *    its sequence, cached + 0, 1, ...; rows past the last get 0;
 *  - *free_count_out: the pages left (may be the same word as free_count).
 * num_pages is the capacity of free_pages and the bound on page numbers;
 * rows <= 2^30.
 * The request is met whole or not at all. If a length is negative, a
 * sequence would exceed max_pages * page_size tokens, the new tokens exceed
 * `rows`, or the stack holds too few pages, then the error word is raised
 * (site -(b+1) for a sequence's length, 201 for rows, 202 for pages), the table
 * and the stack stay as they were, cu_seqlens is all zero, kv_lens is
 * cached_lens, slots are -1 and *free_count_out is *free_count. A page number
 * outside [0, num_pages) in the stack or the table raises site 203; its tokens
 * get slot -1. */
SIGATTN_API int sigattn_paged_reserve(const int32_t* cached_lens, const int32_t* new_lens, int32_t* block_table,
                                      const int32_t* free_pages, const int32_t* free_count, int32_t* free_count_out,
                                      int32_t* cu_seqlens, int32_t* kv_lens, int32_t* slots, int32_t* positions, int B,
                                      int max_pages, int page_size, int num_pages, int rows, void* workspace,
                                      size_t workspace_bytes, void* stream);
/* The same with a bound on the new tokens of one sequence: more than max_new
 * (>= 0) are refused like any other bad length. With the max_seqlen_q of the
 * sigattn_fwd_paged call that follows, a step that this call would refuse in
 * part is refused whole, before its tokens are stored. */
SIGATTN_API int sigattn_paged_reserve_bounded(const int32_t* cached_lens, const int32_t* new_lens,
                                              int32_t* block_table, const int32_t* free_pages,
                                              const int32_t* free_count, int32_t* free_count_out, int32_t* cu_seqlens,
                                              int32_t* kv_lens, int32_t* slots, int32_t* positions, int B,
                                              int max_pages, int page_size, int num_pages, int rows, int max_new,
                                              void* workspace, size_t workspace_bytes, void* stream);

/* Give pages back: sequence b holds kv_lens[b] tokens and keeps the first
 * keep_lens[b] (keep_lens NULL: none). Its pages [ceil(keep / page_size),
 * ceil(kv / page_size)) are pushed on the stack in batch order, each sequence's
 * in order of position, and *free_count_out is the new height (may be the same
 * word as free_count). block_table and kv_lens are not changed. If a length is
 * bad (0 <= keep <= kv <= max_pages * page_size is broken: site -(b+1)) or the
 * stack would exceed num_pages (site 202), nothing is pushed and
 * *free_count_out is *free_count. A page number outside [0, num_pages) in the
 * table is pushed as -1 and raises site 203. */
SIGATTN_API int sigattn_paged_release(const int32_t* kv_lens, const int32_t* keep_lens, const int32_t* block_table,
                                      int32_t* free_pages, const int32_t* free_count, int32_t* free_count_out, int B,
                                      int max_pages, int page_size, int num_pages, void* workspace,
                                      size_t workspace_bytes, void* stream);
/* The same, and what the sequences hold afterwards goes to kv_lens_out (int32
 * [B], may be kv_lens itself): keep_lens (or zeros) if the call was met, else
 * kv_lens. */
SIGATTN_API int sigattn_paged_release_lens(const int32_t* kv_lens, const int32_t* keep_lens,
                                           const int32_t* block_table, int32_t* free_pages,
                                           const int32_t* free_count, int32_t* free_count_out, int32_t* kv_lens_out,
                                           int B, int max_pages, int page_size, int num_pages, void* workspace,
                                           size_t workspace_bytes, void* stream);

/* Store new keys and values in their slots and, with rotary positions, turn
 * the keys (and queries) on the way. k, v: `rows` rows of [Hkv][d]; row t goes to
 * slot slots[t] of k_cache and v_cache; slot -1 stores nothing (another slot
 * outside the cache stores nothing and raises site 204). Slots other than -1
 * must be distinct: which row a repeated slot ends up with is not defined.
 *  - q, q_out (both or neither; `rows` rows of [Hq][d], Hq >= 1, Hq + 2 Hkv <=
 *    4096): q_out
 *    receives the turned queries of every row, whatever its slot; q_out may
 *    be q itself (same stride).
 *  - Rotary positions: `pairs` > 0 pairs of values of each head are turned
 *    (a multiple of 8, 2 * pairs <= d; 0: none, values are copied). Pair i is
 *    values (i, i + pairs), or with `adjacent` (2i, 2i + 1), and becomes
 *    (x1 cos a - x2 sin a, x2 cos a + x1 sin a) with a = p * inv_freq[i], where
 *    p = positions[pair_axis[i]][t] (int32 [axes][rows]; pair_axis int32
 *    [pairs], NULL: all pairs turn with axis 0). Several axes give image and
 *    video tokens their time, height and width. inv_freq: fp32 [pairs].
 *    Values past 2 * pairs are copied. The angle is formed and reduced in 64
 *    bits, so far positions lose nothing; the turn is computed in fp32 and
 *    rounded once. An axis outside [0, axes) counts as 0 and raises site 205.
 *  - k, v, q must not overlap the caches. */
SIGATTN_API int sigattn_paged_write(const void* k, long long k_stride, const void* v, long long v_stride,
                                    const int32_t* slots, void* k_cache, void* v_cache, const void* q,
                                    long long q_stride, void* q_out, long long q_out_stride, const int32_t* positions,
                                    const float* inv_freq, const int32_t* pair_axis, int axes, int pairs, int adjacent,
                                    int rows, int Hq, int Hkv, int d, int page_size, int num_pages, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* Bytes of workspace for sigattn_fwd_paged: a 256-byte header and room for
 * the partial sums of rows whose keys are split over several SMs (does not
 * depend on the batch or on lengths). Returns 0 if the sizes are out of range. */
SIGATTN_API size_t sigattn_paged_workspace_size(int Hq, int Hkv, int d, int max_seqlen_q);

/* Sigmoid attention of a chunk of new tokens over the paged cache. Row i of
 * sequence b's q_b = cu_seqlens[b+1] - cu_seqlens[b] new tokens stands at
 * position p = kv_lens[b] - q_b + i of its sequence and sees N keys: the first
 * p + 1 with `causal`, else all kv_lens[b];
 *     o_i = sum_{j < N} sigma(q_i . k_j / sqrt(d) - ln N) v_j.
 * The bias counts the keys that the row sees, so but for rounding a causal
 * row's result does not depend on how its prompt was cut into chunks, and with
 * causal = 0 and nothing cached before it is sigattn_fwd_varlen's. A row that sees no key
 * (kv_lens[b] = 0, or p < 0 where more rows than tokens are given) is zero.
 *  - q: `total` rows of [Hq][d]; o: [total][Hq][d] bf16, contiguous. Rows
 *    outside every [cu_seqlens[b], cu_seqlens[b+1]) are never written.
 *  - max_seqlen_q >= every q_b (kernel choice, limits). kv_lens[b] <= max_pages
 *    * page_size. A sequence that breaks these rules, or whose cu_seqlens
 *    bounds are out of order or out of [0, total], gets no work: its rows are
 *    left untouched and the error word is raised (site -(b+1)). So does one
 *    whose rows start before the end of an earlier sequence that keeps these
 *    rules (which takes bounds out of order between the two): no row belongs
 *    to two sequences.
 *  - A page number outside [0, num_pages) among a sequence's pages contributes
 *    nothing to its sums and raises site 203. A batch of more than 2^31 key
 *    blocks (128 keys of one query tile) per SM gets no work and raises site 206.
 *  - Cached values of tokens < kv_lens[b] must be finite; whatever else the
 *    pages hold (NaN included) changes no result.
 *  - The keys are cut over the SMs where that balances the work, and the
 *    fp32 partial sums are added in a fixed order: no atomics touch a result,
 *    and a repeated call gives the same bits.
 *  - Arithmetic: operands, sums and roundings as sigattn_fwd (weights are
 *    rounded to bf16 before the second product); sigma itself is taken by an
 *    exponential and a reciprocal, or in the many-row kernel's far tail by a
 *    cubic. Hq / Hkv * max_seqlen_q (<= 64 at d = 64, <= 32 at d = 128, or more)
 *    decides between two kernels, and the batch decides where keys are cut, so
 *    the last bits of a row may differ with max_seqlen_q and with the other
 *    sequences of its batch.
 *  - One launch. Forward only. */
SIGATTN_API int sigattn_fwd_paged(const void* q, long long q_stride, const void* k_cache, const void* v_cache, void* o,
                                  const int32_t* cu_seqlens, const int32_t* kv_lens, const int32_t* block_table, int B,
                                  int Hq, int Hkv, int max_seqlen_q, int total, int max_pages, int page_size,
                                  int num_pages, int d, int causal, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* Run only the ragged tile scheduler for `kind` on the device: afterwards the
 * workspace holds, at byte offset 8, the item count (int32), and at byte
 * offset 256, `count` entries of four int32 (bh = b*H + h, block index, the
 * valid length n_b, 0), ordered longest sequence first (ties in batch order),
 * heads ascending, blocks ascending. Only blocks whose first row is < n_b appear (sec. 2C: fully
 * padded blocks are skipped). */
SIGATTN_API int sigattn_plan(const int32_t* lengths, int B, int H, int Lmax, int d, int kind, void* workspace,
                 size_t workspace_bytes, void* stream);

/* Host-side statement of the same schedule (no GPU needed): writes up to
 * `cap` (bh, block) pairs to `items_out` (2*cap int32) and the full count to
 * `*count`. lengths_host is host memory. */
SIGATTN_API int sigattn_plan_host(const int32_t* lengths_host, int B, int H, int Lmax, int kind, int32_t* items_out, int cap,
                      int* count);

/* Size of the fixed device scratch array used by sigattn_fwd_noalloc. */
#define SIGATTN_NOALLOC_SCRATCH_BYTES (1 << 20)

/* sigattn_fwd for callers that cannot allocate device memory (code that runs
 * where cudaMalloc is unavailable or forbidden, e.g. inside a host framework
 * that owns the whole device pool, or a plugin that may only touch the
 * buffers it is handed). The paper has no counterpart: it is a deployment
 * convenience of this library.
 *  - Same computation, inputs and outputs as sigattn_fwd; instead of a
 *    caller workspace it uses a SIGATTN_NOALLOC_SCRATCH_BYTES array that is
 *    part of the library's device image, held on every GPU that loads the
 *    library until the process exits. It calls no cudaMalloc/cudaFree.
 *  - Size limit: sigattn_workspace_size(B, H, Lmax, d) must not exceed
 *    SIGATTN_NOALLOC_SCRATCH_BYTES, i.e. B*H*ceil(Lmax/128) <= 65520 work
 *    items; larger problems return SIGATTN_ERR_UNSUPPORTED (message in
 *    sigattn_last_error) before anything is enqueued.
 *  - The first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress); make that first call before any stream capture.
 *  - Every call, on every stream, shares the one array: calls that overlap
 *    on the GPU race. Each call clears the array's status words first.
 *  - status_out: optional device int32 (4-byte aligned); if not NULL, it
 *    receives (in stream order) this call's device-side status: 0,
 *    SIGATTN_ERR_INVALID_ARG for an out-of-range length, or
 *    SIGATTN_ERR_TIMEOUT.
 *  - Argument errors (the checks of sigattn_fwd, a misaligned status_out, a
 *    size beyond the array) are returned before anything is enqueued and
 *    leave the array untouched. */
SIGATTN_API int sigattn_fwd_noalloc(const void* q, const void* k, const void* v, void* o, const int32_t* lengths,
                                    int B, int H, int Lmax, int d, int32_t* status_out, void* stream);

/* Text of the last CUDA failure behind a SIGATTN_ERR_CUDA returned to the
 * calling thread (static, thread-local; "no error" if none yet). */
SIGATTN_API const char* sigattn_last_error(void);

/* Diagnostic for the failure path: enqueue a one-warp kernel whose bounded
 * wait on an mbarrier that nothing arrives on must give up after limit_us
 * microseconds (1 .. 10^7). The kernel records SIGATTN_ERR_TIMEOUT with site
 * 901 in the workspace header, exactly as a compute kernel's expired wait
 * does, and returns normally (the context stays usable). Needs only the
 * 256-byte header of a workspace. */
SIGATTN_API int sigattn_selftest_wait_timeout(void* workspace, size_t workspace_bytes, int limit_us, void* stream);

/* Diagnostic: the attention weight of raw scores exactly as the compute
 * kernels evaluate it, P = sigma(s / sqrt(d) - ln n) (sec. 2A: the sigmoid of
 * the scaled score plus the bias b = -ln n), and its derivative
 * P (1 - P) (sec. 2B) as the backward kernels use it. scores, p and slope are
 * device float arrays of `count` elements (4-byte aligned); d is 64 or 128,
 * 1 <= n <= SIGATTN_MAX_LEN. The kernels form x = s / sqrt(d) - ln n and
 * take sigma from one hardware exp2 of -|x| log2(e) and a polynomial for
 * 1/(1 + e^-|x|); this entry point lets a test measure that form's error
 * against the exact function on any set of scores. Stream-ordered, no sync. */
SIGATTN_API int sigattn_eval_sigmoid(const float* scores, float* p, float* slope, int count, int d, int n,
                                     void* stream);

/* Synchronise `stream`, read the workspace's sticky error word, clear it and
 * return it (SIGATTN_OK if no kernel reported a problem). If `site` is not
 * NULL it receives a code naming the failing check or wait (0 if none). Of
 * several errors the first is kept, but SIGATTN_ERR_TIMEOUT replaces any
 * other; after one the whole 256-byte header is cleared. */
SIGATTN_API int sigattn_read_error(void* workspace, int* site, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SIGATTN_H_ */
