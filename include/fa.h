/*
 * fa.h -- C ABI of the GB300 (sm_103a) attention forward library (libfa.so).
 *
 * The operation is the FlashAttention forward pass: for every batch b, head h
 * and query row i,
 *
 *     O[b,h,i,:] = sum_j softmax_j( scale * Q[b,h,i,:] . K[b,h,j,:] + mask(i,j) ) V[b,h,j,:]
 *     LSE[b,h,i] = ln sum_j exp( scale * Q[b,h,i,:] . K[b,h,j,:] + mask(i,j) )
 *
 * with mask(i,j) = 0 for a visible key and -inf for a hidden one. It follows
 * the definition S = QK^T/sqrt(d), P = softmax(S), O = PV of
 * "ai6s.net/6af30f4d40858c2d8819b6d5" §1 with the scale as a parameter, is
 * computed tile by tile with the online-softmax recurrence of §2.2-§2.3 of the
 * same page (running max m, running sum l, rescale of the output accumulator),
 * and writes the saved statistics of §2.4 as one log-sum-exp per row
 * (LSE = m + ln l, natural log, in units of the scaled logits). The three mask
 * variants are those of the (None | causal | (window_left, window_right))
 * attn_mask argument in "ai6s.net/6a0ed07b662f9a54cb761aa2", section
 * "使用：ops-transformer 怎么调 FlashAttention"; the B x H x S x D layout is the
 * one of "aicoding.csdn.net/6a69d3ff10ee7a33f2941f44", table "显存占用计算".
 *
 * All entry points are thread-safe for distinct streams and never throw.
 */
#ifndef TILED_ATTENTION_FA_H
#define TILED_ATTENTION_FA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1, /* a null/misaligned/aliased pointer, a bad size or enum, a bad scale */
    FA_ERR_UNSUPPORTED = 2, /* a valid request this build does not implement (head dim, device) */
    FA_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed (launch, attribute, tensor map) */
    FA_ERR_TIMEOUT = 4,     /* a bounded in-kernel wait ran out (reported by fa_sync_status) */
    FA_ERR_BOUNDS = 5       /* debug builds only: a kernel refused an out-of-range store
                               (reported by fa_sync_status) */
} fa_status;

typedef enum {
    FA_MASK_NONE = 0,   /* every key 0..N-1 is visible */
    FA_MASK_CAUSAL = 1, /* key j visible to query i iff j <= i */
    FA_MASK_WINDOW = 2  /* key j visible to query i iff i - window_left <= j <= i + window_right */
} fa_mask_mode;

typedef enum { FA_DTYPE_FP16 = 0, FA_DTYPE_BF16 = 1 } fa_dtype;

/*
 * fa_forward -- enqueue one attention forward pass on `stream`.
 *
 * Q, K, V : device pointers, contiguous B x H x N x d tensors of `dtype`
 *           (row-major: d fastest, then N, then H, then B). Read only.
 * O       : device pointer, contiguous B x H x N x d of `dtype`. Written with
 *           O/l rounded to nearest-even. Must not overlap Q, K, V or LSE.
 * LSE     : device pointer, contiguous B x H x N float32. Written.
 * B, H, N : >= 1. Any N is accepted (no padding is required of the caller;
 *           rows and keys past N are handled inside the kernel).
 * d       : head dimension: 32, 64, 128 or 256 (else FA_ERR_UNSUPPORTED), in every
 *           forward call. d = 256 runs on a kernel with one 128-row Q tile per unit,
 *           as do d = 64 and 128 when a head's queries, or the queries of one K/V
 *           head's query heads, fit in one tile, and small unsplit problems (whose
 *           256-row units would fill at most half of the SMs). fa_backward takes
 *           32, 64, 128 and 256, and so does fa_backward_varlen.
 * scale   : multiplier of the logits, finite and > 0 (typically 1/sqrt(d)).
 * mask_mode, window_left, window_right : see fa_mask_mode. The window
 *           arguments are read only for FA_MASK_WINDOW and must then be >= 0
 *           (values >= N act as N). Every query sees at least itself.
 * dtype   : element type of Q, K, V and O; the products are exact and every
 *           sum, max, exponent and the accumulator are float32.
 * stream  : a cudaStream_t (NULL = the legacy default stream).
 *
 * Ownership: every pointer is owned by the caller; the library keeps none and
 * allocates no device memory per call. Q, K and V must be 16-byte aligned
 * (they are read by tensor-memory-access copies), O 32-byte aligned (each row is
 * written with 32-byte vector stores); LSE, accessed one float at a time, 4-byte
 * aligned. All on the current device; a pointer that breaks one of these rules is
 * FA_ERR_INVALID_ARG.
 *
 * Errors: arguments are checked before anything is enqueued; an invalid call
 * returns FA_ERR_INVALID_ARG / FA_ERR_UNSUPPORTED and launches nothing. A
 * launch failure returns FA_ERR_CUDA. The call is asynchronous: a device-side
 * timeout of a bounded wait is reported by a later fa_sync_status().
 */
fa_status fa_forward(const void *Q, const void *K, const void *V, void *O, float *LSE,
                     int64_t B, int64_t H, int64_t N, int64_t d, float scale,
                     fa_mask_mode mask_mode, int64_t window_left, int64_t window_right,
                     fa_dtype dtype, void *stream);

/*
 * fa_forward_gqa -- fa_forward with grouped K/V heads (GQA; MQA when H_kv = 1),
 * the "GQA/MQA" adaptation that "ai6s.net/6af30f4d40858c2d8819b6d5" §5 lists
 * among the practical variants. K and V are contiguous B x H_kv x N x d; query
 * head h of batch b attends with K/V head h / (H / H_kv) of batch b. H_kv must
 * divide H (else FA_ERR_INVALID_ARG). Q, O, LSE, every other argument,
 * ownership and errors are as for fa_forward, which equals this call with
 * H_kv = H.
 */
fa_status fa_forward_gqa(const void *Q, const void *K, const void *V, void *O, float *LSE,
                         int64_t B, int64_t H, int64_t H_kv, int64_t N, int64_t d, float scale,
                         fa_mask_mode mask_mode, int64_t window_left, int64_t window_right,
                         fa_dtype dtype, void *stream);

/*
 * fa_forward_splitkv -- attention with the keys of every head cut into
 * `num_splits` contiguous chunks that are processed in parallel and merged
 * (the split variant of FlashAttention for few queries and many keys, the
 * "Flash Decoding" that "ai6s.net/6af30f4d40858c2d8819b6d5" §5 names). Each
 * chunk yields its own normalised output and log-sum-exp; the merge is
 * LSE = ln sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s.
 *
 * Q, O: contiguous B x H x Nq x d; K, V: contiguous B x H_kv x Nk x d; LSE:
 * B x H x Nq float32. Nq and Nk may differ: query i stands at key position
 * i + Nk - Nq (the queries are the last Nq positions, as when decoding), which
 * is what the causal and window masks refer to; masks require Nq <= Nk.
 * num_splits >= 1 (values above the number of 128-key tiles act as that
 * number; fa_splitkv_default_splits suggests one). The result equals
 * fa_forward_gqa's up to rounding.
 *
 * workspace: device memory owned by the caller, 32-byte aligned, at least
 * fa_splitkv_workspace_bytes(B, H, Nq, d, num_splits) bytes, not overlapping
 * the other buffers; its contents are scratch (fp32 partial results) and are
 * overwritten. With num_splits = 1 it is not used (it may then be NULL).
 * Two kernels are enqueued: the split attention and the merge.
 * Errors as for fa_forward, plus FA_ERR_INVALID_ARG for a missing or short
 * workspace, num_splits < 1, or a mask with Nq > Nk.
 */
fa_status fa_forward_splitkv(const void *Q, const void *K, const void *V, void *O, float *LSE,
                             int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t Nk,
                             int64_t d, float scale, fa_mask_mode mask_mode,
                             int64_t window_left, int64_t window_right, fa_dtype dtype,
                             int64_t num_splits, void *workspace, size_t workspace_bytes,
                             void *stream);

/* Workspace bytes fa_forward_splitkv needs (0 for invalid sizes). */
size_t fa_splitkv_workspace_bytes(int64_t B, int64_t H, int64_t Nq, int64_t d,
                                  int64_t num_splits);

/* A split count that fills the current device in one wave: 1 when the query
 * blocks alone give at least one unit per SM, otherwise as many splits as the
 * SMs hold next to those units, each keeping at least four 128-key tiles
 * (1 for invalid sizes). */
int64_t fa_splitkv_default_splits(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t Nk);

/*
 * fa_forward_splitkv_static -- fa_forward_splitkv without a caller workspace,
 * for callers that cannot allocate device memory: runtimes that reserve all of
 * their device memory up front and forbid later allocations (to rule out
 * fragmentation or an out-of-memory failure in the middle of serving), and
 * plug-in hosts that give the library no allocator. The pages have no
 * counterpart: this is an interface choice of this library.
 *
 * The scratch is one fixed array of FA_SPLITKV_STATIC_SCRATCH_BYTES bytes in
 * device memory, part of the library: every GPU that loads the library holds
 * it until the process exits, and this call allocates nothing. Requests whose
 * fa_splitkv_workspace_bytes(B, H, Nq, d, n) exceeds that size are rejected
 * with FA_ERR_UNSUPPORTED before anything is enqueued (use fewer splits, or
 * fa_forward_splitkv with a workspace); n is the split count the call runs,
 * num_splits clamped to the number of 128-key tiles (and lowered further when
 * rounding the tiles per split up leaves a split empty). num_splits >= 1.
 *
 * All calls on a device share the one array and leave their partial results
 * in it; nothing in it needs to start at zero. Calls whose kernels overlap on
 * the GPU (for example on two streams at once) race on the array: order them
 * on one stream, or synchronise between them. The first call on each device
 * looks up the array's device address (with that device current); make that
 * first call before any stream capture. Everything else -- arguments, layout,
 * masks, results and errors -- is as for fa_forward_splitkv.
 */
#define FA_SPLITKV_STATIC_SCRATCH_BYTES (16u << 20)
fa_status fa_forward_splitkv_static(const void *Q, const void *K, const void *V, void *O,
                                    float *LSE, int64_t B, int64_t H, int64_t H_kv, int64_t Nq,
                                    int64_t Nk, int64_t d, float scale, fa_mask_mode mask_mode,
                                    int64_t window_left, int64_t window_right, fa_dtype dtype,
                                    int64_t num_splits, void *stream);

/*
 * fa_forward_varlen -- attention forward over a batch of sequences of different
 * lengths packed back to back (the variable-length batches that
 * "ai6s.net/6af30f4d40858c2d8819b6d5" §4.2 lists among the cases an
 * implementation has to handle). Sequence b owns query tokens
 * cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1 and keys cu_seqlens_k[b] ..
 * cu_seqlens_k[b+1]-1; each sequence is an independent fa_forward_gqa problem
 * whose L_q queries stand at its last L_q key positions (as in
 * fa_forward_splitkv), which is what the masks refer to.
 *
 * Layout (token-major): Q and O total_q x H x d, K and V total_k x H_kv x d, in
 * `dtype`; LSE total_q x H float32; cu_seqlens_q and cu_seqlens_k are B + 1
 * int32 on the device, non-decreasing from 0 to total_q / total_k. All on the
 * current device; Q, K, V 16-byte aligned, O 32-byte, LSE 4-byte. max_seqlen_q >= every L_q (rows
 * past it are not computed). With a mask, every sequence needs L_q <= L_k;
 * every sequence with queries needs L_k >= 1. The device arrays are read by
 * the kernel, not checked on the host; offsets are clamped to the tensors, so
 * inconsistent arrays give wrong results but no access outside them.
 *
 * Errors: as fa_forward. total_q = 0 or max_seqlen_q = 0 returns FA_OK with
 * nothing read, written or enqueued (the pointers may then be NULL).
 */
fa_status fa_forward_varlen(const void *Q, const void *K, const void *V, void *O, float *LSE,
                            const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int64_t B,
                            int64_t H, int64_t H_kv, int64_t total_q, int64_t total_k,
                            int64_t max_seqlen_q, int64_t d, float scale, fa_mask_mode mask_mode,
                            int64_t window_left, int64_t window_right, fa_dtype dtype,
                            void *stream);

/*
 * fa_forward_host -- the forward pass of fa_forward_splitkv over HOST buffers:
 * the inputs are copied to the device, processed and the results copied back,
 * in chunks (one batch entry and a range of K/V heads with their query heads,
 * about chunk_bytes of Q + K + V each; chunk_bytes <= 0 takes 64 MiB). The copy
 * in of chunk c+1, the kernel on chunk c and the copy out of chunk c-1 overlap:
 * the copies run on two streams of the library's own (created once per device),
 * the kernels on `stream`. So only the first copy in and the last copy out are
 * not hidden behind other work.
 *
 * Q, K, V, O, LSE: host memory (page-locked memory makes the copies
 * asynchronous; pageable memory works, with the host waiting on each copy), in
 * the layout of fa_forward_splitkv; O and LSE overlap no input. `workspace`:
 * device memory owned by the caller, 32-byte aligned, at least
 * fa_forward_host_workspace_bytes(...) bytes with the same sizes, num_splits and
 * chunk_bytes; it holds the device copies. num_splits: 0 runs Nq == Nk
 * unsplit and Nq < Nk with fa_splitkv_default_splits per chunk; n >= 1 runs
 * every chunk with n key splits.
 *
 * The call enqueues everything and returns; `stream` then waits for the last
 * copy out, so a stream synchronize (or fa_sync_status(stream)) means O and LSE
 * are in host memory. The host buffers must stay valid until then, and the
 * workspace must not be reused meanwhile. Calls on one device are enqueued one
 * at a time (a lock), so concurrent callers stay correct.
 *
 * Errors: every argument is checked before anything is enqueued (as fa_forward,
 * plus: a device pointer among Q, K, V, O, LSE, or a workspace that is not
 * device memory or is too small, is FA_ERR_INVALID_ARG). A CUDA failure while
 * enqueueing returns FA_ERR_CUDA.
 */
size_t fa_forward_host_workspace_bytes(int64_t B, int64_t H, int64_t H_kv, int64_t Nq,
                                       int64_t Nk, int64_t d, int64_t num_splits,
                                       int64_t chunk_bytes);
fa_status fa_forward_host(const void *Q, const void *K, const void *V, void *O, float *LSE,
                          int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t Nk, int64_t d,
                          float scale, fa_mask_mode mask_mode, int64_t window_left,
                          int64_t window_right, fa_dtype dtype, int64_t num_splits,
                          int64_t chunk_bytes, void *workspace, size_t workspace_bytes,
                          void *stream);

/*
 * fa_backward -- gradients of the forward pass: given Q, K, V, the forward's
 * O and LSE (as fa_forward / fa_forward_gqa wrote them) and dO, the gradient
 * of a loss with respect to O, writes dQ, dK and dV. The forward keeps only O
 * and the row statistics; like the method of "ai6s.net/6af30f4d40858c2d8819b6d5"
 * §2.4 ("重计算(Recomputation)与反向传播"), this call recomputes the scores and
 * probabilities tile by tile from them instead of storing P. With
 * D_i = sum_c dO_ic O_ic and P_ij = exp(scale q_i.k_j - LSE_i) on visible keys:
 *   dV_j = sum_i P_ij dO_i,  dS_ij = P_ij (dO_i . V_j - D_i),
 *   dQ_i = scale sum_j dS_ij K_j,  dK_j = scale sum_i dS_ij Q_i,
 * dK and dV of a K/V head summing over every query head that reads it.
 *
 * Layout: Q, O, dO and dQ are contiguous B x H x N x d; K, V, dK and dV are
 * B x H_kv x N x d (H_kv divides H); LSE is B x H x N float32; all in `dtype`
 * except LSE, on the current device; Q, K, V, O and dO 16-byte aligned, dQ, dK and
 * dV 32-byte aligned (32-byte vector stores), LSE 4-byte. Queries and keys share
 * positions (as in fa_forward); the mask arguments are those of fa_forward.
 * `workspace` is caller-owned device memory of at least
 * fa_backward_workspace_bytes(B, H, N, d) bytes (two fp32 row terms per query
 * row), 32-byte aligned; its contents on entry do not matter. dQ, dK, dV and
 * the workspace overlap no input and no other output. The results are
 * deterministic: no atomics, fixed summation order.
 *
 * d is 32, 64, 128 or 256. At d = 256 each gradient has its own pass (a 128 x 256
 * tile of each operand and both accumulators do not fit one SM's shared and
 * tensor memory): four launches (row terms, dV, dK, dQ) instead of three.
 *
 * Errors: as fa_forward, plus FA_ERR_INVALID_ARG for a missing or small
 * workspace. Asynchronous on `stream` (three kernel launches: row terms, dK/dV,
 * dQ; four at d = 256); timeouts are reported by fa_sync_status.
 */
fa_status fa_backward(const void *Q, const void *K, const void *V, const void *O, const void *dO,
                      const float *LSE, void *dQ, void *dK, void *dV, int64_t B, int64_t H,
                      int64_t H_kv, int64_t N, int64_t d, float scale, fa_mask_mode mask_mode,
                      int64_t window_left, int64_t window_right, fa_dtype dtype, void *workspace,
                      size_t workspace_bytes, void *stream);

/* Workspace bytes fa_backward needs (0 for invalid sizes). */
size_t fa_backward_workspace_bytes(int64_t B, int64_t H, int64_t N, int64_t d);

/*
 * fa_backward_varlen -- fa_backward for a variable-length batch laid out as in
 * fa_forward_varlen (token-major; sequence b owns query tokens cu_seqlens_q[b]
 * .. cu_seqlens_q[b+1]-1 and keys cu_seqlens_k[b] .. cu_seqlens_k[b+1]-1, its
 * queries at its last key positions). O and LSE are fa_forward_varlen's
 * outputs; dO and dQ are total_q x H x d, dK and dV total_k x H_kv x d.
 * max_seqlen_q / max_seqlen_k bound every sequence's lengths. Gradients of
 * keys that no query sees, and of queries that see no key, are zero.
 * `workspace`: fa_backward_varlen_workspace_bytes(B, H, total_q) bytes, 32-byte
 * aligned; pointer alignment as in fa_backward. d is 32, 64, 128 or 256.
 * Deterministic. Errors as fa_backward; the device arrays are clamped to the
 * tensors, as in fa_forward_varlen. Asynchronous on `stream`: three zero-fills
 * of dQ, dK and dV, then four kernel launches (padded row offsets, row terms,
 * dK/dV, dQ), five at d = 256 (one pass per gradient).
 */
fa_status fa_backward_varlen(const void *Q, const void *K, const void *V, const void *O,
                             const void *dO, const float *LSE, const int32_t *cu_seqlens_q,
                             const int32_t *cu_seqlens_k, void *dQ, void *dK, void *dV, int64_t B,
                             int64_t H, int64_t H_kv, int64_t total_q, int64_t total_k,
                             int64_t max_seqlen_q, int64_t max_seqlen_k, int64_t d, float scale,
                             fa_mask_mode mask_mode, int64_t window_left, int64_t window_right,
                             fa_dtype dtype, void *workspace, size_t workspace_bytes,
                             void *stream);

/* Workspace bytes fa_backward_varlen needs (0 for invalid sizes). */
size_t fa_backward_varlen_workspace_bytes(int64_t B, int64_t H, int64_t total_q);

/*
 * ---- Queries and keys on their way to attention: per-head norm, rotary positions,
 * and the paged K/V cache of a serving loop.
 *
 * The calls below take descriptors, plain structs that the caller fills once and
 * keeps; the library reads them during the call only.
 */

/* A (batch, head, token, d) tensor: `data` is the element (0, 0, 0, 0) and the three
 * strides count elements; d is contiguous. Device memory, 16-byte aligned, the strides
 * multiples of 8 elements and >= 0 (what a dimension of one entry has does not matter).
 * data = NULL: the tensor is not there. */
typedef struct {
    void *data;
    int64_t batch, head, token;
} fa_rows;

typedef enum {
    FA_ROPE_HALF = 0,       /* pairs (j, j + rotary_dim / 2) */
    FA_ROPE_INTERLEAVED = 1 /* pairs (2 j, 2 j + 1) */
} fa_rope_layout;

/*
 * What happens to a row x of d elements (one head of one token) at position p, the
 * norm first and the rotation second, all in float32 with one rounding at the end:
 *     n_i = x_i * w_i / sqrt( (x_0^2 + .. + x_{d-1}^2) / d + eps )   (n = x without a weight)
 *     (y_a, y_b) = magnitude * (n_a cos(p f_j) - n_b sin(p f_j),
 *                               n_b cos(p f_j) + n_a sin(p f_j))     for pair j = (a, b)
 *     y_i = n_i                                                      for i >= rotary_dim
 * steps: device memory, rotary_dim / 2 entries, the frequencies f_j as fa_rope_steps
 * writes them; 16-byte aligned. rotary_dim: even, 0 .. d (0: no rotation, steps unused).
 * layout: see fa_rope_layout. magnitude: finite (scalings for long contexts use one; else 1).
 * q_weight, k_weight: device memory, d elements of the call's dtype, 16-byte aligned;
 * NULL: queries (keys) are not normalised. eps: >= 0, finite.
 */
typedef struct {
    const uint64_t *steps;
    int64_t rotary_dim;
    fa_rope_layout layout;
    float magnitude;
    const void *q_weight, *k_weight;
    float eps;
} fa_norm_rope;

/*
 * fa_rope_steps -- the frequencies of n rotary pairs (radians per position) as
 * fractions of a turn in 64-bit fixed point, steps[j] = f_j / (2 pi) * 2^64 mod 2^64,
 * rounded to nearest. Both arrays are host memory. A position times such a step, modulo
 * 2^64, is the exact phase of that position, so far positions lose nothing: the error
 * of an angle stays below 2^-52 f_j p + 2^-22 radians. Scalings of the frequencies for
 * long contexts are applied to f_j by the caller. FA_ERR_INVALID_ARG for NULL, n < 1
 * or a frequency that is not finite or of magnitude 2^20 or more.
 */
fa_status fa_rope_steps(const double *frequencies, int64_t n, uint64_t *steps);

/*
 * fa_qk_norm_rope -- norms of queries and keys per head, and their rotary positions,
 * in one pass: q_out, k_out from q, k as fa_norm_rope says. Queries are B x H x N x d,
 * keys B x H_kv x N x d, by the strides of their descriptors: slices of a fused
 * projection go straight to the layout an attention call takes. Either pair may be
 * absent (data = NULL in both q and q_out, or in both k and k_out).
 * positions: device memory, B x N int32, the position of each token (any value), or
 * NULL: token n of every batch entry stands at n. d: 32, 64, 128 or 256.
 * An output may be its own input (the same data and strides: in place); other
 * overlaps of the buffers are refused when their extents cross, unless they are
 * interleaved slices of one fused buffer with equal token (and batch) strides.
 * One kernel launch, asynchronous on `stream`. Errors as fa_forward.
 */
fa_status fa_qk_norm_rope(const fa_rows *q, const fa_rows *k, const fa_rows *q_out,
                          const fa_rows *k_out, const fa_norm_rope *rope, const int32_t *positions,
                          int64_t B, int64_t H, int64_t H_kv, int64_t N, int64_t d, fa_dtype dtype,
                          void *stream);

/*
 * fa_qk_norm_rope_backward -- gradients of fa_qk_norm_rope: from its inputs q, k and
 * the gradients dq_out, dk_out of its outputs, dq and dk, and dq_weight, dk_weight (d
 * float32 each), the gradients of the weights summed over every token and head. With
 * u the rotation's transpose applied to dy, r = 1 / sqrt(mean(x^2) + eps), z = x r:
 *     dx = r (u w - z mean(u w z)),   dw = sum u z      (dx = u without a weight).
 * q (k) is read only where its weight is given, and dq_weight (dk_weight) is written
 * exactly there; it must be NULL without. dq may be dq_out (in place), likewise dk.
 * workspace: caller-owned device memory of at least
 * fa_qk_norm_rope_backward_workspace_bytes(d) bytes, 16-byte aligned, scratch; needed
 * only with a weight (else it may be NULL). Deterministic: no atomics, fixed order.
 * One kernel launch, two with a weight. Everything else as fa_qk_norm_rope.
 */
fa_status fa_qk_norm_rope_backward(const fa_rows *q, const fa_rows *k, const fa_rows *dq_out,
                                   const fa_rows *dk_out, const fa_rows *dq, const fa_rows *dk,
                                   float *dq_weight, float *dk_weight, const fa_norm_rope *rope,
                                   const int32_t *positions, int64_t B, int64_t H, int64_t H_kv,
                                   int64_t N, int64_t d, fa_dtype dtype, void *workspace,
                                   size_t workspace_bytes, void *stream);

/* Workspace bytes fa_qk_norm_rope_backward needs on the current device (0: invalid d). */
size_t fa_qk_norm_rope_backward_workspace_bytes(int64_t d);

/*
 * A paged K/V cache: num_pages pages of page_size tokens of H_kv heads of d elements,
 * K and V alike, element (page, token, head, i) at data + page * page_stride + token *
 * token_stride + head * head_stride + i. The strides (of dimensions with more than one
 * entry) are multiples of 8 elements, > 0, and place every element somewhere else:
 * token-major pages, head-major pages and K and V interleaved in one buffer are all
 * fine. k, v: device memory, 16-byte aligned. page_size: a power of two, 8 .. 2^20. d: 32,
 * 64, 128 or 256. num_pages < 2^31, and fewer than 2^31 steps of the page and head strides'
 * greatest common divisor from the first to the last page (else FA_ERR_UNSUPPORTED).
 */
typedef struct {
    void *k, *v;
    int64_t page_stride, token_stride, head_stride;
    int64_t num_pages, page_size, H_kv, d;
    fa_dtype dtype;
} fa_paged_cache;

/*
 * The batch of a serving step, as fa_paged_append and fa_forward_paged take it: B
 * sequences with total_q new tokens, packed token-major; sequence b owns tokens
 * cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1 (none, one, or a chunk of a prompt), and
 * seqlens_k[b] keys, its new tokens included: they stand at its last positions. Key
 * position j of sequence b lives in page block_table[b * max_pages + j / page_size], at
 * token j mod page_size. The three arrays are int32 on the device, read by the kernels
 * and not checked on the host: offsets are clamped to the tensors, lengths to max_pages
 * pages, and page numbers outside the cache are not followed (they read as zeros and
 * are not written), so inconsistent arrays give wrong results but no access outside
 * the buffers. Tokens past cu_seqlens_q[B] (a padded batch) belong to no sequence.
 *
 * fa_paged_append -- write the new tokens' keys and values into their pages, the keys
 * (and, when q is given, the queries) normalised and rotated on the way as
 * fa_norm_rope says; a token's rotary position is its key position. rope = NULL: keys
 * are stored, and queries copied, as they are. q, q_out: total_q x H x d, or both with
 * data = NULL (H is then ignored); k, v: total_q x H_kv x d; of all four the descriptor's
 * `head` and `token` strides are used. q_out may be q. Rows of q_out of tokens that belong
 * to no sequence are left as they are. K and V of the cache share no element (the same
 * pointer for both, fine to attend over, is refused). Two sequences that write the same slot of a page
 * leave either's row there. A sequence whose first new tokens would stand before position
 * 0 (more new tokens than keys) stores only the others. One kernel launch.
 */
fa_status fa_paged_append(const fa_rows *q, const fa_rows *k, const fa_rows *v, const fa_rows *q_out,
                          const fa_paged_cache *cache, const int32_t *block_table, int64_t max_pages,
                          const int32_t *cu_seqlens_q, const int32_t *seqlens_k, int64_t B, int64_t H,
                          int64_t total_q, const fa_norm_rope *rope, void *stream);

/*
 * fa_forward_paged -- attention of the new tokens over their sequences' keys in the
 * cache (fa_paged_append first: a token sees its own key). Q, O: total_q x H x d,
 * contiguous, of the cache's dtype; LSE: total_q x H float32; H is a multiple of the
 * cache's H_kv, query head h reads K/V head h / (H / H_kv). Token i of a sequence
 * with L_q new tokens and L_k keys stands at i + L_k - L_q, which is what the masks
 * refer to. A token that sees no key (L_k = 0, or a position before 0 under a mask)
 * gets O = 0 and LSE = -infinity. Rows of O and LSE of tokens that belong to no
 * sequence are left as they are. What pages hold past a sequence's end, or before the
 * window of every query that is processed with it, is not looked at (NaN included); a
 * NaN or infinity in a value row that one query of a sequence sees may reach the
 * outputs of its other new tokens processed in the same tile.
 *
 * Scores, softmax statistics and sums are float32. The weights exp(score - maximum) are rounded
 * to the cache's dtype for their product with V, as in fa_forward; where a batch has few new
 * tokens (at most 16 rows, tokens x query heads of a K/V head, per sequence on average, and 32 of
 * one sequence) they keep twice as many bits.
 *
 * workspace: caller-owned device memory of at least
 * fa_forward_paged_workspace_bytes(d) bytes, 32-byte aligned, scratch: its contents on
 * entry do not matter. It does not depend on the batch. Calls that may overlap on the
 * GPU need a workspace each. Two kernel launches. The results are the same every time on
 * one device. Alignment of Q, O, LSE and errors as fa_forward; the arrays of the
 * batch are 4-byte aligned. total_q = 0 returns FA_OK with nothing enqueued.
 */
fa_status fa_forward_paged(const void *Q, void *O, float *LSE, const fa_paged_cache *cache,
                           const int32_t *block_table, int64_t max_pages,
                           const int32_t *cu_seqlens_q, const int32_t *seqlens_k, int64_t B,
                           int64_t H, int64_t total_q, float scale, fa_mask_mode mask_mode,
                           int64_t window_left, int64_t window_right, void *workspace,
                           size_t workspace_bytes, void *stream);

/* Workspace bytes fa_forward_paged needs on the current device (0: invalid d). */
size_t fa_forward_paged_workspace_bytes(int64_t d);

/*
 * A paged cache of one latent row per token: num_pages pages of page_size rows of
 * d_latent latent elements and d_rope rotary ones behind them, element (page, token, i) at
 * data + page * page_stride + token * token_stride + i. All heads read the same row: it is the
 * key of each, and its latent part the value. Strides, page_size and num_pages as for
 * fa_paged_cache (H_kv = 1). data: device memory, 16-byte aligned. d_latent: 128, 256 or
 * 512; d_rope: 64.
 */
typedef struct {
    void *data;
    int64_t page_stride, token_stride;
    int64_t num_pages, page_size, d_latent, d_rope;
    fa_dtype dtype;
} fa_latent_cache;

/*
 * fa_latent_append -- write the new tokens' latent rows into their pages: the latent c,
 * normalised over its d_latent elements by rope->k_weight (d_latent elements; NULL: as it is),
 * and the key's rotary part k_rope, rotated; and, when q_rope is given, q_out from the
 * rotary parts of the queries, rotated alike. A token's rotary position is its key
 * position. The batch, its arrays and what happens to tokens without a place are as for
 * fa_paged_append. c: total_q rows of d_latent, k_rope: total_q rows of d_rope (their `token`
 * strides are used: the two halves of one projection are fine); q_rope, q_out:
 * total_q x H x d_rope by `head` and `token`, or both with data = NULL (H is then
 * ignored): slices of wider buffers are fine, such as the last d_rope columns of the
 * absorbed queries that fa_forward_latent takes. q_out may be q_rope, and one buffer may
 * hold a token's query heads, c and k_rope beside each other (equal token strides). rope->rotary_dim is
 * at most d_rope, rope->q_weight must be NULL. rope = NULL: rows are stored, and rotary parts of
 * queries copied, as they are. One kernel launch. Errors as fa_forward.
 */
fa_status fa_latent_append(const fa_rows *q_rope, const fa_rows *c, const fa_rows *k_rope,
                           const fa_rows *q_out, const fa_latent_cache *cache,
                           const int32_t *block_table, int64_t max_pages, const int32_t *cu_seqlens_q,
                           const int32_t *seqlens_k, int64_t B, int64_t H, int64_t total_q,
                           const fa_norm_rope *rope, void *stream);

/*
 * fa_forward_latent -- attention of the new tokens over their sequences' latent rows
 * (fa_latent_append first: a token sees its own row), in the absorbed form: for each
 * (token, head) pair with query q of d_latent + d_rope elements
 *     s_j = scale q . row_j + mask,  O = sum_j softmax(s)_j row_j[0 .. d_latent),
 *     LSE = ln sum_j exp(s_j).
 * The caller multiplies its queries with the up-projection of the keys before, and O with that
 * of the values after; with c the stored latent, that is attention with keys (W_k c, k_rope)
 * and values W_v c per head. Q: total_q x H x (d_latent + d_rope), O: total_q x H x d_latent,
 * both contiguous and of the cache's dtype; LSE: total_q x H float32; any H >= 1. scale is that
 * of the heads as the model defines them. Positions, masks, tokens without keys or sequences,
 * what is not looked at, and NaN in rows that are: as for fa_forward_paged. Rows whose scores are all
 * -infinity end as those without keys; a score of +infinity ends in NaN.
 *
 * Scores, softmax statistics and sums are float32. The weights exp(score - reference) are rounded
 * to the cache's dtype for their product with the rows; where a batch has at most 32 rows (tokens x
 * heads) per sequence on average, they keep twice as many bits.
 *
 * workspace: caller-owned device memory of at least
 * fa_forward_latent_workspace_bytes(d_latent) bytes, 32-byte aligned, scratch: its contents on
 * entry do not matter. It does not depend on the batch. Calls that may overlap on the GPU
 * need a workspace each. Two kernel launches. The results are the same every time on one
 * device. total_q * H is at most 2^30. Everything else as fa_forward_paged.
 */
fa_status fa_forward_latent(const void *Q, void *O, float *LSE, const fa_latent_cache *cache,
                            const int32_t *block_table, int64_t max_pages,
                            const int32_t *cu_seqlens_q, const int32_t *seqlens_k, int64_t B,
                            int64_t H, int64_t total_q, float scale, fa_mask_mode mask_mode,
                            int64_t window_left, int64_t window_right, void *workspace,
                            size_t workspace_bytes, void *stream);

/* Workspace bytes fa_forward_latent needs on the current device (0: invalid d_latent). */
size_t fa_forward_latent_workspace_bytes(int64_t d_latent);

/*
 * fa_paged_weights -- the attention weight that a batch's new tokens give to each key, gathered
 * over calls. For key j of sequence b and each K/V head, over the new tokens i that see it and
 * the query heads h of that K/V head,
 *     a_j = sum_{i, h} exp(scale q_{i,h} . k_j - LSE_{i,h})
 * and then weights_j += a_j for a key that was there before the call's tokens, weights_j = a_j for
 * the call's own (the last L_q positions), whose slots need no clearing. Q, cache, batch, scale
 * and mask are those of the fa_forward_paged call that wrote LSE (only the keys of the cache
 * are read). A row whose LSE is -infinity adds nothing. weights: device memory, num_pages x
 * H_kv x page_size float32, contiguous: entry (page, head, token). Entries of keys that no new
 * token sees, and of slots past a sequence's end, are left as they are. A page that several
 * sequences of the batch share gets each one's a_j, added in any order; otherwise the
 * results are the same every time. weights overlaps no other buffer. total_q * H, and H_kv
 * times the tiles of 128 keys that max_pages pages hold, are at most 2^30. Where offsets are in no
 * order, the tokens of a sequence that lie before the furthest end of the sequences before it (of
 * those that have tokens) add nothing. One kernel launch, no workspace. Everything else as
 * fa_forward_paged.
 */
fa_status fa_paged_weights(const void *Q, const float *LSE, float *weights, const fa_paged_cache *cache,
                           const int32_t *block_table, int64_t max_pages, const int32_t *cu_seqlens_q,
                           const int32_t *seqlens_k, int64_t B, int64_t H, int64_t total_q, float scale,
                           fa_mask_mode mask_mode, int64_t window_left, int64_t window_right,
                           void *stream);

/*
 * fa_paged_evict -- cut the sequences of a paged cache back to `budget` keys by the weight
 * that each key has gathered. For sequence b of n = seqlens_k[b] keys, n > budget, every K/V
 * head keeps its first `first` keys, its last `recent` ones, and of those between the
 * budget - first - recent with the largest weights (of equal ones those at lower positions;
 * NaN counts as -infinity). What is kept moves, in its order, to positions 0 .. budget - 1 of
 * the sequence's pages: keys, values and weights alike, each head its own. Shorter sequences, and
 * what the slots behind position budget - 1 hold, are left as they are. seqlens_out[b] =
 * min(n, budget); it must not overlap seqlens_k.
 *
 * Stored keys keep the rotary positions they were stored with, so later tokens' positions are
 * no longer their places in the cache: rotate those with fa_qk_norm_rope and explicit positions,
 * and append with rope = NULL. Masks of later calls count places (causal stays what it is).
 * A page that two sequences of the batch share ends with either's rows. weights as
 * fa_paged_weights leaves it; K and V of the cache share no element. 0 <= first, recent,
 * first + recent <= budget. One kernel launch, no workspace. Everything else as
 * fa_paged_append.
 */
fa_status fa_paged_evict(const fa_paged_cache *cache, float *weights, const int32_t *block_table,
                         int64_t max_pages, const int32_t *seqlens_k, int32_t *seqlens_out, int64_t B,
                         int64_t budget, int64_t first, int64_t recent, void *stream);

/* Static, NUL-terminated description of a status code. Never NULL. */
const char *fa_status_string(fa_status status);

/*
 * fa_sync_status -- synchronise `stream`, then read and clear the device
 * status word of the current device. Returns FA_ERR_TIMEOUT if any kernel
 * since the last call gave up on a bounded wait, FA_ERR_UNSUPPORTED if a
 * kernel reported a shared-memory layout it cannot use (it then did
 * nothing), FA_ERR_CUDA if the synchronisation itself failed, else FA_OK.
 */
fa_status fa_sync_status(void *stream);

/*
 * fa_set_wait_budget_ns -- upper bound, in nanoseconds of GPU global time, of
 * every in-kernel wait of later launches (default 2e9, or the value of the
 * environment variable FA_WAIT_BUDGET_MS read at the first call). 0 restores
 * the default. Process-wide.
 */
void fa_set_wait_budget_ns(uint64_t ns);

/* Number of kernels this library has launched in this process. */
int64_t fa_launch_count(void);

/*
 * fa_test_arm_fault -- test hook for the failure path. The next launch of this
 * process (only that one) makes every CTA skip the TMA load of K at its K/V
 * ring position `kv_position` (counted from 0 over that CTA's work; position 0
 * exists in every CTA that gets any work). Its MMA warp then waits for data
 * that never arrives: the wait runs out after the wait budget, every role of
 * the kernel gives up, drains its copies and MMAs, frees its tensor memory and
 * returns, and fa_sync_status reports FA_ERR_TIMEOUT. The GPU context stays
 * usable. A negative position disarms the hook. When the next call is
 * fa_backward or fa_backward_varlen, the position counts units instead: every
 * CTA of its dK/dV kernel skips the K/V load of its unit number
 * `kv_position`, with the same outcome. fa_forward_paged takes the hook in the kernel
 * that runs chunks of new tokens, fa_forward_latent and fa_paged_weights in theirs (the position
 * counts a CTA's key tiles); calls and kernels without such waits (single steps over the paged
 * cache, the appends, norm and rotation, the eviction) spend it without effect.
 */
void fa_test_arm_fault(int32_t kv_position);

/*
 * Debug builds. The library can be compiled with two checks that release builds
 * leave out (tiled_attention_03_gb300/build.py, debug="serialize" / "bounds"); the
 * pages have no counterpart, they are aids for changing the kernels. They apply
 * to the two-tile forward kernel (every forward at d = 32, and at d = 64 / 128
 * unless the one-tile kernel runs it).
 *  - FA_DEBUG_SERIALIZE: the kernel runs with the least overlap its protocol
 *    allows (K/V rings two deep, the next unit claimed with the current unit's
 *    last K/V tile, every group of matrix products completed before the next is
 *    issued), so that an ordering mistake shows as a wrong result or a timeout.
 *  - FA_DEBUG_BOUNDS: every store of O, LSE and the split buffers is checked
 *    against the output first; an out-of-range row is not stored, and the first
 *    one is recorded in the status word, which fa_sync_status then reports as
 *    FA_ERR_BOUNDS, instead of a memory fault.
 * fa_debug_flags returns which checks the loaded library has (0 in release builds).
 * fa_test_arm_row_shift(rows) is the test hook of the bounds check: the next
 * two-tile forward launch adds `rows` to every row it stores, so that rows at or
 * past the end of the output are refused and reported. Release builds ignore the
 * shift.
 */
#define FA_DEBUG_SERIALIZE_FLAG 1
#define FA_DEBUG_BOUNDS_FLAG 2
int32_t fa_debug_flags(void);
void fa_test_arm_row_shift(int64_t rows);

#ifdef __cplusplus
}
#endif

#endif /* TILED_ATTENTION_FA_H */
