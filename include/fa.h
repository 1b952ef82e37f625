/*
 * fa.h -- C ABI of the exact tiled attention library for GB300 (sm_103a).
 *
 * The library computes, for every head of a [B, H, N, d] batch,
 *
 *     scores  = scale * Q K^T            (scale is normally 1/sqrt(d))
 *     weights = row_softmax(scores + mask)
 *     O       = weights V
 *
 * exactly (up to floating-point rounding order), tile by tile with an online
 * softmax, so the N x N score matrix is never written to device memory.
 * Source of the operation: "FlashAttention Interview Questions: IO
 * Complexity, Tiling, and Numerical Stability", section "What is
 * FlashAttention exact about?" (the three-line definition and the statement
 * that the optimisation keeps the mathematical target, mask included), and
 * "FlashAttention 1, 2 & 3: Memory Tiling & Eliminating the O(N^2) HBM
 * Bottleneck", section 1 (Attention(Q,K,V) = softmax(QK^T/sqrt(d))V).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Layout: every tensor is contiguous row-major [B][H][N][d]; the
 *    log-sum-exp and the backward row term are [B][H][N].  One (b, h) pair
 *    is one head; queries and keys have the same length N (the _varlen
 *    calls take separate query and key lengths and per-sequence lengths).
 *  - Types: Q, K, V and dO are bf16 (raw 16-bit storage, `const void*`);
 *    O, LSE, dQ, dK, dV and the workspace are fp32.
 *  - Mask: causal = 0 means no mask; causal = 1 means query i sees key j iff
 *    j <= i.  With this mask no row is ever fully masked.
 *  - Sizes: B, H, N >= 1; d is 64 or 128; B*H*N < 2^31.
 *  - Alignment: Q, K, V, dO, O, dQ, dK, dV must be 16-byte aligned; LSE and
 *    the workspace 4-byte aligned.
 *  - Ownership: every pointer is device memory owned by the caller.  The
 *    library never frees caller memory and never allocates anything whose
 *    size grows with N^2.
 *  - Streams: work is queued on `stream` (a cudaStream_t; NULL is the legacy
 *    default stream) and the calls return before it runs.
 *  - Errors: argument errors are returned synchronously with nothing queued;
 *    launch errors are returned synchronously.  A device-side failure (a
 *    pipeline wait that ran past its time limit) is recorded in a status word
 *    on the device and reported by fa_sync_status().  Every wait inside the
 *    kernels is bounded (4 s by default; the FA_WAIT_LIMIT_MS environment
 *    variable, read once per process, changes it), so a failing kernel
 *    returns instead of hanging.  For tests of that path only,
 *    fa_test_set_stall(n) (initial value: the FA_TEST_STALL_UNIT environment
 *    variable, read once per process) makes the first CTA of every later
 *    launch leave one tile of its n-th work unit unloaded (fa_fwd_decode and
 *    the few-rows kernel of the paged calls: CTA n leaves its first stage
 *    unloaded): its waits run out and fa_sync_status() then reports
 *    FA_ERR_TIMEOUT.
 *  - Thread safety: calls may be made from several host threads; calls on
 *    different devices are independent.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* fa_stream_t; /* same type as cudaStream_t */

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,   /* null pointer, size out of range, causal not 0/1, scale not finite and > 0 */
  FA_ERR_UNSUPPORTED_D = 2, /* d is not 64 or 128 */
  FA_ERR_MISALIGNED = 3,    /* a pointer breaks the alignment rules above */
  FA_ERR_LAUNCH = 4,        /* the CUDA runtime refused a launch or an allocation */
  FA_ERR_TIMEOUT = 5,       /* a kernel wait ran past its limit; the kernel returned early */
  FA_ERR_DEVICE_FAULT = 6,  /* the stream reported a CUDA error while synchronising */
  FA_ERR_BAD_PAGE = 7       /* a block table names a page outside the cache, or ends before an appended token
                               (reported by fa_sync_status) */
} fa_status;

/* Element type of the forward output O (fa_fwd_ex, fa_bwd_ex). */
typedef enum {
  FA_DTYPE_F32 = 0,  /* fp32 O */
  FA_DTYPE_BF16 = 1  /* bf16 O: the fp32 result rounded to nearest even, half the bytes written */
} fa_dtype;

/*
 * Forward pass.
 *   q, k, v : bf16 [B][H][N][d], read only.
 *   o       : fp32 [B][H][N][d], written: O_i = sum_j softmax(s_i)_j v_j.
 *   lse     : fp32 [B][H][N], written: LSE_i = ln sum_j exp(s_ij) over the
 *             eligible keys (natural log of the scaled scores).  This is the
 *             "compact normalization information" the backward pass keeps
 *             ("FlashAttention Interview Questions ...", section "Why can
 *             recomputation help training?").
 *   scale   : multiplier of q.k, finite and > 0 (1/sqrt(d) in the pages'
 *             definition).
 * The online softmax follows the same page, section "How can softmax be
 * computed across tiles?" (running maximum, rescaled sum and accumulator).
 */
fa_status fa_fwd(const void* q, const void* k, const void* v, float* o, float* lse, int B, int H, int N, int d,
                 float scale, int causal, fa_stream_t stream);

/*
 * Forward pass over unequal query/key lengths and padded batches.
 *   q       : bf16 [B][H][Nq][d];  k, v : bf16 [B][H][Nk][d].
 *   o, lse  : fp32 [B][H][Nq][d] and [B][H][Nq].
 *   seqlens_q, seqlens_k : device arrays of B ints, the valid lengths of
 *             each sequence (values clamped to [0, Nq] and [0, Nk]); rows past
 *             them are padding.  NULL means every row is valid.
 * Sequence b uses its first Lq = seqlens_q[b] queries and Lk = seqlens_k[b]
 * keys.  Causal alignment is bottom-right: query i sees key j iff
 * j <= i + (Lk - Lq), so the last query sits at the last key -- the reading
 * of "FlashAttention Interview Questions ...", section "Does subtracting the
 * maximum solve every numerical issue?", which warns that unequal lengths,
 * padding and packed sequences need an explicit alignment.  With Lq = Lk it
 * is the square rule of fa_fwd; a single query (decoding) sees every key.
 * Rows with no eligible key and padding rows are written as O = 0,
 * LSE = -inf.  Padding rows of q, k and v do not affect the result as long as
 * their values are below 1e18 in magnitude (so that every dot product stays
 * finite in fp32).  fa_fwd(...) equals
 * fa_fwd_varlen(..., NULL, NULL, B, H, N, N, ...).  Errors and conventions
 * as fa_fwd; seqlens pointers must be 4-byte aligned.
 */
fa_status fa_fwd_varlen(const void* q, const void* k, const void* v, float* o, float* lse, const int* seqlens_q,
                        const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale, int causal,
                        fa_stream_t stream);

/*
 * Forward pass with each query tile's keys split over several CTAs: the same
 * result as fa_fwd (to fp32 rounding), for batches with too few query tiles
 * to fill the GPU (one head of a few thousand tokens has a few dozen).  Each
 * split runs the online softmax ("FlashAttention Interview Questions ...",
 * section "How can softmax be computed across tiles?") over its own range of
 * key tiles and leaves a normalised partial output and its log-sum-exp; a
 * second kernel merges the partials by that log-sum-exp -- the same
 * merge-by-rescaling the online softmax applies from tile to tile.  The
 * library picks the number of splits from the device's SM count (at most
 * 16, at least two key tiles each); when one split suffices it runs fa_fwd.
 *   workspace : fp32 scratch of fa_fwd_splitkv_workspace_bytes(B, H, N, d)
 *               bytes, 16-byte aligned; or NULL (a stream-ordered allocation,
 *               freed on the same stream).
 * Other arguments, results and errors as fa_fwd.
 */
fa_status fa_fwd_splitkv(const void* q, const void* k, const void* v, float* o, float* lse, float* workspace, int B,
                         int H, int N, int d, float scale, int causal, fa_stream_t stream);

/* Bytes of the fa_fwd_splitkv workspace (an upper bound that does not depend
 * on the device); 0 on invalid sizes. */
size_t fa_fwd_splitkv_workspace_bytes(int B, int H, int N, int d);

/* Most query rows per head that fa_fwd_decode accepts. */
#define FA_DECODE_MAX_Q 8

/*
 * The general forward: fa_fwd_varlen with a choice of output type.
 *   o       : [B][H][Nq][d] of o_dtype (FA_DTYPE_F32 or FA_DTYPE_BF16),
 *             16-byte aligned.  With FA_DTYPE_BF16 each element is the fp32
 *             result of fa_fwd_varlen rounded to the nearest bf16 (ties to
 *             even); LSE stays fp32.
 * Other arguments, results and errors as fa_fwd_varlen; an o_dtype outside
 * the enum returns FA_ERR_INVALID_ARG.  fa_fwd_varlen(...) equals
 * fa_fwd_ex(..., FA_DTYPE_F32, ...).
 */
fa_status fa_fwd_ex(const void* q, const void* k, const void* v, void* o, int o_dtype, float* lse,
                    const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale,
                    int causal, fa_stream_t stream);

/*
 * Forward pass with a general additive mask: the "+ mask" of the definition
 * weights = row_softmax(scores + mask) ("FlashAttention Interview Questions
 * ...", section "What is FlashAttention exact about?") as a bias added to
 * the scaled scores, s_ij = scale * q_i.k_j + bias_ij.  It is not scaled; an
 * entry of -inf hides the key; it combines with the causal rule and with
 * padding, and a row whose keys are all hidden gets O = 0, LSE = -inf.
 *   bias  : bf16, element (b, h, i, j) at
 *           bias + b*bias_stride_b + h*bias_stride_h + i*bias_stride_q + j,
 *           keys contiguous.  Strides in elements, >= 0; 0 broadcasts over
 *           that index (bias_stride_q = 0: one row of key biases for every
 *           query, e.g. a key-padding mask); otherwise bias_stride_q >= Nk.
 *           2-byte aligned.  Rows that start on a 16-byte boundary (base
 *           16-byte aligned, strides multiples of 8) are read in 16-byte
 *           loads, others element by element (slower).  No +inf, no NaN.
 * Other arguments, results and errors as fa_fwd_ex; a null bias or an
 * invalid stride returns FA_ERR_INVALID_ARG, a bias at an odd address
 * FA_ERR_MISALIGNED.  Gradients of a masked forward: fa_bwd_bias.
 */
fa_status fa_fwd_bias(const void* q, const void* k, const void* v, void* o, int o_dtype, float* lse,
                      const void* bias, long long bias_stride_b, long long bias_stride_h, long long bias_stride_q,
                      const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale,
                      int causal, fa_stream_t stream);

/*
 * FP8 forward: fa_fwd with E4M3 inputs ("FlashAttention 1, 2 & 3", section on
 * FlashAttention-3: FP8 on the tensor cores).  q8, k8: [B][H][N][128] E4M3
 * (one byte each); vt8: V transposed, [B][H][128][N] E4M3; o fp32
 * [B][H][N][128], lse fp32 [B][H][N], as fa_fwd.  Scores and both products
 * accumulate in fp32 from the E4M3 values as given (descale factors of q and
 * k fold into `scale`; one of v multiplies O, which the caller applies);
 * the probabilities P are rounded to E4M3 before O = P V, so O carries an
 * error of up to 2^-4 sum_j P_ij |v_j| plus a subnormal term against the
 * exact result on the same inputs; LSE does not (it sums the unrounded P).
 * d must be 128 (else FA_ERR_UNSUPPORTED_D); N a multiple of 16 (rows of
 * vt8 are whole 16-byte groups; else FA_ERR_INVALID_ARG); square sequences,
 * causal or not.  All pointers 16-byte aligned (lse 4).  Errors and
 * asynchrony as fa_fwd.
 */
fa_status fa_fwd_fp8(const void* q8, const void* k8, const void* vt8, float* o, float* lse, int B, int H, int N,
                     int d, float scale, int causal, fa_stream_t stream);

/*
 * Decode-shaped forward: 1 <= Nq <= FA_DECODE_MAX_Q query rows per head
 * against a long key/value history.  Computes exactly what fa_fwd_varlen
 * computes for the same arguments (same layouts, lengths, bottom-right causal
 * alignment, padding rules and outputs), with a kernel built for this shape:
 * single-token decoding reads all of K and V once per step for one query row,
 * about one FLOP per byte, so it is bound by HBM bandwidth rather than by the
 * tensor cores ("FlashAttention Interview Questions ...", final section, on
 * prefill against single-token decoding).  Each head's keys are split over
 * many CTAs that stream K/V once; a second kernel merges the splits by their
 * log-sum-exp.
 *   workspace : fp32 scratch for the per-split results,
 *               fa_fwd_decode_workspace_bytes(B, H, Nq, Nk, d) bytes,
 *               16-byte aligned; or NULL, in which case the library takes a
 *               stream-ordered allocation when it splits the keys and frees
 *               it on the same stream.
 * Errors as fa_fwd_varlen; Nq outside [1, FA_DECODE_MAX_Q] returns
 * FA_ERR_INVALID_ARG.
 */
fa_status fa_fwd_decode(const void* q, const void* k, const void* v, float* o, float* lse, const int* seqlens_q,
                        const int* seqlens_k, float* workspace, int B, int H, int Nq, int Nk, int d, float scale,
                        int causal, fa_stream_t stream);

/* Bytes of the fa_fwd_decode workspace (an upper bound that does not depend
 * on the device); 0 on invalid sizes. */
size_t fa_fwd_decode_workspace_bytes(int B, int H, int Nq, int Nk, int d);

/*
 * Backward pass by recomputation: attention probabilities are rebuilt from
 * q, k and the saved lse instead of being stored ("FlashAttention Interview
 * Questions ...", section "Why can recomputation help training?").
 *   q, k, v, dO : bf16 [B][H][N][d], read only (dO = dL/dO).
 *   o, lse      : fp32 outputs of fa_fwd for the same q, k, v, scale, causal.
 *   dq, dk, dv  : fp32 [B][H][N][d], overwritten with dL/dQ, dL/dK, dL/dV.
 *   workspace   : fp32 buffer of fa_bwd_workspace_bytes(B, H, N) bytes that
 *                 receives the row term D_i = sum_j P_ij dP_ij (formed from
 *                 rowsum(dO o O) and corrected to the probabilities the
 *                 backward pass recomputes); or NULL, in which case the
 *                 library takes a stream-ordered allocation and frees it on
 *                 the same stream.
 * Computes P_ij = exp(s_ij - LSE_i), dV = P^T dO, dP = dO V^T,
 * dS = P o (dP - D), dQ = scale dS K, dK = scale dS^T Q.
 */
fa_status fa_bwd(const void* q, const void* k, const void* v, const float* o, const float* lse, const void* dO,
                 float* dq, float* dk, float* dv, float* workspace, int B, int H, int N, int d, float scale,
                 int causal, fa_stream_t stream);

/*
 * Backward pass over unequal query/key lengths and padded batches, the
 * gradient of fa_fwd_varlen for the same arguments.
 *   q, dO, o    : [B][H][Nq][d] (q, dO bf16; o fp32);  lse : fp32 [B][H][Nq].
 *   k, v        : bf16 [B][H][Nk][d].
 *   dq          : fp32 [B][H][Nq][d];  dk, dv : fp32 [B][H][Nk][d], overwritten.
 *   workspace   : fp32, fa_bwd_workspace_bytes(B, H, Nq) bytes, or NULL as
 *                 for fa_bwd; it ends holding D for each query row.
 *   seqlens_q, seqlens_k : as fa_fwd_varlen (NULL: every row valid).
 * Alignment and masking follow fa_fwd_varlen.  Padding rows and rows with no
 * eligible key get zero gradients (and D = 0); key rows past the valid length
 * get dK = dV = 0.  Padding rows of q, k, v and dO do not affect the result
 * under the same bound as fa_fwd_varlen.  fa_bwd(...) equals
 * fa_bwd_varlen(..., NULL, NULL, B, H, N, N, ...).
 */
fa_status fa_bwd_varlen(const void* q, const void* k, const void* v, const float* o, const float* lse,
                        const void* dO, float* dq, float* dk, float* dv, float* workspace, const int* seqlens_q,
                        const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale, int causal,
                        fa_stream_t stream);

/*
 * The general backward: fa_bwd_varlen taking O of either output type of
 * fa_fwd_ex (o_dtype as there).  O only enters through the row term
 * D_i = sum_c dO_ic O_ic, which the dQ stage corrects to the exact
 * sum_j P_ij dP_ij of the recomputed probabilities, so a bf16 O leaves the
 * gradients' accuracy unchanged.  fa_bwd_varlen(...) equals
 * fa_bwd_ex(..., FA_DTYPE_F32, ...).
 */
fa_status fa_bwd_ex(const void* q, const void* k, const void* v, const void* o, int o_dtype, const float* lse,
                    const void* dO, float* dq, float* dk, float* dv, float* workspace, const int* seqlens_q,
                    const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale, int causal,
                    fa_stream_t stream);

/* Gradients of fa_fwd_bias ("FlashAttention Interview Questions", sections
 * "What is FlashAttention exact about?" for the mask and "Why can
 * recomputation help training?" for the backward from the saved LSE):
 * fa_bwd_ex with the same additive mask (bias and its strides exactly as
 * passed to the forward call that made o and lse).
 * The mask enters only the recomputed probabilities,
 * P_ij = exp(scale * q_i.k_j + bias_ij - LSE_i); it is a constant of the
 * differentiation, so no gradient of the mask is formed.  Rows whose keys
 * the mask hides entirely (LSE = -inf) get dQ = 0 and add nothing to dK, dV.
 * Mask rows that start on a 16-byte boundary are read in 16-byte loads by the
 * dQ kernel; the dK/dV kernel reads the mask down its columns, one 2-byte
 * load per (query, key) per pass, coalesced over 32 consecutive keys.
 * Errors as fa_bwd_ex and fa_fwd_bias. */
fa_status fa_bwd_bias(const void* q, const void* k, const void* v, const void* o, int o_dtype, const float* lse,
                      const void* dO, const void* bias, long long bias_stride_b, long long bias_stride_h,
                      long long bias_stride_q, float* dq, float* dk, float* dv, float* workspace,
                      const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale,
                      int causal, fa_stream_t stream);

/*
 * Largest B*H*N that fa_bwd_noalloc accepts: 2^20 rows, i.e. 4 MiB of fp32
 * scratch held in a static device array by every GPU that loads the library,
 * for as long as the library stays loaded.
 */
#define FA_NOALLOC_MAX_ROWS (1 << 20)

/*
 * fa_bwd without any allocation.  The pages describe no such call: it exists
 * for callers that cannot allocate device memory when they run the backward
 * pass -- a host framework or inference runtime that owns every byte of
 * device memory through its own pool and forbids libraries to allocate behind
 * its back, or a latency-critical loop that reserved all memory up front and
 * must not risk an allocation (or an out-of-memory failure) on its hot path.
 *
 * Arguments and results are those of fa_bwd, minus the workspace: the row
 * term D lives in a fixed device array inside the library (see
 * FA_NOALLOC_MAX_ROWS).  The call makes no cudaMalloc/cudaFree or other
 * allocating call.  Its first call on a device looks up that array's device
 * address (cudaGetSymbolAddress) with the caller's device current; make that
 * first call before any stream capture on the device.
 *
 * Errors: as fa_bwd; B*H*N above FA_NOALLOC_MAX_ROWS returns
 * FA_ERR_INVALID_ARG with nothing queued.  All calls on one device share the
 * array, and it keeps the last call's contents (every call rewrites all of
 * the rows it uses before reading them): two calls whose work overlaps on the
 * GPU (different streams, not ordered) race on it and give wrong gradients.
 */
fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const float* o, const float* lse,
                         const void* dO, float* dq, float* dk, float* dv, int B, int H, int N, int d, float scale,
                         int causal, fa_stream_t stream);

/*
 * Single-pass backward: the same gradients as fa_bwd_bias (bias NULL: as
 * fa_bwd_varlen), with dQ formed inside the dK/dV sweep instead of by a
 * second sweep that recomputes S and dP ("FlashAttention Interview Questions
 * ...", section "Why can recomputation help training?": P is rebuilt from
 * q, k and the saved lse).  Two kernels run in stream order:
 *   1. the row term D_i = sum_j P_ij dP_ij, formed from the recomputed fp32
 *      probabilities (two tensor-core products per tile, S = q k^T and
 *      dP = dO v^T); it also sets dQ to zero;
 *   2. one CTA per 128-key tile sweeps the query tiles that see it and forms
 *      dV += P^T dO, dK += scale dS^T q and each tile's dQ share
 *      scale dS k, which it adds into dQ in place.
 * The row term comes from P and dP, not from the forward output, so no O is
 * taken.  dQ's sum over key tiles runs in an order that varies between runs,
 * so dQ may differ in its last bits from call to call (dK, dV do not).
 *   q, k, v, dO, lse, dq, dk, dv, seqlens_q, seqlens_k, B, H, Nq, Nk, d,
 *   scale, causal : as fa_bwd_varlen.
 *   bias and its strides : as fa_bwd_bias, or bias = NULL for no mask.
 *   workspace : fp32, fa_bwd_workspace_bytes(B, H, Nq) bytes, ends holding D;
 *               or NULL (a stream-ordered allocation, freed on the stream).
 * Errors as fa_bwd_bias.
 */
fa_status fa_bwd_single_pass(const void* q, const void* k, const void* v, const float* lse, const void* dO,
                             const void* bias, long long bias_stride_b, long long bias_stride_h,
                             long long bias_stride_q, float* dq, float* dk, float* dv, float* workspace,
                             const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq, int Nk, int d,
                             float scale, int causal, fa_stream_t stream);

/*
 * One stage of a backward pass, for callers that time or schedule the
 * kernels separately; the workspace is required (never NULL).
 *   stage 0: dQ; also writes the exact row term D_i = sum_j P_ij dP_ij into
 *            the workspace (formed from rowsum(dO o O) inside the kernel).
 *   stage 1: dK and dV (needs stage 0 first).
 *            Stages 0, 1 in order on one stream are exactly fa_bwd.
 *   stage 2: the row term D from the recomputed P and dP, and dQ = 0
 *            (o is not read and may be NULL).
 *   stage 3: dK, dV, and dQ accumulated into place (needs stage 2 first).
 *            Stages 2, 3 in order are fa_bwd_single_pass without a mask.
 * Arguments as fa_bwd; a stage outside 0..3 returns FA_ERR_INVALID_ARG.
 */
fa_status fa_bwd_stage(int stage, const void* q, const void* k, const void* v, const float* o, const float* lse,
                       const void* dO, float* dq, float* dk, float* dv, float* workspace, int B, int H, int N, int d,
                       float scale, int causal, fa_stream_t stream);

/* Bytes of the fa_bwd workspace: B*H*N fp32 values (0 on invalid sizes);
 * for fa_bwd_varlen pass N = Nq. */
size_t fa_bwd_workspace_bytes(int B, int H, int N);

/* Pairing of the values that fa_rope and fa_kv_append rotate. */
typedef enum {
  FA_ROPE_HALF = 0,        /* pair i is (i, i + rot_dim / 2) */
  FA_ROPE_INTERLEAVED = 1  /* pair i is (2i, 2i + 1) */
} fa_rope_layout;

/* How fa_rope_turns changes the frequencies for contexts longer than the
 * trained one. */
typedef enum {
  FA_ROPE_SCALE_NONE = 0,
  FA_ROPE_SCALE_LINEAR = 1,  /* every frequency divided by factor (interpolated positions) */
  FA_ROPE_SCALE_NTK = 2,     /* base multiplied by factor^(rot_dim / (rot_dim - 2)): the slowest pair is
                                stretched by factor, the fastest kept */
  FA_ROPE_SCALE_PARTS = 3    /* by parts: pairs that turn more than `high` times within original_len keep
                                their frequency, those below `low` turns are divided by factor, a linear
                                ramp in the number of turns between */
} fa_rope_scaling;

/*
 * The frequency table of the rotary calls, computed on the host: turns[i],
 * i in [0, rot_dim / 2), is the angle that pair i turns by from one position
 * to the next, in units of 2^-64 of a full turn.  Pair i's frequency is
 * base^(-2i / rot_dim) radians per position, changed as `scaling` says.
 *   turns    : host memory, rot_dim / 2 values; the device calls take a copy
 *              in device memory.  A caller with frequencies f_i of its own
 *              (radians per position) stores round(f_i / 2 pi * 2^64) mod 2^64.
 *   rot_dim  : a multiple of 16.
 *   factor >= 1 is read for every scaling but NONE; original_len > 0 and
 *   0 <= low < high only for PARTS.
 * Positions multiply these words modulo 2^64, that is modulo a full turn, so
 * at any 32-bit position the phase is the word's to 2^-32 turns; it is then
 * rounded to fp32 for the sine and cosine, by at most 2^-26 turns.  The words
 * of fa_rope_turns carry the roundings of the doubles that they are computed
 * in, about p * 2^-51 radians at position p.
 */
fa_status fa_rope_turns(long long* turns, int rot_dim, double base, int scaling, double factor, double original_len,
                        double low, double high);

/*
 * Rotary positions: y = the first rot_dim values of every row of x rotated
 * pair by pair by its position's angles, the other d - rot_dim values copied.
 * For a pair (a, b) at position p with angle t = p * f_i:
 *     a' = amplitude (a cos t - b sin t),  b' = amplitude (b cos t + a sin t).
 *   x, y      : [B][H][N][d] of x_dtype / y_dtype (FA_DTYPE_F32, FA_DTYPE_BF16),
 *               d contiguous, the other strides in elements (so that the q or
 *               k part of a fused projection [B][N][heads][d] is read where it
 *               lies); bases 16-byte aligned and rows starting on 16-byte
 *               boundaries, strides >= 0, y's such that its rows do not
 *               overlap.  y may be x itself, with its type and strides;
 *               otherwise they must not overlap.
 *   positions : device ints, position of token n of sequence b at
 *               positions[b * positions_stride_b + n] (0: one row for all
 *               sequences; negative positions turn the other way); or NULL:
 *               token n is at position n.
 *   turns     : device memory, rot_dim / 2 words of fa_rope_turns, 8-byte
 *               aligned.  rot_dim: a multiple of 16, at most d.
 *   amplitude : multiplies the rotated values (1 unless the scaling's
 *               recipe calls for more); finite.
 *   inverse   : 0 the forward rotation; 1 the rotation by -t, which is the
 *               gradient with respect to x of the forward call with the same
 *               arguments, given dL/dy as x (the rotation is orthogonal, and
 *               amplitude enters both alike).
 * Computed in fp32 from the angles that fa_rope_turns describes, rounded once
 * when y is bf16.
 */
fa_status fa_rope(const void* x, int x_dtype, long long x_stride_b, long long x_stride_h, long long x_stride_n,
                  void* y, int y_dtype, long long y_stride_b, long long y_stride_h, long long y_stride_n,
                  const int* positions, long long positions_stride_b, const long long* turns, int rot_dim, int layout,
                  float amplitude, int inverse, int B, int H, int N, int d, fa_stream_t stream);

/*
 * The paged key/value cache.  Keys and values live in pages,
 *   k_pages, v_pages : bf16 [num_pages][Hkv][page_size][d], 16-byte aligned,
 *   page_size a multiple of 16, and position p of sequence b is row
 *   p % page_size of page block_table[b * table_stride + p / page_size].
 *   block_table : device ints, max_pages entries a sequence are reachable
 *               (table_stride >= 0 in elements); entries behind a sequence's
 *               last page are never read.
 *   seqlens_k : device ints, the keys of each sequence, the new tokens of
 *               this step among them (negative: 0).  More than max_pages *
 *               page_size: the attention calls read that many; the append
 *               writes the tokens that have a place and reports the others.
 *   seqlens_q : device ints, the new tokens of each sequence (clamped to
 *               [0, N]); NULL: all N (Nq).
 * Token t of a sequence with Lq new tokens and Lk keys is at position
 * Lk - Lq + t, the bottom-right alignment of fa_fwd_varlen, so that one pair
 * of length arrays serves the append and the attention of a step.
 * A table entry outside [0, num_pages) reads or writes nothing: the call
 * reports FA_ERR_BAD_PAGE through fa_sync_status, and the results of the
 * sequences that name it are unspecified.  max_pages * page_size may be up to
 * 2^30; num_pages * Hkv must be below 2^31, and for the attention calls so
 * must B * Hkv * (Hq / Hkv * Nq / 256 + 1) * (max_pages * page_size / 64 + 1).
 */

/*
 * Appends the new tokens' keys and values to the paged cache, the keys
 * rotated by their positions on the way, and (optionally) rotates the
 * queries of the same tokens in the same launch.
 *   k, v  : bf16 [B][Hkv][N][d] with strides as fa_rope's x (stride 0 allowed).
 *   q     : bf16 [B][Hq][N][d] with strides; NULL: keys and values only (then
 *           q_out is NULL and Hq is not read).
 *   q_out : bf16 [B][Hq][N][d], contiguous; q itself if q is contiguous.
 *   positions : as fa_rope, the angles' positions where they are not the
 *           tokens' places in the cache; NULL: the cache position.
 *   turns, rot_dim, layout, amplitude : as fa_rope; turns = NULL appends (and
 *           copies q) without a rotation, and the other three are not read.
 * Rows at or past Lq are padding: neither the cache nor q_out is written for
 * them.  A token whose position is negative (Lq > Lk) has no place in the
 * cache; its q_out row is written.  A token whose position is max_pages *
 * page_size or more has none either, and is reported as FA_ERR_BAD_PAGE; its
 * q_out row is rotated by the position that it would have had.  Two new tokens
 * that a block table puts on one cache row leave either's value there, element
 * by element.
 */
fa_status fa_kv_append(const void* k, long long k_stride_b, long long k_stride_h, long long k_stride_n, const void* v,
                       long long v_stride_b, long long v_stride_h, long long v_stride_n, const void* q,
                       long long q_stride_b, long long q_stride_h, long long q_stride_n, void* q_out, void* k_pages,
                       void* v_pages, int num_pages, int page_size, const int* block_table, long long table_stride,
                       int max_pages, const int* seqlens_q, const int* seqlens_k, const int* positions,
                       long long positions_stride_b, const long long* turns, int rot_dim, int layout, float amplitude,
                       int B, int Hq, int Hkv, int N, int d, fa_stream_t stream);

/*
 * Attention over the paged cache: fa_fwd_varlen for the lengths seqlens_q and
 * seqlens_k, with keys and values read from their pages and query head h
 * reading key head h / (Hq / Hkv) (Hq a multiple of Hkv).
 *   q    : bf16 [B][Hq][Nq][d], contiguous, any Nq >= 1: single tokens,
 *          drafted tokens, chunks of a prompt.
 *   o    : [B][Hq][Nq][d] of o_dtype; lse: fp32 [B][Hq][Nq].
 *   seqlens_k NULL: every sequence has max_pages * page_size keys.
 *   workspace : fp32 scratch of fa_fwd_paged_workspace_bytes(...) bytes,
 *          16-byte aligned, used by one call at a time; or NULL (a
 *          stream-ordered allocation from a pool of the library's that keeps
 *          up to 256 MB a device between calls, freed on the same stream;
 *          inside a stream capture an allocation of the graph's).
 * With up to 16 rows a key head (Hq / Hkv * Nq) the probabilities enter the
 * product with V in 16 significand bits, with more in 8 (bf16, as in fa_fwd).
 * Causal alignment, padding and empty rows as fa_fwd_varlen (O = 0,
 * LSE = -inf).  Rows of a page behind a sequence's last key may hold anything,
 * NaN included; the values of keys that some query of the sequence sees must
 * be finite.  A row with a NaN or +inf score (a NaN in its query or in a key
 * that it sees) has O = NaN and LSE = NaN, however the call is divided; the
 * other rows do not depend on it.  A key with a score of -inf has no weight.
 */
fa_status fa_fwd_paged(const void* q, const void* k_pages, const void* v_pages, int num_pages, int page_size,
                       const int* block_table, long long table_stride, int max_pages, void* o, int o_dtype,
                       float* lse, const int* seqlens_q, const int* seqlens_k, float* workspace, int B, int Hq,
                       int Hkv, int Nq, int d, float scale, int causal, fa_stream_t stream);

/* Bytes of the fa_fwd_paged workspace (an upper bound that does not depend on
 * the device or on the lengths); 0 on invalid sizes. */
size_t fa_fwd_paged_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d);

/*
 * Attention over the paged cache for a batch whose sequences all start with
 * the same prefix_len keys: exactly what fa_fwd_paged computes when every
 * sequence's first prefix_len / page_size block-table entries are
 * prefix_table's, but the prefix's keys and values are read once for the rows
 * of all sequences together, not once a sequence; the rest of each sequence
 * is attended on its own and the two are merged by their log-sum-exp.  It pays
 * for many sequences of few rows a key head (Hq / Hkv * Nq, up to about 64)
 * behind a long prefix; with chunks of a prompt, few sequences or a prefix of
 * about a thousand keys fa_fwd_paged is as fast or faster.
 *   prefix_table : device ints, the prefix's prefix_len / page_size pages;
 *                  block-table entries below prefix_len / page_size are not
 *                  read by this call (positions stay those of the whole
 *                  sequence, so one table serves the append as well).
 *   prefix_len   : a positive multiple of page_size, at most
 *                  max_pages * page_size.  Sequences shorter than it are
 *                  allowed and see their own length's share of the prefix.
 *   workspace    : with more than 32 rows a key head it holds partial results
 *                  of 256 rows (130 KB at d = 128) for every key head of every
 *                  sequence, as many as its rows fill.
 * The prefix's probabilities are bf16, as in fa_fwd, whatever the number of
 * rows.  Other arguments, results and errors as fa_fwd_paged.
 */
fa_status fa_fwd_shared_prefix(const void* q, const void* k_pages, const void* v_pages, int num_pages, int page_size,
                               const int* prefix_table, int prefix_len, const int* block_table,
                               long long table_stride, int max_pages, void* o, int o_dtype, float* lse,
                               const int* seqlens_q, const int* seqlens_k, float* workspace, int B, int Hq, int Hkv,
                               int Nq, int d, float scale, int causal, fa_stream_t stream);

/* Bytes of the fa_fwd_shared_prefix workspace (an upper bound that does not
 * depend on the device or on the lengths); 0 on invalid sizes. */
size_t fa_fwd_shared_prefix_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d);

/*
 * Synchronises `stream`, then reads and clears the device status word of the
 * current device.  Returns FA_ERR_DEVICE_FAULT if the stream reported a CUDA
 * error, FA_ERR_TIMEOUT if a kernel wait ran out since the last call,
 * FA_ERR_BAD_PAGE if a paged call met a table entry that names no page, FA_OK
 * otherwise.
 */
fa_status fa_sync_status(fa_stream_t stream);

/*
 * Details of the last device-side failure read by fa_sync_status():
 * out[0] status code, out[1] wait site, out[2] block index, out[3] work unit.
 * Wait sites: 1-7 forward, 11-20 dK/dV, 21-32 dQ, 35-36 decode, 41-47 FP8
 * forward, 51-59 the single-pass row-term pass, 61-63 the single-pass dK/dV
 * sweep, 71-81 the paged calls (each kernel's source names them).  After
 * FA_ERR_BAD_PAGE: out[2] the sequence (0 for a prefix), out[3] the table
 * entry, or where out[1] is 81 the position of an appended token that is
 * behind the table's last one.
 * Returns FA_OK, or FA_ERR_INVALID_ARG if out is NULL.
 */
fa_status fa_last_failure(int out[4]);

/*
 * Testing hook of the timeout path (see "Errors" above): from the next call
 * on, the first CTA of each launch leaves one tile of its unit-th work unit
 * unloaded, so that the waits on it run out and fa_sync_status() reports
 * FA_ERR_TIMEOUT; unit = -1 switches the hook off (the default unless
 * FA_TEST_STALL_UNIT was set when the library first launched work).  Nothing
 * faults or hangs.  Returns FA_OK, or FA_ERR_INVALID_ARG for unit < -1.
 */
fa_status fa_test_set_stall(int unit);

/* Testing hook: how many tensor maps the library has had the driver encode
 * since it was loaded.  A call on tensors that it has seen adds none. */
long long fa_test_map_encodes(void);

/* Static, human-readable name of a status code; never NULL. */
const char* fa_status_string(fa_status s);

/*
 * Host-only view of the persistent scheduler, for tests and tools (no GPU
 * needed).  Deals the ceil(N/256) two-tile work units of each of `heads`
 * heads to `grid` CTAs exactly as the forward kernel does.  Writes up to
 * `capacity` triples (cta, head, pair) in dealing order and returns how many
 * units exist in total, or -1 on invalid arguments.  l2_budget_bytes sets how
 * many heads share an L2 group (0 = the library default).
 */
long long fa_sched_enumerate(int heads, int N, int d, int causal, int grid, long long l2_budget_bytes,
                             int* out_cta, int* out_head, int* out_pair, long long capacity);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
