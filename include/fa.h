/*
 * fa.h -- C ABI of the GB300 (sm_103a) exact-attention library, libfa.so.
 *
 * The operation is exact scaled-dot-product attention computed tile by tile
 * with online softmax, so the N x N score and probability matrices never reach
 * device memory:
 *
 *     S = scale * Q K^T  (causal: S_ij = -inf for key j > query i),
 *     P = rowsoftmax(S),  O = P V,  lse_i = log sum_j exp(S_ij)
 *
 * ("FlashAttention-1", jshn9515 deep-learning-notes 10.2.1-10.2.3, for the
 * definition and the online-softmax rescaling; "Flash Attention V1/V2/V3演进",
 * sections V1分块原理 / 在线Softmax / V2并行优化, for tiling, the running
 * max/sum/output state and the one-time final normalisation; "5.4
 * FlashAttention", listing 3-1, for the alpha = exp(m_old - m_new) rescale.)
 * The backward recomputes P from the saved lse instead of storing it
 * ("FlashAttention-1", 10.2.4).
 *
 * Conventions shared by every entry point
 *   - Tensors are dense, contiguous, row-major [B][H][N][d]; lse and delta are
 *     [B][H][N].  There are no strides.  Every device pointer must be 16-byte
 *     aligned (tensor-memory-accelerator copies need it); a misaligned pointer
 *     is FA_ERR_INVALID_ARG.
 *   - All pointers are DEVICE pointers on the current CUDA device unless a
 *     comment says otherwise.  The caller owns every buffer, including the
 *     backward workspace; the library allocates no device memory per call.  It
 *     owns only one status word per device, created on first use.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Calls are asynchronous on that stream: they enqueue kernels and
 *     return without synchronising.
 *   - Return value: an fa_status.  Argument problems are detected on the host
 *     before anything is launched.  Errors that happen inside a kernel (a
 *     bounded wait that ran out) are recorded in the per-device status word and
 *     reported by fa_last_device_error().
 *   - `scale` multiplies Q K^T (the configurations use 1/sqrt(d)).
 *   - Any N >= 1 is accepted (tiles past N are zero-filled and masked).
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FA_F32 = 0, FA_BF16 = 1, FA_E4M3 = 2 } fa_dtype;

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,     /* null/misaligned pointer, N < 1, B/H < 1, bad dtype */
    FA_ERR_UNSUPPORTED = 2,     /* valid request this build does not implement      */
    FA_ERR_CUDA = 3,            /* a CUDA runtime/driver call or launch failed      */
    FA_ERR_DEVICE_TIMEOUT = 4,  /* a kernel's bounded wait ran out (device-side)    */
    FA_ERR_DEVICE_INDEX = 5     /* a page, position or length outside the 4-bit cache
                                   (device-side; the access was left out)           */
} fa_status;

/*
 * Size limits shared by every entry point: B*H (heads, or query heads) at most
 * 2^24, N (rows of one head) at most 2^24, and B*H*ceil(N/128) at most 2^31 - 1,
 * so that the kernels' work items (128-row blocks of one head) can be counted in
 * an int.  Larger sizes are refused with FA_ERR_UNSUPPORTED before anything runs.
 */

/*
 * Forward pass.  O = softmax(scale Q K^T [causal mask]) V and
 * lse_i = m_i + ln l_i (natural log, in units of the scaled score; m_i the row
 * max, l_i the row sum of exp(S_ij - m_i)), as on the "FlashAttention-1" page
 * 10.2.1 (standard attention, stable softmax) and 10.2.2 (online update).
 *
 *   q, k, v : [B][H][N][d] of `dtype`, read only.
 *   o       : [B][H][N][d] of `dtype`, written (fully overwritten).
 *   lse     : [B][H][N] float32, written.  May be NULL if not wanted.
 *   dtype   : FA_F32 (d = 64 or 128; exact fp32 CUDA-core kernel) or
 *             FA_BF16 (d = 64 or 128; tensor-core kernel with fp32
 *             accumulation; O rounded to bf16 to nearest even).
 *             FA_E4M3 is FA_ERR_INVALID_ARG here: use fa_fwd_fp8().
 *   causal  : 0 = full attention; 1 = key j attends only to queries i >= j.
 * Errors: FA_ERR_INVALID_ARG (null q/k/v/o, misalignment, B,H,N < 1, bad
 * dtype), FA_ERR_UNSUPPORTED (other d), FA_ERR_CUDA (launch failure).
 */
int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
           int B, int H, int N, int d, float scale, int causal, int dtype, void* stream);

/*
 * FP8 forward ("Flash Attention V1/V2/V3演进", section V3增强: FP8 matrix
 * inputs, FP32 accumulation, scale factors).  Inputs are OCP E4M3 codes with
 * one float32 dequantisation factor per tensor: the real value of element x is
 * e4m3(x) * x_descale.  The kernel computes the same O and lse as fa_fwd on the
 * dequantised inputs; P is re-quantised to E4M3 inside the kernel for the P V
 * product (accumulation stays fp32).
 *
 *   q8, k8, v8 : [B][H][N][d] uint8 E4M3 codes.
 *   o          : [B][H][N][d] bfloat16, written.
 *   lse        : [B][H][N] float32, written (may be NULL).
 *   d          : 128.
 * Errors: as fa_fwd; FA_ERR_INVALID_ARG also for a non-finite or <= 0 descale.
 */
int fa_fwd_fp8(const void* q8, const void* k8, const void* v8, void* o, float* lse,
               float q_descale, float k_descale, float v_descale,
               int B, int H, int N, int d, float scale, int causal, void* stream);

/*
 * Grouped-query forward: groups of H / H_kv query heads share one K/V head
 * (the "GQA" of the "5.4 FlashAttention" page's heading; the arithmetic per query
 * head is exactly fa_fwd's).  Query head h of batch b reads K/V head
 * b*H_kv + h / (H / H_kv).
 *
 *   q, o : [B][H][N][d] bfloat16;  k, v : [B][H_kv][N][d] bfloat16;  lse [B][H][N].
 *   dtype : FA_BF16.  d : 64 or 128.
 * Errors: as fa_fwd; FA_ERR_INVALID_ARG also for H_kv < 1 or H % H_kv != 0;
 * FA_ERR_UNSUPPORTED for FA_F32.
 */
int fa_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
               int H_kv, int N, int d, float scale, int causal, int dtype, void* stream);

/*
 * FP8 forward with one dequantisation factor per (batch, head) instead of per
 * tensor: finer scale factors ("Flash Attention V1/V2/V3演进", section V3增强).
 * Element x of head (b, h) has the real value e4m3(x) * x_descale[b*H + h].
 *
 *   q_descale, k_descale, v_descale : DEVICE float32 arrays of B*H factors.
 *   Other arguments as fa_fwd_fp8.
 * Errors: as fa_fwd_fp8; FA_ERR_INVALID_ARG also for a null descale array.  The
 * factors themselves are read on the device and not validated.
 */
int fa_fwd_fp8_per_head(const void* q8, const void* k8, const void* v8, void* o, float* lse,
                        const float* q_descale, const float* k_descale, const float* v_descale,
                        int B, int H, int N, int d, float scale, int causal, void* stream);

/*
 * FP8 forward with one dequantisation factor per 128-row block of each head, the
 * finest scale granularity here ("Flash Attention V1/V2/V3演进", section V3增强:
 * fine-grained scale factors).  Row i of head (b, h) of Q has the real value
 * e4m3(q8[b][h][i]) * q_descale[(b*H + h) * nb + i / 128], nb = ceil(N / 128), and the
 * same for K and V with their own arrays.  The result is the attention of the real
 * values, as fa_fwd_fp8.
 *
 *   q_descale, k_descale, v_descale : DEVICE float32 arrays of B*H*ceil(N/128)
 *                                     factors, positive and finite (read on the
 *                                     device, not validated).
 *   Other arguments as fa_fwd_fp8.
 * Method: the Q and K factors fold into the score constant per (query tile, key
 * block); V's factor for key block j scales P before its E4M3 rounding by
 * v_j / max_j v_j (at most 1), and the row sum and O are corrected exactly.
 * Errors: as fa_fwd_fp8_per_head.
 */
int fa_fwd_fp8_per_block(const void* q8, const void* k8, const void* v8, void* o, float* lse,
                         const float* q_descale, const float* k_descale, const float* v_descale,
                         int B, int H, int N, int d, float scale, int causal, void* stream);

/*
 * Forward over one shard of the keys, the per-shard step of sequence-sharded
 * attention: N_q queries at global positions q_offset + i against N_kv keys at
 * global positions kv_offset + j.  It is the forward of "FlashAttention-1",
 * 10.2.1-10.2.3, on the keys the shard holds; its normalised output and lse are
 * what fa_lse_merge combines across shards (the two-state combination of 10.2.2).
 *
 *   q        : [B][H][N_q][d] bfloat16.   k, v : [B][H_kv][N_kv][d] bfloat16
 *              (H_kv divides H; query head h reads K/V head h / (H / H_kv)).
 *   o_part   : [B][H][N_q][d] FLOAT32, written (the shard's normalised output).
 *   lse_part : [B][H][N_q] float32, written, required.
 *   causal   : 0, or 1: key j reaches query i iff kv_offset + j <= q_offset + i.
 *              A row that reaches no key of the shard gets O = 0, lse = -inf.
 *   dtype    : FA_BF16.  d : 64 or 128.  Offsets are only compared, never used
 *              to address memory: k and v start at the shard's first key.
 * Errors: as fa_fwd; FA_ERR_INVALID_ARG also for lse_part null, N_kv < 1, or
 * H_kv not dividing H.
 */
int fa_fwd_kv_shard(const void* q, const void* k, const void* v, float* o_part,
                    float* lse_part, int B, int H, int H_kv, int N_q, int N_kv, int d,
                    float scale, int causal, long long q_offset, long long kv_offset,
                    int dtype, void* stream);

/*
 * Merge n_parts shard outputs of the same queries over disjoint key sets
 * ("FlashAttention-1", 10.2.2: partial states combine through their maxima and
 * sums; with normalised parts the weight of part s is exp(lse_s - lse)):
 *     lse = ln sum_s exp(lse_s),   O = sum_s exp(lse_s - lse) O_s.
 * Parts with lse_s = -inf add nothing; a row with every lse_s = -inf gives O = 0
 * and lse = -inf.  The result equals the forward over the union of the keys up to
 * rounding.
 *
 *   o_parts   : [n_parts][B][H][N][d] float32 (the fa_fwd_kv_shard outputs,
 *               stacked), read only.   lse_parts : [n_parts][B][H][N] float32.
 *   o         : [B][H][N][d] written, bfloat16 (dtype FA_BF16) or float32
 *               (FA_F32).   lse : [B][H][N] float32, written, or NULL.
 *   n_parts   : 1 to 16.   d : 64 or 128.  Every pointer 16-byte aligned.
 * Errors: FA_ERR_INVALID_ARG (null/misaligned pointers, n_parts < 1, bad sizes or
 * dtype), FA_ERR_UNSUPPORTED (other d, n_parts > 16), FA_ERR_CUDA (launch failure).
 */
int fa_lse_merge(const float* o_parts, const float* lse_parts, int n_parts, void* o,
                 float* lse, int B, int H, int N, int d, int dtype, void* stream);

/*
 * Bytes of device workspace that fa_bwd needs for these sizes: the per-row
 * delta_i = dO_i . O_i and the pre-scaled lse (float32, N rounded up to 128
 * per head), plus for d = 64 the float32 dQ accumulator
 * ([B][H][N rounded up to 128][d]).
 * Returns 0 for invalid sizes and for sizes the backward refuses (beyond the
 * size limits above), whose byte count could overflow.
 */
size_t fa_bwd_workspace_size(int B, int H, int N, int d);

/*
 * Backward pass by recomputation ("FlashAttention-1", 10.2.4): with
 * P_ij = exp(S_ij - lse_i) rebuilt tile by tile from the saved lse,
 *     dV = P^T dO,   dP = dO V^T,   delta_i = dO_i . O_i,
 *     dS = P o (dP - delta),   dQ = scale dS K,   dK = scale dS^T Q.
 *
 *   q, k, v, o, dO : [B][H][N][d] bfloat16, read only (o from fa_fwd).
 *   lse            : [B][H][N] float32 from fa_fwd, read only.
 *   dq, dk, dv     : [B][H][N][d] bfloat16, written.
 *   workspace      : device buffer of at least fa_bwd_workspace_size() bytes,
 *                    owned by the caller; its contents on entry do not matter
 *                    and on return are unspecified.  Calls that overlap in time
 *                    must not share one workspace.
 *   dtype          : FA_BF16.   d : 64 or 128 (d = 64 accumulates dQ with fp32
 *                    atomics in the workspace; d = 128 computes dQ in a second,
 *                    query-parallel kernel, and its workspace holds no accumulator).
 *   causal         : 0, or 1 for the causal mask of the forward (key j reaches
 *                    only queries i >= j; lse must come from a causal forward).
 * Errors: FA_ERR_INVALID_ARG (null/misaligned pointers, workspace too small,
 * bad sizes), FA_ERR_UNSUPPORTED (other dtype or d),
 * FA_ERR_CUDA (launch failure).
 */
int fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
           const void* dO, void* dq, void* dk, void* dv, void* workspace,
           size_t workspace_bytes, int B, int H, int N, int d, float scale, int causal,
           int dtype, void* stream);

/*
 * Grouped-query backward, the gradient of fa_fwd_gqa: query head h of batch b
 * reads K/V head b*H_kv + h / (H / H_kv), so each K/V head's dK and dV are the
 * sums of the per-query-head gradients over the H / H_kv query heads sharing it
 * (the chain rule through the shared operand; the pages give the forward
 * grouping under "5.4 FlashAttention" and the per-head backward in
 * "FlashAttention-1", 10.2.4).  With H_kv = H this is fa_bwd.
 *
 *   q, o, dO : [B][H][N][d] bfloat16;  lse [B][H][N] float32 (from fa_fwd_gqa).
 *   k, v     : [B][H_kv][N][d] bfloat16.
 *   dq       : [B][H][N][d] bfloat16, written.
 *   dk, dv   : [B][H_kv][N][d] bfloat16, written (the group sums, accumulated
 *              in fp32 on chip and rounded once).
 *   workspace: at least fa_bwd_workspace_size(B, H, N, d) bytes (query heads).
 *   Other arguments as fa_bwd.
 * Errors: as fa_bwd; FA_ERR_INVALID_ARG also for H_kv < 1 or H % H_kv != 0.
 */
int fa_bwd_gqa(const void* q, const void* k, const void* v, const void* o, const float* lse,
               const void* dO, void* dq, void* dk, void* dv, void* workspace,
               size_t workspace_bytes, int B, int H, int H_kv, int N, int d, float scale,
               int causal, int dtype, void* stream);

/*
 * fa_bwd without a caller-supplied workspace, for callers that cannot allocate
 * device memory when they run the backward -- for example a plug-in called
 * from a host framework that owns the device memory budget and forbids
 * allocation inside its execution hook, or a latency-critical caller that
 * cannot afford cudaMalloc's implicit device synchronisation.  The pages have
 * no counterpart to this entry point; it is a deployment convenience.
 *
 * Arguments and results are those of fa_bwd minus (workspace,
 * workspace_bytes).  The scratch is a fixed 64 MiB array inside the library
 * (a file-scope __device__ array that every GPU loading the library holds until
 * the process exits); the call allocates nothing.  Sizes whose
 * fa_bwd_workspace_size() exceeds 64 MiB are refused with FA_ERR_UNSUPPORTED
 * before anything is launched (at d = 64 that allows B*H*ceil128(N) up to
 * 254,200 rows, e.g. B=4, H=16, N=2048).
 *
 * The first call on a device looks up the array's device address for that
 * device (with that device current); make that first call before any stream
 * capture.  All calls on a device share the one array and it keeps the last
 * call's contents: each call writes every scratch region it reads before
 * reading it, so nothing carries over, but calls that overlap in time on the
 * GPU (different streams, or other host threads) race on the array and give
 * wrong results.  FA_ERR_CUDA if the address lookup fails.
 */
int fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const float* lse,
                   const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                   float scale, int causal, int dtype, void* stream);

/* ------------------------------------------------------------------------
 * A layer's work around the attention call.
 * ------------------------------------------------------------------------ */

/*
 * Norm and rotation of the query and key heads, from a layer's projections to the
 * operands of the attention calls in one pass.  For each head row x of Q or K at
 * position t, with that operand's weights w:
 *     y = w o x / sqrt(mean(x^2) + eps),
 *     (y_a, y_b) -> (y_a cos A - y_b sin A,  y_b cos A + y_a sin A),  A = t inv_freq[p],
 * for the rot / 2 pairs p of its first `rot` elements: (a, b) = (p, p + rot / 2), or with
 * `interleaved` (2 p, 2 p + 1).  V is moved only.
 *
 *   qkv       : [B][N][H + 2 H_kv][d] of `dtype`: a token's query heads, then its key heads,
 *               then its value heads (the one tensor here that is not [B][H][N][d]).
 *   q_weight, k_weight : [d] float32, or NULL (ones).
 *   positions : [B][N] int32 (negative ones turn backwards), or NULL: the index in the
 *               sequence.
 *   inv_freq  : HOST array of rot / 2 doubles, radians per position, of up to 2^64 in magnitude;
 *               read before the call returns.  May be NULL if rot is 0.  Angles are exact to
 *               2^-24 of a turn at every int32 position.
 *   q, k, v   : [B][H][N][d] and twice [B][H_kv][N][d] of `dtype`, written; they must not
 *               overlap qkv.
 *   d : 64 or 128.  rot : a multiple of 16, 0 to d.  eps : finite, >= 0.
 *   dtype : FA_BF16 or FA_F32 (arithmetic in float32 either way: x^2 is summed in it, so that a
 *   row's largest magnitude has to be below 2^60, and with eps below 2^-100 above 2^-60).
 * Errors: FA_ERR_INVALID_ARG (null or misaligned pointers, B, H, H_kv, N < 1, bad rot, eps,
 * frequencies or dtype), FA_ERR_UNSUPPORTED (other d, sizes beyond the limits above, B*N
 * beyond 2^31 - 1), FA_ERR_CUDA (launch failure).
 */
int fa_qk_norm_rope(const void* qkv, const float* q_weight, const float* k_weight,
                    const int* positions, const double* inv_freq, void* q, void* k, void* v, int B,
                    int H, int H_kv, int N, int d, int rot, int interleaved, float eps, int dtype,
                    void* stream);

/*
 * Gradient of fa_qk_norm_rope.  With g the incoming row turned back by its angles and
 * r = (mean(x^2) + eps)^(-1/2):
 *     dx = r (w g - r^2 x mean(w g x)),    dw = sum over all rows of g r x.
 *
 *   dq, dk, dv : gradients of q, k, v, in their layouts, read only.
 *   dqkv       : gradient of qkv, in its layout, written; it must not overlap the inputs.
 *   dq_weight, dk_weight : [d] float32, written (the sum over all rows), or NULL if not
 *                wanted.  The sums have a fixed order: the same bits every time.
 *   workspace  : at least fa_qk_norm_rope_bwd_workspace_size() bytes of device memory; NULL
 *                with 0 bytes is accepted when neither weight gradient is wanted.  Calls that
 *                overlap in time must not share one.
 *   Other arguments as fa_qk_norm_rope; nothing of the forward is needed.
 * Errors: as fa_qk_norm_rope; FA_ERR_INVALID_ARG also for a workspace that is too small.
 */
int fa_qk_norm_rope_bwd(const void* qkv, const float* q_weight, const float* k_weight,
                        const int* positions, const double* inv_freq, const void* dq,
                        const void* dk, const void* dv, void* dqkv, float* dq_weight,
                        float* dk_weight, void* workspace, size_t workspace_bytes, int B, int H,
                        int H_kv, int N, int d, int rot, int interleaved, float eps, int dtype,
                        void* stream);
/* Bytes for any call with these sizes; 0 for sizes that the call refuses. */
size_t fa_qk_norm_rope_bwd_workspace_size(int B, int H, int H_kv, int N, int d);

/*
 * Norm and rotation as fa_qk_norm_rope with positions of several axes, such as the frame, row and
 * column of a video's tokens: pair p turns by A = t[axis[p]] inv_freq[p].
 *
 *   positions : [n_axes][B][N] int32 (may be NULL if rot is 0).
 *   axis      : HOST array of rot / 2 ints, the axis 0 .. n_axes - 1 of each pair; read before the
 *               call returns.  May be NULL if rot is 0.
 *   n_axes    : 1 to 8.
 *   Other arguments as fa_qk_norm_rope, with whose results these agree to the bit where all axes hold
 *   the same positions.
 * Errors: as fa_qk_norm_rope; FA_ERR_INVALID_ARG also for a bad axis or n_axes.
 */
int fa_qk_norm_rope_axes(const void* qkv, const float* q_weight, const float* k_weight,
                         const int* positions, const double* inv_freq, const int* axis, void* q,
                         void* k, void* v, int B, int H, int H_kv, int N, int d, int rot, int n_axes,
                         int interleaved, float eps, int dtype, void* stream);

/*
 * Gradient of fa_qk_norm_rope_axes, as fa_qk_norm_rope_bwd, whose workspace size holds here too.  The same
 * bits every time; against fa_qk_norm_rope_bwd's the weights' gradients may add up in another order.
 */
int fa_qk_norm_rope_axes_bwd(const void* qkv, const float* q_weight, const float* k_weight,
                             const int* positions, const double* inv_freq, const int* axis,
                             const void* dq, const void* dk, const void* dv, void* dqkv,
                             float* dq_weight, float* dk_weight, void* workspace,
                             size_t workspace_bytes, int B, int H, int H_kv, int N, int d, int rot,
                             int n_axes, int interleaved, float eps, int dtype, void* stream);

/*
 * Forward under a causal sliding window with sinks: query i sees key j iff j <= i and
 * (j > i - window or j < n_sink), the `window` newest keys (its own among them) and the
 * first n_sink ones.  O, lse and the grouping of heads as fa_fwd_gqa; only key blocks that
 * hold a visible key are read.
 *
 *   q, o : [B][H][N][d] bfloat16;  k, v : [B][H_kv][N][d] bfloat16;  lse : [B][H][N] float32,
 *   or NULL.   window >= 1 (N or more: plain causal), n_sink >= 0.   dtype : FA_BF16.
 * K and V are read in blocks of 128 keys: a NaN or an infinity in V reaches every query whose
 * blocks hold it (0 * NaN), hidden or not, as in fa_fwd.
 * Errors: as fa_fwd_gqa; FA_ERR_INVALID_ARG also for window < 1 or n_sink < 0.
 */
int fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                  int H_kv, int N, int d, float scale, int window, int n_sink, int dtype,
                  void* stream);

/*
 * Backward of fa_fwd_window, by recomputation from its lse, as fa_bwd_gqa over the pairs that
 * the forward saw.
 *   o, lse      : from fa_fwd_window with the same window and n_sink.
 *   dq          : [B][H][N][d];  dk, dv : [B][H_kv][N][d] bfloat16, written.
 *   workspace   : at least fa_bwd_window_workspace_size() bytes; its contents on entry do not
 *                 matter.  Calls that overlap in time must not share one.
 * Nothing is summed by atomics: the same bits every time.  A NaN or an infinity in q, k, v, o or dO
 * reaches the gradients of the rows whose 128-row blocks meet its own, hidden pairs or not (0 * NaN).
 * Errors: as fa_fwd_window; FA_ERR_INVALID_ARG also for a null lse and a workspace that is
 * too small.
 */
int fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse,
                  const void* dO, void* dq, void* dk, void* dv, void* workspace,
                  size_t workspace_bytes, int B, int H, int H_kv, int N, int d, float scale,
                  int window, int n_sink, int dtype, void* stream);
/* 0 for sizes that the call refuses. */
size_t fa_bwd_window_workspace_size(int B, int H, int H_kv, int N, int d, int window, int n_sink);

/*
 * Cross attention: N_q queries a batch to the N_kv keys of another sequence, such as an encoder's
 * states or a prompt that several samples continue.  Query batch b reads K/V batch
 * b / (B / B_kv) (B_kv = B: each its own) and query head h K/V head h / (H / H_kv); of a K/V
 * batch's keys the first kv_lengths[b] are seen by every query.  O and lse as fa_fwd; a sequence
 * of length 0 gives O = 0, lse = -inf.
 *
 *   q, o       : [B][H][N_q][d] bfloat16;  k, v : [B_kv][H_kv][N_kv][d] bfloat16;
 *                lse : [B][H][N_q] float32, or NULL.
 *   kv_lengths : [B_kv] int32, device, or NULL (all of N_kv).  Negative ones are taken as 0, those
 *                beyond N_kv as N_kv.  K and V from there on may hold anything, NaN too.
 *   workspace  : at least fa_fwd_cross_workspace_size() bytes (NULL if that is 0); its contents
 *                on entry do not matter.  Calls that overlap in time must not share one.
 *   dtype      : FA_BF16.   d : 64 or 128.
 * The work is divided by the lengths that the kernel reads, so that a captured call follows them;
 * the result depends on the inputs and the device alone.
 * Errors: FA_ERR_INVALID_ARG (null or misaligned pointers, sizes < 1, B % B_kv or H % H_kv not 0,
 * a scale that is not finite, bad dtype, a workspace that is too small), FA_ERR_UNSUPPORTED (other
 * dtype or d, sizes beyond the limits above for queries or keys, H / H_kv * N_q beyond 2^31 - 257),
 * FA_ERR_CUDA.
 */
int fa_fwd_cross(const void* q, const void* k, const void* v, const int* kv_lengths, void* o,
                 float* lse, void* workspace, size_t workspace_bytes, int B, int B_kv, int H,
                 int H_kv, int N_q, int N_kv, int d, float scale, int dtype, void* stream);
/* 0 for sizes that the call refuses, and where none is needed. */
size_t fa_fwd_cross_workspace_size(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d);

/*
 * Backward of fa_fwd_cross, by recomputation from its lse.  dK and dV are summed over the query heads
 * and the batches that share a K/V head, in float32 and rounded once; those of keys that no query
 * sees (from kv_lengths[b] on) are zeros, and so is dQ of queries without keys.
 *
 *   o, lse     : from fa_fwd_cross with the same kv_lengths.
 *   dO, dq     : [B][H][N_q][d] bfloat16;  dk, dv : [B_kv][H_kv][N_kv][d] bfloat16, written.
 *   workspace  : at least fa_bwd_cross_workspace_size() bytes; its contents on entry do not matter.
 *                Calls that overlap in time must not share one.
 * Nothing is summed by atomics: the same bits every time.  A NaN or an infinity in q, o or dO reaches the
 * gradients of the keys of its head that are seen, and may reach those of hidden keys.
 * Errors: as fa_fwd_cross; FA_ERR_INVALID_ARG also for a null lse.
 */
int fa_bwd_cross(const void* q, const void* k, const void* v, const int* kv_lengths, const void* o,
                 const float* lse, const void* dO, void* dq, void* dk, void* dv, void* workspace,
                 size_t workspace_bytes, int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d,
                 float scale, int dtype, void* stream);
/* 0 for sizes that the call refuses. */
size_t fa_bwd_cross_workspace_size(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d);

/*
 * Attention to a shared prefix and to each request's own tokens: fa_fwd_cross merged with
 * (o_own, lse_own), the same queries' attention to keys outside of k (from fa_decode_kv4, fa_fwd_window,
 * fa_fwd_gqa, ...):  lse = ln(e^lse_prefix + e^lse_own),
 * O = e^(lse_prefix - lse) O_prefix + e^(lse_own - lse) o_own.  The prefix is read once for all
 * batches that share it, whose rows fill tiles together.
 *
 *   o_own, lse_own : as o and lse, read; a row with lse_own = -inf has no keys of its own, and its o_own is
 *                    not used.  Finite lse_own are of up to 2^127 in magnitude; the lowest float is
 *                    taken as -inf.  o may be o_own and lse may be lse_own (in place); they must not
 *                    overlap otherwise.
 *   lse            : may be NULL.   Other arguments and errors as fa_fwd_cross.
 */
int fa_fwd_prefix(const void* q, const void* k, const void* v, const int* kv_lengths,
                  const void* o_own, const float* lse_own, void* o, float* lse, void* workspace,
                  size_t workspace_bytes, int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d,
                  float scale, int dtype, void* stream);
/* 0 for sizes that the call refuses, and where none is needed. */
size_t fa_fwd_prefix_workspace_size(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d);

/*
 * A paged K/V cache in 4 bits.  32 neighbouring values of a head share one scale
 * s = bf16(max|x| / 7); a value is held as the nearest integer to x / s (ties to even) in
 * -7 .. 7, as the nibble code + 8.  A group of zeros has s = 0; a group that holds an
 * infinity or a NaN has a NaN scale and reads back as NaN.  4.5 bits a value.
 *
 *   k_codes, v_codes   : [n_pages][H_kv][page][d / 2] bytes.
 *   k_scales, v_scales : [n_pages][H_kv][page][d / 32] bfloat16.
 * These are sizes; within a page the nibbles lie in the order in which the decode kernel
 * reads them (kv4.cuh), so that only these functions and code written to that order
 * address single values.  Zero-initialised pages are valid.
 *   block_table        : [B][max_blocks] int32: token i of request b is token i % page of
 *                        page block_table[b][i / page].  Entries past a request's tokens are
 *                        not read.
 *   page : 16, 32, 64, 128 or 256 tokens.   d : 64 or 128.
 * A page, position or length outside the cache that a kernel meets is left out (not written;
 * read as zeros; hidden from attention) and recorded as FA_ERR_DEVICE_INDEX.  A negative length
 * or count is taken as 0, a length beyond max_blocks * page as that, in all three calls.
 */

/*
 * Store rows of K and V: row i of request b becomes its token first[b] + i, for
 * i < count[b] (count NULL, or N and more: all N).  Two rows of one call must not name the same
 * token.
 *   k, v  : [B][H_kv][N][d] bfloat16, read only.
 *   first : [B] int32, device: tokens that the requests had before.   count : [B] int32 or NULL.
 * Errors: FA_ERR_INVALID_ARG (null or misaligned pointers, sizes < 1, bad page),
 * FA_ERR_UNSUPPORTED (other d, sizes beyond the limits above, max_blocks * page beyond
 * 2^31 - 256, B*H_kv*N beyond 2^31 - 1), FA_ERR_CUDA.
 */
int fa_kv4_append(const void* k, const void* v, void* k_codes, void* k_scales, void* v_codes,
                  void* v_scales, const int* block_table, const int* first, const int* count, int B,
                  int H_kv, int N, int d, int page, int n_pages, int max_blocks, void* stream);

/*
 * Read tokens 0 .. N - 1 of every request back as bfloat16 rows [B][H_kv][N][d] (code * s,
 * rounded to nearest even): the dense prefix that a chunked prompt attends to, for
 * fa_fwd_kv_shard.  Rows from lengths[b] on are written as zeros.  Errors: as fa_kv4_append.
 */
int fa_kv4_read(const void* k_codes, const void* k_scales, const void* v_codes,
                const void* v_scales, const int* block_table, const int* lengths, void* k, void* v,
                int B, int H_kv, int N, int d, int page, int n_pages, int max_blocks, void* stream);

/*
 * Attention of the N_q newest tokens of every request over the cache (their own keys and
 * values stored before the call): query i of request b is at position
 * p = lengths[b] - N_q + i and sees token j iff j <= p and, for window > 0,
 * (j > p - window or j < n_sink).  window = 0: every j <= p.  Query head h reads K/V head
 * h / (H / H_kv).  A query at a negative position (a request shorter than N_q, or empty) sees
 * nothing: O = 0, lse = -inf.
 *
 *   q, o  : [B][H][N_q][d] bfloat16.   lse : [B][H][N_q] float32, or NULL.  The scores take
 *           q to 2^-28 of its row's largest magnitude, which has to lie between 2^-85 and
 *           2^115 (or be 0).
 *   V       : P times V's scales is rounded to bfloat16 in that type's range: values above 2^100 in
 *           magnitude may overflow, groups of 32 below 2^-100 lose bits.
 *   lengths : [B] int32, device.
 *   workspace : at least fa_decode_kv4_workspace_size() bytes; its contents on entry do not
 *           matter.  Calls that overlap in time must not share one.
 * The work is divided by the lengths that the kernel reads, so that a captured call follows
 * them; the result depends on the inputs and the device alone.
 * Errors: as fa_kv4_append; FA_ERR_INVALID_ARG also for H % H_kv != 0, a scale that is not
 * finite, window < 0, n_sink < 0, or a workspace that is too small.
 */
int fa_decode_kv4(const void* q, const void* k_codes, const void* k_scales, const void* v_codes,
                  const void* v_scales, const int* block_table, const int* lengths, void* o,
                  float* lse, void* workspace, size_t workspace_bytes, int B, int H, int H_kv,
                  int N_q, int d, int page, int n_pages, int max_blocks, float scale, int window,
                  int n_sink, void* stream);
/* 0 for sizes that the call refuses. */
size_t fa_decode_kv4_workspace_size(int B, int H, int H_kv, int N_q, int d);

/*
 * Synchronise `stream`, then return and clear the current device's status
 * word: FA_OK, or the first device-side error recorded since the last call
 * (FA_ERR_DEVICE_TIMEOUT when a kernel's bounded wait ran out; that kernel
 * returned early and its outputs are undefined.  FA_ERR_DEVICE_INDEX: see the
 * 4-bit cache).  FA_ERR_CUDA if the synchronisation itself failed.
 */
int fa_last_device_error(void* stream);

/*
 * Upper bound, in nanoseconds of %globaltimer, on any single wait inside a
 * kernel launched after this call on any device (default 2e9 = 2 s; 0 restores
 * the default).  After it runs out the kernel records FA_ERR_DEVICE_TIMEOUT,
 * drains its own in-flight copies and matrix operations (with a fixed 1 s
 * bound), frees its tensor memory and returns.  Tests use a tiny limit to
 * exercise that path; it is not a tuning knob.
 */
void fa_set_wait_timeout_ns(uint64_t ns);

/*
 * Failure-path self test: launch a one-warp kernel whose single wait can never
 * be satisfied (nothing arrives on its barrier).  The bounded wait gives up
 * after the fa_set_wait_timeout_ns() limit and records FA_ERR_DEVICE_TIMEOUT,
 * which the next fa_last_device_error() returns.  Nothing faults or hangs.
 * Returns FA_OK if the kernel was launched.
 */
int fa_selftest_wait_timeout(void* stream);

/* Human-readable name of an fa_status value (static string). */
const char* fa_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
