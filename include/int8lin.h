/*
 * int8lin.h — C ABI of an LLM.int8-style row-wise quantized linear layer for
 * AMD Instinct MI355X (gfx950).
 *
 * The operations follow bitsandbytes PR #33 "Memory efficient backward"
 * (public pull request page):
 *   - PR description: int8 weights kept row-major; forward on int8; backward
 *     turns the int8 weights into fp16 weights on the fly and multiplies them
 *     with the fp16 output gradient, never storing fp16 weights; inputs are
 *     cast to fp16 and outputs back to the input dtype.
 *   - review "Cast A to fp16" and commit "cast to half before double_quant":
 *     the quantizer sees the fp16 cast of the activation.
 *   - review on the bias add and "4. Mixed-precision decomposition matmul":
 *     dequantized int8 product + bias + fp16 product of the outlier columns.
 *   - author notes: grad_bias from the un-cast gradient; frozen weight (no
 *     weight gradient).
 *   - review on the backward dequantization: CB * (SCB * (1/127)).
 *   - the has_fp16_weights option beside the memory-efficient one (a trainable
 *     weight re-quantized on each forward): int8_linear_backward_weight.
 * and EasyDeL discussion #66 ("Run and find Out": fwd_bits=8, bwd_bits=8), an
 * 8-bit backward dot product: int8_linear_backward_input_int8.
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller (the library
 *     never allocates, frees or synchronises, except int8_linear_forward_check
 *     which synchronises by definition). Every call only enqueues work on
 *     `stream` (a hipStream_t passed as void*; NULL = the default stream).
 *     Kernels run on the calling thread's current device, which must be the
 *     one of `stream` and of the tensors (the Python binding sees to it).
 *   - Tensors are dense and row-major (last dimension contiguous); leading
 *     batch dimensions are flattened into the row count by the caller.
 *   - dtype: I8L_F32, I8L_F16 or I8L_BF16 (bf16 passed as raw 16-bit words).
 *     fp16 casts and narrowing casts round to nearest even.
 *   - Workspaces are caller-owned device buffers of at least the size the
 *     matching *_workspace_bytes() function returns, 256-byte aligned. Their
 *     contents need no initialisation and are overwritten by each call.
 *   - Return value: I8L_OK (0) or a negative error code. Argument errors are
 *     detected on the host BEFORE any HIP call (nothing is enqueued); launch
 *     errors are reported as I8L_EHIP. Faults inside kernels surface, as in
 *     HIP, at the caller's next synchronisation.
 *   - Calls are stateless and reentrant; results are bitwise deterministic.
 *   - Graph capture: every call except int8_linear_forward_check enqueues
 *     kernels only (no allocation, memset or synchronisation), so it can be
 *     recorded by HIP stream capture and replayed; the pointers are captured,
 *     so a replay reads whatever the buffers hold then. The first call of a
 *     kernel family on a device raises that kernel's LDS limit
 *     (hipFuncSetAttribute); make one ordinary call before capturing.
 *   - Outlier threshold tau: a feature column is an outlier column when any
 *     row of the (flattened) input has |fp16(x)| > tau (strict, compared in
 *     fp32). tau <= 0, tau = +inf or NaN disables the split.
 */
#ifndef INT8LIN_H
#define INT8LIN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { I8L_F32 = 0, I8L_F16 = 1, I8L_BF16 = 2 } i8l_dtype;

enum {
  I8L_OK = 0,
  I8L_EINVAL = -1,     /* NULL pointer, negative size, misaligned workspace */
  I8L_EDTYPE = -2,     /* dtype not one of i8l_dtype */
  I8L_ESHAPE = -3,     /* size beyond what the kernels index, or K > I8L_MAX_K */
  I8L_EWORKSPACE = -4, /* workspace NULL or smaller than required */
  I8L_EHIP = -5,       /* a HIP launch or copy failed */
  I8L_EOVERFLOW = -6,  /* reserved: no call returns it (the forward handles any number of
                          outlier columns; int8_quantize_rowwise reports |O| > cap
                          through its count) */
  I8L_ESCRATCH = -7    /* problem larger than the static scratch of the allocation-free
                          forward */
};

/* Largest contraction length whose int32 accumulator cannot overflow:
 * 127 * 127 * K < 2^31. */
#define I8L_MAX_K 133144
/* Widest row int8_quantize_rowwise accepts (column flags kept on chip). */
#define I8L_MAX_COLS 262144

/* Short text for an error code (static storage). */
const char* int8_linear_strerror(int code);

/* ------------------------------------------------------------------------ *
 * Row-wise quantization (bitsandbytes PR #33: "Cast A to fp16" review, commit
 * "cast to half before double_quant"; the 127 scale of the dequantization
 * review). For X (rows x cols):
 *   X16       = fp16(X)
 *   O         = ascending outlier columns of X16 (see tau above)
 *   s[r]      = max over c not in O of |X16[r, c]|        (0 if none)
 *   codes     = clamp(rint(fl32(X16 * fl32(127 / s[r]))), -127, 127), 0 on O
 *               and on rows with s[r] = 0; -128 is never produced
 *   sub[r, j] = X16[r, O[j]] for j < min(|O|, cap)
 * Outputs (device): codes rows x cols int8; row_scale rows fp32 (s, exact);
 * outlier_idx cap int32 (first min(|O|, cap) entries written);
 * outlier_count 1 int32 (= |O|, may exceed cap: overflow is then visible);
 * sub rows x cap fp16 bits (leading dimension cap; only columns j < |O| are
 * written). outlier_idx / sub may be NULL when cap = 0.
 * cols <= I8L_MAX_COLS, else I8L_ESHAPE.
 * Weights are quantized with this call and tau off: CB = codes, SCB = s.
 * ------------------------------------------------------------------------ */
size_t int8_quantize_rowwise_workspace_bytes(int64_t rows, int64_t cols);

int int8_quantize_rowwise(const void* X, int dtype, int64_t rows, int64_t cols, float threshold,
                          int8_t* codes, float* row_scale, int32_t* outlier_idx, int32_t* outlier_count,
                          uint16_t* sub, int32_t cap, void* workspace, size_t workspace_bytes,
                          void* stream);

/* ------------------------------------------------------------------------ *
 * Forward (bitsandbytes PR #33, review on the bias add and
 * "4. Mixed-precision decomposition matmul"):
 *   (CA, SCA, O, subA) = quantize(A, tau)                      (as above)
 *   C32[m, n] = sum_k CA[m, k] * CB[n, k]                      (exact int32)
 *   Wdq[n, k] = fp16(fl32(CB[n, k] * fl32(SCB[n] * fl32(1/127))))
 *   out[m, n] = D(C32 * SCA[m] * SCB[n] / 127^2 + sum_j subA[m, j] * Wdq[n, O[j]]
 *                 + bias[n])                                    (fp32 accumulate)
 * A: M x K of `dtype`; CB: N x K int8 row-major; SCB: N fp32; bias: N of
 * `dtype` or NULL; out: M x N of `dtype`; c32_debug: M x N int32 or NULL
 * (exports C32). K <= I8L_MAX_K.
 * cap (>= 0): columns of the workspace's fp16 outlier sub-matrix subA. The
 * values of the first cap outlier columns are staged there by the quantizer;
 * the epilogue reads those of any further outlier column from A itself (the
 * same fp16 cast), so every |O| <= K is handled and the output is complete
 * for any cap. The row pass also writes the dequantized weight values of
 * the first wcap outlier columns, wcap = cap rounded up to a multiple of 8
 * and at most 256 (N x wcap fp16: the weight side of the outlier product,
 * rebuilt from CB on every call), so that the epilogue reads both operands
 * of that product as contiguous rows; the weight values of further columns
 * are rebuilt from CB by the epilogue. A small cap (a few times the expected
 * |O|) keeps the workspace at about M*K + 2*(M + N)*cap bytes.
 * The workspace holds the quantized activation (CA, SCA), the full outlier
 * list (K entries), subA, the weight slice and the quantizer's flag words;
 * its layout is
 * reported by int8_linear_forward_workspace_layout so that tests can read it
 * back. A must stay unchanged until the call has run (it is read twice by the
 * quantizer and again by the epilogue).
 * ------------------------------------------------------------------------ */
typedef struct {
  size_t count;   /* int32 |O| */
  size_t idx;     /* int32[K] outlier columns, ascending (first |O| valid) */
  size_t scale;   /* fp32[M] SCA */
  size_t codes;   /* int8[M*K] CA */
  size_t sub;     /* fp16[M*cap] subA: A16[:, O[j]] for j < min(|O|, cap) */
  size_t wsub;    /* fp16[N*wcap] (wcap above): Wdq[n, O[j]] for j < min(|O|, wcap) */
  size_t total;   /* bytes required */
} i8l_forward_layout;

size_t int8_linear_forward_workspace_bytes(int64_t M, int64_t K, int64_t N, int32_t cap);
int int8_linear_forward_workspace_layout(int64_t M, int64_t K, int64_t N, int32_t cap, i8l_forward_layout* layout);

int int8_linear_forward(const void* A, int dtype, int64_t M, int64_t K, const int8_t* CB, const float* SCB,
                        int64_t N, const void* bias, float threshold, int32_t cap, void* out, int32_t* c32_debug,
                        void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ *
 * Allocation-free forward, for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): int8_linear_forward with the same inputs, outputs, arithmetic
 * and errors, but its workspace is a static array inside the library
 * (I8L_NOALLOC_SCRATCH_BYTES = 64 MiB per GPU, reserved on each GPU the
 * library runs on until the process ends) and the outlier staging width is
 * min(K, 64) (further outlier columns are read from A, as in the forward).
 * The call allocates nothing and calls no allocating routine.
 *   int8_linear_forward_noalloc_bytes(M, K, N): scratch bytes a call needs
 *     (the forward workspace at that staging width);
 *   int8_linear_forward_noalloc_max_bytes(): the limit, I8L_NOALLOC_SCRATCH_BYTES.
 * A problem needing more (about M*K + 128*(M + N) bytes above 64 MiB) is
 * rejected with I8L_ESCRATCH on the host, before any HIP call. The first call
 * on a GPU looks up that GPU's copy of the array (the current device must be
 * the stream's). Every call on one GPU shares that copy: calls that overlap
 * on one GPU (different streams, or different host threads without
 * ordering) race and give wrong results; calls in one stream are ordered and
 * safe. Nothing in the array needs to start at zero.
 * ------------------------------------------------------------------------ */
#define I8L_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

size_t int8_linear_forward_noalloc_bytes(int64_t M, int64_t K, int64_t N);
size_t int8_linear_forward_noalloc_max_bytes(void);

int int8_linear_forward_noalloc(const void* A, int dtype, int64_t M, int64_t K, const int8_t* CB, const float* SCB,
                                int64_t N, const void* bias, float threshold, void* out, void* stream);

/* ------------------------------------------------------------------------ *
 * Outlier flags handed over by the producer of the input (EasyDeL discussion
 * #66, "Run and find Out": Dense -> SiLU -> Dense). The outlier columns of a
 * layer input are a property of all its rows, so the quantizer normally reads
 * the input once to flag them and once to quantize. When the input is made
 * by the activation kernel below, that kernel flags the columns as it writes
 * them and the flagged forward skips the flagging read.
 *
 * int8_outlier_flags_words(rows, cols): size of the flag buffer in uint32
 * words for an input of rows x cols (row slabs x ceil(cols / 32) words).
 *
 * int8_silu_outlier_flags: A = D(SiLU(H)) elementwise, SiLU(x) = x / (1 +
 * exp(-x)) evaluated in fp32 (within four fp32 units in the last place) and
 * rounded once to `dtype`; flags = the
 * outlier-column flags of A for `threshold` (a column is flagged when any row
 * has |fp16(A)| > threshold; threshold <= 0, +inf or NaN flags nothing).
 * H, A: rows x cols of `dtype` (A may not overlap H); flags: the caller's
 * buffer of flag_words >= int8_outlier_flags_words(rows, cols) words, fully
 * overwritten (I8L_EWORKSPACE when smaller).
 *
 * int8_linear_forward_flagged: int8_linear_forward with the outlier columns
 * given by `flags` (from int8_silu_outlier_flags on the same rows x K shape;
 * the threshold is the one the flags were made with) instead of found by a
 * pass over A. Same workspace, outputs and errors as int8_linear_forward;
 * flags NULL (with M, K > 0) is I8L_EINVAL, flag_words below
 * int8_outlier_flags_words(M, K) is I8L_EWORKSPACE.
 * ------------------------------------------------------------------------ */
size_t int8_outlier_flags_words(int64_t rows, int64_t cols);

int int8_silu_outlier_flags(const void* H, int dtype, int64_t rows, int64_t cols, float threshold, void* A,
                            uint32_t* flags, size_t flag_words, void* stream);

int int8_linear_forward_flagged(const void* A, int dtype, int64_t M, int64_t K, const uint32_t* flags,
                                size_t flag_words, const int8_t* CB, const float* SCB, int64_t N, const void* bias,
                                int32_t cap, void* out, int32_t* c32_debug, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Synchronises `stream` and reads the outlier count |O| of the last forward
 * that used `workspace` (laid out for M, K, N, cap) into *count (if non-NULL).
 * Returns I8L_OK, or I8L_EINVAL / I8L_EHIP. The forward's output is complete
 * for every count, so this call is a diagnostic, not a required check. */
int int8_linear_forward_check(const void* workspace, int64_t M, int64_t K, int64_t N, int32_t cap, void* stream,
                              int32_t* count);

/* Which GEMM kernel a call of this shape launches, for operands with the
 * alignment of device allocations (host only: no HIP call, no device
 * memory). int8_linear_forward_plan(dtype, M, K, N) for the forward product
 * (also the int8 backward's, with K and N exchanged) and
 * int8_linear_backward_plan(dtype, M, N, K) for the input gradient:
 * 0 nothing to compute (empty output), 1 the generic 128 x 128 tile kernel,
 * 2 the large pipelined kernel with 256 x 256 tiles, 3 the large kernel with
 * 256 x 128 tiles (chosen where 256 x 256 tiles would fill at most half of the
 * chip's 256 compute units). Negative: the error the call itself would
 * return for these sizes or dtype. Used by tests to check the dispatch. */
int int8_linear_forward_plan(int dtype, int64_t M, int64_t K, int64_t N);
int int8_linear_backward_plan(int dtype, int64_t M, int64_t N, int64_t K);

/* ------------------------------------------------------------------------ *
 * Memory-efficient backward, input gradient only (bitsandbytes PR #33, PR
 * description, backward-dequantization review, author notes):
 *   grad_A[m, k]  = D(sum_n fp16(G[m, n]) * Wdq[n, k])   (fp32 accumulate)
 *   grad_bias[n]  = D(sum_m G[m, n])   on the un-cast G    (fp32 accumulate)
 * G: M x N of `dtype`; CB: N x K int8 row-major; SCB: N fp32; grad_A: M x K
 * of `dtype`; grad_bias: N of `dtype` or NULL (then no workspace is needed).
 * No weight gradient exists: the int8 weight is frozen.
 * ------------------------------------------------------------------------ */
size_t int8_linear_backward_workspace_bytes(int64_t M, int64_t N, int with_grad_bias);

int int8_linear_backward_input(const void* G, int dtype, int64_t M, int64_t N, const int8_t* CB, const float* SCB,
                               int64_t K, void* grad_A, void* grad_bias, void* workspace, size_t workspace_bytes,
                               void* stream);

/* ------------------------------------------------------------------------ *
 * int8 backward variant (EasyDeL discussion #66, "Run and find Out": a Dense
 * layer with fwd_bits=8, bwd_bits=8 computes its backward dot product in 8
 * bits). Not the memory-efficient backward above: here both operands of the
 * input-gradient product are int8, with scales constant along the
 * contraction N:
 *   (CG, SG)     = quantize(G, tau off)                    (row-wise, per token)
 *   C32[m, k]    = sum_n CG[m, n] * CBt[k, n]              (exact int32)
 *   grad_A[m, k] = D(C32 * SG[m] * SCBt[k] / 127^2)        (fp32 arithmetic)
 *   grad_bias[n] = D(sum_m G[m, n])   on the un-cast G       (fp32 accumulate)
 * CBt / SCBt: a second offline int8 copy of the weight, W^T (K x N, row-major)
 * quantized with int8_quantize_rowwise and tau off (one scale per input
 * feature k). G: M x N of `dtype`; grad_A: M x K of `dtype`; grad_bias: N of
 * `dtype` or NULL; c32_debug: M x K int32 or NULL (exports C32).
 * N <= I8L_MAX_K. The workspace holds CG, SG and the quantizer's scratch.
 * ------------------------------------------------------------------------ */
size_t int8_linear_backward_int8_workspace_bytes(int64_t M, int64_t N, int with_grad_bias);

int int8_linear_backward_input_int8(const void* G, int dtype, int64_t M, int64_t N, const int8_t* CBt,
                                    const float* SCBt, int64_t K, void* grad_A, void* grad_bias, int32_t* c32_debug,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ *
 * Weight gradient of the trainable-weight mode (bitsandbytes PR #33 names a
 * has_fp16_weights option beside the memory-efficient backward; the weight
 * then stays a trainable tensor that is re-quantized on each forward):
 *   grad_W[n, k] = D(sum_m fp16(G[m, n]) * fp16(A[m, k]))   (fp32 accumulate)
 * G: M x N and A: M x K of `dtype` (the output gradient and the layer input,
 * both row-major); grad_W: N x K of `dtype`, row-major (the weight's layout).
 * M = 0 writes zeros. Needs no workspace. Errors: I8L_EDTYPE, I8L_EINVAL
 * (negative size, NULL pointer where data is needed), I8L_ESHAPE (a size
 * beyond INT32_MAX or a product beyond 2^40), I8L_EHIP (launch failure).
 * ------------------------------------------------------------------------ */
int int8_linear_backward_weight(const void* G, const void* A, int dtype, int64_t M, int64_t N, int64_t K,
                                void* grad_W, void* stream);

/* ------------------------------------------------------------------------ *
 * Low-rank adapters of many requests beside a shared projection (lit-gpt PR
 * #275 fine-tunes low-rank adapters beside frozen quantized weights). The T
 * token rows lie in n_seg consecutive segments (requests or sequences):
 * segment j holds rows seg_offsets[j] .. seg_offsets[j + 1] - 1 and uses
 * adapter seg_adapter[j]. For a row t of adapter a, with factor s[a]:
 *   V[t, r]   = sum_k A[a, r, k] X[t, k]                           (fp32)
 *   out[t, n] = D(base[t, n] + s[a] sum_r B[a, n, r] V[t, r])      (fp32 accumulate)
 * and the gradients
 *   dV[t, r]     = s[a] sum_n B[a, n, r] G[t, n]                   (fp32)
 *   grad_X[t, k] = D(base_grad[t, k] + sum_r A[a, r, k] dV[t, r])
 *   grad_A[a, r, k] = D(sum over the rows t of adapter a of dV[t, r] X[t, k])
 *   grad_B[a, n, r] = D(s[a] sum over the rows t of adapter a of G[t, n] V[t, r])
 * V and dV are never rounded below fp32's 24 bits except for the matrix
 * products with 16-bit operands, where they enter as the sum of two values of
 * that type, within 2^-17 of the value. In fp16 these are scaled by a power of
 * two, and a value below 2^-22 of the largest of its set is off by up to 2^-39
 * of that one instead; the set is one row of V or dV for out and grad_X (no row
 * depends on another), and the rows of a tile for grad_A and grad_B.
 * An infinity or NaN in an operand reaches the outputs that the formulas say
 * and no others; with 16-bit operands an infinity in A, B, X or G can arrive as
 * a NaN (it meets both parts of V or dV, one of which may be 0).
 *   X: T x K, out / base: T x N, A: n_adapters x R x K, B: n_adapters x N x R,
 *   G: T x N, grad_X / base_grad: T x K, all of `dtype`; grad_A, grad_B: as A
 *   and B; scaling: n_adapters fp32; V: T x R fp32.
 *   seg_offsets: n_seg + 1 int32 on the device, non-decreasing from 0 to T
 *   (the first and last are taken as 0 and T; may be NULL when n_seg <= 1).
 *   Contents that are not non-decreasing give undefined values in the outputs
 *   but no access outside the tensors. seg_adapter: n_seg int32 on the device,
 *   NULL for segment j using adapter j. A segment whose adapter lies outside
 *   [0, n_adapters) has none: out = D(base), V = 0, grad_X = D(base_grad). Empty
 *   segments are fine; one token per segment is the form for serving single
 *   tokens.
 *   base, base_grad: NULL for 0; may be the output itself (updated in place).
 *   Adapters of different ranks are stored with the largest, padded with zeros.
 * Forward: V may be NULL (kept for the backward otherwise). Backward: grad_X,
 * grad_A and grad_B may each be NULL (not computed); V is the forward's. An
 * adapter without rows gets a zero gradient.
 * R <= I8L_LORA_MAX_RANK, K and N <= I8L_MAX_COLS, n_adapters <= 65535,
 * T <= 2^24, n_seg <= 2^20, and n_adapters * max(K, N) * (R rounded up to 16,
 * 32, 64 or 128) <= 2^33, else I8L_ESHAPE. Apart from base and base_grad no
 * output may overlap an input. Forward and backward may return 0 as their
 * workspace's size; workspace may then be NULL.
 * ------------------------------------------------------------------------ */
#define I8L_LORA_MAX_RANK 128

size_t int8_lora_forward_workspace_bytes(int64_t T, int64_t K, int64_t N, int64_t R, int64_t n_seg);

int int8_lora_forward(const void* X, int dtype, int64_t T, int64_t K, const void* A, const void* B,
                      const float* scaling, int64_t n_adapters, int64_t R, int64_t N, const int32_t* seg_offsets,
                      const int32_t* seg_adapter, int64_t n_seg, const void* base, void* out, float* V,
                      void* workspace, size_t workspace_bytes, void* stream);

size_t int8_lora_backward_workspace_bytes(int64_t T, int64_t K, int64_t N, int64_t R, int64_t n_adapters,
                                          int64_t n_seg);

int int8_lora_backward(const void* G, const void* X, const float* V, int dtype, int64_t T, int64_t K, const void* A,
                       const void* B, const float* scaling, int64_t n_adapters, int64_t R, int64_t N,
                       const int32_t* seg_offsets, const int32_t* seg_adapter, int64_t n_seg, const void* base_grad,
                       void* grad_X, void* grad_A, void* grad_B, void* workspace, size_t workspace_bytes,
                       void* stream);

/* ------------------------------------------------------------------------ *
 * Layer norm in front of a projection, and its gradient. Per row of X (T x C):
 *   mean = sum x / C, rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)      (fp32)
 *   out  = D((x - mean) rstd w + b)
 * and with h = (x - mean) rstd, u = G w:
 *   grad_X = D(rstd (u - mean(u) - h mean(u h)))
 *   grad_w = Dw(sum over rows of G h), grad_b = Dw(sum over rows of G)
 * X, out, G, grad_X: T x C of `dtype`; weight, bias and their gradients: C of
 * `weight_dtype`, which is `dtype` or I8L_F32. bias may be NULL. mean, rstd: T
 * fp32, written by the forward (each may be NULL) and read by the backward.
 * grad_X, grad_weight and grad_bias may each be NULL (not computed). out may be
 * X; grad_X may be G unless a weight or bias gradient is asked for too. T = 0
 * writes zero weight gradients. C <= I8L_MAX_COLS, T <= 2^24, else I8L_ESHAPE; an
 * eps that is negative or NaN is I8L_EINVAL. A few rows need no workspace (its
 * size is 0, it may be NULL).
 * ------------------------------------------------------------------------ */
int int8_layer_norm_forward(const void* X, int dtype, int64_t T, int64_t C, const void* weight, const void* bias,
                            int weight_dtype, float eps, void* out, float* mean, float* rstd, void* stream);

size_t int8_layer_norm_backward_workspace_bytes(int64_t T, int64_t C);

int int8_layer_norm_backward(const void* G, const void* X, int dtype, int64_t T, int64_t C, const float* mean,
                             const float* rstd, const void* weight, int weight_dtype, void* grad_X,
                             void* grad_weight, void* grad_bias, void* workspace, size_t workspace_bytes,
                             void* stream);

/* ------------------------------------------------------------------------ *
 * AdamW over many tensors in one launch, states in 32 or in 8 bits (lit-gpt PR
 * #275 reports its runs with an 8-bit optimizer). Per value, with g' = c g
 * (c = *grad_scale, 1 without):
 *   m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2
 *   w = w (1 - lr weight_decay) - lr / (1 - beta1^step) m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * every operation rounded to fp32. w is `master` where that is non-NULL (then
 * p = D(w)), else p itself.
 * state_bits 32: m, v are n fp32. state_bits 8: m and v are n bytes of e4m3
 * codes in blocks of 256 values from the tensor's start, m_scale and v_scale
 * ceil(n / 256) fp32, one scale per block: m = code * scale, and v's codes hold
 * its root, sqrt(v) = code * scale. The scale is the least power of two, 2^-126
 * or more, with the block's largest magnitude / scale <= 448; codes round to
 * nearest even, and a sqrt(v) over 0 keeps at least the smallest code over 0
 * (2^-9). The step uses m and v before that rounding. A block with an infinity
 * or NaN in it gets the scale NaN. All-zero bytes and scales are the state
 * before the first step.
 * The tensors are described on the host, checked and laid out once:
 *   int8_adamw_table_bytes: size of the table of these tensors (0: invalid)
 *   int8_adamw_table_fill: checks them, writes the table to host memory and the
 *     number of workgroups to *chunks. The caller copies it to device memory
 *     (16-byte aligned) and keeps it, and the tensors, while steps use it.
 *   int8_adamw_step: one step of every tensor in the table; `count` and
 *     `chunks` as they were filled in. step >= 1 counts the steps, this one
 *     included. grad_scale, found_inf: device fp32, or NULL; *found_inf != 0
 *     leaves everything as it is.
 * A beta outside [0, 1), or a negative or non-finite lr, eps or weight_decay is
 * I8L_EINVAL. Each value is read and written by one thread: no two tensors
 * may overlap. A captured step keeps the lr, step and other numbers of its
 * capture; grad_scale and found_inf are read at each replay.
 * ------------------------------------------------------------------------ */
typedef struct {
  void* p;           /* n of dtype */
  const void* g;     /* n of dtype */
  void* m;
  void* v;
  float* m_scale;    /* state_bits 8 only */
  float* v_scale;    /* state_bits 8 only */
  float* master;     /* n fp32 or NULL */
  int64_t n;
  int32_t dtype;
  int32_t state_bits;
} i8l_adamw_tensor;

size_t int8_adamw_table_bytes(const i8l_adamw_tensor* tensors, int64_t count);
int int8_adamw_table_fill(const i8l_adamw_tensor* tensors, int64_t count, void* table, size_t table_bytes,
                          int64_t* chunks);
int int8_adamw_step(const void* table, int64_t count, int64_t chunks, double lr, double beta1, double beta2,
                    double eps, double weight_decay, int64_t step, const float* grad_scale, const float* found_inf,
                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* INT8LIN_H */
