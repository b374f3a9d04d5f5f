// Internal launch interface between the C-ABI layer and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace i8l {

// Quantizer: X (rows x cols, dtype dt) -> codes, scale, outlier list (first
// idx_cap entries; idx_cap < 0 means cap), count, sub (rows x cap fp16: the
// values of the first cap outlier columns). scratch: quant_scratch_words()
// 32-bit words.
// preflags: column flag words ([slabs][words], the layout of the scratch)
// handed over by the producer of X; the flags pass is then skipped.
//
// Columns of the weight's dequantized outlier slice kept for a staging width
// cap: a multiple of 8 (16-byte rows), at most 256.
inline int wsub_width(int cap) {
  if (cap <= 0) return 0;
  const int w = (cap + 7) & ~7;
  return w < 256 ? w : 256;
}
// With ow (forward only), the row pass also writes ow->wsub[n * wcap + j] =
// fp16(CB[n, O[j]] * (SCB[n] * (1/127))) for n < N, j < min(|O|, wcap): the
// dequantized weight values of the outlier columns (cols = the weight's K).
struct OutlierWeights {
  const int8_t* CB;
  const float* SCB;
  int N, K;
  uint16_t* wsub;
  int wcap;
};
size_t quant_scratch_words(int64_t rows, int64_t cols);
hipError_t launch_quantize(int dt, const void* X, int64_t rows, int cols, float tau, int8_t* codes, float* scale,
                           int32_t* idx, int32_t* count, uint16_t* sub, int cap, uint32_t* scratch,
                           hipStream_t st, const uint32_t* preflags = nullptr, int idx_cap = -1,
                           const OutlierWeights* ow = nullptr);

// Producer of a quantizer input: A = D(SiLU(H)) and A's column flag words
// (quant_scratch_words(rows, cols) words) for tau.
hipError_t launch_silu_flags(int dt, const void* H, int64_t rows, int cols, float tau, void* A, uint32_t* flags,
                             hipStream_t st);

// Forward GEMM with fused epilogue: out = D(CA.CB^T * SCA SCB / 127^2
// + A16[:, idx] . Wdq[:, idx]^T + bias); optional int32 export of CA.CB^T.
// The outlier values of the first cap columns come from subA (M x cap fp16),
// those of later columns straight from A (M x K of dt, fp16 cast on the fly);
// the weight values of the first wcap (wsub_width) columns from wsub (N x
// wcap fp16), later ones rebuilt from CB; idx holds all *count columns.
hipError_t launch_gemm_fwd(int dt, const int8_t* CA, const float* SCA, int M, const int8_t* CB, const float* SCB,
                           int N, int K, const uint16_t* subA, int cap, const uint16_t* wsub, int wcap,
                           const void* A, const int32_t* idx, const int32_t* count, const void* bias, void* out,
                           int32_t* c32, hipStream_t st);

// Kernel chosen for a forward / backward GEMM of this shape (operands 16-byte
// aligned): 0 none (empty output), 1 the generic 128 x 128 kernel, 2 the
// large 256 x 256 tile kernel, 3 the large kernel with 256 x 128 tiles.
int gemm_fwd_plan(int dt, int64_t M, int64_t N, int64_t K, bool aligned);
int gemm_bwd_plan(int dt, int64_t M, int64_t N, int64_t K, bool aligned);

// Backward-input GEMM: grad_A = D(fp16(G) . Wdq), Wdq built from CB on the fly.
hipError_t launch_gemm_bwd(int dt, const void* G, int M, int N, const int8_t* CB, const float* SCB, int K,
                           void* grad_A, hipStream_t st);

// Weight gradient of the trainable-weight mode: grad_W = D(fp16(G)^T . fp16(A)).
hipError_t launch_gemm_wgrad(int dt, const void* G, const void* A, int M, int N, int K, void* grad_W,
                             hipStream_t st);

// grad_bias[n] = D(sum_m G[m, n]) (fp32 accumulation, fixed order).
size_t grad_bias_partial_floats(int M, int N);
hipError_t launch_grad_bias(int dt, const void* G, int M, int N, float* partial, void* grad_bias, hipStream_t st);

// Adapters beside a shared projection: the tokens 0 .. T - 1 lie in n_seg
// consecutive segments; segment s holds tokens off[s] .. off[s + 1] - 1 (off[0]
// and off[n_seg] are taken as 0 and T) of adapter ids[s] (s itself when ids is
// NULL; none when outside [0, n_adapters)).
struct LoraSegs {
  const int32_t* off;
  const int32_t* ids;
  int n_seg, n_adapters;
};
size_t lora_forward_floats(int T, int K, int N, int R, int n_seg);
size_t lora_backward_floats(int T, int K, int N, int R, int n_adapters, int n_seg);
// Forward: T >= 1, V (T x R fp32) or NULL. ws: lora_*_floats() floats. S.n_adapters
// is 0 where nothing is to be read of the adapters (no rank); the backward's
// n_adapters is the one its workspace was sized with.
hipError_t launch_lora_forward(int dt, const void* X, int T, int K, const void* A, const void* B,
                               const float* scaling, int R, int N, const LoraSegs& S, const void* base, void* out,
                               float* V, float* ws, hipStream_t st);
hipError_t launch_lora_backward(int dt, const void* G, const void* X, const float* V, int T, int K, const void* A,
                                const void* B, const float* scaling, int R, int N, const LoraSegs& S,
                                int n_adapters, const void* base_grad, void* gX, void* gA, void* gB, float* ws,
                                hipStream_t st);

// Layer norm, T x C of dt, weight and bias of wdt (dt or fp32).
hipError_t launch_norm_forward(int dt, int wdt, const void* X, int T, int C, const void* w, const void* b, float eps,
                               void* Y, float* mean, float* rstd, hipStream_t st);
size_t norm_backward_floats(int T, int C);
hipError_t launch_norm_backward(int dt, int wdt, const void* G, const void* X, const float* mean, const float* rstd,
                                int T, int C, const void* w, void* gX, void* gw, void* gb, float* ws,
                                hipStream_t st);

// AdamW over a table of tensors: chunk c is values [chunk * adamw_chunk(), ...)
// of its tensor, one workgroup each.
struct AdamWTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  int64_t n;
  int32_t dtype, bits;
  int32_t vec, pad;   // vec: every pointer on a 16-byte border (codes 8)
};
struct AdamWChunk {
  int32_t tensor, chunk;
};
struct AdamWScalars {
  float beta1, one_beta1, beta2, one_beta2, keep, step_size, inv_root_bc2, eps;
};
int adamw_chunk();
hipError_t launch_adamw(const AdamWTensor* tensors, const AdamWChunk* chunks, int64_t n_chunks, const AdamWScalars& h,
                        const float* grad_scale, const float* found_inf, hipStream_t st);

}  // namespace i8l
