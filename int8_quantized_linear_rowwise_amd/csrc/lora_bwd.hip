// Low-rank adapters of many requests beside a shared projection.
//
// Token t of adapter a: V[t] = A[a] x[t] (R values, fp32) and
//   y[t] = D(base[t] + s[a] B[a] V[t]);
// backward, g = dL/dy:
//   dV[t] = s[a] B[a]^T g[t],  dx[t] = D(base_grad[t] + A[a]^T dV[t]),
//   dA[a] = D(sum_t dV[t] x[t]^T),  dB[a] = D(s[a] sum_t g[t] V[t]^T).
#include "lora.hpp"

namespace i8l {

constexpr int TM = 16;

// P[t, r] = f sum_k X[t, k] W(r, k); W(r, k) = W[a][r][k], or W[a][k][r] if WT.
template <int DT, bool WT>
__global__ __launch_bounds__(256) void k_lora_shrink(const typename Elem<DT>::T* __restrict__ X, int T, int K,
                                                     const typename Elem<DT>::T* __restrict__ W, int R,
                                                     const float* __restrict__ scaling, LoraSegs S,
                                                     float* __restrict__ P) {
  const LoraTile tl = lora_tile(S, blockIdx.x + 1, T, TM);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = tl.t1 - tl.t0;
  const float f = (tl.adapter >= 0 && scaling) ? scaling[tl.adapter] : 1.0f;
  const typename Elem<DT>::T* Wa = W + (int64_t)max(tl.adapter, 0) * R * K;
  for (int j = wave; j < n * R; j += 4) {
    const int t = tl.t0 + j / R, r = j % R;
    float s = 0.0f;
    if (tl.adapter >= 0)
      for (int k = lane; k < K; k += 64)
        s = __builtin_fmaf(Elem<DT>::to_f32(X[(int64_t)t * K + k]),
                           Elem<DT>::to_f32(Wa[WT ? (int64_t)k * R + r : (int64_t)r * K + k]), s);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
    if (lane == 0) P[(int64_t)t * R + r] = s * f;
  }
}

// out[t, n] = D(base[t, n] + f sum_r P[t, r] W(n, r)); W(n, r) = W[a][n][r], or W[a][r][n] if WT.
template <int DT, bool WT>
__global__ __launch_bounds__(256) void k_lora_expand(const float* __restrict__ P, int T, int N,
                                                     const typename Elem<DT>::T* __restrict__ W, int R,
                                                     const float* __restrict__ scaling, LoraSegs S,
                                                     const typename Elem<DT>::T* base, typename Elem<DT>::T* out) {
  const LoraTile tl = lora_tile(S, blockIdx.x + 1, T, TM);
  const float f = (tl.adapter >= 0 && scaling) ? scaling[tl.adapter] : 1.0f;
  const typename Elem<DT>::T* Wa = W + (int64_t)max(tl.adapter, 0) * R * N;
  const int n = blockIdx.y * 256 + threadIdx.x;
  if (n >= N) return;
  for (int t = tl.t0; t < tl.t1; ++t) {
    float s = 0.0f;
    if (tl.adapter >= 0)
      for (int r = 0; r < R; ++r)
        s = __builtin_fmaf(P[(int64_t)t * R + r], Elem<DT>::to_f32(Wa[WT ? (int64_t)r * N + n : (int64_t)n * R + r]),
                           s);
    const int64_t at = (int64_t)t * N + n;
    out[at] = Elem<DT>::from_f32((base ? Elem<DT>::to_f32(base[at]) : 0.0f) + f * s);
  }
}

// gW(r, k) = D(f sum_{t of adapter a} P[t, r] X[t, k]), written to gW[a][r][k], or gW[a][k][r] if WT.
template <int DT, bool WT>
__global__ __launch_bounds__(256) void k_lora_wgrad(const float* __restrict__ P,
                                                    const typename Elem<DT>::T* __restrict__ X, int T, int K, int R,
                                                    const float* __restrict__ scaling, LoraSegs S,
                                                    typename Elem<DT>::T* __restrict__ gW) {
  const int a = blockIdx.z, r = blockIdx.y, k = blockIdx.x * 256 + threadIdx.x;
  float s = 0.0f;
  for (int g = 0; g < S.n_seg; ++g) {
    if (seg_adapter(S, g) != a) continue;
    const int t1 = seg_start(S, g + 1, T);
    for (int t = seg_start(S, g, T); t < t1; ++t)
      if (k < K) s = __builtin_fmaf(P[(int64_t)t * R + r], Elem<DT>::to_f32(X[(int64_t)t * K + k]), s);
  }
  if (scaling) s *= scaling[a];
  if (k < K) gW[(int64_t)a * R * K + (WT ? (int64_t)k * R + r : (int64_t)r * K + k)] = Elem<DT>::from_f32(s);
}


size_t lora_backward_floats(int T, int K, int N, int R, int n_adapters, int n_seg) { return (size_t)T * R; }

template <int DT>
static hipError_t backward_t(const void* Gv, const void* Xv, const float* V, int T, int K, const void* A,
                             const void* B, const float* scaling, int R, int N, const LoraSegs& S,
                             const void* base_grad, void* gX, void* gA, void* gB, float* ws, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  const E* G = static_cast<const E*>(Gv);
  const E* X = static_cast<const E*>(Xv);
  const int nt = lora_tiles(T, S, TM), na = S.n_adapters;
  if (T > 0 && R > 0 && (gX || gA))
    hipLaunchKernelGGL((k_lora_shrink<DT, true>), dim3(nt), dim3(256), 0, st, G, T, N, static_cast<const E*>(B), R,
                       scaling, S, ws);
  if (T > 0 && K > 0 && gX)
    hipLaunchKernelGGL((k_lora_expand<DT, true>), dim3(nt, (K + 255) / 256), dim3(256), 0, st, ws, T, K,
                       static_cast<const E*>(A), R, nullptr, S, static_cast<const E*>(base_grad), static_cast<E*>(gX));
  if (gA && na > 0 && R > 0 && K > 0)
    hipLaunchKernelGGL((k_lora_wgrad<DT, false>), dim3((K + 255) / 256, R, na), dim3(256), 0, st, ws, X, T, K, R,
                       nullptr, S, static_cast<E*>(gA));
  if (gB && na > 0 && R > 0 && N > 0)
    hipLaunchKernelGGL((k_lora_wgrad<DT, true>), dim3((N + 255) / 256, R, na), dim3(256), 0, st, V, G, T, N, R,
                       scaling, S, static_cast<E*>(gB));
  return hipGetLastError();
}

hipError_t launch_lora_backward(int dt, const void* G, const void* X, const float* V, int T, int K, const void* A,
                                const void* B, const float* scaling, int R, int N, const LoraSegs& S,
                                const void* base_grad, void* gX, void* gA, void* gB, float* ws, hipStream_t st) {
  switch (dt) {
    case DT_F32: return backward_t<DT_F32>(G, X, V, T, K, A, B, scaling, R, N, S, base_grad, gX, gA, gB, ws, st);
    case DT_F16: return backward_t<DT_F16>(G, X, V, T, K, A, B, scaling, R, N, S, base_grad, gX, gA, gB, ws, st);
    default: return backward_t<DT_BF16>(G, X, V, T, K, A, B, scaling, R, N, S, base_grad, gX, gA, gB, ws, st);
  }
}

}  // namespace i8l
