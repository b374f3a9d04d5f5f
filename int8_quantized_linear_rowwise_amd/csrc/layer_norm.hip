// Layer norm of the rows of X (T x C), and its gradient.
//
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), y = D((x - mu) r w + b)
// and, with h = (x - mu) r and u = g w,
//   dx = D(r (u - mean(u) - h mean(u h))),  dw = sum_t g h,  db = sum_t g.
#include "common.hpp"
#include "kernels.hpp"

namespace i8l {

// Sum of a block's 256 values, returned to every thread.
__device__ __forceinline__ float block_sum(float v, float* sm) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
  __syncthreads();
  return (sm[0] + sm[1]) + (sm[2] + sm[3]);
}

template <int DT, int WDT>
__global__ __launch_bounds__(256) void k_norm_fwd(const typename Elem<DT>::T* __restrict__ X, int C, float eps,
                                                  const typename Elem<WDT>::T* __restrict__ w,
                                                  const typename Elem<WDT>::T* __restrict__ b,
                                                  typename Elem<DT>::T* __restrict__ Y, float* __restrict__ mean,
                                                  float* __restrict__ rstd) {
  __shared__ float sm[4];
  const int64_t t = blockIdx.x;
  const typename Elem<DT>::T* x = X + t * C;
  float s = 0.0f;
  for (int c = threadIdx.x; c < C; c += 256) s += Elem<DT>::to_f32(x[c]);
  const float mu = block_sum(s, sm) / C;
  s = 0.0f;
  for (int c = threadIdx.x; c < C; c += 256) {
    const float d = Elem<DT>::to_f32(x[c]) - mu;
    s += d * d;
  }
  const float r = 1.0f / __builtin_sqrtf(block_sum(s, sm) / C + eps);
  for (int c = threadIdx.x; c < C; c += 256) {
    const float h = (Elem<DT>::to_f32(x[c]) - mu) * r;
    Y[t * C + c] = Elem<DT>::from_f32(h * Elem<WDT>::to_f32(w[c]) + (b ? Elem<WDT>::to_f32(b[c]) : 0.0f));
  }
  if (threadIdx.x == 0) {
    if (mean) mean[t] = mu;
    if (rstd) rstd[t] = r;
  }
}

template <int DT, int WDT>
__global__ __launch_bounds__(256) void k_norm_bwd(const typename Elem<DT>::T* __restrict__ G,
                                                  const typename Elem<DT>::T* __restrict__ X,
                                                  const float* __restrict__ mean, const float* __restrict__ rstd,
                                                  int C, const typename Elem<WDT>::T* __restrict__ w,
                                                  typename Elem<DT>::T* __restrict__ gX) {
  __shared__ float sm[4];
  const int64_t t = blockIdx.x;
  const float mu = mean[t], r = rstd[t];
  float s1 = 0.0f, s2 = 0.0f;
  for (int c = threadIdx.x; c < C; c += 256) {
    const float u = Elem<DT>::to_f32(G[t * C + c]) * Elem<WDT>::to_f32(w[c]);
    s1 += u;
    s2 += u * ((Elem<DT>::to_f32(X[t * C + c]) - mu) * r);
  }
  const float m1 = block_sum(s1, sm) / C, m2 = block_sum(s2, sm) / C;
  for (int c = threadIdx.x; c < C; c += 256) {
    const float u = Elem<DT>::to_f32(G[t * C + c]) * Elem<WDT>::to_f32(w[c]);
    const float h = (Elem<DT>::to_f32(X[t * C + c]) - mu) * r;
    gX[t * C + c] = Elem<DT>::from_f32(r * (u - m1 - h * m2));
  }
}

// dw and db of 64 columns: four waves take every fourth row, summed in a fixed order.
template <int DT, int WDT>
__global__ __launch_bounds__(256) void k_norm_wgrad(const typename Elem<DT>::T* __restrict__ G,
                                                    const typename Elem<DT>::T* __restrict__ X,
                                                    const float* __restrict__ mean, const float* __restrict__ rstd,
                                                    int T, int C, typename Elem<WDT>::T* __restrict__ gw,
                                                    typename Elem<WDT>::T* __restrict__ gb) {
  __shared__ float sw[4][64], sb[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  float dw = 0.0f, db = 0.0f;
  for (int64_t t = wave; t < T; t += 4)
    if (c < C) {
      const float g = Elem<DT>::to_f32(G[t * C + c]);
      dw += g * ((Elem<DT>::to_f32(X[t * C + c]) - mean[t]) * rstd[t]);
      db += g;
    }
  sw[wave][lane] = dw;
  sb[wave][lane] = db;
  __syncthreads();
  if (wave == 0 && c < C) {
    if (gw) gw[c] = Elem<WDT>::from_f32((sw[0][lane] + sw[1][lane]) + (sw[2][lane] + sw[3][lane]));
    if (gb) gb[c] = Elem<WDT>::from_f32((sb[0][lane] + sb[1][lane]) + (sb[2][lane] + sb[3][lane]));
  }
}

size_t norm_backward_floats(int T, int C) { return 0; }

template <int DT, int WDT>
static hipError_t fwd_t(const void* X, int T, int C, const void* w, const void* b, float eps, void* Y, float* mean,
                        float* rstd, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  typedef typename Elem<WDT>::T W;
  hipLaunchKernelGGL((k_norm_fwd<DT, WDT>), dim3(T), dim3(256), 0, st, static_cast<const E*>(X), C, eps,
                     static_cast<const W*>(w), static_cast<const W*>(b), static_cast<E*>(Y), mean, rstd);
  return hipGetLastError();
}

template <int DT, int WDT>
static hipError_t bwd_t(const void* G, const void* X, const float* mean, const float* rstd, int T, int C,
                        const void* w, void* gX, void* gw, void* gb, float* ws, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  typedef typename Elem<WDT>::T W;
  if (T > 0 && gX)
    hipLaunchKernelGGL((k_norm_bwd<DT, WDT>), dim3(T), dim3(256), 0, st, static_cast<const E*>(G),
                       static_cast<const E*>(X), mean, rstd, C, static_cast<const W*>(w), static_cast<E*>(gX));
  if (gw || gb)
    hipLaunchKernelGGL((k_norm_wgrad<DT, WDT>), dim3((C + 63) / 64), dim3(256), 0, st, static_cast<const E*>(G),
                       static_cast<const E*>(X), mean, rstd, T, C, static_cast<W*>(gw), static_cast<W*>(gb));
  return hipGetLastError();
}

#define I8L_NORM_TYPES(F, ...)                                                    \
  switch (dt * 3 + wdt) {                                                         \
    case DT_F32 * 3 + DT_F32: return F<DT_F32, DT_F32>(__VA_ARGS__);               \
    case DT_F16 * 3 + DT_F32: return F<DT_F16, DT_F32>(__VA_ARGS__);               \
    case DT_F16 * 3 + DT_F16: return F<DT_F16, DT_F16>(__VA_ARGS__);               \
    case DT_BF16 * 3 + DT_F32: return F<DT_BF16, DT_F32>(__VA_ARGS__);             \
    case DT_BF16 * 3 + DT_BF16: return F<DT_BF16, DT_BF16>(__VA_ARGS__);           \
    default: return hipErrorInvalidValue;                                         \
  }

hipError_t launch_norm_forward(int dt, int wdt, const void* X, int T, int C, const void* w, const void* b, float eps,
                               void* Y, float* mean, float* rstd, hipStream_t st) {
  I8L_NORM_TYPES(fwd_t, X, T, C, w, b, eps, Y, mean, rstd, st)
}

hipError_t launch_norm_backward(int dt, int wdt, const void* G, const void* X, const float* mean, const float* rstd,
                                int T, int C, const void* w, void* gX, void* gw, void* gb, float* ws,
                                hipStream_t st) {
  I8L_NORM_TYPES(bwd_t, G, X, mean, rstd, T, C, w, gX, gw, gb, ws, st)
}

}  // namespace i8l
