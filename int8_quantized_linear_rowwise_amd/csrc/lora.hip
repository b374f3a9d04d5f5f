// Low-rank adapters of many requests beside a shared projection.
//
// Token t of adapter a: V[t] = A[a] x[t] (R values, fp32) and
//   y[t] = D(base[t] + s[a] B[a] V[t]);
// backward, g = dL/dy:
//   dV[t] = s[a] B[a]^T g[t],  dx[t] = D(base_grad[t] + A[a]^T dV[t]),
//   dA[a] = D(sum_t dV[t] x[t]^T),  dB[a] = D(s[a] sum_t g[t] V[t]^T).
#include "common.hpp"
#include "kernels.hpp"

namespace i8l {

// Start of segment s: the caller's offsets held inside [0, T], so that no
// content of the array leads to an access outside the token rows.
__device__ __forceinline__ int seg_start(const LoraSegs& S, int s, int T) {
  return s <= 0 ? 0 : s >= S.n_seg ? T : min(max(S.off[s], 0), T);
}

// Adapter of segment s, -1 for none (any value outside [0, n_adapters)).
__device__ __forceinline__ int seg_adapter(const LoraSegs& S, int s) {
  if (s >= S.n_seg) return -1;
  const int a = S.ids ? S.ids[s] : s;
  return (a >= 0 && a < S.n_adapters) ? a : -1;
}

// Token tiles: the tokens are cut at every multiple of `tm` and at every
// segment start. The cuts in ascending order (a multiple of tm before a
// segment start at the same token) number the tiles 0 .. nb + n_seg - 1; tile
// d runs from cut d to cut d + 1 and lies in one segment. Tile 0 is empty.
// Segment s is cut number s + min(start(s) / tm + 1, nb), so the segments
// begun by tile d are counted by a search 64 wide (every lane of the wave).
struct LoraTile {
  int t0, t1, adapter;
};
__device__ __forceinline__ LoraTile lora_tile(const LoraSegs& S, int d, int T, int tm) {
  const int lane = threadIdx.x & 63;
  const int nb = (T + tm - 1) / tm, ns = max(S.n_seg, 1);
  int lo = 0, len = ns;
  while (len > 0) {
    const int step = (len + 63) >> 6;
    const int off = (lane + 1) * step - 1;
    const int s = lo + off;
    const bool in = off < len && s + min(seg_start(S, s, T) / tm + 1, nb) <= d;
    const int c = __popcll(__ballot(in));
    lo += c * step;
    len = min(step - 1, len - c * step);
  }
  const int i = d + 1 - lo;
  LoraTile r;
  r.t0 = min(max((i - 1) * tm, lo > 0 ? seg_start(S, lo - 1, T) : 0), T);
  r.t1 = min(min((int64_t)i * tm, (int64_t)T), (int64_t)(lo < ns ? seg_start(S, lo, T) : T));
  if (lo <= 0 || i <= 0) r.t1 = r.t0;
  r.adapter = lo > 0 ? seg_adapter(S, lo - 1) : -1;
  return r;
}

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

static int tiles(int T, const LoraSegs& S, int tm) { return (T + tm - 1) / tm + (S.n_seg > 1 ? S.n_seg : 1) - 1; }

size_t lora_forward_floats(int T, int K, int N, int R, int n_seg) { return (size_t)T * R; }
size_t lora_backward_floats(int T, int K, int N, int R, int n_adapters, int n_seg) { return (size_t)T * R; }

template <int DT>
static hipError_t forward_t(const void* Xv, int T, int K, const void* A, const void* B, const float* scaling, int R,
                            int N, const LoraSegs& S, const void* base, void* out, float* V, float* ws,
                            hipStream_t st) {
  typedef typename Elem<DT>::T E;
  float* P = V ? V : ws;
  const int nt = tiles(T, S, TM);
  if (R > 0)
    hipLaunchKernelGGL((k_lora_shrink<DT, false>), dim3(nt), dim3(256), 0, st, static_cast<const E*>(Xv), T, K,
                       static_cast<const E*>(A), R, nullptr, S, P);
  if (N > 0)
    hipLaunchKernelGGL((k_lora_expand<DT, false>), dim3(nt, (N + 255) / 256), dim3(256), 0, st, P, T, N,
                       static_cast<const E*>(B), R, scaling, S, static_cast<const E*>(base), static_cast<E*>(out));
  return hipGetLastError();
}

hipError_t launch_lora_forward(int dt, const void* X, int T, int K, const void* A, const void* B,
                               const float* scaling, int R, int N, const LoraSegs& S, const void* base, void* out,
                               float* V, float* ws, hipStream_t st) {
  switch (dt) {
    case DT_F32: return forward_t<DT_F32>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
    case DT_F16: return forward_t<DT_F16>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
    default: return forward_t<DT_BF16>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
  }
}

template <int DT>
static hipError_t backward_t(const void* Gv, const void* Xv, const float* V, int T, int K, const void* A,
                             const void* B, const float* scaling, int R, int N, const LoraSegs& S,
                             const void* base_grad, void* gX, void* gA, void* gB, float* ws, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  const E* G = static_cast<const E*>(Gv);
  const E* X = static_cast<const E*>(Xv);
  const int nt = tiles(T, S, TM), na = S.n_adapters;
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
