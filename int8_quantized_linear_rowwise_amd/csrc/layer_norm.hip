// Layer norm of the rows of X (T x C), and its gradient.
//
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), y = D((x - mu) r w + b)
// and, with h = (x - mu) r and u = g w,
//   dx = D(r (u - mean(u) - h mean(u h))),  dw = sum_t g h,  db = sum_t g.
// Bound by memory: 2 T C elements forward, 3 T C backward. A row lives in the
// registers of TPR threads (up to 16 values each), so it is read once (4096 x
// 4096 bf16: 14 us, 4.8 TB/s, against 29 us with three reads of each row); the
// variance is the mean of squared differences to the mean, which a sum of
// squares would lose for rows far from zero. A workgroup keeps w and b (and the
// gradients dw and db of its rows) in registers and walks rows with the next
// row's loads in flight. dw and db leave as one partial row per workgroup and
// are added up by a second launch in a fixed order (16384 x 8192 bf16 with fp32
// weights: 150 + 6 us, 5.2 TB/s; one thread a column walking all rows took 1.9
// ms for dw and db alone). Rows wider than 16384 are
// read from memory (and cache) in several passes.
#include "lora.hpp"

namespace i8l {

namespace {

// Sum over the TPR threads of a row, returned to all of them. Rows of more than
// a wave meet in LDS; `turn` alternates the place, so one barrier is enough.
template <int TPR>
__device__ __forceinline__ v2f row_sum(float a, float b, v2f (*sm)[16], int turn) {
#pragma unroll
  for (int o = (TPR < 64 ? TPR : 64) / 2; o >= 1; o >>= 1) {
    a += __shfl_xor(a, o, 64);
    b += __shfl_xor(b, o, 64);
  }
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) sm[turn][threadIdx.x >> 6] = v2f{a, b};
    __syncthreads();
    v2f s = sm[turn][0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) {
      s[0] += sm[turn][i][0];
      s[1] += sm[turn][i][1];
    }
    return s;
  }
  return v2f{a, b};
}

// EL values of the weights at p in fp32, zeros from `left` on.
template <int WDT, int EL>
__device__ __forceinline__ void ld_weights(const typename Elem<WDT>::T* p, int left, float (&f)[EL]) {
  constexpr int N = Mx<WDT>::EL;
#pragma unroll
  for (int i = 0; i < EL; i += N) {
    float x[N];
    frag_f32<WDT>(ld_frag<WDT>(p + i, left - i), x);
#pragma unroll
    for (int j = 0; j < N; ++j) f[i + j] = x[j];
  }
}

}  // namespace

constexpr int block_of(int tpr) { return tpr < 256 ? 256 : tpr; }

template <int DT, int WDT, int TPR, int NV>
__global__ __launch_bounds__(block_of(TPR)) void k_norm_fwd(const typename Elem<DT>::T* X, int T, int C, float eps,
                                                            const typename Elem<WDT>::T* __restrict__ w,
                                                            const typename Elem<WDT>::T* __restrict__ b,
                                                            typename Elem<DT>::T* Y, float* __restrict__ mean,
                                                            float* __restrict__ rstd) {
  constexpr int EL = Mx<DT>::EL, RPB = block_of(TPR) / TPR;
  __shared__ v2f sm[2][16];
  const int lane = threadIdx.x % TPR;
  const float inv_c = 1.0f / (float)C;
  int left[NV];
  float fw[NV][EL], fb[NV][EL];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + lane) * EL;
    left[i] = C - c;
    ld_weights<WDT>(w + c, left[i], fw[i]);
#pragma unroll
    for (int j = 0; j < EL; ++j) fb[i][j] = 0.0f;
    if (b) ld_weights<WDT>(b + c, left[i], fb[i]);
  }
  // every thread of the workgroup walks the same number of rows (barriers);
  // those past the end repeat the last one and store nothing
  const int stride = gridDim.x * RPB, t0 = blockIdx.x * RPB + threadIdx.x / TPR;
  v4u raw[NV];
  auto load = [&](int t) {
    const typename Elem<DT>::T* x = X + (int64_t)min(t, T - 1) * C;
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i] = ld_frag<DT>(x + (i * TPR + lane) * EL, left[i]);
  };
  load(t0);
  for (int it = 0, t = t0; it * stride + (int)blockIdx.x * RPB < T; ++it, t += stride) {
    float x[NV][EL];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      frag_f32<DT>(raw[i], x[i]);
#pragma unroll
      for (int j = 0; j < EL; ++j) s += x[i][j];
    }
    if (t + stride < T) load(t + stride);
    const float mu = row_sum<TPR>(s, 0.0f, sm, 0)[0] * inv_c;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < EL; ++j) {
        x[i][j] = j < left[i] ? x[i][j] - mu : 0.0f;
        s = __builtin_fmaf(x[i][j], x[i][j], s);
      }
    const float r = 1.0f / __builtin_sqrtf(row_sum<TPR>(s, 0.0f, sm, 1)[0] * inv_c + eps);
    if (t < T) {
      typename Elem<DT>::T* y = Y + (int64_t)t * C;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < EL; ++j) x[i][j] = __builtin_fmaf(x[i][j] * r, fw[i][j], fb[i][j]);
        st_frag<DT>(y + (i * TPR + lane) * EL, frag_of<DT>(x[i]), left[i]);
      }
      if (lane == 0) {
        if (mean) mean[t] = mu;
        if (rstd) rstd[t] = r;
      }
    }
  }
}

// part: [workgroup][2][Cp] partial dw and db; NULL for a single workgroup, which
// writes gw and gb itself, or where neither is wanted. gX, gw, gb may be NULL.
template <int DT, int WDT, int TPR, int NV>
__global__ __launch_bounds__(block_of(TPR)) void k_norm_bwd(const typename Elem<DT>::T* G,
                                                            const typename Elem<DT>::T* __restrict__ X,
                                                            const float* __restrict__ mean,
                                                            const float* __restrict__ rstd, int T, int C,
                                                            const typename Elem<WDT>::T* __restrict__ w,
                                                            typename Elem<DT>::T* gX, float* __restrict__ part,
                                                            int Cp, typename Elem<WDT>::T* __restrict__ gw,
                                                            typename Elem<WDT>::T* __restrict__ gb) {
  constexpr int EL = Mx<DT>::EL, RPB = block_of(TPR) / TPR;
  // 1024 threads have 128 registers each: no loads in flight for the next row,
  // and w comes from the cache for every row
  constexpr bool ROOMY = TPR < 1024;
  __shared__ v2f sm[2][16];
  __shared__ float meet[RPB > 1 ? 2 * 256 * NV * EL : 1];
  const int lane = threadIdx.x % TPR;
  const float inv_c = 1.0f / (float)C;
  int left[NV];
  float fw[NV][EL], dw[NV][EL], db[NV][EL];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + lane) * EL;
    left[i] = C - c;
#pragma unroll
    for (int j = 0; j < EL; ++j) fw[i][j] = dw[i][j] = db[i][j] = 0.0f;
    if (gX && ROOMY) ld_weights<WDT>(w + c, left[i], fw[i]);
  }
  const int stride = gridDim.x * RPB, t0 = blockIdx.x * RPB + threadIdx.x / TPR;
  v4u rg[NV], rx[NV];
  float mu_next, r_next;
  auto load = [&](int t) {
    const int64_t at = (int64_t)min(t, T - 1) * C;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      rg[i] = ld_frag<DT>(G + at + (i * TPR + lane) * EL, left[i]);
      rx[i] = ld_frag<DT>(X + at + (i * TPR + lane) * EL, left[i]);
    }
    mu_next = mean[min(t, T - 1)];
    r_next = rstd[min(t, T - 1)];
  };
  if (ROOMY) load(t0);
  for (int it = 0, t = t0; it * stride + (int)blockIdx.x * RPB < T; ++it, t += stride) {
    if (!ROOMY) load(t);
    const float mu = mu_next, r = r_next;
    float g[NV][EL], h[NV][EL];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      frag_f32<DT>(rg[i], g[i]);
      frag_f32<DT>(rx[i], h[i]);
    }
    if (ROOMY && t + stride < T) load(t + stride);
    if (!ROOMY && gX)
#pragma unroll
      for (int i = 0; i < NV; ++i) ld_weights<WDT>(w + (i * TPR + lane) * EL, left[i], fw[i]);
    const bool row = t < T;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < EL; ++j) {
        h[i][j] = j < left[i] ? (h[i][j] - mu) * r : 0.0f;
        if (row) {
          dw[i][j] = __builtin_fmaf(g[i][j], h[i][j], dw[i][j]);
          db[i][j] += g[i][j];
        }
        g[i][j] *= fw[i][j];
        s1 += g[i][j];
        s2 = __builtin_fmaf(g[i][j], h[i][j], s2);
      }
    if (gX) {
      const v2f s = row_sum<TPR>(s1, s2, sm, it & 1);
      const float m1 = s[0] * inv_c, m2 = s[1] * inv_c;
      if (row) {
        typename Elem<DT>::T* o = gX + (int64_t)t * C;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int j = 0; j < EL; ++j) g[i][j] = r * (g[i][j] - m1 - h[i][j] * m2);
          st_frag<DT>(o + (i * TPR + lane) * EL, frag_of<DT>(g[i]), left[i]);
        }
      }
    }
  }
  if (part == nullptr && gw == nullptr && gb == nullptr) return;
  float* p = part + (int64_t)blockIdx.x * 2 * Cp;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * EL;
      if (part == nullptr) {
#pragma unroll
        for (int j = 0; j < EL; ++j)
          if (j < left[i]) {
            if (gw) gw[c + j] = Elem<WDT>::from_f32(dw[i][j]);
            if (gb) gb[c + j] = Elem<WDT>::from_f32(db[i][j]);
          }
        continue;
      }
#pragma unroll
      for (int j = 0; j < EL; j += 4)
        if (c + j < Cp) {
          *reinterpret_cast<v4f*>(p + c + j) = v4f{dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]};
          *reinterpret_cast<v4f*>(p + Cp + c + j) = v4f{db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]};
        }
    }
  } else {
    constexpr int W = TPR * NV * EL;   // columns of a row's threads
    const int grp = threadIdx.x / TPR;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < EL; ++j) {
        const int c = (i * TPR + lane) * EL + j;
        meet[(2 * grp) * W + c] = dw[i][j];
        meet[(2 * grp + 1) * W + c] = db[i][j];
      }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * W; e += 256) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < RPB; ++k) s += meet[2 * k * W + e];
      const int c = e % W;
      if (part == nullptr) {
        typename Elem<WDT>::T* o = e < W ? gw : gb;
        if (o && c < C) o[c] = Elem<WDT>::from_f32(s);
      } else if (c < Cp) {
        p[(e / W) * Cp + c] = s;
      }
    }
  }
}

// dw (blockIdx.y 0) and db (1) of 64 columns: 16 threads a group of 4 columns, each every 16th partial row.
template <int WDT>
__global__ __launch_bounds__(256) void k_norm_sum(const float* __restrict__ part, int n, int C, int Cp,
                                                  typename Elem<WDT>::T* gw, typename Elem<WDT>::T* gb) {
  __shared__ v4f sm[16][16];
  typename Elem<WDT>::T* out = blockIdx.y ? gb : gw;
  if (out == nullptr) return;
  const int cg = threadIdx.x & 15, rs = threadIdx.x >> 4, c = blockIdx.x * 64 + 4 * cg;
  const float* p = part + (int64_t)blockIdx.y * Cp + min(c, Cp - 4);
  v4f s = {};
#pragma unroll 8
  for (int i = rs; i < n; i += 16) s += *reinterpret_cast<const v4f*>(p + (int64_t)i * 2 * Cp);
  sm[rs][cg] = s;
  __syncthreads();
  if (rs == 0) {
    s = sm[0][cg];
#pragma unroll
    for (int i = 1; i < 16; ++i) s += sm[i][cg];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < C) out[c + j] = Elem<WDT>::from_f32(s[j]);
  }
}

// Rows of any width, in passes over memory: 1024 threads a row.
template <int DT, int WDT>
__global__ __launch_bounds__(1024) void k_norm_fwd_wide(const typename Elem<DT>::T* X, int T, int C, float eps,
                                                        const typename Elem<WDT>::T* __restrict__ w,
                                                        const typename Elem<WDT>::T* __restrict__ b,
                                                        typename Elem<DT>::T* Y, float* __restrict__ mean,
                                                        float* __restrict__ rstd) {
  constexpr int EL = Mx<DT>::EL;
  __shared__ v2f sm[2][16];
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const typename Elem<DT>::T* x = X + (int64_t)t * C;
    typename Elem<DT>::T* y = Y + (int64_t)t * C;
    float s = 0.0f;
    for (int c = threadIdx.x * EL; c < C; c += 1024 * EL) {
      float f[EL];
      frag_f32<DT>(ld_frag<DT>(x + c, C - c), f);
#pragma unroll
      for (int j = 0; j < EL; ++j) s += f[j];
    }
    const float mu = row_sum<1024>(s, 0.0f, sm, 0)[0] / (float)C;
    s = 0.0f;
    for (int c = threadIdx.x * EL; c < C; c += 1024 * EL) {
      float f[EL];
      frag_f32<DT>(ld_frag<DT>(x + c, C - c), f);
#pragma unroll
      for (int j = 0; j < EL; ++j) {
        const float d = j < C - c ? f[j] - mu : 0.0f;
        s = __builtin_fmaf(d, d, s);
      }
    }
    const float r = 1.0f / __builtin_sqrtf(row_sum<1024>(s, 0.0f, sm, 1)[0] / (float)C + eps);
    for (int c = threadIdx.x * EL; c < C; c += 1024 * EL) {
      float f[EL], fw[EL], fb[EL] = {};
      frag_f32<DT>(ld_frag<DT>(x + c, C - c), f);
      ld_weights<WDT>(w + c, C - c, fw);
      if (b) ld_weights<WDT>(b + c, C - c, fb);
#pragma unroll
      for (int j = 0; j < EL; ++j) f[j] = __builtin_fmaf((f[j] - mu) * r, fw[j], fb[j]);
      st_frag<DT>(y + c, frag_of<DT>(f), C - c);
    }
    if (threadIdx.x == 0) {
      if (mean) mean[t] = mu;
      if (rstd) rstd[t] = r;
    }
  }
}

template <int DT, int WDT>
__global__ __launch_bounds__(1024) void k_norm_bwd_wide(const typename Elem<DT>::T* G,
                                                        const typename Elem<DT>::T* __restrict__ X,
                                                        const float* __restrict__ mean,
                                                        const float* __restrict__ rstd, int T, int C,
                                                        const typename Elem<WDT>::T* __restrict__ w,
                                                        typename Elem<DT>::T* gX) {
  constexpr int EL = Mx<DT>::EL;
  __shared__ v2f sm[2][16];
  for (int t = blockIdx.x, it = 0; t < T; t += gridDim.x, ++it) {
    const int64_t at = (int64_t)t * C;
    const float mu = mean[t], r = rstd[t];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x * EL; c < C; c += 1024 * EL) {
      float g[EL], x[EL], fw[EL];
      frag_f32<DT>(ld_frag<DT>(G + at + c, C - c), g);
      frag_f32<DT>(ld_frag<DT>(X + at + c, C - c), x);
      ld_weights<WDT>(w + c, C - c, fw);
#pragma unroll
      for (int j = 0; j < EL; ++j) {   // past the row u is 0
        const float u = g[j] * fw[j];
        s1 += u;
        s2 = __builtin_fmaf(u, j < C - c ? (x[j] - mu) * r : 0.0f, s2);
      }
    }
    const v2f s = row_sum<1024>(s1, s2, sm, it & 1);
    const float m1 = s[0] / (float)C, m2 = s[1] / (float)C;
    for (int c = threadIdx.x * EL; c < C; c += 1024 * EL) {
      float g[EL], x[EL], fw[EL];
      frag_f32<DT>(ld_frag<DT>(G + at + c, C - c), g);
      frag_f32<DT>(ld_frag<DT>(X + at + c, C - c), x);
      ld_weights<WDT>(w + c, C - c, fw);
#pragma unroll
      for (int j = 0; j < EL; ++j) g[j] = r * (g[j] * fw[j] - m1 - (x[j] - mu) * r * m2);
      st_frag<DT>(gX + at + c, frag_of<DT>(g), C - c);
    }
  }
}

// Partial dw and db of 128 EL columns and the rows of part blockIdx.y.
template <int DT>
__global__ __launch_bounds__(128) void k_norm_wgrad_wide(const typename Elem<DT>::T* __restrict__ G,
                                                         const typename Elem<DT>::T* __restrict__ X,
                                                         const float* __restrict__ mean,
                                                         const float* __restrict__ rstd, int T, int C,
                                                         float* __restrict__ part, int Cp) {
  constexpr int EL = Mx<DT>::EL;
  const int c = (blockIdx.x * 128 + threadIdx.x) * EL;
  const int n = gridDim.y, t0 = (int)((int64_t)T * blockIdx.y / n), t1 = (int)((int64_t)T * (blockIdx.y + 1) / n);
  if (c >= C) return;
  float dw[EL] = {}, db[EL] = {};
#pragma unroll 4
  for (int t = t0; t < t1; ++t) {
    float g[EL], x[EL];
    frag_f32<DT>(ld_frag<DT>(G + (int64_t)t * C + c, C - c), g);
    frag_f32<DT>(ld_frag<DT>(X + (int64_t)t * C + c, C - c), x);
    const float mu = mean[t], r = rstd[t];
#pragma unroll
    for (int j = 0; j < EL; ++j) {
      dw[j] = __builtin_fmaf(g[j], (x[j] - mu) * r, dw[j]);
      db[j] += g[j];
    }
  }
  float* p = part + (int64_t)blockIdx.y * 2 * Cp;
#pragma unroll
  for (int j = 0; j < EL; ++j)
    if (c + j < C) {
      p[c + j] = dw[j];
      p[Cp + c + j] = db[j];
    }
}

namespace {

constexpr int WIDEST = 16384;
int pad_cols(int C) { return (C + 63) / 64 * 64; }

// Rows of partial sums: one a workgroup of the backward, as many as are resident
// together (one a compute unit from 512 threads on, else two; more would only
// lengthen the second launch: 16384 x 8192 takes 156, 164 and 173 us with 256,
// 512 and 1024), or parts of the rows for wide ones.
int norm_parts(int T, int C) {
  if (C > WIDEST) {
    const int n = T / 32;
    return n < 1 ? 1 : n > 32 ? 32 : n;
  }
  const int rows = C <= 128 ? 16 : C <= 1024 ? 4 : 1;    // rows a workgroup takes at once
  // One workgroup walks few narrow rows and needs no second launch and no
  // workspace (6 us on the host). On the GPU 8 x 1024 bf16 takes 5.1 us against
  // 6.8, 16 x 1024 6.9 and 6.9, 4 x 4096, the bound, 10 and 6.8, where a call's
  // host side takes 10.5 and 16.5. More than that outlasts what it saves: 8 x
  // 4096 takes 15 us, 8 x 16384 36 against 8.6, 128 x 64 9.6 against 7.0.
  if (T <= 4 * rows && T * C <= 16384) return 1;
  const int n = (T + rows - 1) / rows;
  const int most = C > 4096 ? 256 : 512;
  return n < 1 ? 1 : n < most ? n : most;
}

template <int DT, int WDT, int TPR, int NV>
hipError_t fwd_run(const void* X, int T, int C, const void* w, const void* b, float eps, void* Y, float* mean,
                   float* rstd, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  typedef typename Elem<WDT>::T W;
  constexpr int RPB = block_of(TPR) / TPR;
  const int need = (T + RPB - 1) / RPB, most = 2048 * 256 / block_of(TPR);
  hipLaunchKernelGGL((k_norm_fwd<DT, WDT, TPR, NV>), dim3(need < most ? need : most), dim3(block_of(TPR)), 0, st,
                     static_cast<const E*>(X), T, C, eps, static_cast<const W*>(w), static_cast<const W*>(b),
                     static_cast<E*>(Y), mean, rstd);
  return hipGetLastError();
}

template <int DT, int WDT, int TPR, int NV>
hipError_t bwd_run(const void* G, const void* X, const float* mean, const float* rstd, int T, int C, const void* w,
                   void* gX, float* part, void* gw, void* gb, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  typedef typename Elem<WDT>::T W;
  hipLaunchKernelGGL((k_norm_bwd<DT, WDT, TPR, NV>), dim3(norm_parts(T, C)), dim3(block_of(TPR)), 0, st,
                     static_cast<const E*>(G), static_cast<const E*>(X), mean, rstd, T, C, static_cast<const W*>(w),
                     static_cast<E*>(gX), part, pad_cols(C), static_cast<W*>(gw), static_cast<W*>(gb));
  return hipGetLastError();
}

// Threads of a row by its width, 8 or 16 values each.
#define I8L_NORM_WIDTHS(F, ...)                                               \
  constexpr int V = 8 / Mx<DT>::EL;                                           \
  if (C <= 128) return F<DT, WDT, 16, V>(__VA_ARGS__);                        \
  if (C <= 512) return F<DT, WDT, 64, V>(__VA_ARGS__);                        \
  if (C <= 1024) return F<DT, WDT, 64, 2 * V>(__VA_ARGS__);                   \
  if (C <= 2048) return F<DT, WDT, 256, V>(__VA_ARGS__);                      \
  if (C <= 4096) return F<DT, WDT, 256, 2 * V>(__VA_ARGS__);                  \
  if (C <= 8192) return F<DT, WDT, 512, 2 * V>(__VA_ARGS__);                  \
  return F<DT, WDT, 1024, 2 * V>(__VA_ARGS__);

template <int DT, int WDT>
hipError_t fwd_width(const void* X, int T, int C, const void* w, const void* b, float eps, void* Y, float* mean,
                     float* rstd, hipStream_t st) {
  I8L_NORM_WIDTHS(fwd_run, X, T, C, w, b, eps, Y, mean, rstd, st)
}
template <int DT, int WDT>
hipError_t bwd_width(const void* G, const void* X, const float* mean, const float* rstd, int T, int C, const void* w,
                     void* gX, float* part, void* gw, void* gb, hipStream_t st) {
  I8L_NORM_WIDTHS(bwd_run, G, X, mean, rstd, T, C, w, gX, part, gw, gb, st)
}

template <int DT, int WDT>
hipError_t fwd_t(const void* X, int T, int C, const void* w, const void* b, float eps, void* Y, float* mean,
                 float* rstd, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  typedef typename Elem<WDT>::T W;
  if (C <= WIDEST) return fwd_width<DT, WDT>(X, T, C, w, b, eps, Y, mean, rstd, st);
  hipLaunchKernelGGL((k_norm_fwd_wide<DT, WDT>), dim3(T < 512 ? T : 512), dim3(1024), 0, st, static_cast<const E*>(X),
                     T, C, eps, static_cast<const W*>(w), static_cast<const W*>(b), static_cast<E*>(Y), mean, rstd);
  return hipGetLastError();
}

template <int DT, int WDT>
hipError_t bwd_t(const void* G, const void* X, const float* mean, const float* rstd, int T, int C, const void* w,
                 void* gX, void* gw, void* gb, float* ws, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  typedef typename Elem<WDT>::T W;
  const bool sums = gw || gb;
  int n = 0;   // partial rows
  if (T > 0) {
    n = norm_parts(T, C);
    if (C <= WIDEST) {
      const bool whole = n == 1;
      const hipError_t e = bwd_width<DT, WDT>(G, X, mean, rstd, T, C, w, gX, sums && !whole ? ws : nullptr,
                                              whole ? gw : nullptr, whole ? gb : nullptr, st);
      if (e != hipSuccess || whole) return e;
    } else {
      // the weight gradient first: gX may be G only where there is none
      if (sums)
        hipLaunchKernelGGL((k_norm_wgrad_wide<DT>), dim3((C + 128 * Mx<DT>::EL - 1) / (128 * Mx<DT>::EL), n),
                           dim3(128), 0, st, static_cast<const E*>(G), static_cast<const E*>(X), mean, rstd, T, C, ws,
                           pad_cols(C));
      if (gX)
        hipLaunchKernelGGL((k_norm_bwd_wide<DT, WDT>), dim3(T < 512 ? T : 512), dim3(1024), 0, st,
                           static_cast<const E*>(G), static_cast<const E*>(X), mean, rstd, T, C,
                           static_cast<const W*>(w), static_cast<E*>(gX));
    }
  }
  if (sums)
    hipLaunchKernelGGL(k_norm_sum<WDT>, dim3((C + 63) / 64, 2), dim3(256), 0, st, ws, n, C, pad_cols(C),
                       static_cast<W*>(gw), static_cast<W*>(gb));
  return hipGetLastError();
}

}  // namespace

size_t norm_backward_floats(int T, int C) {
  const int n = norm_parts(T, C);
  return n == 1 && C <= WIDEST ? 0 : (size_t)2 * pad_cols(C) * n;
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
