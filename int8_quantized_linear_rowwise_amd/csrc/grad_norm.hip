// Norm of all gradients, the factor that clips them, and the clipping.
//
//   norm = c sqrt(sum g^2)  or  c max |g|,   c = *grad_scale (1 without)
//   factor = c min(1, max_norm / (norm + 1e-6)),   found_inf = norm is not finite
// Squares are formed and added in 64 bits, so that no finite gradient overflows
// or vanishes and the sum of any number of values keeps fp32's 24 bits. (The
// chip's 64-bit vector rate is half its 32-bit rate, far over what memory
// delivers.) Workgroups add up their chunks in a fixed order, one more
// workgroup the workgroups' sums: the result is the same on every run.
//
// Bound by memory. The list of tensors travels in the kernels' arguments and
// is put into LDS by every workgroup, so a call needs no table on the device:
// nothing to lay out, nothing to keep between calls. The norm of 202 M
// bf16 values takes 67 us and 4.8 to add the workgroups' sums (6.0 TB/s). Clipping
// 40 M bf16 values of 448 tensors: launches of 280 tensors with 18 M values and of
// 168 with 22 M, 10.0 and 10.8 us for their sums (3.7 and 4.0 TB/s), 3.6 to add them
// up, 15.1 and 15.4 for the scaling (4.9 and 5.6 TB/s).
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace i8l {

constexpr int GN_VALUES = 32;                 // values of a thread in one chunk
constexpr int GN_CHUNK = 256 * GN_VALUES;
constexpr int GN_GROUPS = 1024;               // workgroups of a launch: as many as are at work at once

int grad_chunk() { return GN_CHUNK; }
int grad_groups(int64_t chunks) { return (int)(chunks < GN_GROUPS ? chunks : GN_GROUPS); }

// The list in LDS, and the tensor of a chunk.
struct ListLds {
  const void* p[GRAD_LIST];
  int32_t start[GRAD_LIST + 1];
  uint16_t last[GRAD_LIST];
  __device__ __forceinline__ int64_t values(int t) const {
    return (int64_t)(start[t + 1] - start[t] - 1) * GN_CHUNK + (last[t] >> 2);
  }
};
static_assert(GN_CHUNK << 2 < 65536 && sizeof(GradList) + 64 <= 4096, "packed sizes");
__device__ __forceinline__ void list_to_lds(const GradList& list, ListLds& s) {
  for (int i = threadIdx.x; i < list.count; i += blockDim.x) {
    s.p[i] = list.p[i];
    s.last[i] = list.last[i];
  }
  for (int i = threadIdx.x; i <= list.count; i += blockDim.x) s.start[i] = list.start[i];
  __syncthreads();
}
// Tensor of chunk c: the last one that starts at or before it (empty tensors have no chunk).
__device__ __forceinline__ int tensor_of(const ListLds& s, int count, int c) {
  const int lane = threadIdx.x & 63;
  int n = 0;
#pragma unroll
  for (int b = 0; b < GRAD_LIST; b += 64) n += __popcll(__ballot(b + lane < count && s.start[b + lane] <= c));
  return __builtin_amdgcn_readfirstlane(n - 1);
}

// f(group of 8 values, how many of them are in the tensor, their place) for this thread's values of a chunk, which 256
// threads take together.
template <int DT, typename F>
__device__ __forceinline__ void chunk_values(const void* base, int64_t first, int64_t n, bool vec, F f) {
  typedef typename Elem<DT>::T T;
  const int tid = threadIdx.x & 255;
  const T* p = static_cast<const T*>(base);
  if (vec && first + GN_CHUNK <= n) {
    T e[GN_VALUES / 8][8];
#pragma unroll
    for (int i = 0; i < GN_VALUES / 8; ++i) load8<DT>(p + first + (i * 256 + tid) * 8, e[i]);
#pragma unroll
    for (int i = 0; i < GN_VALUES / 8; ++i) f(e[i], 8, first + (i * 256 + tid) * 8);
  } else {
    for (int i = 0; i < GN_VALUES / 8; ++i) {
      const int64_t at = first + (i * 256 + tid) * 8;
      const int m = (int)min((int64_t)8, n - at);
      if (m <= 0) break;
      T e[8] = {};
      if (vec && m == 8) load8<DT>(p + at, e);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < m) e[j] = p[at + j];
      f(e, m, at);
    }
  }
}

template <bool INF>
__device__ __forceinline__ double join(double a, double b) {
  if constexpr (INF) return a != a ? a : (b != b ? b : (a > b ? a : b));   // NaN stays
  else return a + b;
}
// All threads of the workgroup; the result in thread 0.
template <bool INF>
__device__ __forceinline__ double join_block(double v, double* lds) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = join<INF>(v, __shfl_xor(v, o, 64));
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < waves; ++w) v = join<INF>(v, lds[w]);
  return v;
}

// Chunks first, first + step, ... of the list, by 256 threads: this thread's sum (INF: largest magnitude).
template <bool INF>
__device__ __forceinline__ double sum_chunks(const ListLds& s, int count, int first, int step) {
  const int total = s.start[count];
  double sum = 0.0;
  for (int c = first; c < total; c += step) {
    const int t = tensor_of(s, count, c);
    const int64_t n = s.values(t), at = (int64_t)(c - s.start[t]) * GN_CHUNK;
    const bool vec = (uintptr_t)s.p[t] % 16 == 0;
    auto one = [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      chunk_values<DT>(s.p[t], at, n, vec, [&](const typename Elem<DT>::T(&e)[8], int, int64_t) {
        if constexpr (INF) {
          uint32_t top = 0u;   // magnitudes as integers: infinities and NaN on top
#pragma unroll
          for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(Elem<DT>::to_f32(e[j])) & 0x7fffffffu);
          sum = join<true>(sum, (double)__uint_as_float(top));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const double x = (double)Elem<DT>::to_f32(e[j]);
            sum = __builtin_fma(x, x, sum);
          }
        }
      });
    };
    switch (s.last[t] & 3) {
      case DT_F32: one(std::integral_constant<int, DT_F32>{}); break;
      case DT_F16: one(std::integral_constant<int, DT_F16>{}); break;
      default: one(std::integral_constant<int, DT_BF16>{}); break;
    }
  }
  return sum;
}

// g = D(f g) in those chunks.
__device__ __forceinline__ void scale_chunks(const ListLds& s, int count, int first, int step, float f) {
  const int total = s.start[count];
  for (int c = first; c < total; c += step) {
    const int t = tensor_of(s, count, c);
    const int64_t n = s.values(t), from = (int64_t)(c - s.start[t]) * GN_CHUNK;
    const bool vec = (uintptr_t)s.p[t] % 16 == 0;
    auto one = [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      typedef typename Elem<DT>::T T;
      T* p = static_cast<T*>(const_cast<void*>(s.p[t]));
      chunk_values<DT>(s.p[t], from, n, vec, [&](const T(&e)[8], int m, int64_t at) {
        T o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = Elem<DT>::from_f32(Elem<DT>::to_f32(e[j]) * f);
        if (vec && m == 8) {
          if constexpr (DT == DT_F32) {
            reinterpret_cast<v4f*>(p + at)[0] = v4f{o[0], o[1], o[2], o[3]};
            reinterpret_cast<v4f*>(p + at)[1] = v4f{o[4], o[5], o[6], o[7]};
          } else {
            v4u w;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[j] = (uint32_t)__builtin_bit_cast(uint16_t, o[2 * j]) |
                     ((uint32_t)__builtin_bit_cast(uint16_t, o[2 * j + 1]) << 16);
            *reinterpret_cast<v4u*>(p + at) = w;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < m) p[at + j] = o[j];
        }
      });
    };
    switch (s.last[t] & 3) {
      case DT_F32: one(std::integral_constant<int, DT_F32>{}); break;
      case DT_F16: one(std::integral_constant<int, DT_F16>{}); break;
      default: one(std::integral_constant<int, DT_BF16>{}); break;
    }
  }
}

// The three results from the sum of squares (INF: the largest magnitude).
struct GradOut {
  float norm, factor, found_inf;
};
template <bool INF>
__device__ __forceinline__ GradOut grad_out(double v, double max_norm, const float* __restrict__ grad_scale) {
  const double c = grad_scale ? (double)grad_scale[0] : 1.0;
  const double x = (INF ? v : __builtin_sqrt(v)) * fabs(c);
  const double r = max_norm / (x + 1e-6);
  GradOut o;
  o.norm = (float)x;
  o.factor = (float)(max_norm < __builtin_huge_val() && !(r >= 1.0) ? c * r : c);   // a NaN norm: NaN
  o.found_inf = (o.norm - o.norm == 0.0f) ? 0.0f : 1.0f;
  return o;
}

template <bool INF>
__global__ __launch_bounds__(256) void k_grad_partial(const GradList list, double* __restrict__ partial) {
  __shared__ ListLds s;
  __shared__ double red[4];
  list_to_lds(list, s);
  const double v = join_block<INF>(sum_chunks<INF>(s, list.count, blockIdx.x, gridDim.x), red);
  if (threadIdx.x == 0) partial[blockIdx.x] = v;
}

// A few chunks (GN_SMALL) take one launch and one workgroup: four chunks at a time, the results, and the clipping. 4096
// bf16 values, clipped: 8.3 us against 19 in three launches, nearly all of it the host's.
constexpr int GN_SMALL = 16;
int grad_small_chunks() { return GN_SMALL; }
template <bool INF>
__global__ __launch_bounds__(1024) void k_grad_small(const GradList list, double max_norm,
                                                     const float* __restrict__ grad_scale, int clip,
                                                     float* __restrict__ norm, float* __restrict__ factor,
                                                     float* __restrict__ found_inf) {
  __shared__ ListLds s;
  __shared__ double red[16];
  __shared__ float f;
  list_to_lds(list, s);
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const double v = join_block<INF>(sum_chunks<INF>(s, list.count, group, 4), red);
  if (threadIdx.x == 0) {
    const GradOut o = grad_out<INF>(v, max_norm, grad_scale);
    *norm = o.norm;
    *factor = f = o.factor;
    *found_inf = o.found_inf;
  }
  if (!clip) return;
  __syncthreads();
  if (f != 1.0f) scale_chunks(s, list.count, group, 4, f);
}

template <bool INF>
__global__ __launch_bounds__(1024) void k_grad_final(const double* __restrict__ partial, int n, double max_norm,
                                                     const float* __restrict__ grad_scale, float* __restrict__ norm,
                                                     float* __restrict__ factor, float* __restrict__ found_inf) {
  __shared__ double red[16];
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) v = join<INF>(v, partial[i]);
  v = join_block<INF>(v, red);
  if (threadIdx.x == 0) {
    const GradOut o = grad_out<INF>(v, max_norm, grad_scale);
    *norm = o.norm;
    *factor = o.factor;
    *found_inf = o.found_inf;
  }
}

// g = D(factor g), nothing where factor is 1.
__global__ __launch_bounds__(256) void k_grad_scale(const GradList list, const float* __restrict__ factor) {
  const float f = factor[0];
  if (f == 1.0f) return;
  __shared__ ListLds s;
  list_to_lds(list, s);
  scale_chunks(s, list.count, blockIdx.x, gridDim.x, f);
}

hipError_t launch_grad_partial(const GradList& list, bool inf, double* partial, hipStream_t st) {
  const int g = grad_groups(list.start[list.count]);
  if (g == 0) return hipSuccess;
  if (inf) hipLaunchKernelGGL(k_grad_partial<true>, dim3(g), dim3(256), 0, st, list, partial);
  else hipLaunchKernelGGL(k_grad_partial<false>, dim3(g), dim3(256), 0, st, list, partial);
  return hipGetLastError();
}

hipError_t launch_grad_final(const double* partial, int n, bool inf, double max_norm, const float* grad_scale,
                             float* norm, float* factor, float* found_inf, hipStream_t st) {
  if (inf)
    hipLaunchKernelGGL(k_grad_final<true>, dim3(1), dim3(1024), 0, st, partial, n, max_norm, grad_scale, norm, factor,
                       found_inf);
  else
    hipLaunchKernelGGL(k_grad_final<false>, dim3(1), dim3(1024), 0, st, partial, n, max_norm, grad_scale, norm, factor,
                       found_inf);
  return hipGetLastError();
}

hipError_t launch_grad_small(const GradList& list, bool inf, double max_norm, const float* grad_scale, int clip,
                             float* norm, float* factor, float* found_inf, hipStream_t st) {
  auto kern = inf ? k_grad_small<true> : k_grad_small<false>;
  hipLaunchKernelGGL(kern, dim3(1), dim3(1024), 0, st, list, max_norm, grad_scale, clip, norm, factor, found_inf);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const GradList& list, const float* factor, hipStream_t st) {
  const int g = grad_groups(list.start[list.count]);
  if (g == 0) return hipSuccess;
  hipLaunchKernelGGL(k_grad_scale, dim3(g), dim3(256), 0, st, list, factor);
  return hipGetLastError();
}

}  // namespace i8l
