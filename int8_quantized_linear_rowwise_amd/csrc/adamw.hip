// AdamW step over many tensors in one launch, states in 32 or 8 bits.
//
//   g' = c g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2,
//   w = w (1 - lr wd) - m / (sqrt(v) / sqrt(1 - b2^t) + eps) * lr / (1 - b1^t)
// w is the fp32 master copy where there is one (p = D(w)), else p. Every
// operation is rounded to fp32 by itself (no fused multiply-add), so the
// result does not depend on the path a tensor takes.
//
// Bound by memory. A workgroup takes 2048 values of one tensor, 8 a thread, so
// that bf16 moves 16 bytes a lane and a block of 256 8-bit states is half a
// wave's; it finds its tensor through a table, so any number of tensors is one
// launch. 202 M bf16 values with 32-bit states: 777 us, 5.7 TB/s; 41 M in 448
// tensors with 8-bit states and fp32 masters: 117 us, 5.4 TB/s (a large copy
// reaches 4.8 to 5.4).
//
// 8-bit states: blocks of 256 values, each with one scale; codes are e4m3.
// m is held as it is, v as its root q = sqrt(v): e4m3 spans a factor of 2^17,
// of which the square covers 2^35. The scale is the least power of two with
// absmax / scale <= 448 (e4m3's largest value), 2^-126 at least, so scaling is
// exact and the conversion rounds once (to nearest even, at most 2^-4
// relative for normal codes). A q over zero keeps at least the smallest code,
// 2^-9 scale: m's block can have a far smaller scale than q's after one large
// gradient, and a q of zero beside an m over zero would divide by eps. The
// step uses m and q before they are rounded to 8 bits.
#include "common.hpp"
#include "kernels.hpp"

#pragma clang fp contract(off)

namespace i8l {

constexpr int EPT = 8;               // values a thread takes: 32 lanes share one block of 256
constexpr int CHUNK = 256 * EPT;     // values of one workgroup

int adamw_chunk() { return CHUNK; }

template <int DT>
__device__ __forceinline__ void ld(const void* p, int64_t i, int n, bool vec, float (&f)[EPT]) {
  typedef typename Elem<DT>::T T;
  const T* q = static_cast<const T*>(p) + i;
  if (vec && n == EPT) {
    T e[EPT];
    load8<DT>(q, e);
#pragma unroll
    for (int j = 0; j < EPT; ++j) f[j] = Elem<DT>::to_f32(e[j]);
  } else {
#pragma unroll
    for (int j = 0; j < EPT; ++j) f[j] = j < n ? Elem<DT>::to_f32(q[j]) : 0.0f;
  }
}

template <int DT>
__device__ __forceinline__ void stv(void* p, int64_t i, int n, bool vec, const float (&f)[EPT]) {
  typedef typename Elem<DT>::T T;
  T* q = static_cast<T*>(p) + i;
  if (vec && n == EPT) {
    if constexpr (DT == DT_F32) {
      v4f* o = reinterpret_cast<v4f*>(q);
      o[0] = v4f{f[0], f[1], f[2], f[3]};
      o[1] = v4f{f[4], f[5], f[6], f[7]};
    } else {
      v4u o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = (uint32_t)__builtin_bit_cast(uint16_t, Elem<DT>::from_f32(f[2 * j])) |
               ((uint32_t)__builtin_bit_cast(uint16_t, Elem<DT>::from_f32(f[2 * j + 1])) << 16);
      *reinterpret_cast<v4u*>(q) = o;
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPT; ++j)
      if (j < n) q[j] = Elem<DT>::from_f32(f[j]);
  }
}

__device__ __forceinline__ void ld_any(int dt, const void* p, int64_t i, int n, bool vec, float (&f)[EPT]) {
  if (dt == DT_F32) ld<DT_F32>(p, i, n, vec, f);
  else if (dt == DT_F16) ld<DT_F16>(p, i, n, vec, f);
  else ld<DT_BF16>(p, i, n, vec, f);
}
__device__ __forceinline__ void st_any(int dt, void* p, int64_t i, int n, bool vec, const float (&f)[EPT]) {
  if (dt == DT_F32) stv<DT_F32>(p, i, n, vec, f);
  else if (dt == DT_F16) stv<DT_F16>(p, i, n, vec, f);
  else stv<DT_BF16>(p, i, n, vec, f);
}

__device__ __forceinline__ void ld_codes(const uint8_t* p, int64_t i, int n, bool vec, float scale, float (&f)[EPT]) {
  uint32_t w[2] = {0u, 0u};
  if (vec && n == EPT) {
    const v2u q = *reinterpret_cast<const v2u*>(p + i);
    w[0] = q[0];
    w[1] = q[1];
  } else {
#pragma unroll
    for (int j = 0; j < EPT; ++j)
      if (j < n) w[j >> 2] |= (uint32_t)p[i + j] << (8 * (j & 3));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f[4 * h + 0] = __builtin_amdgcn_cvt_f32_fp8((int)w[h], 0) * scale;
    f[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8((int)w[h], 1) * scale;
    f[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8((int)w[h], 2) * scale;
    f[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8((int)w[h], 3) * scale;
  }
}

// Codes and scale of the block that this half wave's 32 lanes hold.
template <bool POSITIVE>
__device__ __forceinline__ void st_codes(uint8_t* p, float* scale, int64_t i, int n, bool vec, const float (&f)[EPT]) {
  uint32_t top = 0u;   // magnitudes as integers: infinities and NaN stay on top
#pragma unroll
  for (int j = 0; j < EPT; ++j) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 32));
  // top = 1.m 2^E: 448 = 1.75 2^8, so the scale's exponent is E - 8, one more when 1.m > 1.75
  int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, 1);
  const bool bad = top >= 0x7f800000u;
  const float nan = __uint_as_float(0x7fc00000u);
  const float sc = bad ? nan : __uint_as_float((uint32_t)e << 23);
  const float inv = bad ? nan : __uint_as_float((uint32_t)(254 - e) << 23);
  float y[EPT];
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    y[j] = f[j] * inv;
    if (POSITIVE && f[j] > 0.0f && !bad) y[j] = fmaxf(y[j], 0.001953125f);
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h], y[4 * h + 1], 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h + 2], y[4 * h + 3], c, true);
    w[h] = (uint32_t)c;
  }
  if (vec && n == EPT) {
    *reinterpret_cast<v2u*>(p + i) = v2u{w[0], w[1]};
  } else {
#pragma unroll
    for (int j = 0; j < EPT; ++j)
      if (j < n) p[i + j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
  }
  if ((threadIdx.x & 31) == 0 && n > 0) scale[i / 256] = sc;
}

__global__ __launch_bounds__(256) void k_adamw(const AdamWTensor* __restrict__ tensors,
                                               const AdamWChunk* __restrict__ chunks, AdamWScalars h,
                                               const float* __restrict__ grad_scale,
                                               const float* __restrict__ found_inf) {
  if (found_inf && found_inf[0] != 0.0f) return;
  const AdamWChunk ch = chunks[blockIdx.x];
  const AdamWTensor t = tensors[ch.tensor];
  const int64_t i = (int64_t)ch.chunk * CHUNK + threadIdx.x * EPT;
  const int n = (int)min((int64_t)EPT, max((int64_t)0, t.n - i));
  const bool vec = t.vec != 0;
  const int64_t at = min(i, t.n);     // lanes past the end take part in the block's maximum only
  float w[EPT], g[EPT], m[EPT], v[EPT];
  ld_any(t.dtype, t.g, at, n, vec, g);
  if (t.master) ld<DT_F32>(t.master, at, n, vec, w);
  else ld_any(t.dtype, t.p, at, n, vec, w);
  if (t.bits == 8) {
    const int64_t blk = min(at, t.n - 1) / 256;
    ld_codes(static_cast<const uint8_t*>(t.m), at, n, vec, t.m_scale[blk], m);
    ld_codes(static_cast<const uint8_t*>(t.v), at, n, vec, t.v_scale[blk], v);
#pragma unroll
    for (int j = 0; j < EPT; ++j) v[j] = v[j] * v[j];
  } else {
    ld<DT_F32>(t.m, at, n, vec, m);
    ld<DT_F32>(t.v, at, n, vec, v);
  }
  const float gs = grad_scale ? grad_scale[0] : 1.0f;
  float q[EPT];
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const float gj = g[j] * gs;
    m[j] = m[j] * h.beta1 + gj * h.one_beta1;
    v[j] = v[j] * h.beta2 + (gj * gj) * h.one_beta2;
    q[j] = __builtin_sqrtf(v[j]);
    w[j] = w[j] * h.keep - (m[j] / (q[j] * h.inv_root_bc2 + h.eps)) * h.step_size;
  }
  st_any(t.dtype, t.p, at, n, vec, w);
  if (t.master) stv<DT_F32>(t.master, at, n, vec, w);
  if (t.bits == 8) {
    st_codes<false>(static_cast<uint8_t*>(t.m), t.m_scale, at, n, vec, m);
    st_codes<true>(static_cast<uint8_t*>(t.v), t.v_scale, at, n, vec, q);
  } else {
    stv<DT_F32>(t.m, at, n, vec, m);
    stv<DT_F32>(t.v, at, n, vec, v);
  }
}

hipError_t launch_adamw(const AdamWTensor* tensors, const AdamWChunk* chunks, int64_t n_chunks, const AdamWScalars& h,
                        const float* grad_scale, const float* found_inf, hipStream_t st) {
  hipLaunchKernelGGL(k_adamw, dim3((unsigned)n_chunks), dim3(256), 0, st, tensors, chunks, h, grad_scale, found_inf);
  return hipGetLastError();
}

}  // namespace i8l
