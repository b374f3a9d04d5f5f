// Pieces of the quantizer's kernels: chunks of 8 consecutive values of a row.
#pragma once

#include "common.hpp"

namespace i8l {

typedef unsigned short us2 __attribute__((ext_vector_type(2)));

// Load 8 consecutive elements of row r (cols c0..c0+7) as raw words, zero
// past the end of the row. vec: rows are 16-byte aligned and cols % 8 == 0. Other
// rows are read 16 bytes at a time too, at any address: 4096 x 4095 bf16 values
// quantized in 24 us against 48 with a load for each.
template <int DT>
__device__ __forceinline__ void load_raw8(const typename Elem<DT>::T* __restrict__ row, int c0, int cols, bool vec,
                                          v4u& a, v4u& b) {
  typedef typename Elem<DT>::T T;
  if (vec && c0 + 8 <= cols) {
    a = *reinterpret_cast<const v4u*>(row + c0);
    if constexpr (DT == DT_F32) b = *reinterpret_cast<const v4u*>(row + c0 + 4);
    return;
  }
  if (c0 + 8 <= cols) {      // at any address
    __builtin_memcpy(&a, row + c0, 16);
    if constexpr (DT == DT_F32) __builtin_memcpy(&b, row + c0 + 4, 16);
    return;
  }
  uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (c0 + e < cols) {
      if constexpr (DT == DT_F32) {
        w[e] = __float_as_uint(row[c0 + e]);
      } else {
        const uint32_t h = (uint32_t)__builtin_bit_cast(uint16_t, row[c0 + e]);
        w[e >> 1] |= h << (16 * (e & 1));
      }
    }
  }
  a = v4u{w[0], w[1], w[2], w[3]};
  if constexpr (DT == DT_F32) b = v4u{w[4], w[5], w[6], w[7]};
}

// fp16 value (as fp32) of element e of a raw 8-element chunk
template <int DT>
__device__ __forceinline__ float chunk_val(const v4u& a, const v4u& b, int e) {
  if constexpr (DT == DT_F32) {
    const uint32_t w = (e < 4) ? a[e] : b[e - 4];
    return (float)(_Float16)__uint_as_float(w);
  } else {
    const uint32_t w = a[e >> 1];
    const uint16_t h = (uint16_t)((e & 1) ? (w >> 16) : (w & 0xffffu));
    if constexpr (DT == DT_F16) return (float)__builtin_bit_cast(_Float16, h);
    else return (float)(_Float16)bf16_to_f32(h);
  }
}

// magnitude bits of element e of a raw chunk, in the storage format
template <int DT>
__device__ __forceinline__ uint32_t chunk_mag(const v4u& a, const v4u& b, int e) {
  if constexpr (DT == DT_F32) return ((e < 4) ? a[e] : b[e - 4]) & 0x7fffffffu;
  else return ((e & 1) ? (a[e >> 1] >> 16) : a[e >> 1]) & 0x7fffu;
}

template <int DT>
__device__ __forceinline__ float mag_to_half_value(uint32_t m) {
  if constexpr (DT == DT_F32) return (float)(_Float16)__uint_as_float(m);
  else if constexpr (DT == DT_F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)m);
  else return (float)(_Float16)bf16_to_f32((uint16_t)m);
}
// column-mask bits of chunk ci
__device__ __forceinline__ uint32_t chunk_mask_bits(const uint32_t* smask, int ci) {
  const int c0 = ci * 8;
  return (smask[c0 >> 5] >> (c0 & 31)) & 0xffu;
}

// largest magnitude (storage-format bits) of the chunk's non-outlier
// elements; om: the chunk's outlier-column bits; any: some lane of the wave
// has an outlier column in this chunk (wave-uniform, so that the common case
// skips all masking)
template <int DT, bool VEC>
__device__ __forceinline__ uint32_t chunk_absmax(const v4u& a, const v4u& b, uint32_t om, bool any) {
  if constexpr (VEC && DT != DT_F32) {
    us2 mx = {0, 0};
    if (!any) {
#pragma unroll
      for (int d = 0; d < 4; ++d) mx = __builtin_elementwise_max(mx, __builtin_bit_cast(us2, a[d] & 0x7fff7fffu));
    } else {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t keep = (((om >> (2 * d)) & 1u) ? 0u : 0x0000ffffu) | (((om >> (2 * d + 1)) & 1u) ? 0u : 0xffff0000u);
        mx = __builtin_elementwise_max(mx, __builtin_bit_cast(us2, a[d] & 0x7fff7fffu & keep));
      }
    }
    return max((uint32_t)mx[0], (uint32_t)mx[1]);
  } else {
    uint32_t mx = 0u;
    if (!any) {
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = max(mx, chunk_mag<DT>(a, b, e));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t m = chunk_mag<DT>(a, b, e);
        mx = ((om >> e) & 1u) ? mx : max(mx, m);
      }
    }
    return mx;
  }
}

// codes of one chunk, packed little-endian into two words: x16 = fp16(x),
// code = rint(fl32(x16 * inv)) by the exact fp32 add of 1.5 * 2^23
template <int DT>
__device__ __forceinline__ void chunk_quant8(const v4u& a, const v4u& b, float inv, uint32_t& lo, uint32_t& hi) {
#pragma clang fp contract(off)
  uint32_t h[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if constexpr (DT == DT_F16) h[d] = a[d];
    else if constexpr (DT == DT_BF16) h[d] = bf16x2_to_f16x2(a[d]);
    else h[d] = f32x2_to_f16x2(__uint_as_float(d < 2 ? a[2 * d] : b[2 * d - 4]),
                               __uint_as_float(d < 2 ? a[2 * d + 1] : b[2 * d - 3]));
  }
  uint32_t q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const _Float16 x = __builtin_bit_cast(_Float16, (uint16_t)(h[e >> 1] >> (16 * (e & 1))));
    const float p = (float)x * inv;
    q[e] = __float_as_uint(p + 12582912.0f);
  }
  lo = __builtin_amdgcn_perm(q[1], q[0], 0x0c0c0400u) | __builtin_amdgcn_perm(q[3], q[2], 0x04000c0cu);
  hi = __builtin_amdgcn_perm(q[5], q[4], 0x0c0c0400u) | __builtin_amdgcn_perm(q[7], q[6], 0x04000c0cu);
}

}  // namespace i8l
