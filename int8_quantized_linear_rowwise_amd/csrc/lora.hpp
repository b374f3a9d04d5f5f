// What the adapter kernels share: token tiles, matrix-core fragments of the
// three dtypes, and the two-part form of fp32 values.
#pragma once

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
// begun by tile d are counted by a search 64 wide (every lane of the wave):
// one load for up to 64 segments, two for up to 4096.
// Up to 64 segments are held one a lane, so that any tile is found without
// another access to memory.
struct LoraTile {
  int t0, t1, adapter;
};
struct SegLanes {
  int start, adapter;   // of segment min(lane, n_seg - 1)
};
__device__ __forceinline__ SegLanes seg_lanes(const LoraSegs& S, int T) {
  const int s = min((int)(threadIdx.x & 63), max(S.n_seg, 1) - 1);
  return SegLanes{seg_start(S, s, T), seg_adapter(S, s)};
}

// How many of the ns segments (in order) satisfy a predicate that holds for a
// first part of them: pred(start, segment).
template <typename F>
__device__ __forceinline__ int count_segments(const LoraSegs& S, const SegLanes& L, int T, F pred) {
  const int lane = threadIdx.x & 63, ns = max(S.n_seg, 1);
  if (ns <= 64) return __popcll(__ballot(lane < ns && pred(L.start, lane)));
  int lo = 0, len = ns;
  while (len > 0) {
    const int step = (len + 63) >> 6;
    const int off = (lane + 1) * step - 1;
    const bool in = off < len && pred(seg_start(S, lo + off, T), lo + off);
    const int c = __popcll(__ballot(in));
    lo += c * step;
    len = min(step - 1, len - c * step);
  }
  return lo;
}

__device__ __forceinline__ LoraTile lora_tile(const LoraSegs& S, const SegLanes& L, int d, int T, int tm) {
  const int nb = (T + tm - 1) / tm, ns = max(S.n_seg, 1);
  const int lo = __builtin_amdgcn_readfirstlane(
      count_segments(S, L, T, [&](int start, int s) { return s + min(start / tm + 1, nb) <= d; }));
  int first, last, adapter;
  if (ns <= 64) {
    first = __builtin_amdgcn_readlane(L.start, max(lo - 1, 0));
    last = lo < ns ? __builtin_amdgcn_readlane(L.start, min(lo, 63)) : T;
    adapter = __builtin_amdgcn_readlane(L.adapter, max(lo - 1, 0));
  } else {
    first = seg_start(S, lo - 1, T);
    last = lo < ns ? seg_start(S, lo, T) : T;
    adapter = seg_adapter(S, max(lo - 1, 0));
  }
  const int i = d + 1 - lo;
  LoraTile r;
  r.t0 = min(max((i - 1) * tm, first), T);
  r.t1 = min(min(i * tm, T), last);
  if (lo <= 0 || i <= 0) r.t1 = r.t0;
  r.adapter = lo > 0 ? adapter : -1;
  r.t0 = __builtin_amdgcn_readfirstlane(r.t0);
  r.t1 = __builtin_amdgcn_readfirstlane(r.t1);
  r.adapter = __builtin_amdgcn_readfirstlane(r.adapter);
  return r;
}
// Number of the first tile of tokens [i tm, (i + 1) tm): i and the segments that start before.
__device__ __forceinline__ int first_tile(const LoraSegs& S, const SegLanes& L, int i, int T, int tm) {
  const int64_t at = (int64_t)i * tm;
  if (at >= T) return (T + tm - 1) / tm + max(S.n_seg, 1);
  const int lo = count_segments(S, L, T, [&](int start, int) { return start < at; });
  return __builtin_amdgcn_readfirstlane(i + lo);
}
// Tiles 1 .. lora_tiles() are the ones that can hold rows.
inline int lora_tiles(int T, const LoraSegs& S, int tm) {
  return (T + tm - 1) / tm + (S.n_seg > 1 ? S.n_seg : 1) - 1;
}

// The rank's class, in parts of 16.
inline int rank_tiles(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

// Workgroup `bid` of tiles * slices: the eight XCDs take workgroups in turn, so
// each gets one run of neighbouring tiles, whose rows share an adapter more
// often than not: its A and B then come through one L2 instead of all eight.
__device__ __forceinline__ void xcd_order(int bid, int total, int slices, int& tile, int& slice) {
  const int x = bid & 7, base = total >> 3, rem = total & 7;
  const int id = x * base + min(x, rem) + (bid >> 3);
  tile = id / slices;
  slice = id - tile * slices;
}

// Matrix-core fragments: 16 bytes a lane. Lane l of a 16-row operand holds row
// l & 15 and elements EL (l >> 4) .. of one step of KS along the contraction;
// the product's lane l holds column l & 15 (the second operand's row) and rows
// 4 (l >> 4) .. + 3 (the first's). A 16-bit step is one v_mfma_f32_16x16x32; an
// fp32 step is four v_mfma_f32_16x16x4, element j of every lane in product j
// (both operands order the contraction alike, so any order is right).
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

template <int DT>
struct Mx {
  static constexpr bool F32 = DT == DT_F32;
  static constexpr int EL = F32 ? 4 : 8;    // elements of a fragment
  static constexpr int KS = 4 * EL;         // contraction of a step
  static constexpr int NC = F32 ? 1 : 2;    // parts of an fp32 value
  __device__ static __forceinline__ v4f mma(v4u a, v4u b, v4f c) {
    if constexpr (DT == DT_BF16) {
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0,
                                                     0);
    } else if constexpr (DT == DT_F16) {
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
    } else {
      const v4f x = __builtin_bit_cast(v4f, a), y = __builtin_bit_cast(v4f, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[j], y[j], c, 0, 0, 0);
      return c;
    }
  }
};

// Element bits of a fragment, one at a time (tails and gathers).
template <int DT>
__device__ __forceinline__ void frag_set(v4u& f, int j, typename Elem<DT>::T e) {
  if constexpr (DT == DT_F32) f[j] = __float_as_uint(e);
  else f[j >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, e) << (16 * (j & 1));
}

// 16 bytes at any element boundary. Global loads and stores of 16 bytes need
// no alignment on gfx950; the type says so to the compiler.
typedef unsigned int v4u_any __attribute__((ext_vector_type(4), aligned(2)));
template <int DT>
__device__ __forceinline__ v4u ld16(const typename Elem<DT>::T* p) {
  return *reinterpret_cast<const v4u_any*>(p);
}
template <int DT>
__device__ __forceinline__ void st16(typename Elem<DT>::T* p, v4u v) {
  *reinterpret_cast<v4u_any*>(p) = v;
}

// The EL elements at p, those from `left` on taken as zero and not read.
template <int DT>
__device__ __forceinline__ v4u ld_frag(const typename Elem<DT>::T* p, int left) {
  if (left >= Mx<DT>::EL) return ld16<DT>(p);
  v4u f = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < Mx<DT>::EL; ++j)
    if (j < left) frag_set<DT>(f, j, p[j]);
  return f;
}
template <int DT>
__device__ __forceinline__ void st_frag(typename Elem<DT>::T* p, v4u f, int left) {
  if (left >= Mx<DT>::EL) {
    st16<DT>(p, f);
    return;
  }
#pragma unroll
  for (int j = 0; j < Mx<DT>::EL; ++j)
    if (j < left) {
      if constexpr (DT == DT_F32) p[j] = __uint_as_float(f[j]);
      else p[j] = __builtin_bit_cast(typename Elem<DT>::T, (uint16_t)(f[j >> 1] >> (16 * (j & 1))));
    }
}

// Fragment values as fp32 and back (one rounding).
template <int DT>
__device__ __forceinline__ void frag_f32(v4u f, float (&x)[Mx<DT>::EL]) {
#pragma unroll
  for (int j = 0; j < Mx<DT>::EL; ++j) {
    if constexpr (DT == DT_F32) x[j] = __uint_as_float(f[j]);
    else
      x[j] = Elem<DT>::to_f32(
          __builtin_bit_cast(typename Elem<DT>::T, (uint16_t)(j & 1 ? f[j >> 1] >> 16 : f[j >> 1] & 0xffffu)));
  }
}
template <int DT>
__device__ __forceinline__ v4u frag_of(const float (&x)[Mx<DT>::EL]) {
  v4u f;
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __float_as_uint(x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f[j] = (uint32_t)__builtin_bit_cast(uint16_t, Elem<DT>::from_f32(x[2 * j])) |
             ((uint32_t)__builtin_bit_cast(uint16_t, Elem<DT>::from_f32(x[2 * j + 1])) << 16);
  }
  return f;
}

// Rows of CW 16-byte chunks in LDS, chunk ch of row r at ch ^ (r / W): the rows
// of a fragment read (8 lanes, one chunk of 8 rows) and the chunks of a row
// written side by side fall on distinct banks.
template <int CW>
struct Rows {
  static constexpr int W = CW < 16 ? 16 / CW : 1, MASK = (CW < 16 ? CW : 16) - 1;
  __device__ static __forceinline__ v4u& at(char* p, int r, int ch) {
    return *reinterpret_cast<v4u*>(p + (r * CW + (ch ^ ((r / W) & MASK))) * 16);
  }
};

// V and dV are fp32 and enter products with 16-bit operands as hi + lo, two
// values of that type: hi is v rounded, lo the rest rounded, together within
// 2^-17 of v (bf16; 2^-22 in fp16). Rounding V to 16 bits once instead would
// add an error of the output's own rounding to every adapter product. An fp16
// pair covers fp32's range by a power of two that puts the largest magnitude
// of its set at 2^14: values down to 2^-17 of that keep 22 bits, to 2^-22 17
// bits, and below that an absolute 2^-39 of it; products with fp16 values stay
// far inside fp32. In products along r (out, grad_X) the set is one token's
// values, so no token depends on its neighbours. Along the tokens (grad_A,
// grad_B) one sum meets values of many tokens, and the set is what the tile
// has met so far.
template <int DT>
__device__ __forceinline__ uint32_t split2(float v, float unit) {
  if constexpr (DT == DT_F16) v *= unit;
  const typename Elem<DT>::T hi = Elem<DT>::from_f32(v);
  const float r = v - Elem<DT>::to_f32(hi);
  // an infinity has no rest (inf - inf would make it a NaN in `lo` alone)
  const typename Elem<DT>::T lo = Elem<DT>::from_f32(__builtin_isfinite(v) ? r : 0.0f);
  return (uint32_t)__builtin_bit_cast(uint16_t, hi) | ((uint32_t)__builtin_bit_cast(uint16_t, lo) << 16);
}
// Largest of the W lanes (16, 32 or 64 side by side, all active) that a lane
// belongs to, of values of 0 or more, whose bits order as they do.
template <int W>
__device__ __forceinline__ float lanes_max(float f) {
  uint32_t v = __float_as_uint(f);
  if constexpr (W == 64) {
    v = wave_umax(v);
  } else {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xB1, 0xf, 0xf, false));   // quad_perm 1,0,3,2
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4E, 0xf, 0xf, false));   // quad_perm 2,3,0,1
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x141, 0xf, 0xf, false));  // row_half_mirror
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x140, 0xf, 0xf, false));  // row_mirror
    if constexpr (W == 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
  }
  return __uint_as_float(v);
}

// Power of two that takes a largest magnitude `top` to [2^14, 2^15), and its
// inverse; 1 for zero, infinities and NaN. Both stay normal fp32 values.
__device__ __forceinline__ float unit_for(float top) {
  const int e = (int)((__float_as_uint(top) >> 23) & 0xff);
  if (e == 0xff || top == 0.0f) return 1.0f;
  return __uint_as_float((uint32_t)min(max(127 + 14 + 127 - e, 2), 252) << 23);
}
__device__ __forceinline__ float inv_pow2(float u) { return __uint_as_float((254u << 23) - __float_as_uint(u)); }

}  // namespace i8l
