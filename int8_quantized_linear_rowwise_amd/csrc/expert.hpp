// What the expert kernels share: row tiles of segments, gathered rows, and the
// fp16 operands of the outlier product.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace i8l {

// Start of segment s, held inside [0, R] whatever the caller's offsets are.
// Segment n_seg holds the rows behind the last offset and has no expert.
__device__ __forceinline__ int expert_start(const ExpertSegs& S, int s, int R) {
  return s <= 0 ? 0 : s > S.n_seg ? R : min(max(S.off[s], 0), R);
}

__device__ __forceinline__ int expert_of(const ExpertSegs& S, int s) {
  if (s >= S.n_seg) return -1;
  const int e = S.ids ? S.ids[s] : s;
  return (e >= 0 && e < S.n_experts) ? e : -1;
}

// Row tiles: every segment is cut into tiles of tm rows from its own start, so
// a tile lies in one segment. Segment s owns the slots from start(s) / tm + s
// on: ceil(len / tm) of them never reach the next segment's, so a slot is found
// from the offsets alone, without a prefix sum of the tile counts. The search
// is 64 wide (every lane of the wave): one load for up to 64 segments, two for
// up to 4096.
struct ExpertTile {
  int r0, r1, expert;   // rows [r0, r1), none where r1 <= r0; expert -1: rows of zeros
};
__device__ __forceinline__ ExpertTile expert_tile(const ExpertSegs& S, int slot, int R, int tm) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = S.n_seg + 1;     // segments whose first slot is <= slot
  while (len > 0) {
    const int step = (len + 63) >> 6;
    const int o = (lane + 1) * step - 1;
    const bool in = o < len && expert_start(S, lo + o, R) / tm + lo + o <= slot;
    const int c = __popcll(__ballot(in));
    lo += c * step;
    len = min(step - 1, len - c * step);
  }
  const int s = __builtin_amdgcn_readfirstlane(max(lo - 1, 0));
  const int start = expert_start(S, s, R), end = expert_start(S, s + 1, R);
  const int i = slot - (start / tm + s);
  ExpertTile t;
  t.r0 = __builtin_amdgcn_readfirstlane(start + i * tm);
  t.r1 = __builtin_amdgcn_readfirstlane(i < 0 ? start + i * tm : min(start + (i + 1) * tm, end));
  t.expert = __builtin_amdgcn_readfirstlane(expert_of(S, s));
  return t;
}
// Slots of R rows: 0 .. expert_slots() - 1.
inline int64_t expert_slots(int64_t R, int64_t n_seg, int tm) { return R / tm + n_seg + 1; }

// Grid of `total` workgroups in two dimensions (a grid axis holds fewer than 2^32 threads).
inline dim3 expert_grid(int64_t total) {
  const int64_t x = total < (1 << 20) ? total : (1 << 20);
  return dim3((unsigned)x, (unsigned)((total + x - 1) / x));
}
__device__ __forceinline__ int64_t expert_block() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Token of row r (any r inside the tile): -1 where the caller's index lies outside [0, T).
__device__ __forceinline__ int row_token(const int32_t* __restrict__ rows, int r, int T) {
  const int t = rows ? rows[r] : r;
  return (t >= 0 && t < T) ? t : -1;
}

// fp16 outlier values j0 .. j0 + 7 of token t (zero at and past cnt, or for no
// token): from the quantizer's staged copy for the first cap columns, beyond
// them from the input itself.
template <int DT>
__device__ __forceinline__ v8h expert_out_a8(const uint16_t* __restrict__ sub, int cap,
                                             const typename Elem<DT>::T* __restrict__ X, int K,
                                             const int32_t* __restrict__ idx, int t, int j0, int cnt) {
  v8h q = {};
  if (t >= 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = j0 + e;
      if (j < cnt)
        q[e] = j < cap ? __builtin_bit_cast(_Float16, sub[(int64_t)t * cap + j])
                       : to_half<DT>(X[(int64_t)t * K + idx[j]]);
    }
  }
  return q;
}
// Dequantized weights of those columns, row n of an expert's weight: fp16(CB * fl32(SCB * fl32(1/127))).
__device__ __forceinline__ v8h expert_out_w8(const int8_t* __restrict__ CB, const float* __restrict__ SCB, int K,
                                             const int32_t* __restrict__ idx, int n, bool ok, int j0, int cnt) {
  v8h p = {};
  if (ok) {
    const float sig = SCB[n] * (1.0f / 127.0f);
    const int8_t* row = CB + (int64_t)n * K;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j0 + e < cnt) p[e] = half_of_f32((float)row[idx[j0 + e]] * sig);
  }
  return p;
}

}  // namespace i8l
