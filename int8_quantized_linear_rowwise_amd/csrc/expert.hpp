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
// a tile lies in one segment. Every wave finds its tile from the offsets alone.
// Up to 255 segments: a scan of the tile counts, 64 segments at a time, so that
// only tiles with rows are launched for (but for those of a bound on their
// number). More: segment s owns the slots from start(s) / tm + s on; its
// ceil(len / tm) tiles never reach the next segment's, so a search 64 wide finds
// the segment in two or three loads, and slots that hold no tile end at once.
struct ExpertTile {
  int r0, r1, expert;   // rows [r0, r1), none where r1 <= r0; expert -1: rows of zeros
};
constexpr int SCAN_SEGMENTS = 256;
__device__ __forceinline__ ExpertTile expert_tile(const ExpertSegs& S, int slot, int R, int tm) {
  const int lane = threadIdx.x & 63;
  int s, i;      // segment, and the tile's number in it
  if (S.n_seg < SCAN_SEGMENTS) {
    int before = 0;
    s = S.n_seg + 1;
    i = 0;
    for (int s0 = 0; s0 <= S.n_seg; s0 += 64) {
      const int mine = s0 + lane;
      const int len = mine <= S.n_seg ? expert_start(S, mine + 1, R) - expert_start(S, mine, R) : 0;
      const int tiles = len > 0 ? (len + tm - 1) / tm : 0;
      int incl = tiles;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(incl, o, 64);
        incl += lane >= o ? v : 0;
      }
      const int total = __builtin_amdgcn_readlane(incl, 63);
      if (slot < before + total) {
        const int l = __popcll(__ballot(before + incl <= slot));
        s = s0 + l;
        i = slot - before - (l > 0 ? __builtin_amdgcn_readlane(incl, l - 1) : 0);
        break;
      }
      before += total;
    }
    if (s > S.n_seg) return ExpertTile{0, 0, -1};
  } else {
    int lo = 0, len = S.n_seg + 1;     // segments whose first slot is <= slot
    while (len > 0) {
      const int step = (len + 63) >> 6;
      const int o = (lane + 1) * step - 1;
      const bool in = o < len && expert_start(S, lo + o, R) / tm + lo + o <= slot;
      const int c = __popcll(__ballot(in));
      lo += c * step;
      len = min(step - 1, len - c * step);
    }
    s = max(lo - 1, 0);
    i = slot - (expert_start(S, s, R) / tm + s);
  }
  s = __builtin_amdgcn_readfirstlane(s);
  i = __builtin_amdgcn_readfirstlane(i);
  const int start = expert_start(S, s, R), end = expert_start(S, s + 1, R);
  ExpertTile t;
  t.r0 = __builtin_amdgcn_readfirstlane(start + i * tm);
  t.r1 = __builtin_amdgcn_readfirstlane(i < 0 ? start + i * tm : min(start + (i + 1) * tm, end));
  t.expert = __builtin_amdgcn_readfirstlane(expert_of(S, s));
  return t;
}
// Tiles to launch for: at most one per non-empty segment is not full.
inline int64_t expert_slots(int64_t R, int64_t n_seg, int tm) {
  if (n_seg >= SCAN_SEGMENTS) return R / tm + n_seg + 1;
  const int64_t parts = n_seg + 1 < R ? n_seg + 1 : R;
  return (R + parts * (tm - 1)) / tm;
}

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

// Bytes k .. k + 15 of a row of K bytes at any address, zero past its end: one
// load of 16 bytes, which global memory takes unaligned; the last piece of a row
// is loaded so that it ends with the row and shifted into place.
__device__ __forceinline__ v4i bytes16(const int8_t* row, int k, int K) {
  unsigned __int128 v = 0;
  if (k + 16 <= K) {
    __builtin_memcpy(&v, row + k, 16);
  } else if (k < K) {
    if (K >= 16) {
      __builtin_memcpy(&v, row + K - 16, 16);
      v >>= 8 * (k + 16 - K);
    } else {
      for (int b = 0; b < K; ++b) v |= (unsigned __int128)(uint8_t)row[b] << (8 * b);   // k is 0
    }
  }
  return __builtin_bit_cast(v4i, v);
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
