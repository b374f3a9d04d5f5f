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
// Up to 255 segments: a scan of the tile counts, four times 64 segments, so that
// the number of tiles is known in the kernel and only tiles with rows are worked
// on. Tiles of rows without an expert, which only get zeros, come behind all
// others: left in their places, they would leave the work of a rank that holds one
// of eight experts to one XCD of eight (8192 rows, 4096 -> 11008, bf16: 303 us
// against 117, the gradient 502 against 142). More: segment s owns the slots from start(s) / tm + s on; its
// ceil(len / tm) tiles never reach the next segment's, so a search 64 wide finds
// the segment in two or three loads, and slots that hold no tile end at once. There
// the tiles of rows without an expert stay in the rows' order and the empty slots
// count as tiles: 4096 tokens, eight of 255 experts against eight of 256, 2048 ->
// 1408, bf16: 266 us against 270, gradient 394 against 431, but on a rank that holds
// an eighth of them 90 against 220 and 108 against 370.
struct ExpertTile {
  int r0, r1, expert;   // rows [r0, r1), none where r1 <= r0; expert -1: rows of zeros
};
constexpr int SCAN_SEGMENTS = 256;
// Sum over the lanes up to and with this one.
__device__ __forceinline__ int lane_scan(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    v += lane >= o ? u : 0;
  }
  return v;
}
struct ExpertScan {
  int total, zeros;                 // slots with an expert, and without one behind them
  int incl[4], none[4];             // of lane l's segment 64 b + l: slots of either kind up to and with it
  int start[4], end[4];             // and its rows
};
__device__ __forceinline__ ExpertScan expert_scan(const ExpertSegs& S, int R, int tm) {
  const int lane = threadIdx.x & 63;
  ExpertScan c;
  if (S.n_seg >= SCAN_SEGMENTS) {
    c.total = R / tm + S.n_seg + 1;
    c.zeros = 0;
    return c;
  }
  c.total = 0;
  c.zeros = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    c.incl[b] = c.total;
    c.none[b] = c.zeros;
    if (64 * b <= S.n_seg) {
      const int s = 64 * b + lane;
      c.start[b] = expert_start(S, s, R);
      c.end[b] = expert_start(S, s + 1, R);
      const int len = s <= S.n_seg ? c.end[b] - c.start[b] : 0;
      const int tiles = len > 0 ? (len + tm - 1) / tm : 0;
      const bool has = tiles > 0 && expert_of(S, s) >= 0;
      c.incl[b] += lane_scan(has ? tiles : 0);
      c.none[b] += lane_scan(has ? 0 : tiles);
      c.total = __builtin_amdgcn_readlane(c.incl[b], 63);
      c.zeros = __builtin_amdgcn_readlane(c.none[b], 63);
    }
  }
  // offsets that are not non-decreasing can count rows twice: no more tiles than were launched for
  const int most = (R + min(S.n_seg + 1, R) * (tm - 1)) / tm;
  c.total = min(c.total, most);
  c.zeros = min(c.zeros, most - c.total);
  return c;
}
// Slot 0 <= slot < total + zeros.
__device__ __forceinline__ ExpertTile expert_tile(const ExpertSegs& S, const ExpertScan& c, int slot, int R, int tm) {
  const int lane = threadIdx.x & 63;
  int s = 0, i, start = 0, end = 0;      // segment, the tile's number in it, and its rows
  if (S.n_seg < SCAN_SEGMENTS) {
    int before = 0;
    const bool none = slot >= c.total;
    if (none) slot -= c.total;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (64 * b <= S.n_seg) {
        const int incl = none ? c.none[b] : c.incl[b];
        const int l = __popcll(__ballot(incl <= slot));      // segments that end before the slot: a first part
        if (l > 0) before = __builtin_amdgcn_readlane(incl, l - 1);
        if (s == 64 * b) {      // all of the blocks before
          start = __builtin_amdgcn_readlane(c.start[b], min(l, 63));
          end = __builtin_amdgcn_readlane(c.end[b], min(l, 63));
        }
        s += l;
      }
    i = slot - before;
  } else {
    int lo = 0, len = S.n_seg + 1;     // segments whose first slot is <= slot
    while (len > 0) {
      const int step = (len + 63) >> 6;
      const int o = (lane + 1) * step - 1;
      const bool in = o < len && expert_start(S, lo + o, R) / tm + lo + o <= slot;
      const int n = __popcll(__ballot(in));
      lo += n * step;
      len = min(step - 1, len - n * step);
    }
    s = max(lo - 1, 0);
    start = expert_start(S, s, R);
    end = expert_start(S, s + 1, R);
    i = slot - (start / tm + s);
  }
  s = __builtin_amdgcn_readfirstlane(s);
  i = __builtin_amdgcn_readfirstlane(i);
  ExpertTile t;
  t.r0 = __builtin_amdgcn_readfirstlane(start + i * tm);
  t.r1 = __builtin_amdgcn_readfirstlane(i < 0 ? start + i * tm : min(start + (i + 1) * tm, end));
  t.expert = __builtin_amdgcn_readfirstlane(expert_of(S, s));
  return t;
}
// Slots to launch for, at least as many as the scan finds: at most one tile of a segment is not full.
inline int64_t expert_slots(int64_t R, int64_t n_seg, int tm) {
  if (n_seg >= SCAN_SEGMENTS) return R / tm + n_seg + 1;
  const int64_t parts = n_seg + 1 < R ? n_seg + 1 : R;
  return (R + parts * (tm - 1)) / tm;
}

// Work of a workgroup of the large-tile kernels: tile (slot, column tile), or
// one of `parts` column parts of it. One workgroup runs on a compute unit at a
// time, so tiles run in rounds of 256, and a last round of a few tiles takes as
// long as a full one. Up to SPLIT_2 tiles over the full rounds are cut in two,
// up to SPLIT_4 in four, which spreads them over idle units.
// The XCDs take workgroups in turn; each gets one run of neighbouring tiles, in
// groups of four slots by all columns, whose weights and rows meet in its L2.
constexpr int ROUND = 256, SPLIT_4 = 64, SPLIT_2 = 128;
struct ExpertWork {
  int slot, tc, part, parts;     // slot -1: none
};
// Behind them come the tiles of rows without an expert.
template <bool CUT>
__device__ __forceinline__ ExpertWork expert_work(int64_t bid, const ExpertScan& c, int tiles_c) {
  const int slots = c.total;
  const int nt = slots * tiles_c, rem = CUT ? nt % ROUND : 0;
  ExpertWork w = {-1, 0, 0, rem == 0 || rem > SPLIT_2 ? 1 : rem > SPLIT_4 ? 2 : 4};
  const int full = w.parts > 1 ? nt - rem : nt;      // tiles worked on whole
  int id;
  if (bid < full) {
    const int b = (int)bid, x = b & 7, base = full >> 3, r = full & 7;
    id = x * base + min(x, r) + (b >> 3);
    w.parts = 1;
  } else {
    const int64_t q = bid - full;
    const int64_t z = q - (int64_t)(nt - full) * w.parts;
    if (z >= 0) {
      w.parts = 1;
      if (z >= (int64_t)c.zeros * tiles_c) return w;
      w.slot = slots + (int)(z / tiles_c);
      w.tc = (int)(z % tiles_c);
      return w;
    }
    id = full + (int)q / w.parts;
    w.part = (int)q % w.parts;
  }
  constexpr int GRP = 4;
  const int group = id / (GRP * tiles_c), first = group * GRP, gsz = min(slots - first, GRP);
  const int in = id - group * GRP * tiles_c;
  w.slot = first + in % gsz;
  w.tc = in / gsz;
  return w;
}
// Workgroups for that with CUT: cut tiles take at most 3 SPLIT_4 more.
inline int64_t expert_groups(int64_t slots, int64_t tiles_c) { return slots * tiles_c + 3 * SPLIT_4; }

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

// 16 bytes at any address (global memory takes unaligned loads).
__device__ __forceinline__ v4u bytes16(const int8_t* p) {
  v4u v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
// Rows of K >= 16 bytes at any address: the last piece is loaded so that it ends
// with the row (at tail_at(k)), in both operands alike; in the codes, the bytes
// that the piece before holds already are cleared.
__device__ __forceinline__ int tail_at(int k, int K) { return min(k, K - 16); }
__device__ __forceinline__ v4u tail_clear(v4u v, int k, int K) {
  const int d = k - tail_at(k, K);      // bytes to clear
#pragma unroll
  for (int x = 0; x < 4; ++x) v[x] &= (uint32_t)(0xffffffffull << min(max(8 * (d - 4 * x), 0), 32));
  return v;
}
// Bytes k .. k + 15 of a row of fewer than 16, zero past its end.
__device__ __forceinline__ v4u short_row(const int8_t* row, int k, int K) {
  v4u v = {0u, 0u, 0u, 0u};
  for (int b = k; b < K; ++b) v[b >> 2] |= (uint32_t)(uint8_t)row[b] << (8 * (b & 3));
  return v;
}

// Outlier columns j0 .. j0 + 7 (0 at and past cnt). They and their number belong
// to no tile: the kernels ask for the first ones before anything else.
struct OutlierCols {
  int c[8];
};
__device__ __forceinline__ OutlierCols expert_out_cols(const int32_t* __restrict__ idx, int j0, int cnt) {
  OutlierCols o;
#pragma unroll
  for (int e = 0; e < 8; ++e) o.c[e] = j0 + e < cnt ? idx[j0 + e] : 0;
  return o;
}
// fp16 outlier values j0 .. j0 + 7 of token t (zero at and past cnt, or for no
// token): from the quantizer's staged copy for the first cap columns, beyond
// them from the input itself.
template <int DT>
__device__ __forceinline__ v8h expert_out_a8(const uint16_t* __restrict__ sub, int cap,
                                             const typename Elem<DT>::T* __restrict__ X, int K, const OutlierCols& o,
                                             int t, int j0, int cnt) {
  v8h q = {};
  if (t >= 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = j0 + e;
      if (j < cnt)
        q[e] = j < cap ? __builtin_bit_cast(_Float16, sub[(int64_t)t * cap + j])
                       : to_half<DT>(X[(int64_t)t * K + o.c[e]]);
    }
  }
  return q;
}
// Dequantized weights of those columns, row n of an expert's weight: fp16(CB * fl32(SCB * fl32(1/127))).
__device__ __forceinline__ v8h expert_out_w8(const int8_t* __restrict__ CB, const float* __restrict__ SCB, int K,
                                             const OutlierCols& o, int n, bool ok, int j0, int cnt) {
  v8h p = {};
  if (ok) {
    const float sig = SCB[n] * (1.0f / 127.0f);
    const int8_t* row = CB + (int64_t)n * K;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j0 + e < cnt) p[e] = half_of_f32((float)row[o.c[e]] * sig);
  }
  return p;
}

// Zeros into columns [c0, c1) of rows [r0, r1), by the whole workgroup: rows without an expert.
template <typename E>
__device__ __forceinline__ void expert_zeros(E* out, int64_t ld, int r0, int r1, int c0, int c1) {
  constexpr int V = 16 / sizeof(E);
  const int step = blockDim.x;
  if (ld % V == 0 && (uintptr_t)out % 16 == 0 && (c1 - c0) % V == 0) {      // c0 is on a border of 16 values
    const int w = (c1 - c0) / V, n = (r1 - r0) * w;
    for (int i = threadIdx.x; i < n; i += step)
      *reinterpret_cast<v4u*>(out + (int64_t)(r0 + i / w) * ld + c0 + i % w * V) = v4u{0u, 0u, 0u, 0u};
  } else {
    const int w = c1 - c0, n = (r1 - r0) * w;
    for (int i = threadIdx.x; i < n; i += step) out[(int64_t)(r0 + i / w) * ld + c0 + i % w] = E{};
  }
}

// Scale of a row without a token: such a row is zeros, whatever its expert's weights hold.
constexpr float NO_TOKEN = -0.0f;
__device__ __forceinline__ bool no_token(float sa) { return __float_as_uint(sa) == 0x80000000u; }

// Output tiles in LDS, so that global stores cover whole rows: 16-byte chunk c of
// row r (RB bytes) at chunk position c ^ (r mod RB / 16). Where rows start on
// 16-byte borders a lane stores 8 values, else one or two, with lanes side by
// side: products of 4096 tokens with two of eight 4096 -> 11007 experts, bf16 478 us
// against 543 with 8 stores a lane, fp32 533 against 691 straight from registers.
template <int RB>
__device__ __forceinline__ int etile_off(int row, int chunk) {
  return row * RB + 16 * (chunk ^ (row & (RB / 16 - 1)));
}
// BM rows by BN 16-bit values. Rows whose scale in `lsa` (if any) says that they have no token are stored as zeros.
template <int BM, int BN, int THREADS, typename E>
__device__ __forceinline__ void etile_store(const char* ot, const float* lsa, E* __restrict__ dst, int64_t ld, int r0,
                                            int c0, int r1, int c1) {
  static_assert(sizeof(E) == 2, "16-bit outputs");
  constexpr int CPR = BN / 8;
  const int rows = min(BM, r1 - r0);
  if (ld % 8 == 0 && (uintptr_t)dst % 16 == 0) {      // c1 is ld, or a tile's border
#pragma unroll 4
    for (int i = threadIdx.x; i < rows * CPR; i += THREADS) {
      const int row = i / CPR, ch = i % CPR, c = c0 + ch * 8;
      v4u v = *reinterpret_cast<const v4u*>(ot + etile_off<2 * BN>(row, ch));
      if (lsa != nullptr && no_token(lsa[row])) v = v4u{0u, 0u, 0u, 0u};
      if (c < c1) *reinterpret_cast<v4u*>(dst + (int64_t)(r0 + row) * ld + c) = v;
    }
  } else if (ld % 2 == 0 && (uintptr_t)dst % 4 == 0) {
#pragma unroll 4
    for (int i = threadIdx.x; i < rows * (BN / 2); i += THREADS) {
      const int row = i / (BN / 2), col = i % (BN / 2) * 2, c = c0 + col;
      uint32_t v = *reinterpret_cast<const uint32_t*>(ot + etile_off<2 * BN>(row, col >> 3) + 2 * (col & 7));
      if (lsa != nullptr && no_token(lsa[row])) v = 0u;
      if (c < c1) *reinterpret_cast<uint32_t*>(dst + (int64_t)(r0 + row) * ld + c) = v;
    }
  } else {
#pragma unroll 4
    for (int i = threadIdx.x; i < rows * BN; i += THREADS) {
      const int row = i / BN, col = i % BN, c = c0 + col;
      uint16_t v = *reinterpret_cast<const uint16_t*>(ot + etile_off<2 * BN>(row, col >> 3) + 2 * (col & 7));
      if (lsa != nullptr && no_token(lsa[row])) v = 0;
      if (c < c1) dst[(int64_t)(r0 + row) * ld + c] = __builtin_bit_cast(E, v);
    }
  }
}
// BM rows by BN fp32 values, rows that start anywhere, through `bytes` of LDS, in
// two parts where they do not fit at once. value(i, j, q): the lane's four values
// of columns wn BN / 2 + 32 i + 8 q + 4 lg .. + 3 and row 64 wm + 32 j + lr.
template <int BM, int BN, int THREADS, int BYTES, typename V>
__device__ __forceinline__ void etile_f32(char* ot, V value, const float* lsa, float* __restrict__ dst, int64_t ld,
                                          int r0, int c0, int r1, int c1, int wn, int wm, int lr, int lg) {
  constexpr int PARTS = BM * BN * 4 > BYTES ? 2 : 1, TIP = BN / 64 / PARTS, CP = BN / PARTS, HALF = CP / 2;
  static_assert(BM * CP * 4 <= BYTES && TIP > 0, "a part fits");
  const int rows = min(BM, r1 - r0);
#pragma unroll
  for (int h = 0; h < PARTS; ++h) {
    __syncthreads();   // what lay there is no longer read
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < TIP; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<v4f*>(
              ot + etile_off<4 * CP>(wm * 64 + j * 32 + lr, (wn * HALF + i * 32 + q * 8) / 4 + lg)) =
              value(h * TIP + i, j, q);
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < rows * CP; i += THREADS) {
      const int row = i / CP, col = i % CP, c = c0 + col / HALF * (BN / 2) + h * HALF + col % HALF;
      float v = *reinterpret_cast<const float*>(ot + etile_off<4 * CP>(row, col >> 2) + 4 * (col & 3));
      if (lsa != nullptr && no_token(lsa[row])) v = 0.0f;
      if (c < c1) dst[(int64_t)(r0 + row) * ld + c] = v;
    }
  }
}

// Four results of one row to p[0 .. 3], of which m lie inside the row; vec: p is on a border of four.
template <int DT>
__device__ __forceinline__ void expert_store4(typename Elem<DT>::T* p, const float (&y)[4], int m, bool vec) {
  typename Elem<DT>::T v[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) v[x] = Elem<DT>::from_f32(y[x]);
  if (vec && m >= 4) {
    if constexpr (DT == DT_F32)
      *reinterpret_cast<v4f*>(p) = v4f{y[0], y[1], y[2], y[3]};
    else
      *reinterpret_cast<v2u*>(p) =
          v2u{(uint32_t)__builtin_bit_cast(uint16_t, v[0]) | ((uint32_t)__builtin_bit_cast(uint16_t, v[1]) << 16),
              (uint32_t)__builtin_bit_cast(uint16_t, v[2]) | ((uint32_t)__builtin_bit_cast(uint16_t, v[3]) << 16)};
  } else {
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (x < m) p[x] = v[x];
  }
}

}  // namespace i8l
