// Low-rank adapters of many requests beside a shared projection: forward.
//
// Token t of adapter a: V[t] = A[a] x[t] (R values, fp32) and
//   y[t] = D(base[t] + s[a] B[a] V[t]).
// Bound by memory: T (K + 2 N) elements and the adapters in use once, against
// 2 T R (K + N) flops. Two launches, each reading its large operand once:
// `shrink` (X and A to V) and `expand` (V, B and base to out). The token rows
// are cut into tiles of one adapter each (lora_tile), 64 tokens in long
// batches and 16 otherwise, so a decoding step of single tokens runs one tile a
// token and every launch is filled by splitting the other axis.
#include <type_traits>

#include "lora.hpp"

namespace i8l {

namespace {

constexpr int MAX_SPLITS = 8;

// acc[i][j] += X's rows 16 i .. of the tile times A[a]'s rows 16 j .., over the
// contraction steps s0 .. s1 - 1 that fall to `wave` of NW. A wave takes pairs
// of steps: 128 bytes of each row, eight lanes side by side, UU pairs with all
// their loads in flight; they reach the fragments' layout through the wave's
// 2 KB a 16 rows in LDS. (Fragments loaded straight from memory, 16 rows at
// once, run at about one 16-byte request a nanosecond and compute unit: 4096
// tokens of 4096 features at rank 64 took 43 us.) Rows past the tile or the
// rank only reach products that are not used.
//
// fp16 weights below 2^-14 are denormals, whose products the matrix core sums
// with the absolute error of products of 2^-14: V of an adapter that is small
// throughout lost up to 10 of its 24 bits. So A is multiplied by 2^14 (exact)
// until a value of 2 or more is met, from where the sums go on without.
template <int DT, int RT, int TMT, int NW, int U>
__device__ __forceinline__ void shrink_steps(const typename Elem<DT>::T* __restrict__ X, int K,
                                             const typename Elem<DT>::T* __restrict__ A, int R, const LoraTile& tl,
                                             int s0, int s1, int wave, int lane, char* mine, v4f (&acc)[TMT][RT]) {
  typedef Mx<DT> M;
  typedef typename Elem<DT>::T E;
  constexpr int KS = M::KS, EL = M::EL;
  const int c = lane & 15, q = lane >> 4, lrow = lane >> 3, lch = lane & 7;
  const int n_tok = tl.t1 - tl.t0;
  const E* Xt = X + (int64_t)tl.t0 * K;
  const E* Aa = A + (int64_t)tl.adapter * R * K;
#pragma unroll
  for (int i = 0; i < TMT; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = v4f{};

  bool lifted = DT == DT_F16;
  auto lift = [&](v4u (&f)[RT]) {
    if constexpr (DT == DT_F16) {
      if (!lifted) return;
      uint32_t any = 0u;
#pragma unroll
      for (int j = 0; j < RT; ++j) any |= (f[j][0] | f[j][1]) | (f[j][2] | f[j][3]);
      if (__any((any & 0x40004000u) != 0u)) {   // an exponent of 16 or more: |a| >= 2, infinities and NaN
        lifted = false;
#pragma unroll
        for (int i = 0; i < TMT; ++i)
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[i][j] *= 0x1p-14f;
        return;
      }
#pragma unroll
      for (int j = 0; j < RT; ++j) f[j] = __builtin_bit_cast(v4u, __builtin_bit_cast(v8h, f[j]) * (_Float16)0x1p14f);
    }
  };
  auto products = [&](v4u (&fx)[TMT], v4u (&fw)[RT]) {
    lift(fw);
#pragma unroll
    for (int i = 0; i < TMT; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[i][j] = M::mma(fx[i], fw[j], acc[i][j]);
  };
  const int np = max(min(s1, K / KS) - s0, 0) / 2;   // whole pairs
  int p = wave;
  auto pairs = [&](auto uu) {
    constexpr int UU = decltype(uu)::value;
    for (; p + NW * (UU - 1) < np; p += NW * UU) {
      v4u lx[UU][2 * TMT], lw[UU][2 * RT];
#pragma unroll
      for (int u = 0; u < UU; ++u) {
        const int k = (s0 + 2 * (p + NW * u)) * KS + EL * lch;
#pragma unroll
        for (int i = 0; i < 2 * TMT; ++i)
          lx[u][i] = 8 * i + lrow < n_tok ? ld16<DT>(Xt + (int64_t)(8 * i + lrow) * K + k) : v4u{0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 2 * RT; ++j)
          lw[u][j] = 8 * j + lrow < R ? ld16<DT>(Aa + (int64_t)(8 * j + lrow) * K + k) : v4u{0u, 0u, 0u, 0u};
      }
      __builtin_amdgcn_sched_barrier(0);   // else the loads move to their products, a few in flight at a time
#pragma unroll
      for (int u = 0; u < UU; ++u) {
#pragma unroll
        for (int i = 0; i < 2 * TMT; ++i) Rows<8>::at(mine, 8 * i + lrow, lch) = lx[u][i];
#pragma unroll
        for (int j = 0; j < 2 * RT; ++j) Rows<8>::at(mine, 16 * TMT + 8 * j + lrow, lch) = lw[u][j];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v4u fx[TMT], fw[RT];
#pragma unroll
          for (int i = 0; i < TMT; ++i) fx[i] = Rows<8>::at(mine, 16 * i + c, 4 * h + q);
#pragma unroll
          for (int j = 0; j < RT; ++j) fw[j] = Rows<8>::at(mine, 16 * (TMT + j) + c, 4 * h + q);
          products(fx, fw);
        }
      }
    }
  };
  pairs(std::integral_constant<int, U>{});
  if constexpr (U > 4) pairs(std::integral_constant<int, 4>{});
  if constexpr (U > 2) pairs(std::integral_constant<int, 2>{});
  if constexpr (U > 1) pairs(std::integral_constant<int, 1>{});
  // what is left of the range: a step without its pair, and k's end
#pragma unroll 1
  for (int s = s0 + 2 * np + wave; s < s1; s += NW) {
    const int k = s * KS + EL * q, left = K - k;
    v4u fx[TMT], fw[RT];
#pragma unroll
    for (int i = 0; i < TMT; ++i) fx[i] = ld_frag<DT>(Xt + (int64_t)min(16 * i + c, n_tok - 1) * K + k, left);
#pragma unroll
    for (int j = 0; j < RT; ++j) fw[j] = ld_frag<DT>(Aa + (int64_t)min(16 * j + c, R - 1) * K + k, left);
    products(fx, fw);
  }
  if (lifted)   // every wave its own state: the sums meet in common units
#pragma unroll
    for (int i = 0; i < TMT; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[i][j] *= 0x1p-14f;
}

// The columns of a tile's output: out[t, n] = D(base[t, n] + f sum_r V[t, r]
// B[a][n][r]) in groups of GC columns, 128 bytes of a row, of one wave. base, B
// and out cross the wave's LDS between memory's order (lanes side by side on a
// row) and the product's. The product is taken transposed (rows n, columns t),
// so that a lane holds consecutive n of one token: with row m of product u
// standing for n = 8 (m / 4) + 4 u + m % 4 two 16-bit products give a lane 8
// consecutive n, 16 bytes. The contraction runs over both parts of V against
// the same B fragments; at rank 16 both parts fill one step. FULL: whole groups
// and a rank of whole tiles; otherwise B's fragments come straight from memory.
template <int DT, int RT, int TMT, bool FULL>
struct Columns {
  typedef Mx<DT> M;
  typedef typename Elem<DT>::T E;
  static constexpr int KS = M::KS, EL = M::EL, TM = 16 * TMT, RP = 16 * RT;
  static constexpr int GC = 8 * EL;                               // columns of a group: two blocks of KS
  static constexpr int UN = M::F32 ? 1 : 2;                       // products of one block
  static constexpr int NB = M::F32 ? RT : (RT + 1) / 2;           // B fragments of a row
  static constexpr int NS = M::F32 ? RT : RT == 1 ? 1 : RT;       // contraction steps over all parts of V
  static constexpr int LD = M::F32 ? RP + 4 : RP + 8;             // V's row in LDS, in elements
  static constexpr int CB = RP / EL;                              // chunks of a row of B
  static constexpr int LDS = TM * 128 + (FULL ? GC * RP * (int)sizeof(E) : 0);   // a wave's
  struct Group {
    v4u base[2 * TMT], b[FULL ? 2 * RT : 1];
  };
  const E* Ba;
  const E* base;
  E* out;
  int64_t row0;
  int N, R, n_tok, lane, c, q, lrow, lch;
  char* mine;
  v4u vf[TMT][NS];
  float f[TMT];

  __device__ __forceinline__ Columns(const LoraTile& tl, const E* B, const E* base_, E* out_, int N_, int R_, int lane_,
                                     char* lds)
      : Ba(B + (int64_t)max(tl.adapter, 0) * N_ * R_), base(base_), out(out_), row0((int64_t)tl.t0 * N_), N(N_), R(R_),
        n_tok(tl.t1 - tl.t0), lane(lane_), c(lane_ & 15), q(lane_ >> 4), lrow(lane_ >> 3), lch(lane_ & 7), mine(lds) {}
  __device__ static __forceinline__ int r_of(int s, int q) {
    return M::F32 ? 16 * s + 4 * q : RT == 1 ? 8 * (q & 1) : 32 * s + 8 * q;
  }
  __device__ __forceinline__ void load_base(int grp, v4u (&b)[2 * TMT]) const {
    const int n = grp * GC + EL * lch;
#pragma unroll
    for (int i = 0; i < 2 * TMT; ++i) {
      b[i] = v4u{0u, 0u, 0u, 0u};
      if (base && 8 * i + lrow < n_tok) {
        const E* p = base + row0 + (int64_t)(8 * i + lrow) * N + n;
        b[i] = FULL ? ld16<DT>(p) : ld_frag<DT>(p, N - n);
      }
    }
  }
  __device__ __forceinline__ void load(int grp, Group& k) const {
    load_base(grp, k.base);
    if constexpr (FULL) {   // GC rows of B are one piece of memory
      const E* b = Ba + (int64_t)grp * GC * RP + EL * lane;
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i) k.b[i] = ld16<DT>(b + 64 * EL * i);
    }
  }
  __device__ __forceinline__ void store(int grp, int i, v4u y) const {
    const int n = grp * GC + EL * lch;
    if (8 * i + lrow < n_tok) {
      E* p = out + row0 + (int64_t)(8 * i + lrow) * N + n;
      if (FULL) st16<DT>(p, y);
      else st_frag<DT>(p, y, N - n);
    }
  }
  // V's fragments from LDS [part][token][LD]
  __device__ __forceinline__ void take_v(const E* sv) {
#pragma unroll
    for (int i = 0; i < TMT; ++i)
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int part = M::F32 ? 0 : RT == 1 ? q >> 1 : s / NB;
        vf[i][s] = *reinterpret_cast<const v4u*>(sv + (part * TM + 16 * i + c) * LD + r_of(s % NB, q));
      }
  }
  // the group's base and B to LDS, from where `finish` takes them
  __device__ __forceinline__ void stage(const Group& k) const {
#pragma unroll
    for (int i = 0; i < 2 * TMT; ++i) Rows<8>::at(mine, 8 * i + lrow, lch) = k.base[i];
    if constexpr (FULL) {
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i) {
        const int id = 64 * i + lane;
        Rows<CB>::at(mine + TM * 128, id / CB, id % CB) = k.b[i];
      }
    }
  }
  __device__ __forceinline__ void finish(int grp) const {
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      v4u b[UN][NB];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int n = blk * KS + (M::F32 ? c : 8 * (c >> 2) + 4 * u + (c & 3));
#pragma unroll
        for (int s = 0; s < NB; ++s) {
          const int r = r_of(s, q);
          if constexpr (FULL) b[u][s] = Rows<CB>::at(mine + TM * 128, n, r / EL);
          else b[u][s] = ld_frag<DT>(Ba + (int64_t)min(grp * GC + n, N - 1) * R + r, R - r);
        }
      }
#pragma unroll
      for (int i = 0; i < TMT; ++i) {
        v4f acc[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          acc[u] = v4f{};
#pragma unroll
          for (int s = 0; s < NS; ++s) acc[u] = M::mma(b[u][s % NB], vf[i][s], acc[u]);
        }
        v4u& place = Rows<8>::at(mine, 16 * i + c, 4 * blk + q);
        float y[EL];
        frag_f32<DT>(place, y);
#pragma unroll
        for (int j = 0; j < EL; ++j) y[j] = __builtin_fmaf(f[i], acc[j >> 2][j & 3], y[j]);
        place = frag_of<DT>(y);
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * TMT; ++i) store(grp, i, Rows<8>::at(mine, 8 * i + lrow, lch));
  }
  // groups g0, g0 + step .. of a wave, the first PD of them loaded before
  template <int PD>
  __device__ __forceinline__ void prefetch(int g0, int g1, int step, Group (&k)[PD]) const {
#pragma unroll
    for (int i = 0; i < PD; ++i)
      if (g0 + step * i < g1) load(g0 + step * i, k[i]);
  }
  template <int PD>
  __device__ __forceinline__ void all(int g0, int g1, int step, Group (&k)[PD]) const {
    for (int g = g0; g < g1; g += step * PD)
#pragma unroll
      for (int i = 0; i < PD; ++i)
        if (g + step * i < g1) {
          stage(k[i]);
          if (g + step * (i + PD) < g1) load(g + step * (i + PD), k[i]);
          finish(g + step * i);
        }
  }
  // a tile without an adapter
  __device__ __forceinline__ void copy(int g0, int g1, int step) const {
    if (base == out) return;
    for (int g = g0; g < g1; g += step) {
      v4u b[2 * TMT];
      load_base(g, b);
#pragma unroll
      for (int i = 0; i < 2 * TMT; ++i) store(g, i, b[i]);
    }
  }
};

}  // namespace

// P[split][t][r] = sum over the split's part of k of X[t, k] A[a][r][k], Rp =
// 16 RT columns (columns past R hold values that are not read). NW waves share
// a tile; their sums are added in LDS in a fixed order.
template <int DT, int RT, int TMT, int NW>
__global__ __launch_bounds__(NW * 64) void k_lora_shrink(const typename Elem<DT>::T* __restrict__ X, int T, int K,
                                                         const typename Elem<DT>::T* __restrict__ A, int R,
                                                         LoraSegs S, float* __restrict__ P, int splits) {
  int tile, split;
  xcd_order(blockIdx.x, gridDim.x, splits, tile, split);
  constexpr int KS = Mx<DT>::KS, U = TMT + RT <= 2 ? 4 : TMT + RT <= 6 ? 2 : 1;
  extern __shared__ __attribute__((aligned(16))) char sm[];
  v4f(*red)[TMT * RT][64] = reinterpret_cast<v4f(*)[TMT * RT][64]>(sm);
  const LoraTile tl = lora_tile(S, seg_lanes(S, T), tile + 1, T, 16 * TMT);
  if (tl.t1 <= tl.t0 || tl.adapter < 0) return;
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int steps = (K + KS - 1) / KS, pairs = (steps + 1) / 2;
  const int s0 = 2 * (int)((int64_t)pairs * split / splits);
  const int s1 = min(2 * (int)((int64_t)pairs * (split + 1) / splits), steps);
  v4f acc[TMT][RT];
  shrink_steps<DT, RT, TMT, NW, U>(X, K, A, R, tl, s0, s1, wave, lane, sm + wave * (TMT + RT) * 2048, acc);
#pragma unroll
  for (int half = NW / 2; half >= 1; half >>= 1) {
    __syncthreads();
    if (wave >= half && wave < 2 * half)
#pragma unroll
      for (int i = 0; i < TMT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) red[wave - half][i * RT + j][lane] = acc[i][j];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int i = 0; i < TMT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[i][j] += red[wave][i * RT + j][lane];
  }
  if (wave == 0) {
    float* p = P + (int64_t)split * T * (16 * RT);
#pragma unroll
    for (int i = 0; i < TMT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = tl.t0 + 16 * i + 4 * q + e;
        if (t < tl.t1)
#pragma unroll
          for (int j = 0; j < RT; ++j) p[(int64_t)t * (16 * RT) + 16 * j + c] = acc[i][j][e];
      }
  }
}

// The columns of a tile from V = the sum of the splits of P (also written to
// `V` by the first column slice). The first groups of base and B are loaded
// before V.
template <int DT, int RT, int TMT, bool FULL>
__global__ __launch_bounds__(256) void k_lora_expand(const float* __restrict__ P, int splits, int T, int N,
                                                     const typename Elem<DT>::T* __restrict__ B, int R,
                                                     const float* __restrict__ scaling, LoraSegs S,
                                                     const typename Elem<DT>::T* base, typename Elem<DT>::T* out,
                                                     float* __restrict__ V, int groups_per_wave, int slices) {
  int tile, slice;
  xcd_order(blockIdx.x, gridDim.x, slices, tile, slice);
  typedef Columns<DT, RT, TMT, FULL> C;
  typedef typename Elem<DT>::T E;
  constexpr int TM = C::TM, RP = C::RP, LD = C::LD;
  constexpr bool F32 = DT == DT_F32;
  constexpr int PD = TMT == 1 ? (RT <= 2 ? 3 : RT == 4 ? 2 : 1) : 1;
  extern __shared__ __attribute__((aligned(16))) char sm[];
  E* sv = reinterpret_cast<E*>(sm);                                    // [part][TM][LD], before the waves' stages
  float* sunit = reinterpret_cast<float*>(sv + Mx<DT>::NC * TM * LD);   // [TM]
  const LoraTile tl = lora_tile(S, seg_lanes(S, T), tile + 1, T, TM);
  const int n_tok = tl.t1 - tl.t0;
  if (n_tok <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int first = slice * 4 * groups_per_wave;
  const int g0 = first + wave, g1 = min(first + 4 * groups_per_wave, (N + C::GC - 1) / C::GC);
  C col(tl, B, base, out, N, R, lane, sm + wave * C::LDS);

  if (tl.adapter < 0) {
    if (V && slice == 0)
      for (int64_t e = (int64_t)tl.t0 * R + tid; e < (int64_t)tl.t1 * R; e += 256) V[e] = 0.0f;
    col.copy(g0, g1, 4);
    return;
  }
  const float scale = scaling[tl.adapter];
  typename C::Group k[PD];
  col.prefetch(g0, g1, 4, k);

  // V's parts into LDS: four consecutive r a thread, the threads of a token side by side
  for (int e = tid; e < TM * RP / 4; e += 256) {
    const int t = e / (RP / 4), r = e % (RP / 4) * 4;
    v4f v = {};
    if (t < n_tok) {
      const float* p = P + (int64_t)(tl.t0 + t) * RP + r;
      v4f part[MAX_SPLITS];
#pragma unroll
      for (int s = 0; s < MAX_SPLITS; ++s)
        part[s] = s < splits ? *reinterpret_cast<const v4f*>(p + (int64_t)s * T * RP) : v4f{};
#pragma unroll
      for (int s = 0; s < MAX_SPLITS; ++s) v += part[s];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (r + j >= R) v[j] = 0.0f;
      else if (V && slice == 0 && t < n_tok) V[(int64_t)(tl.t0 + t) * R + r + j] = v[j];
    }
    E* o = sv + t * LD + r;
    if constexpr (F32) {
      *reinterpret_cast<v4f*>(o) = v;
    } else {
      float unit = 1.0f;
      if constexpr (DT == DT_F16) {
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, __builtin_isfinite(v[j]) ? __builtin_fabsf(v[j]) : 0.0f);
#pragma unroll
        for (int x = 1; x < RP / 4; x <<= 1) top = fmaxf(top, __shfl_xor(top, x, 64));
        unit = unit_for(top);
        if (r == 0) sunit[t] = inv_pow2(unit);
      }
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = split2<DT>(v[j], unit);
      *reinterpret_cast<v2u*>(o) = v2u{(h[0] & 0xffffu) | (h[1] << 16), (h[2] & 0xffffu) | (h[3] << 16)};
      *reinterpret_cast<v2u*>(o + TM * LD) =
          v2u{(h[0] >> 16) | (h[1] & 0xffff0000u), (h[2] >> 16) | (h[3] & 0xffff0000u)};
    }
  }
  __syncthreads();
  col.take_v(sv);
#pragma unroll
  for (int i = 0; i < TMT; ++i) {
    col.f[i] = scale;
    if constexpr (DT == DT_F16) col.f[i] *= sunit[16 * i + (lane & 15)];
  }
  __syncthreads();
  col.all(g0, g1, 4, k);
}

// Both in one launch, for tiles of 16 tokens: every workgroup computes the whole
// V of its tile, which the workgroups of one tile repeat (X and A come from the
// caches), and its slice of the columns. The first groups of base and B are
// loaded before V's contraction.
template <int DT, int RT, bool FULL>
__global__ __launch_bounds__(512, 1) void k_lora_short(const typename Elem<DT>::T* __restrict__ X, int T, int K,
                                                       const typename Elem<DT>::T* __restrict__ A, int R,
                                                       const float* __restrict__ scaling, LoraSegs S,
                                                       const typename Elem<DT>::T* __restrict__ B, int N,
                                                       const typename Elem<DT>::T* base, typename Elem<DT>::T* out,
                                                       float* __restrict__ V, int groups_per_wave) {
  typedef Columns<DT, RT, 1, FULL> C;
  typedef typename Elem<DT>::T E;
  constexpr int LD = C::LD, PD = RT <= 2 ? 3 : RT == 4 ? 2 : 1;
  constexpr int STAGE = (1 + RT) * 2048 > C::LDS ? (1 + RT) * 2048 : C::LDS;
  extern __shared__ __attribute__((aligned(16))) char sm[];
  v4f(*red)[RT][64] = reinterpret_cast<v4f(*)[RT][64]>(sm);              // over the waves' stages, between their uses
  E* sv = reinterpret_cast<E*>(sm + 8 * STAGE);                          // [part][16][LD]
  float* tops = reinterpret_cast<float*>(sv + Mx<DT>::NC * 16 * LD);     // fp16: [RT][16], a wave's largest of each token
  const LoraTile tl = lora_tile(S, seg_lanes(S, T), blockIdx.x + 1, T, 16);
  const int n_tok = tl.t1 - tl.t0;
  if (n_tok <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  char* mine = sm + wave * STAGE;
  const int first = blockIdx.y * 8 * groups_per_wave;
  const int g0 = first + wave, g1 = min(first + 8 * groups_per_wave, (N + C::GC - 1) / C::GC);
  C col(tl, B, base, out, N, R, lane, mine);
  if (tl.adapter < 0) {
    if (V && blockIdx.y == 0)
      for (int64_t e = (int64_t)tl.t0 * R + tid; e < (int64_t)tl.t1 * R; e += 512) V[e] = 0.0f;
    col.copy(g0, g1, 8);
    return;
  }
  const float scale = scaling[tl.adapter];
  typename C::Group k[PD];
  col.prefetch(g0, g1, 8, k);
  {
    v4f acc[1][RT];
    shrink_steps<DT, RT, 1, 8, RT == 1 ? 8 : RT == 2 ? 4 : RT == 4 ? 2 : 1>(X, K, A, R, tl, 0, (K + C::KS - 1) / C::KS,
                                                                            wave, lane, mine, acc);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < RT; ++j) red[wave][j][lane] = acc[0][j];
  }
  __syncthreads();
  // thread: four tokens of one r
  v4f v = {};
  const int c = lane & 15, q = lane >> 4, r = 16 * wave + c;
  if (wave < RT) {
#pragma unroll
    for (int w = 0; w < 8; ++w) v += red[w][wave][lane];
    if (r >= R) v = v4f{};
    else if (V && blockIdx.y == 0)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * q + e < n_tok) V[(int64_t)(tl.t0 + 4 * q + e) * R + r] = v[e];
  }
  // fp16: the power of two of token t
  auto unit_of = [&](int t) {
    float top = 0.0f;
#pragma unroll
    for (int w = 0; w < RT; ++w) top = fmaxf(top, tops[16 * w + t]);
    return unit_for(top);
  };
  if constexpr (DT == DT_F16) {
    if (wave < RT)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float top = lanes_max<16>(__builtin_isfinite(v[e]) ? __builtin_fabsf(v[e]) : 0.0f);
        if (c == 0) tops[16 * wave + 4 * q + e] = top;
      }
    __syncthreads();
  }
  if (wave < RT) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      E* o = sv + (4 * q + e) * LD + r;
      if constexpr (DT == DT_F32) {
        *o = v[e];
      } else {
        const uint32_t h = split2<DT>(v[e], DT == DT_F16 ? unit_of(4 * q + e) : 1.0f);
        o[0] = __builtin_bit_cast(E, (uint16_t)(h & 0xffffu));
        o[16 * LD] = __builtin_bit_cast(E, (uint16_t)(h >> 16));
      }
    }
  }
  __syncthreads();
  col.take_v(sv);
  col.f[0] = scale;
  if constexpr (DT == DT_F16) col.f[0] *= inv_pow2(unit_of(c));
  col.all(g0, g1, 8, k);
}

namespace {

// 64-token tiles read B once for 64 tokens; they need segments that fill them.
bool long_tiles(int T, int n_seg) { return T >= 1024 && T / 48 >= n_seg; }

// Splits of the contraction: as many workgroups as run together (one a compute
// unit with 64 tokens), each with two pairs of steps or more for each of its
// waves. 4096 tokens of 4096 features at rank 64: tiles of 64 tokens in three
// splits take 15 us, of 32 in two 22 us, of 16 whole 26 us, as A is read once a
// tile (from L2 at best: 512 KB against 128 KB of X for 16 tokens).
int shrink_splits(int T, int K, int n_seg) {
  const LoraSegs S = {nullptr, nullptr, n_seg, 0};
  const bool big = long_tiles(T, n_seg);
  const int tiles = lora_tiles(T, S, big ? 64 : 16);
  const int most = K / 512 < MAX_SPLITS ? K / 512 : MAX_SPLITS;
  const int want = (big ? 256 : 384) / (tiles > 0 ? tiles : 1);
  return want < 1 || most < 1 ? 1 : want < most ? want : most;
}

// One launch for up to 32 tiles with an A of up to 81920 values (it needs no
// workspace). Every workgroup reads A[a] whole, at the 25 GB/s or so that one
// compute unit gets from memory, but a second launch and a workspace cost the
// host 5 us. 16-bit, on the GPU, one launch against two: one token, 4096 -> 4096
// at rank 16, 6.3 and 7.2 us; 64 of 16 adapters, 4096 -> 11008, 7.5 and 8.4; 512
// of one, 1024 -> 11008 at rank 64, 10.9 and 13.5; at the bound, 5120 at rank
// 16, 7.2 and 7.2 for one token, 9.0 and 8.3 for the 64. fp32 reads twice the
// bytes: 10.2 and 7.4, 16 and 10, 23 and 24; there only the host's side gains at
// the bound, and the workspace's size does not depend on the type. With 64
// tiles and 11008 columns one launch took 22 us against 6 + 10.
bool one_launch(int T, int K, int R, int n_seg) {
  const LoraSegs S = {nullptr, nullptr, n_seg, 0};
  return lora_tiles(T, S, 16) <= 32 && (int64_t)K * R <= 81920;
}

// A launch with `lds` bytes of dynamic LDS; over 64 KB the kernel's limit is raised first.
template <typename... P, typename... Q>
hipError_t launch(void (*kern)(P...), std::atomic<uint64_t>& done, dim3 grid, int threads, int lds, hipStream_t st,
                  Q... args) {
  if (lds > 64 * 1024) {
    const hipError_t e = lds_limit_once((const void*)kern, lds, done);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, grid, dim3(threads), lds, st, args...);
  return hipGetLastError();
}

template <int DT, int RT, bool FULL>
hipError_t run_short(const void* Xv, int T, int K, const void* Av, const void* Bv, const float* scaling, int R, int N,
                     const LoraSegs& S, const void* base, void* out, float* V, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  typedef Columns<DT, RT, 1, FULL> C;
  constexpr int stage = (1 + RT) * 2048 > C::LDS ? (1 + RT) * 2048 : C::LDS;
  constexpr int lds = 8 * stage + Mx<DT>::NC * 16 * C::LD * (int)sizeof(E) + RT * 16 * 4;
  static std::atomic<uint64_t> done{0};
  const int tiles = lora_tiles(T, S, 16), groups = (N + C::GC - 1) / C::GC;
  // at most 256 workgroups, one a compute unit: a second round would compute V again
  const int most = 256 / tiles, gpw = groups > 0 ? (groups + 8 * most - 1) / (8 * most) : 1;
  const int slices = groups > 0 ? (groups + 8 * gpw - 1) / (8 * gpw) : V ? 1 : 0;
  if (slices == 0) return hipSuccess;
  return launch(k_lora_short<DT, RT, FULL>, done, dim3(tiles, slices), 512, lds, st, static_cast<const E*>(Xv), T, K,
                static_cast<const E*>(Av), R, scaling, S, static_cast<const E*>(Bv), N, static_cast<const E*>(base),
                static_cast<E*>(out), V, gpw);
}

template <int DT, int RT, int TMT, bool FULL>
hipError_t run(const void* Xv, int T, int K, const void* Av, const void* Bv, const float* scaling, int R, int N,
               const LoraSegs& S, const void* base, void* out, float* V, float* ws, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  typedef Columns<DT, RT, TMT, FULL> C;
  constexpr int NW = RT < 8 ? 8 : 4, ST = TMT == 1 ? 1 : 4;   // shrink: its waves and 16-token parts
  const int splits = shrink_splits(T, K, S.n_seg);
  if (S.n_adapters > 0) {
    constexpr int stage = NW * (ST + RT) * 2048, red = NW / 2 * ST * RT * 1024;
    static std::atomic<uint64_t> done{0};
    const hipError_t e = launch(k_lora_shrink<DT, RT, ST, NW>, done, dim3((unsigned)lora_tiles(T, S, 16 * ST) * splits), NW * 64,
                                stage > red ? stage : red, st, static_cast<const E*>(Xv), T, K,
                                static_cast<const E*>(Av), R, S, ws, splits);
    if (e != hipSuccess) return e;
  }
  const int tiles = lora_tiles(T, S, 16 * TMT), groups = (N + C::GC - 1) / C::GC;
  // workgroups that are resident together: two a compute unit in long batches, four with 16 tokens
  constexpr int want = TMT == 1 ? 1024 : 512;
  int64_t gpw = ((int64_t)tiles * groups + 4 * want - 1) / (4 * want);
  gpw = gpw < 1 ? 1 : gpw;
  const int slices = groups > 0 ? (int)((groups + 4 * gpw - 1) / (4 * gpw)) : V ? 1 : 0;
  if (slices == 0) return hipSuccess;
  constexpr int small = Mx<DT>::NC * C::TM * C::LD * (int)sizeof(E) + C::TM * 4;
  constexpr int lds = 4 * C::LDS > small ? 4 * C::LDS : small;
  static std::atomic<uint64_t> done{0};
  return launch(k_lora_expand<DT, RT, TMT, FULL>, done, dim3((unsigned)tiles * slices), 256, lds, st, (const float*)ws, splits, T,
                N, static_cast<const E*>(Bv), R, scaling, S, static_cast<const E*>(base), static_cast<E*>(out), V,
                (int)gpw, slices);
}

template <int DT, int RT, bool FULL>
hipError_t run_rank(const void* X, int T, int K, const void* A, const void* B, const float* scaling, int R, int N,
              const LoraSegs& S, const void* base, void* out, float* V, float* ws, hipStream_t st) {
  if (one_launch(T, K, R, S.n_seg))
    return run_short<DT, RT, FULL>(X, T, K, A, B, scaling, R, N, S, base, out, V, st);
  // 32 tokens at rank 128: B's part in LDS leaves room for two workgroups a compute unit
  if (long_tiles(T, S.n_seg)) return run<DT, RT, RT == 8 ? 2 : 4, FULL>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
  return run<DT, RT, 1, FULL>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
}

template <int DT, int RT>
hipError_t run_size(const void* X, int T, int K, const void* A, const void* B, const float* scaling, int R, int N,
                    const LoraSegs& S, const void* base, void* out, float* V, float* ws, hipStream_t st) {
  if (N % (8 * Mx<DT>::EL) == 0 && R == 16 * RT)
    return run_rank<DT, RT, true>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
  return run_rank<DT, RT, false>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
}

template <int DT>
hipError_t forward_t(const void* X, int T, int K, const void* A, const void* B, const float* scaling, int R, int N,
                     const LoraSegs& S, const void* base, void* out, float* V, float* ws, hipStream_t st) {
  switch (rank_tiles(R)) {
    case 1: return run_size<DT, 1>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
    case 2: return run_size<DT, 2>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
    case 4: return run_size<DT, 4>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
    default: return run_size<DT, 8>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
  }
}

}  // namespace

size_t lora_forward_floats(int T, int K, int N, int R, int n_seg) {
  if (one_launch(T, K, R, n_seg)) return 0;
  return (size_t)shrink_splits(T, K, n_seg) * T * 16 * rank_tiles(R);
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

}  // namespace i8l
