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
// contraction steps s0 .. s1 - 1 that fall to `wave` of NW: pairs of steps in
// turn, 128 bytes of each row. Fragments come straight from memory, as both
// operands lie along k. Rows past the tile or the rank repeat the last one:
// they only reach products that are not used.
//
// fp16 weights below 2^-14 are denormals, whose products the matrix core sums
// with the absolute error of products of 2^-14: V of an adapter that is small
// throughout lost up to 10 of its 24 bits. So A is multiplied by 2^14 (exact)
// until a value of 2 or more is met, from where the sums go on without.
template <int DT, int RT, int TMT, int NW, int U, bool FULL>
__device__ __forceinline__ void shrink_steps(const typename Elem<DT>::T* __restrict__ X, int K,
                                             const typename Elem<DT>::T* __restrict__ A, int R, const LoraTile& tl,
                                             int s0, int s1, int wave, int lane, v4f (&acc)[TMT][RT]) {
  typedef Mx<DT> M;
  typedef typename Elem<DT>::T E;
  constexpr int KS = M::KS, EL = M::EL;
  const int c = lane & 15, q = lane >> 4;
  const E* x[TMT];
  const E* w[RT];
#pragma unroll
  for (int i = 0; i < TMT; ++i) x[i] = X + (int64_t)min(tl.t0 + 16 * i + c, tl.t1 - 1) * K + EL * q;
#pragma unroll
  for (int j = 0; j < RT; ++j) w[j] = A + ((int64_t)tl.adapter * R + min(16 * j + c, R - 1)) * K + EL * q;
#pragma unroll
  for (int i = 0; i < TMT; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = v4f{};

  bool lifted = DT == DT_F16;
  auto lift = [&](auto& f, int count) {
    if constexpr (DT == DT_F16) {
      if (!lifted) return;
      uint32_t any = 0u;
      for (int u = 0; u < count; ++u)
#pragma unroll
        for (int j = 0; j < RT; ++j) any |= (f[u][j][0] | f[u][j][1]) | (f[u][j][2] | f[u][j][3]);
      if (__any((any & 0x40004000u) != 0u)) {   // an exponent of 16 or more: |a| >= 2, infinities and NaN
        lifted = false;
#pragma unroll
        for (int i = 0; i < TMT; ++i)
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[i][j] *= 0x1p-14f;
        return;
      }
      for (int u = 0; u < count; ++u)
#pragma unroll
        for (int j = 0; j < RT; ++j) f[u][j] = __builtin_bit_cast(v4u, __builtin_bit_cast(v8h, f[u][j]) * (_Float16)0x1p14f);
    }
  };
  // Whole pairs of steps, wave after wave, UU of a wave with all their loads in
  // flight. Tiles begin at different pairs: with all of them at k = 0 rows of a
  // power-of-two width would meet in a few of the memory's channels.
  const int whole = FULL ? s1 : min(s1, K / KS), np = max(whole - s0, 0) / 2;
  const int turn = np > 0 ? (int)((unsigned)(tl.t0 / 16 * 5) % (unsigned)np) : 0;
  int p = wave;
  auto pairs = [&](auto uu) {
    constexpr int UU = decltype(uu)::value;
    for (; p + NW * (UU - 1) < np; p += NW * UU) {
      v4u fx[2 * UU][TMT], fw[2 * UU][RT];
#pragma unroll
      for (int u = 0; u < UU; ++u) {
        int at = p + NW * u + turn;
        if (at >= np) at -= np;
        const int k = (s0 + 2 * at) * KS;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < TMT; ++i) fx[2 * u + h][i] = ld16<DT>(x[i] + k + h * KS);
#pragma unroll
          for (int j = 0; j < RT; ++j) fw[2 * u + h][j] = ld16<DT>(w[j] + k + h * KS);
        }
      }
      __builtin_amdgcn_sched_barrier(0);   // else the loads move to their products, a few in flight at a time
      lift(fw, 2 * UU);
#pragma unroll
      for (int u = 0; u < 2 * UU; ++u)
#pragma unroll
        for (int i = 0; i < TMT; ++i)
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[i][j] = M::mma(fx[u][i], fw[u][j], acc[i][j]);
    }
  };
  pairs(std::integral_constant<int, U>{});
  if constexpr (U > 4) pairs(std::integral_constant<int, 4>{});
  if constexpr (U > 2) pairs(std::integral_constant<int, 2>{});
  if constexpr (U > 1) pairs(std::integral_constant<int, 1>{});
  // what is left of the range: a step without its pair, and k's end
#pragma unroll 1
  for (int s = s0 + 2 * np + wave; s < s1; s += NW) {
    const int left = K - s * KS - EL * q;
    v4u fx[TMT], fw[1][RT];
#pragma unroll
    for (int i = 0; i < TMT; ++i) fx[i] = FULL ? ld16<DT>(x[i] + s * KS) : ld_frag<DT>(x[i] + s * KS, left);
#pragma unroll
    for (int j = 0; j < RT; ++j) fw[0][j] = FULL ? ld16<DT>(w[j] + s * KS) : ld_frag<DT>(w[j] + s * KS, left);
    lift(fw, 1);
#pragma unroll
    for (int i = 0; i < TMT; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[i][j] = M::mma(fx[i], fw[0][j], acc[i][j]);
  }
  if (lifted)   // every wave its own state: the sums meet in common units
#pragma unroll
    for (int i = 0; i < TMT; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[i][j] *= 0x1p-14f;
}

// The columns of a tile's output: out[t, n] = D(base[t, n] + f sum_r V[t, r]
// B[a][n][r]) in blocks of KS columns. The product is taken transposed (rows n,
// columns t), so that a lane holds consecutive n of one token: with row m of
// product u standing for n = 8 (m / 4) + 4 u + m % 4 two 16-bit products give a
// lane 8 consecutive n, 16 bytes of base and out. The contraction runs over
// both parts of V against the same B fragments; at rank 16 both parts fill one
// step.
template <int DT, int RT, int TMT, bool FULL>
struct Columns {
  typedef Mx<DT> M;
  typedef typename Elem<DT>::T E;
  static constexpr int KS = M::KS, EL = M::EL, TM = 16 * TMT, RP = 16 * RT;
  static constexpr int UN = M::F32 ? 1 : 2;                       // products of one block
  static constexpr int NB = M::F32 ? RT : (RT + 1) / 2;           // B fragments of a row
  static constexpr int NS = M::F32 ? RT : RT == 1 ? 1 : RT;       // contraction steps over all parts of V
  static constexpr int LD = M::F32 ? RP + 4 : RP + 8;             // V's row in LDS, in elements
  struct Block {
    v4u b[UN][NB], base[TMT];
  };
  const E* Ba;
  const E* base;
  E* out;
  int64_t row[TMT];
  int N, R, n_tok, c, q;
  v4u vf[TMT][NS];
  float f[TMT];

  __device__ __forceinline__ Columns(const LoraTile& tl, const E* B, const E* base_, E* out_, int N_, int R_, int lane)
      : Ba(B + (int64_t)max(tl.adapter, 0) * N_ * R_), base(base_), out(out_), N(N_), R(R_), n_tok(tl.t1 - tl.t0),
        c(lane & 15), q(lane >> 4) {
#pragma unroll
    for (int i = 0; i < TMT; ++i) row[i] = (int64_t)min(tl.t0 + 16 * i + c, tl.t1 - 1) * N;
  }
  __device__ static __forceinline__ int r_of(int s, int q) {
    return M::F32 ? 16 * s + 4 * q : RT == 1 ? 8 * (q & 1) : 32 * s + 8 * q;
  }
  __device__ __forceinline__ void load_base(int blk, Block& k) const {
    const int n = blk * KS + EL * q;
    if (base == nullptr) {
#pragma unroll
      for (int i = 0; i < TMT; ++i) k.base[i] = v4u{0u, 0u, 0u, 0u};
    } else if (FULL || (blk + 1) * KS <= N) {
#pragma unroll
      for (int i = 0; i < TMT; ++i) k.base[i] = ld16<DT>(base + row[i] + n);
    } else {
#pragma unroll
      for (int i = 0; i < TMT; ++i) k.base[i] = ld_frag<DT>(base + row[i] + n, N - n);
    }
  }
  __device__ __forceinline__ void load(int blk, Block& k) const {
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int n = blk * KS + (M::F32 ? c : 8 * (c >> 2) + 4 * u + (c & 3));
      const E* b = Ba + (int64_t)(FULL ? n : min(n, N - 1)) * R;
#pragma unroll
      for (int s = 0; s < NB; ++s) {
        const int r = r_of(s, q);
        if (FULL || R == RP) k.b[u][s] = ld16<DT>(b + r);
        else k.b[u][s] = ld_frag<DT>(b + r, R - r);
      }
    }
    load_base(blk, k);
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
  __device__ __forceinline__ void store(int blk, int i, v4u y) const {
    const int n = blk * KS + EL * q;
    if (16 * i + c < n_tok) {
      if (FULL || (blk + 1) * KS <= N) st16<DT>(out + row[i] + n, y);
      else st_frag<DT>(out + row[i] + n, y, N - n);
    }
  }
  __device__ __forceinline__ void finish(int blk, const Block& k) const {
#pragma unroll
    for (int i = 0; i < TMT; ++i) {
      v4f acc[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        acc[u] = v4f{};
#pragma unroll
        for (int s = 0; s < NS; ++s) acc[u] = M::mma(k.b[u][s % NB], vf[i][s], acc[u]);
      }
      float y[EL];
      frag_f32<DT>(k.base[i], y);
#pragma unroll
      for (int j = 0; j < EL; ++j) y[j] = __builtin_fmaf(f[i], acc[j >> 2][j & 3], y[j]);
      store(blk, i, frag_of<DT>(y));
    }
  }
  // a tile without an adapter
  __device__ __forceinline__ void copy(int b0, int b1, int step) const {
    if (base == out) return;
    for (int b = b0; b < b1; b += step) {
      Block k;
      load_base(b, k);
#pragma unroll
      for (int i = 0; i < TMT; ++i) store(b, i, k.base[i]);
    }
  }
};

}  // namespace

// P[split][t][r] = sum over the split's part of k of X[t, k] A[a][r][k], Rp =
// 16 RT columns (columns past R hold values that are not read). NW waves share
// a tile; their sums are added in LDS in a fixed order.
template <int DT, int RT, int TMT, int NW, bool FULL>
__global__ __launch_bounds__(NW * 64) void k_lora_shrink(const typename Elem<DT>::T* __restrict__ X, int T, int K,
                                                         const typename Elem<DT>::T* __restrict__ A, int R,
                                                         LoraSegs S, float* __restrict__ P) {
  constexpr int KS = Mx<DT>::KS;
  __shared__ v4f red[NW / 2][TMT * RT][64];
  const LoraTile tl = lora_tile(S, seg_lanes(S, T), blockIdx.x + 1, T, 16 * TMT);
  if (tl.t1 <= tl.t0 || tl.adapter < 0) return;
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int steps = (K + KS - 1) / KS;
  const int s0 = (int)((int64_t)steps * blockIdx.y / gridDim.y), s1 = (int)((int64_t)steps * (blockIdx.y + 1) / gridDim.y);
  v4f acc[TMT][RT];
  shrink_steps<DT, RT, TMT, NW, TMT + RT <= 2 ? 4 : TMT + RT <= 5 ? 2 : 1, FULL>(X, K, A, R, tl, s0, s1, wave, lane, acc);
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
    float* p = P + (int64_t)blockIdx.y * T * (16 * RT);
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
// `V` by the first column slice).
template <int DT, int RT, int TMT, bool FULL>
__global__ __launch_bounds__(256) void k_lora_expand(const float* __restrict__ P, int splits, int T, int N,
                                                     const typename Elem<DT>::T* __restrict__ B, int R,
                                                     const float* __restrict__ scaling, LoraSegs S,
                                                     const typename Elem<DT>::T* base, typename Elem<DT>::T* out,
                                                     float* __restrict__ V, int blocks_per_wave) {
  typedef Columns<DT, RT, TMT, FULL> C;
  typedef typename Elem<DT>::T E;
  constexpr int TM = C::TM, RP = C::RP, LD = C::LD;
  constexpr bool F32 = DT == DT_F32;
  __shared__ __attribute__((aligned(16))) E sv[Mx<DT>::NC][TM][LD];
  __shared__ float sunit[TM];
  const LoraTile tl = lora_tile(S, seg_lanes(S, T), blockIdx.x + 1, T, TM);
  const int n_tok = tl.t1 - tl.t0;
  if (n_tok <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int blk0 = blockIdx.y * 4 * blocks_per_wave + wave, n_blk = (N + C::KS - 1) / C::KS;
  const int blk_end = min(blk0 - wave + 4 * blocks_per_wave, n_blk);
  C col(tl, B, base, out, N, R, lane);

  if (tl.adapter < 0) {
    if (V && blockIdx.y == 0)
      for (int64_t e = (int64_t)tl.t0 * R + tid; e < (int64_t)tl.t1 * R; e += 256) V[e] = 0.0f;
    col.copy(blk0, blk_end, 4);
    return;
  }

  constexpr int PD = TMT == 1 ? (RT <= 2 ? 6 : RT == 4 ? 3 : 2) : RT == 8 ? 1 : 2;   // blocks in flight
  const float scale = scaling[tl.adapter];
  typename C::Block k[PD];
#pragma unroll
  for (int i = 0; i < PD; ++i)
    if (blk0 + 4 * i < blk_end) col.load(blk0 + 4 * i, k[i]);

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
      else if (V && blockIdx.y == 0 && t < n_tok) V[(int64_t)(tl.t0 + t) * R + r + j] = v[j];
    }
    if constexpr (F32) {
      *reinterpret_cast<v4f*>(&sv[0][t][r]) = v;
    } else {
      float unit = 1.0f;
      if constexpr (DT == DT_F16) {
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, __builtin_isfinite(v[j]) ? __builtin_fabsf(v[j]) : 0.0f);
#pragma unroll
        for (int o = 1; o < RP / 4; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
        unit = unit_for(top);
        if (r == 0) sunit[t] = inv_pow2(unit);
      }
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = split2<DT>(v[j], unit);
      *reinterpret_cast<v2u*>(&sv[0][t][r]) =
          v2u{(h[0] & 0xffffu) | (h[1] << 16), (h[2] & 0xffffu) | (h[3] << 16)};
      *reinterpret_cast<v2u*>(&sv[Mx<DT>::NC - 1][t][r]) =
          v2u{(h[0] >> 16) | (h[1] & 0xffff0000u), (h[2] >> 16) | (h[3] & 0xffff0000u)};
    }
  }
  __syncthreads();
  if (blk0 >= blk_end) return;
  col.take_v(&sv[0][0][0]);
#pragma unroll
  for (int i = 0; i < TMT; ++i) {
    col.f[i] = scale;
    if constexpr (DT == DT_F16) col.f[i] *= sunit[16 * i + (lane & 15)];
  }
  for (int b = blk0; b < blk_end; b += 4 * PD)
#pragma unroll
    for (int i = 0; i < PD; ++i)
      if (b + 4 * i < blk_end) {
        col.finish(b + 4 * i, k[i]);
        if (b + 4 * (i + PD) < blk_end) col.load(b + 4 * (i + PD), k[i]);
      }
}

// Both in one launch, for tiles of 16 tokens: every workgroup computes the whole
// V of its tile, which the workgroups of one tile repeat (X and A come from the
// caches), and its slice of the columns. The first block of base and B is
// loaded before V's contraction. One request of one token, 4096 x 4096 at rank
// 16: 4.8 us against 3.9 + 4.4 us and a second launch.
template <int DT, int RT, bool FULL>
__global__ __launch_bounds__(512, 1) void k_lora_short(const typename Elem<DT>::T* __restrict__ X, int T, int K,
                                                    const typename Elem<DT>::T* __restrict__ A, int R,
                                                    const float* __restrict__ scaling, LoraSegs S,
                                                    const typename Elem<DT>::T* __restrict__ B, int N,
                                                    const typename Elem<DT>::T* base, typename Elem<DT>::T* out,
                                                    float* __restrict__ V, int blocks_per_wave) {
  typedef Columns<DT, RT, 1, FULL> C;
  typedef typename Elem<DT>::T E;
  constexpr int LD = C::LD;
  __shared__ v4f red[8][RT][64];
  __shared__ __attribute__((aligned(16))) E sv[Mx<DT>::NC][16][LD];
  __shared__ float top8[8];
  const LoraTile tl = lora_tile(S, seg_lanes(S, T), blockIdx.x + 1, T, 16);
  const int n_tok = tl.t1 - tl.t0;
  if (n_tok <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int first = blockIdx.y * 8 * blocks_per_wave, n_blk = (N + C::KS - 1) / C::KS;
  const int blk0 = first + wave, blk_end = min(first + 8 * blocks_per_wave, n_blk);
  C col(tl, B, base, out, N, R, lane);
  if (tl.adapter < 0) {
    if (V && blockIdx.y == 0)
      for (int64_t e = (int64_t)tl.t0 * R + tid; e < (int64_t)tl.t1 * R; e += 512) V[e] = 0.0f;
    col.copy(blk0, blk_end, 8);
    return;
  }
  constexpr int PD = RT <= 2 ? 6 : RT == 4 ? 3 : 2;   // blocks in flight
  const float scale = scaling[tl.adapter];
  typename C::Block k[PD];
#pragma unroll
  for (int i = 0; i < PD; ++i)
    if (blk0 + 8 * i < blk_end) col.load(blk0 + 8 * i, k[i]);
  {
    v4f acc[1][RT];
    shrink_steps<DT, RT, 1, 8, RT == 1 ? 8 : RT == 2 ? 4 : RT == 4 ? 2 : 1, FULL>(X, K, A, R, tl, 0, (K + C::KS - 1) / C::KS, wave, lane, acc);
#pragma unroll
    for (int j = 0; j < RT; ++j) red[wave][j][lane] = acc[0][j];
  }
  __syncthreads();
  // thread: four tokens of one r
  v4f v = {};
  const int c = lane & 15, q = lane >> 4, r = 16 * wave + c;
  float unit = 1.0f;
  if (wave < RT) {
#pragma unroll
    for (int w = 0; w < 8; ++w) v += red[w][wave][lane];
    if (r >= R) v = v4f{};
    else if (V && blockIdx.y == 0)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * q + e < n_tok) V[(int64_t)(tl.t0 + 4 * q + e) * R + r] = v[e];
  }
  if constexpr (DT == DT_F16) {
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e)   // rows past the tile repeat its last
      top = fmaxf(top, __builtin_isfinite(v[e]) ? __builtin_fabsf(v[e]) : 0.0f);
    top = wave_max(top);
    if (lane == 0) top8[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) top = fmaxf(top, top8[w]);
    unit = unit_for(top);
  }
  if (wave < RT) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (DT == DT_F32) {
        sv[0][4 * q + e][r] = v[e];
      } else {
        const uint32_t h = split2<DT>(v[e], unit);
        sv[0][4 * q + e][r] = __builtin_bit_cast(E, (uint16_t)(h & 0xffffu));
        sv[Mx<DT>::NC - 1][4 * q + e][r] = __builtin_bit_cast(E, (uint16_t)(h >> 16));
      }
    }
  }
  __syncthreads();
  if (blk0 >= blk_end) return;
  col.take_v(&sv[0][0][0]);
  col.f[0] = scale;
  if constexpr (DT == DT_F16) col.f[0] *= inv_pow2(unit);
  for (int b = blk0; b < blk_end; b += 8 * PD)
#pragma unroll
    for (int i = 0; i < PD; ++i)
      if (b + 8 * i < blk_end) {
        col.finish(b + 8 * i, k[i]);
        if (b + 8 * (i + PD) < blk_end) col.load(b + 8 * (i + PD), k[i]);
      }
}

namespace {

int rank_tiles(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

// 64-token tiles read B once for 64 tokens; they need segments that fill them.
bool long_tiles(int T, int n_seg) { return T >= 1024 && T / 48 >= n_seg; }

// Tokens of a shrink tile. 16 fill the chip without splitting k from 4096
// tokens on, and A, read once a tile, comes from L2 (a rank-64 A of 4096
// features: 512 KB a tile against 128 KB of X from memory); at rank 128 that
// would be the larger part, so long batches take 64.
int shrink_tokens(int T, int R, int n_seg) { return R > 64 && long_tiles(T, n_seg) ? 64 : 16; }

// Splits of the contraction: about 256 workgroups, each with two steps or more for each of its waves.
int shrink_splits(int T, int K, int R, int n_seg) {
  const LoraSegs S = {nullptr, nullptr, n_seg, 0};
  const int tiles = lora_tiles(T, S, shrink_tokens(T, R, n_seg));
  const int most = K / 512 < MAX_SPLITS ? K / 512 : MAX_SPLITS;
  const int want = 384 / (tiles > 0 ? tiles : 1);
  return want < 1 || most < 1 ? 1 : want < most ? want : most;
}

// One launch for up to 32 tiles with an A of up to 160 KB. Every workgroup
// reads A[a] whole, at the 15 to 25 GB/s that one compute unit gets from
// memory: 128 KB take as long as two launches that split k (8 us), but the
// second launch costs the host 4 us. With 64 tiles and 11008 columns one launch
// takes 22 us against 7 + 9.
bool one_launch(int T, int K, int R, int elem, int n_seg) {
  const LoraSegs S = {nullptr, nullptr, n_seg, 0};
  return lora_tiles(T, S, 16) <= 32 && (int64_t)K * R * elem <= 160 * 1024;
}

template <int DT, int RT, bool FULL>
void run_short(const void* Xv, int T, int K, const void* Av, const void* Bv, const float* scaling, int R, int N,
               const LoraSegs& S, const void* base, void* out, float* V, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  const int tiles = lora_tiles(T, S, 16), blocks = (N + Mx<DT>::KS - 1) / Mx<DT>::KS;
  int64_t bpw = (int64_t)tiles * blocks / (8 * 256);     // about 256 workgroups: few repeat V
  bpw = bpw < 1 ? 1 : bpw > 64 ? 64 : bpw;
  const int slices = blocks > 0 ? (int)((blocks + 8 * bpw - 1) / (8 * bpw)) : V ? 1 : 0;
  if (slices > 0)
    hipLaunchKernelGGL((k_lora_short<DT, RT, FULL>), dim3(tiles, slices), dim3(512), 0, st, static_cast<const E*>(Xv), T, K,
                       static_cast<const E*>(Av), R, scaling, S, static_cast<const E*>(Bv), N,
                       static_cast<const E*>(base), static_cast<E*>(out), V, (int)bpw);
}

template <int DT, int RT, int TMT, bool FULL>
void run(const void* Xv, int T, int K, const void* Av, const void* Bv, const float* scaling, int R, int N,
         const LoraSegs& S, const void* base, void* out, float* V, float* ws, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  constexpr int KS = Mx<DT>::KS, ST = RT == 8 ? TMT : 1, NW = RT < 8 ? 16 : ST == 4 ? 4 : 8;
  const int tiles = lora_tiles(T, S, 16 * TMT);
  const int splits = shrink_splits(T, K, R, S.n_seg);
  if (S.n_adapters > 0)
    hipLaunchKernelGGL((k_lora_shrink<DT, RT, ST, NW, FULL>), dim3(lora_tiles(T, S, 16 * ST), splits), dim3(NW * 64),
                       0, st, static_cast<const E*>(Xv), T, K, static_cast<const E*>(Av), R, S, ws);
  const int blocks = (N + KS - 1) / KS;
  int64_t bpw = (int64_t)tiles * blocks / (4 * 1024);
  bpw = bpw < 1 ? 1 : bpw > 8 ? 8 : bpw;
  const int slices = blocks > 0 ? (int)((blocks + 4 * bpw - 1) / (4 * bpw)) : V ? 1 : 0;
  if (slices > 0)
    hipLaunchKernelGGL((k_lora_expand<DT, RT, TMT, FULL>), dim3(tiles, slices), dim3(256), 0, st, ws, splits, T, N,
                       static_cast<const E*>(Bv), R, scaling, S, static_cast<const E*>(base), static_cast<E*>(out), V,
                       (int)bpw);
}

template <int DT, int RT, bool FULL>
void run_rank(const void* X, int T, int K, const void* A, const void* B, const float* scaling, int R, int N,
              const LoraSegs& S, const void* base, void* out, float* V, float* ws, hipStream_t st) {
  if (one_launch(T, K, R, Elem<DT>::size, S.n_seg))
    run_short<DT, RT, FULL>(X, T, K, A, B, scaling, R, N, S, base, out, V, st);
  else if (long_tiles(T, S.n_seg))
    run<DT, RT, 4, FULL>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
  else
    run<DT, RT, 1, FULL>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
}

// Widths of whole steps and a rank of whole tiles run kernels without the code
// for their ends: a short launch waits for its instructions as for its data.
template <int DT, int RT>
void run_size(const void* X, int T, int K, const void* A, const void* B, const float* scaling, int R, int N,
              const LoraSegs& S, const void* base, void* out, float* V, float* ws, hipStream_t st) {
  if (K % Mx<DT>::KS == 0 && N % Mx<DT>::KS == 0 && R == 16 * RT)
    run_rank<DT, RT, true>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
  else
    run_rank<DT, RT, false>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
}

template <int DT>
hipError_t forward_t(const void* X, int T, int K, const void* A, const void* B, const float* scaling, int R, int N,
                     const LoraSegs& S, const void* base, void* out, float* V, float* ws, hipStream_t st) {
  switch (rank_tiles(R)) {
    case 1: run_size<DT, 1>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st); break;
    case 2: run_size<DT, 2>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st); break;
    case 4: run_size<DT, 4>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st); break;
    default: run_size<DT, 8>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st);
  }
  return hipGetLastError();
}

}  // namespace

size_t lora_forward_floats(int T, int K, int N, int R, int n_seg) {
  return (size_t)shrink_splits(T, K, R, n_seg) * T * 16 * rank_tiles(R);
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
