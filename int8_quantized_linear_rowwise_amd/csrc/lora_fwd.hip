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
#include "lora.hpp"

namespace i8l {

// P[split][t][r] = sum over the split's part of k of X[t, k] A[a][r][k], Rp =
// 16 RT columns (columns past R hold values that are not read). NW waves share
// a tile and take pairs of contraction steps in turn (128 bytes of each row);
// fragments come straight from memory, as both operands lie along k; the waves'
// sums are added in LDS in a fixed order.
//
// fp16 weights below 2^-14 are denormals, whose products the matrix core sums
// with the absolute error of products of 2^-14: V of an adapter that is small
// throughout lost up to 10 of its 24 bits. So A is multiplied by 2^14 (exact)
// until a value of 2 or more is met, from where the sums go on without.
template <int DT, int RT, int TMT, int NW>
__global__ __launch_bounds__(NW * 64) void k_lora_shrink(const typename Elem<DT>::T* __restrict__ X, int T, int K,
                                                         const typename Elem<DT>::T* __restrict__ A, int R,
                                                         LoraSegs S, float* __restrict__ P) {
  typedef Mx<DT> M;
  typedef typename Elem<DT>::T E;
  constexpr int KS = M::KS, EL = M::EL;
  constexpr int U = TMT + RT <= 2 ? 4 : TMT + RT <= 5 ? 2 : 1;   // pairs of steps in flight
  __shared__ v4f red[NW / 2][TMT * RT][64];
  const LoraTile tl = lora_tile(S, blockIdx.x + 1, T, 16 * TMT);
  if (tl.t1 <= tl.t0 || tl.adapter < 0) return;
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // rows past the tile or the rank repeat the last one: they only reach
  // products that are not stored
  const E* x[TMT];
  const E* w[RT];
#pragma unroll
  for (int i = 0; i < TMT; ++i) x[i] = X + (int64_t)min(tl.t0 + 16 * i + c, tl.t1 - 1) * K + EL * q;
#pragma unroll
  for (int j = 0; j < RT; ++j) w[j] = A + ((int64_t)tl.adapter * R + min(16 * j + c, R - 1)) * K + EL * q;

  v4f acc[TMT][RT];
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
  const int steps = (K + KS - 1) / KS;
  const int s0 = (int)((int64_t)steps * blockIdx.y / gridDim.y), s1 = (int)((int64_t)steps * (blockIdx.y + 1) / gridDim.y);
  int s = s0 + 2 * wave;
  for (; s + 2 * NW * (U - 1) + 2 <= s1 && (s + 2 * NW * (U - 1) + 2) * KS <= K; s += 2 * NW * U) {
    v4u fx[2 * U][TMT], fw[2 * U][RT];
#pragma unroll
    for (int u = 0; u < 2 * U; ++u) {
      const int k = (s + 2 * NW * (u >> 1) + (u & 1)) * KS;
#pragma unroll
      for (int i = 0; i < TMT; ++i) fx[u][i] = ld16<DT>(x[i] + k);
#pragma unroll
      for (int j = 0; j < RT; ++j) fw[u][j] = ld16<DT>(w[j] + k);
    }
    lift(fw, 2 * U);
#pragma unroll
    for (int u = 0; u < 2 * U; ++u)
#pragma unroll
      for (int i = 0; i < TMT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[i][j] = M::mma(fx[u][i], fw[u][j], acc[i][j]);
  }
  for (; s < s1; s += 2 * NW)
    for (int h = s; h < min(s + 2, s1); ++h) {
      const int left = K - h * KS - EL * q;
      v4u fx[TMT], fw[1][RT];
#pragma unroll
      for (int i = 0; i < TMT; ++i) fx[i] = ld_frag<DT>(x[i] + h * KS, left);
#pragma unroll
      for (int j = 0; j < RT; ++j) fw[0][j] = ld_frag<DT>(w[j] + h * KS, left);
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

// out[t, n] = D(base[t, n] + s[a] sum_r V[t, r] B[a][n][r]), V = the sum of the
// splits of P (also written to `V` by the first column slice). The product is
// taken transposed (rows n, columns t), so that a lane holds consecutive n of
// one token: with row m of product u standing for n = 8 (m / 4) + 4 u + m % 4
// two 16-bit products give a lane 8 consecutive n, 16 bytes of base and out.
// The contraction runs over both parts of V against the same B fragments; at
// rank 16 both parts fill one step.
template <int DT, int RT, int TMT>
__global__ __launch_bounds__(256) void k_lora_expand(const float* __restrict__ P, int splits, int T, int N,
                                                     const typename Elem<DT>::T* __restrict__ B, int R,
                                                     const float* __restrict__ scaling, LoraSegs S,
                                                     const typename Elem<DT>::T* base, typename Elem<DT>::T* out,
                                                     float* __restrict__ V, int blocks_per_wave) {
  typedef Mx<DT> M;
  typedef typename Elem<DT>::T E;
  constexpr int KS = M::KS, EL = M::EL, TM = 16 * TMT, RP = 16 * RT;
  constexpr int UN = M::F32 ? 1 : 2;                              // products of one block of KS columns
  constexpr int NB = M::F32 ? RT : (RT + 1) / 2;                  // B fragments of a row
  constexpr int NS = M::F32 ? RT : RT == 1 ? 1 : RT;              // contraction steps over all parts of V
  constexpr int LD = M::F32 ? RP + 4 : RP + 8;                    // LDS row, in elements
  __shared__ __attribute__((aligned(16))) E sv[M::NC][TM][LD];
  __shared__ float sunit[TM];
  const LoraTile tl = lora_tile(S, blockIdx.x + 1, T, TM);
  const int n_tok = tl.t1 - tl.t0;
  if (n_tok <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int blk0 = blockIdx.y * 4 * blocks_per_wave + wave, n_blk = (N + KS - 1) / KS;
  const int blk_end = min(blk0 + 4 * blocks_per_wave, n_blk);

  const E* bp[TMT];
  int64_t row[TMT];
#pragma unroll
  for (int i = 0; i < TMT; ++i) {
    row[i] = (int64_t)min(tl.t0 + 16 * i + c, tl.t1 - 1) * N;
    bp[i] = base + row[i];
  }

  if (tl.adapter < 0) {
    if (V && blockIdx.y == 0)
      for (int64_t e = (int64_t)tl.t0 * R + tid; e < (int64_t)tl.t1 * R; e += 256) V[e] = 0.0f;
    if (base == out) return;
    for (int b = blk0; b < blk_end; b += 4) {
      const int n = b * KS + EL * q;
#pragma unroll
      for (int i = 0; i < TMT; ++i) {
        const v4u f = base ? ld_frag<DT>(bp[i] + n, N - n) : v4u{0u, 0u, 0u, 0u};
        if (16 * i + c < n_tok) st_frag<DT>(out + row[i] + n, f, N - n);
      }
    }
    return;
  }

  // V's parts into LDS: four consecutive r a thread, the threads of a token side by side
  for (int e = tid; e < TM * RP / 4; e += 256) {
    const int t = e / (RP / 4), r = e % (RP / 4) * 4;
    v4f v = {};
    if (t < n_tok) {
      const float* p = P + (int64_t)(tl.t0 + t) * RP + r;
      for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const v4f*>(p + (int64_t)s * T * RP);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (r + j >= R) v[j] = 0.0f;
      else if (V && blockIdx.y == 0 && t < n_tok) V[(int64_t)(tl.t0 + t) * R + r + j] = v[j];
    }
    if constexpr (M::F32) {
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
      *reinterpret_cast<v2u*>(&sv[M::NC - 1][t][r]) =
          v2u{(h[0] >> 16) | (h[1] & 0xffff0000u), (h[2] >> 16) | (h[3] & 0xffff0000u)};
    }
  }
  __syncthreads();

  v4u vf[TMT][NS];
  float f[TMT];
#pragma unroll
  for (int i = 0; i < TMT; ++i) {
    f[i] = scaling[tl.adapter];
    if constexpr (DT == DT_F16) f[i] *= sunit[16 * i + c];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int part = M::F32 ? 0 : RT == 1 ? q >> 1 : s / NB;
      const int r = M::F32 ? 16 * s + 4 * q : RT == 1 ? 8 * (q & 1) : 32 * (s % NB) + 8 * q;
      vf[i][s] = *reinterpret_cast<const v4u*>(&sv[part][16 * i + c][r]);
    }
  }

  const E* Ba = B + (int64_t)tl.adapter * N * R;
  const bool full = R == RP;
  struct Block {
    v4u b[UN][NB], base[TMT];
  };
  auto load = [&](int blk, Block& k) {
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int n = min(blk * KS + (M::F32 ? c : 8 * (c >> 2) + 4 * u + (c & 3)), N - 1);
#pragma unroll
      for (int s = 0; s < NB; ++s) {
        const int r = M::F32 ? 16 * s + 4 * q : RT == 1 ? 8 * (q & 1) : 32 * s + 8 * q;
        if (full) k.b[u][s] = ld16<DT>(Ba + (int64_t)n * R + r);
        else k.b[u][s] = ld_frag<DT>(Ba + (int64_t)n * R + r, R - r);
      }
    }
    const int n = blk * KS + EL * q;
    if (base == nullptr) {
#pragma unroll
      for (int i = 0; i < TMT; ++i) k.base[i] = v4u{0u, 0u, 0u, 0u};
    } else if ((blk + 1) * KS <= N) {
#pragma unroll
      for (int i = 0; i < TMT; ++i) k.base[i] = ld16<DT>(bp[i] + n);
    } else {
#pragma unroll
      for (int i = 0; i < TMT; ++i) k.base[i] = ld_frag<DT>(bp[i] + n, N - n);
    }
  };
  auto finish = [&](int blk, const Block& k) {
    const int n = blk * KS + EL * q;
    const bool whole = (blk + 1) * KS <= N;
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
      if (16 * i + c < n_tok) {
        if (whole) st16<DT>(out + row[i] + n, frag_of<DT>(y));
        else st_frag<DT>(out + row[i] + n, frag_of<DT>(y), N - n);
      }
    }
  };
  if (blk0 >= blk_end) return;
  Block k;
  load(blk0, k);
  for (int b = blk0; b < blk_end; b += 4) {
    const Block cur = k;
    if (b + 4 < blk_end) load(b + 4, k);
    finish(b, cur);
  }
}

namespace {

int rank_tiles(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

// 64-token tiles read A once for 64 tokens; they need segments that fill them.
bool long_tiles(int T, int n_seg) { return T >= 1024 && T / 48 >= n_seg; }

// Splits of the contraction: about 512 workgroups, each with two steps or more for each of its waves.
int shrink_splits(int T, int K, int n_seg) {
  const LoraSegs S = {nullptr, nullptr, n_seg, 0};
  const int tiles = lora_tiles(T, S, long_tiles(T, n_seg) ? 64 : 16);
  const int most = K / 512 < 8 ? K / 512 : 8;
  const int want = 512 / (tiles > 0 ? tiles : 1);
  return want < 1 || most < 1 ? 1 : want < most ? want : most;
}

template <int DT, int RT, int TMT>
void run(const void* Xv, int T, int K, const void* Av, const void* Bv, const float* scaling, int R, int N,
         const LoraSegs& S, const void* base, void* out, float* V, float* ws, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  constexpr int NW = TMT * RT > 16 ? 4 : 8, KS = Mx<DT>::KS;
  const int tiles = lora_tiles(T, S, 16 * TMT);
  const int splits = shrink_splits(T, K, S.n_seg);
  if (S.n_adapters > 0)
    hipLaunchKernelGGL((k_lora_shrink<DT, RT, TMT, NW>), dim3(tiles, splits), dim3(NW * 64), 0, st,
                       static_cast<const E*>(Xv), T, K, static_cast<const E*>(Av), R, S, ws);
  const int blocks = (N + KS - 1) / KS;
  int64_t bpw = (int64_t)tiles * blocks / (4 * 1024);
  bpw = bpw < 1 ? 1 : bpw > 8 ? 8 : bpw;
  const int slices = blocks > 0 ? (int)((blocks + 4 * bpw - 1) / (4 * bpw)) : V ? 1 : 0;
  if (slices > 0)
    hipLaunchKernelGGL((k_lora_expand<DT, RT, TMT>), dim3(tiles, slices), dim3(256), 0, st, ws, splits, T, N,
                       static_cast<const E*>(Bv), R, scaling, S, static_cast<const E*>(base), static_cast<E*>(out), V,
                       (int)bpw);
}

template <int DT>
hipError_t forward_t(const void* X, int T, int K, const void* A, const void* B, const float* scaling, int R, int N,
                     const LoraSegs& S, const void* base, void* out, float* V, float* ws, hipStream_t st) {
#define I8L_RUN(RT)                                                                           \
  if (long_tiles(T, S.n_seg)) run<DT, RT, 4>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st); \
  else run<DT, RT, 1>(X, T, K, A, B, scaling, R, N, S, base, out, V, ws, st)
  switch (rank_tiles(R)) {
    case 1: I8L_RUN(1); break;
    case 2: I8L_RUN(2); break;
    case 4: I8L_RUN(4); break;
    default: I8L_RUN(8);
  }
#undef I8L_RUN
  return hipGetLastError();
}

}  // namespace

size_t lora_forward_floats(int T, int K, int N, int R, int n_seg) {
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
