// Low-rank adapters of many requests beside a shared projection: gradients.
//
// With g = dL/dy, token t of adapter a:
//   dV[t] = s[a] B[a]^T g[t],  dx[t] = D(base_grad[t] + A[a]^T dV[t]),
//   dA[a] = D(sum_t dV[t] x[t]^T),  dB[a] = D(s[a] sum_t g[t] V[t]^T).
// Bound by memory: G, X, base_grad and dx once, T (N + 3 K) elements, against
// 4 T R (K + N) flops. Each large operand serves two products, one along the
// features and one along the tokens, so each is read once for both:
//   g pass: G gives dV (partial sums by column slice) and dB (by token tile);
//   sum of the slices of dV and of the tiles of dB, in a fixed order;
//   x pass: X and base_grad give dx and dA (partial sums by token tile);
//   sum of the tiles of dA.
// Small batches skip the first sum: the x pass adds the slices up itself. 4096
// tokens, 4096 -> 11008 at rank 16: 27 + 6 + 28 + 6 us; 16384 tokens of 16
// sequences, 8192 -> 28672 at rank 32: 235 + 40 + 167 + 7 us, of which the
// partial sums (300 MB beside 1.77 GB of operands) are about a sixth.
// A workgroup takes a slice of columns and a token tile (tokens of one adapter),
// or a block of tokens that it walks tile by tile; its eight waves split the
// columns, and each holds its part of the weight gradient in registers while it
// walks the tokens 32 (fp32: 16) at a time. The rows go through LDS, from where
// they are read along the features for the one product and transposed for the
// one along the tokens.
#include "lora.hpp"

namespace i8l {

typedef short v4s __attribute__((ext_vector_type(4)));
#define I8L_LDS(p) ((__attribute__((address_space(3))) v4s*)(p))

namespace {

// A wave's tile of ST token rows x WN columns in LDS. 16-bit rows are stored in
// pairs of 16-byte chunks (16 columns), pair p of row t at p ^ swz(t): the
// eight rows of one write by eight lanes and the eight rows of a half wave's
// transposed read fall on distinct banks. fp32 rows are padded by 16 bytes.
template <int DT, int WN>
struct Tile {
  static constexpr int ST = DT == DT_F32 ? 16 : 32;
  static constexpr int TT = ST / 16;
  static constexpr int ROWB = DT == DT_F32 ? (WN + 4) * 4 : WN * 2;
  static constexpr int BYTES = ST * ROWB;
  static constexpr int PAIRS = WN / 16, ROWS = PAIRS >= 8 ? 1 : 8 / PAIRS;   // rows that span all banks
  __device__ static __forceinline__ int swz(int t) {
    return ((t / ROWS) & (PAIRS - 1)) ^ (((t >> 3) & 1) * (PAIRS / 2));
  }
  // 16-byte chunk ch of row t
  __device__ static __forceinline__ v4u& at(char* w, int t, int ch) {
    if constexpr (DT == DT_F32) return *reinterpret_cast<v4u*>(w + t * ROWB + 16 * ch);
    else return *reinterpret_cast<v4u*>(w + t * ROWB + 32 * ((ch >> 1) ^ swz(t)) + 16 * (ch & 1));
  }
  // The tile as it lies in memory: load i of NI takes RPI rows, CPR lanes side by
  // side on one row. (A fragment's lanes lie on 16 rows each; loading
  // fragments straight from memory, 16 bytes a request, held these kernels to
  // about one request a nanosecond and compute unit.)
  static constexpr int CPR = WN / Mx<DT>::EL, RPI = 64 / CPR, NI = ST / RPI;
  // Rows r0 + (8 | 4) q .. along the contraction, columns `col` .. of 4 lanes each as rows: with rows that are ranks,
  // the operand of a product along the ranks. 16-bit: lane c's column is col(c / 4) + c % 4; fp32: col(0) + c.
  template <typename F>
  __device__ static __forceinline__ v4u get_cols(const char* w, int r0, F col, int lane) {
    const int c = lane & 15;
    if constexpr (DT == DT_F32) {
      v4u f;
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = *reinterpret_cast<const uint32_t*>(w + (r0 + j) * ROWB + 4 * (col(0) + c));
      return f;
    } else {
      v4s h[2];
      const int x = col(c & 3);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = r0 + 4 * i + (c >> 2);
        h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(I8L_LDS(w + t * ROWB + 32 * ((x >> 4) ^ swz(t)) + 2 * (x & 15)));
      }
      return __builtin_bit_cast(v4u, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
  // columns 16 nt .. + 15 as rows, the tokens along the contraction
  __device__ static __forceinline__ v4u get(const char* w, int nt, int lane) {
    const int c = lane & 15, q = lane >> 4;
    if constexpr (DT == DT_F32) {
      v4u f;
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = *reinterpret_cast<const uint32_t*>(w + (4 * q + j) * ROWB + 4 * (16 * nt + c));
      return f;
    } else {
      v4s h[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 8 * q + 4 * i + (c >> 2);
        h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(I8L_LDS(w + t * ROWB + 32 * (nt ^ swz(t)) + 8 * (c & 3)));
      }
      return __builtin_bit_cast(v4u, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// fp32 values [token][r] in LDS as operands: `vt` [part][r][token] (rows of 80
// bytes) for products along the tokens, `vr` [part][token][r] along r.
template <int DT, int RT>
struct Small {
  typedef typename Elem<DT>::T E;
  static constexpr int ST = DT == DT_F32 ? 16 : 32, RP = 16 * RT, NC = Mx<DT>::NC;
  static constexpr int LDT = 80 / (int)sizeof(E), LDR = RP + 16 / (int)sizeof(E);
  static constexpr int VT = NC * RP * LDT * (int)sizeof(E), VR = NC * ST * LDR * (int)sizeof(E);
  static constexpr int PAIRS = ST / 2 * RP;                  // two tokens of one r
  static constexpr int PER = (PAIRS + 511) / 512;            // pairs a thread holds
  __device__ static __forceinline__ void put_t(char* vt, int r, int tp, float a, float b, float unit) {
    E* p = reinterpret_cast<E*>(vt) + r * LDT + 2 * tp;
    if constexpr (DT == DT_F32) {
      *reinterpret_cast<v2f*>(p) = v2f{a, b};
    } else {
      const uint32_t x = split2<DT>(a, unit), y = split2<DT>(b, unit);
      *reinterpret_cast<uint32_t*>(p) = (x & 0xffffu) | (y << 16);
      *reinterpret_cast<uint32_t*>(p + RP * LDT) = (x >> 16) | (y & 0xffff0000u);
    }
  }
  __device__ static __forceinline__ void put_r(char* vr, int r, int t, float a, float unit) {
    E* p = reinterpret_cast<E*>(vr) + t * LDR + r;
    if constexpr (DT == DT_F32) {
      *p = a;
    } else {
      const uint32_t x = split2<DT>(a, unit);
      p[0] = __builtin_bit_cast(E, (uint16_t)(x & 0xffffu));
      p[ST * LDR] = __builtin_bit_cast(E, (uint16_t)(x >> 16));
    }
  }
  __device__ static __forceinline__ v4u get_t(const char* vt, int part, int rt, int lane) {
    return *reinterpret_cast<const v4u*>(reinterpret_cast<const E*>(vt) + (part * RP + 16 * rt + (lane & 15)) * LDT +
                                         Mx<DT>::EL * (lane >> 4));
  }
  __device__ static __forceinline__ v4u get_r(const char* vr, int part, int t, int r) {
    return *reinterpret_cast<const v4u*>(reinterpret_cast<const E*>(vr) + (part * ST + t) * LDR + r);
  }
};

// acc[j][n] += the tile's columns 16 n .. times vt's r 16 j .., along the
// tokens; the operand with fewer fragments stays in registers.
template <int DT, int RT, int WN>
__device__ __forceinline__ void along_tokens(const char* tile, const char* vt, int lane, v4f (&acc)[RT][WN / 16]) {
  typedef Mx<DT> M;
  constexpr int NT = WN / 16;
  if constexpr (NT <= M::NC * RT) {
    v4u f[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) f[n] = Tile<DT, WN>::get(tile, n, lane);
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int p = 0; p < M::NC; ++p) {
        const v4u fv = Small<DT, RT>::get_t(vt, p, j, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[j][n] = M::mma(f[n], fv, acc[j][n]);
      }
  } else {
    v4u fv[M::NC][RT];
#pragma unroll
    for (int p = 0; p < M::NC; ++p)
#pragma unroll
      for (int j = 0; j < RT; ++j) fv[p][j] = Small<DT, RT>::get_t(vt, p, j, lane);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const v4u f = Tile<DT, WN>::get(tile, n, lane);
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int p = 0; p < M::NC; ++p) acc[j][n] = M::mma(f, fv[p][j], acc[j][n]);
    }
  }
}

// Row of sorted position i: the rows themselves without a permutation. A
// permutation of offsets that make no sense can have holes: its entries are
// held inside the tensor.
__device__ __forceinline__ int row_of(const int32_t* perm, int i, int T) {
  return perm ? (int)min((uint32_t)perm[i], (uint32_t)(T - 1)) : i;
}

__device__ __forceinline__ float finite_abs(float v) { return __builtin_isfinite(v) ? __builtin_fabsf(v) : 0.0f; }

}  // namespace

// One tile of k_lora_gpass.
template <int DT, int RT, int WN>
__device__ __forceinline__ void g_tile(const typename Elem<DT>::T* __restrict__ G, int N, int T,
                                       const float* __restrict__ V, const typename Elem<DT>::T* __restrict__ B, int R,
                                       const float* __restrict__ scaling, const LoraSegs& S,
                                       const SegLanes& L, const int32_t* __restrict__ perm, int tm,
                                       float* __restrict__ P,
                                       float* __restrict__ dBp, int32_t* __restrict__ tile_adapter, int slice, int d) {
  typedef Mx<DT> M;
  typedef typename Elem<DT>::T E;
  typedef Tile<DT, WN> TL;
  typedef Small<DT, RT> SM;
  constexpr int KS = M::KS, EL = M::EL, ST = TL::ST, TT = TL::TT, NK = WN / KS, NT = WN / 16, RP = 16 * RT;
  constexpr int RW = RP < 64 ? RP : 64, RH = RP / RW, RTH = RW / 16;   // dV meets in LDS up to 64 columns at a time
  constexpr int LDV = RW + 4;
  extern __shared__ __attribute__((aligned(16))) char sm[];
  char* vt = sm + 8 * TL::BYTES;
  float* red = reinterpret_cast<float*>(vt + SM::VT);
  float* top8 = red + 8 * ST * LDV;

  const LoraTile tl = lora_tile(S, L, d, T, tm);
  const bool none = tl.t1 <= tl.t0 || tl.adapter < 0;
  // opaque per tile: hoisted out of the tile loop, the addresses made from it cost 50 registers
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, c = lane & 15, q = lane >> 4;
  if (slice == 0 && tid == 0) tile_adapter[d - 1] = none ? -1 : tl.adapter;
  if (none) return;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  char* mine = sm + wave * TL::BYTES;
  const int n0 = slice * 8 * WN + wave * WN;
  const bool whole = n0 + WN <= N;
  const float scale = scaling[tl.adapter];

  v4f acc[RT][NT];
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[j][n] = v4f{};
  float run_top = 0.0f, unit = 1.0f;

  v4u g[TL::NI];
  float v[SM::PER][2];
  const int lrow = lane / TL::CPR, lch = lane % TL::CPR;
  auto load = [&](int at) {
    const int left = N - n0 - EL * lch;
#pragma unroll
    for (int i = 0; i < TL::NI; ++i) {
      const int row = row_of(perm, min(at + TL::RPI * i + lrow, tl.t1 - 1), T);
      const E* p = G + (int64_t)row * N + n0 + EL * lch;
      g[i] = whole ? ld16<DT>(p) : ld_frag<DT>(p, left);
    }
    if (dBp) {
#pragma unroll
      for (int x = 0; x < SM::PER; ++x) {
        const int e = tid + 512 * x, r = e % RP, t = at + 2 * (e / RP);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[x][h] = e < SM::PAIRS && r < R && t + h < tl.t1 ? V[(int64_t)row_of(perm, t + h, T) * R + r] : 0.0f;
      }
    }
  };
  typedef Tile<DT, RP> TB;
  constexpr bool BYLDS = TB::BYTES <= ST * LDV * 4;
  v4u lb[BYLDS ? NK : 1][BYLDS ? TB::NI : 1];
  if constexpr (BYLDS) {
    const int ch = EL * (lane % TB::CPR);
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
      for (int i = 0; i < TB::NI; ++i) {
        const int n = n0 + k * KS + TB::RPI * i + lane / TB::CPR;
        lb[k][i] = v4u{0u, 0u, 0u, 0u};
        if (P && n < N) lb[k][i] = ld_frag<DT>(B + ((int64_t)tl.adapter * N + n) * R + ch, R - ch);
      }
  }
  load(tl.t0);

  // B[a][n][r] with n along the contraction: its rows through the wave's part of
  // `red`, read transposed (fp32 at rank 128, where that is too small: gathered)
  v4u fb[RT][NK];
  float bunit = 1.0f;
  if (P) {
    const E* Ba = B + (int64_t)tl.adapter * N * R;
    if constexpr (BYLDS) {
      char* w = reinterpret_cast<char*>(red + wave * ST * LDV);
#pragma unroll
      for (int k = 0; k < NK; ++k) {
#pragma unroll
        for (int i = 0; i < TB::NI; ++i) TB::at(w, TB::RPI * i + lane / TB::CPR, lane % TB::CPR) = lb[k][i];
#pragma unroll
        for (int j = 0; j < RT; ++j) fb[j][k] = TB::get(w, j, lane);
      }
    } else {
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          fb[j][k] = v4u{0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < EL; ++e) {
            const int n = n0 + k * KS + EL * q + e, r = 16 * j + c;
            const E w = Ba[(int64_t)min(n, N - 1) * R + min(r, R - 1)];
            frag_set<DT>(fb[j][k], e, n < N && r < R ? w : Elem<DT>::from_f32(0.0f));
          }
        }
    }
    if constexpr (DT == DT_F16) {
      // denormal weights lose bits in the matrix core (see the forward's
      // shrink): a power of two takes the wave's largest to 2^14
      uint32_t top = 0u;   // magnitude bits order as the values do
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
          for (int e = 0; e < EL; ++e) {
            const uint32_t m = (fb[j][k][e >> 1] >> (16 * (e & 1))) & 0x7fffu;
            top = max(top, m < 0x7c00u ? m : 0u);
          }
      const float most = (float)__builtin_bit_cast(_Float16, (uint16_t)wave_umax(top));
      bunit = fminf(fmaxf(unit_for(most), 1.0f), 0x1p15f);   // an fp16 value; never shrinks a weight
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int k = 0; k < NK; ++k)
          fb[j][k] = __builtin_bit_cast(v4u, __builtin_bit_cast(v8h, fb[j][k]) * (_Float16)bunit);
    }
  }

  for (int at = tl.t0; at < tl.t1; at += ST) {
    if (dBp) {
      if constexpr (DT == DT_F16) {
        float top = 0.0f;
#pragma unroll
        for (int x = 0; x < SM::PER; ++x) top = fmaxf(top, fmaxf(finite_abs(v[x][0]), finite_abs(v[x][1])));
        top = wave_max(top);
        if (lane == 0) top8[wave] = top;
        __syncthreads();
        float all = run_top;
#pragma unroll
        for (int w = 0; w < 8; ++w) all = fmaxf(all, top8[w]);
        if (all > run_top) {
          const float u = unit_for(all), f = u * inv_pow2(unit);
#pragma unroll
          for (int j = 0; j < RT; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[j][n] *= f;
          unit = u;
          run_top = all;
        }
      }
#pragma unroll
      for (int x = 0; x < SM::PER; ++x) {
        const int e = tid + 512 * x;
        if (e < SM::PAIRS) SM::put_t(vt, e % RP, e / RP, v[x][0], v[x][1], unit);
      }
    }
    // rows past the tile are zeros: a NaN there must not meet their zeros in V
#pragma unroll
    for (int i = 0; i < TL::NI; ++i) {
      const int t = TL::RPI * i + lrow;
      TL::at(mine, t, lch) = at + t < tl.t1 ? g[i] : v4u{0u, 0u, 0u, 0u};
    }
    if (at + ST < tl.t1) load(at + ST);
    if (P) {
      const float f = DT == DT_F16 ? inv_pow2(bunit) : 1.0f;
#pragma unroll
      for (int h = 0; h < RH; ++h) {
        v4f dv[TT][RTH];
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
          for (int j = 0; j < RTH; ++j) {
            dv[i][j] = v4f{};
#pragma unroll
            for (int k = 0; k < NK; ++k) dv[i][j] = M::mma(TL::at(mine, 16 * i + c, 4 * k + q), fb[h * RTH + j][k], dv[i][j]);
          }
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
          for (int j = 0; j < RTH; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              red[(wave * ST + 16 * i + 4 * q + e) * LDV + 16 * j + c] = dv[i][j][e] * f;
        __syncthreads();
        for (int e = tid; e < ST * RW / 4; e += 512) {
          const int t = e / (RW / 4), r = e % (RW / 4) * 4;
          v4f s = {};
#pragma unroll
          for (int w = 0; w < 8; ++w) s += *reinterpret_cast<const v4f*>(&red[(w * ST + t) * LDV + r]);
          if (at + t < tl.t1)
            *reinterpret_cast<v4f*>(P + ((int64_t)slice * T + at + t) * RP + h * RW + r) = s * scale;
        }
        if (h + 1 < RH) __syncthreads();
      }
    } else {
      __syncthreads();
    }
    if (dBp) {
      along_tokens<DT, RT, WN>(mine, vt, lane, acc);
    }
    __syncthreads();
  }
  if (dBp) {
    const float f = DT == DT_F16 ? scale * inv_pow2(unit) : scale;
    float* o = dBp + (int64_t)(d - 1) * N * RP;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = n0 + 16 * n + 4 * q + e;
        if (at < N)
#pragma unroll
          for (int j = 0; j < RT; ++j) o[(int64_t)at * RP + 16 * j + c] = acc[j][n][e] * f;
      }
  }
}

// dV partial sums P[slice][position][Rp] and dB partial sums dBp[tile][n][Rp] of
// 8 WN columns of G and one tile of tokens, or with BLOCKS tokens [y tm, (y + 1)
// tm) tile by tile. Workgroup y * slices + slice (y as a grid axis of its own
// would end at 65535). B's fragments
// for dV stay in registers; the eight waves' parts of dV meet in LDS.
template <int DT, int RT, int WN, bool BLOCKS>
__global__ __launch_bounds__(512, RT == 1 ? 4 : 2) void k_lora_gpass(const typename Elem<DT>::T* __restrict__ G, int N, int T,
                                                    const float* __restrict__ V,
                                                    const typename Elem<DT>::T* __restrict__ B, int R,
                                                    const float* __restrict__ scaling, LoraSegs S,
                                                    const int32_t* __restrict__ perm, int tm, float* __restrict__ P,
                                                    float* __restrict__ dBp, int32_t* __restrict__ tile_adapter,
                                                    int n_slices) {
  const SegLanes L = seg_lanes(S, T);
  const int y = blockIdx.x / n_slices, slice = blockIdx.x - y * n_slices;
  if constexpr (!BLOCKS) {
    g_tile<DT, RT, WN>(G, N, T, V, B, R, scaling, S, L, perm, tm, P, dBp, tile_adapter, slice, y + 1);
  } else {
    const int d1 = first_tile(S, L, y + 1, T, tm);
    for (int d = max(first_tile(S, L, y, T, tm), 1); d < d1; ++d) {
      g_tile<DT, RT, WN>(G, N, T, V, B, R, scaling, S, L, perm, tm, P, dBp, tile_adapter, slice, d);
      __syncthreads();
    }
  }
}

// One tile of k_lora_xpass.
template <int DT, int RT, int WN>
__device__ __forceinline__ void x_tile(const typename Elem<DT>::T* __restrict__ X, int K, int T,
                                       const float* __restrict__ dV, int slices, const typename Elem<DT>::T* __restrict__ A, int R,
                                       const LoraSegs& S, const SegLanes& L, const int32_t* __restrict__ perm, int tm,
                                       const typename Elem<DT>::T* base, typename Elem<DT>::T* out,
                                       float* __restrict__ dAp, int Kp, int32_t* __restrict__ tile_adapter, int slice,
                                       int d) {
  typedef Mx<DT> M;
  typedef typename Elem<DT>::T E;
  typedef Tile<DT, WN> TL;
  typedef Small<DT, RT> SM;
  constexpr int KS = M::KS, EL = M::EL, ST = TL::ST, TT = TL::TT, NK = WN / KS, NT = WN / 16, RP = 16 * RT;
  constexpr int UN = M::F32 ? 1 : 2;
  constexpr int NB = M::F32 ? RT : (RT + 1) / 2, NS = M::F32 ? RT : RT == 1 ? 1 : RT;
  extern __shared__ __attribute__((aligned(16))) char sm[];
  char* vt = sm + 8 * TL::BYTES;
  char* vr = vt + SM::VT;
  float* top8 = reinterpret_cast<float*>(vr + SM::VR);
  float* tops = top8 + 8;   // fp16: [part][token], the largest of up to 64 of a token's values
  constexpr int W = RP < 64 ? RP : 64, NP = RP / W;
  // fp16: the power of two of the tile's token t, and of t and t + 1
  auto unit_of = [&](int t) { return unit_for(NP == 1 ? tops[t] : fmaxf(tops[t], tops[ST + t])); };
  auto units_of = [&](int t) {
    v2f m = *reinterpret_cast<const v2f*>(tops + t);
    if constexpr (NP == 2) {
      const v2f o = *reinterpret_cast<const v2f*>(tops + ST + t);
      m = v2f{fmaxf(m[0], o[0]), fmaxf(m[1], o[1])};
    }
    return v2f{unit_for(m[0]), unit_for(m[1])};
  };

  const LoraTile tl = lora_tile(S, L, d, T, tm);
  const bool none = tl.t1 <= tl.t0 || tl.adapter < 0;
  // opaque per tile: hoisted out of the tile loop, the addresses made from it cost 50 registers
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, c = lane & 15, q = lane >> 4;
  if (dAp && slice == 0 && tid == 0) tile_adapter[d - 1] = none ? -1 : tl.adapter;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  char* mine = sm + wave * TL::BYTES;
  const int k0 = slice * 8 * WN + wave * WN;
  const bool whole = k0 + WN <= K;

  v4u x[TL::NI], b[TL::NI];
  float v[SM::PER][2];
  const int lrow = lane / TL::CPR, lch = lane % TL::CPR, left = K - k0 - EL * lch;
  auto spot = [&](int at, int i) {
    return (int64_t)row_of(perm, min(at + TL::RPI * i + lrow, tl.t1 - 1), T) * K + k0 + EL * lch;
  };
  auto load_rows = [&](const E* from, int at, v4u (&f)[TL::NI]) {
#pragma unroll
    for (int i = 0; i < TL::NI; ++i) {
      const E* p = from + spot(at, i);
      f[i] = whole ? ld16<DT>(p) : ld_frag<DT>(p, left);
    }
  };
  auto store_row = [&](int at, int i, v4u f) {
    if (at + TL::RPI * i + lrow < tl.t1) {
      E* p = out + spot(at, i);
      if (whole) st16<DT>(p, f);
      else st_frag<DT>(p, f, left);
    }
  };

  if (none) {
    if (out == nullptr || base == out) return;
    for (int at = tl.t0; at < tl.t1; at += ST) {
      if (base) load_rows(base, at, b);
#pragma unroll
      for (int i = 0; i < TL::NI; ++i) store_row(at, i, base ? b[i] : v4u{0u, 0u, 0u, 0u});
    }
    return;
  }

  v4f acc[RT][NT];
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[j][n] = v4f{};
  float run_top = 0.0f, unit = 1.0f;

  auto load_v = [&](int at) {
#pragma unroll
    for (int y = 0; y < SM::PER; ++y) {
      const int e = tid + 512 * y, r = e % RP, t = at + 2 * (e / RP);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v[y][h] = 0.0f;
        if (e < SM::PAIRS && r < R && t + h < tl.t1) {
          const float* p = dV + (int64_t)(t + h) * RP + r;
          v[y][h] = p[0];
          if constexpr (WN == 32) {   // the small batches' form: dV still in slices
#pragma unroll 4
            for (int s = 1; s < slices; ++s) v[y][h] += p[(int64_t)s * T * RP];
          }
        }
      }
    }
  };
  if (dAp) load_rows(X, tl.t0, x);
  if (out && base) load_rows(base, tl.t0, b);
  load_v(tl.t0);

  // A[a][r][k] with r along the contraction, rows k in the order that gives a
  // lane consecutive k of the product: rows of A through the wave's tile, read
  // transposed
  v4u fa[NK][UN][NB];
  if (out) {
    const E* Aa = A + (int64_t)tl.adapter * R * K + k0 + EL * lch;
#pragma unroll
    for (int r0 = 0; r0 < RP; r0 += ST) {
#pragma unroll
      for (int i = 0; i < TL::NI; ++i) {
        const int r = r0 + TL::RPI * i + lrow;
        v4u f = {0u, 0u, 0u, 0u};
        if (r < R) f = whole ? ld16<DT>(Aa + (int64_t)r * K) : ld_frag<DT>(Aa + (int64_t)r * K, left);
        TL::at(mine, TL::RPI * i + lrow, lch) = f;
      }
#pragma unroll
      for (int blk = 0; blk < NK; ++blk)
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          auto col = [&](int g) { return blk * KS + (M::F32 ? 0 : 8 * g + 4 * u); };
          fa[blk][u][r0 / ST] = TL::get_cols(mine, M::F32 ? 4 * q : RT == 1 ? 8 * (q & 1) : 8 * q, col, lane);
        }
    }
  }

  for (int at = tl.t0; at < tl.t1; at += ST) {
    if constexpr (DT == DT_F16) {
      float top = 0.0f;
#pragma unroll
      for (int y = 0; y < SM::PER; ++y) {
        const int e = tid + 512 * y;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float m = lanes_max<W>(finite_abs(v[y][h]));
          if (e < SM::PAIRS && lane % W == 0) tops[e % RP / W * ST + 2 * (e / RP) + h] = m;
          top = fmaxf(top, m);
        }
      }
      if constexpr (W < 64) top = lanes_max<64>(top);
      if (lane == 0) top8[wave] = top;
      __syncthreads();
      float all = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) all = fmaxf(all, top8[w]);
      if (all > run_top) {   // dA: the scale of all tokens so far
        const float u = unit_for(all), f = u * inv_pow2(unit);
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[j][n] *= f;
        unit = u;
        run_top = all;
      }
    }
#pragma unroll
    for (int y = 0; y < SM::PER; ++y) {
      const int e = tid + 512 * y;
      if (e < SM::PAIRS) {
        if (dAp) SM::put_t(vt, e % RP, e / RP, v[y][0], v[y][1], unit);
        if (out) {   // dx: the scale of the token
          const int t = 2 * (e / RP);
          v2f u = {1.0f, 1.0f};
          if constexpr (DT == DT_F16) u = units_of(t);
          SM::put_r(vr, e % RP, t, v[y][0], u[0]);
          SM::put_r(vr, e % RP, t + 1, v[y][1], u[1]);
        }
      }
    }
    if (dAp) {
#pragma unroll
      for (int i = 0; i < TL::NI; ++i) {
        const int t = TL::RPI * i + lrow;
        TL::at(mine, t, lch) = at + t < tl.t1 ? x[i] : v4u{0u, 0u, 0u, 0u};
      }
    }
    const bool more = at + ST < tl.t1;
    if (more) {
      if (dAp) load_rows(X, at + ST, x);
      load_v(at + ST);
    }
    __syncthreads();
    if (dAp) along_tokens<DT, RT, WN>(mine, vt, lane, acc);
    if (out) {
      // base through the wave's tile into the product's layout, dx back the same way
      if (base) {
#pragma unroll
        for (int i = 0; i < TL::NI; ++i) TL::at(mine, TL::RPI * i + lrow, lch) = b[i];
        if (more) load_rows(base, at + ST, b);
      }
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const float f = DT == DT_F16 ? inv_pow2(unit_of(16 * i + c)) : 1.0f;
        v4u fv[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s)
          fv[s] = SM::get_r(vr, M::F32 ? 0 : RT == 1 ? q >> 1 : s / NB, 16 * i + c,
                            M::F32 ? 16 * s + 4 * q : RT == 1 ? 8 * (q & 1) : 32 * (s % NB) + 8 * q);
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          v4f w[UN];
#pragma unroll
          for (int u = 0; u < UN; ++u) {
            w[u] = v4f{};
#pragma unroll
            for (int s = 0; s < NS; ++s) w[u] = M::mma(fa[k][u][s % NB], fv[s], w[u]);
          }
          v4u& place = TL::at(mine, 16 * i + c, 4 * k + q);
          float y[EL];
          frag_f32<DT>(base ? place : v4u{0u, 0u, 0u, 0u}, y);
#pragma unroll
          for (int e = 0; e < EL; ++e) y[e] = __builtin_fmaf(f, w[e >> 2][e & 3], y[e]);
          place = frag_of<DT>(y);
        }
      }
#pragma unroll
      for (int i = 0; i < TL::NI; ++i) store_row(at, i, TL::at(mine, TL::RPI * i + lrow, lch));
    }
    __syncthreads();
  }
  if (dAp) {
    const float f = DT == DT_F16 ? inv_pow2(unit) : 1.0f;
    float* o = dAp + (int64_t)(d - 1) * R * Kp;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int r = 16 * j + c;
      if (r < R)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int k = k0 + 16 * n + 4 * q;
          if (k < Kp) *reinterpret_cast<v4f*>(o + (int64_t)r * Kp + k) = acc[j][n] * f;
        }
    }
  }
}

// dx and the partial sums dAp[tile][r][Kp] of 8 WN columns of X and the same tokens. dx is taken transposed, as the forward's expand,
// with A's fragments in registers.
template <int DT, int RT, int WN, bool BLOCKS>
__global__ __launch_bounds__(512, RT == 1 && DT != DT_F16 ? 4 : 2) void k_lora_xpass(const typename Elem<DT>::T* __restrict__ X, int K, int T,
                                                    const float* __restrict__ dV, int slices,
                                                    const typename Elem<DT>::T* __restrict__ A, int R, LoraSegs S,
                                                    const int32_t* __restrict__ perm, int tm,
                                                    const typename Elem<DT>::T* base, typename Elem<DT>::T* out,
                                                    float* __restrict__ dAp, int Kp,
                                                    int32_t* __restrict__ tile_adapter, int n_slices) {
  const SegLanes L = seg_lanes(S, T);
  const int y = blockIdx.x / n_slices, slice = blockIdx.x - y * n_slices;
  if constexpr (!BLOCKS) {
    x_tile<DT, RT, WN>(X, K, T, dV, slices, A, R, S, L, perm, tm, base, out, dAp, Kp, tile_adapter, slice, y + 1);
  } else {
    const int d1 = first_tile(S, L, y + 1, T, tm);
    for (int d = max(first_tile(S, L, y, T, tm), 1); d < d1; ++d) {
      x_tile<DT, RT, WN>(X, K, T, dV, slices, A, R, S, L, perm, tm, base, out, dAp, Kp, tile_adapter, slice, d);
      __syncthreads();
    }
  }
}

// One weight gradient: sums of tiles [tile][rows][ld] into out
// [adapter][rows][width], in tile order.
struct TileSum {
  const float* part;
  const int32_t* adapter;
  void* out;
  int tiles, rows, ld, width, blocks;   // blocks: workgroups of 1024 values for an adapter
};
// dV: the sum of P's slices, four values a thread.
struct SliceSum {
  const float* part;
  float* out;
  int64_t n4;
  int slices, blocks;   // blocks: workgroups of 1024 values
};
// Workgroups: the slices' first, then a's and b's tiles, adapter after adapter.
template <int DT>
__global__ __launch_bounds__(256) void k_lora_sum(SliceSum v, TileSum a, TileSum b, int adapters) {
  typedef typename Elem<DT>::T E;
  __shared__ int list[256];
  __shared__ int count;
  if ((int)blockIdx.x < v.blocks) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= v.n4) return;
    const v4f* p = reinterpret_cast<const v4f*>(v.part) + i;
    v4f sum = {};
#pragma unroll 8
    for (int k = 0; k < v.slices; ++k) sum += p[k * v.n4];
    reinterpret_cast<v4f*>(v.out)[i] = sum;
    return;
  }
  const int at = blockIdx.x - v.blocks;
  const bool first = at < a.blocks * adapters;
  const TileSum s = first ? a : b;
  const int id = first ? at : at - a.blocks * adapters, ad = id / s.blocks;
  const int64_t e = ((int64_t)(id - ad * s.blocks) * 256 + threadIdx.x) * 4;
  const int64_t each = (int64_t)s.rows * s.ld;
  const float* p = s.part + min(e, each - 4);
  v4f sum = {};
  for (int t0 = 0; t0 < s.tiles; t0 += 256) {
    // this adapter's tiles among 256, in order
    __syncthreads();
    if (threadIdx.x < 64) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = t0 + 64 * i + threadIdx.x;
        const bool mine = t < s.tiles && s.adapter[t] == ad;
        const uint64_t m = __ballot(mine);
        if (mine) list[n + __popcll(m & ((1ull << threadIdx.x) - 1))] = t;
        n += __popcll(m);
      }
      if (threadIdx.x == 0) count = n;
    }
    __syncthreads();
    const int n = count;
#pragma unroll 8
    for (int i = 0; i < n; ++i) sum += *reinterpret_cast<const v4f*>(p + list[i] * each);
  }
  if (e >= each) return;
  const int row = (int)(e / s.ld), col = (int)(e % s.ld);
  E* o = static_cast<E*>(s.out) + ((int64_t)ad * s.rows + row) * s.width + col;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (col + j < s.width) o[j] = Elem<DT>::from_f32(sum[j]);
}

// Rows sorted by adapter (in their order within one; rows without an adapter
// last): workgroup a writes the positions of adapter a's rows, a = n_adapters
// those without. Every workgroup reads all segments once.
__global__ __launch_bounds__(256) void k_lora_sort(LoraSegs S, int T, int32_t* __restrict__ perm,
                                                   int32_t* __restrict__ starts) {
  __shared__ int64_t part[4];
  __shared__ int64_t before[257];
  __shared__ int own[256], first[256], len[256];
  const int a = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto adapter = [&](int s) {
    const int x = seg_adapter(S, s);
    return x < 0 ? S.n_adapters : x;
  };
  int64_t less = 0;
  for (int s = tid; s < S.n_seg; s += 256)
    if (adapter(s) < a) less += max(seg_start(S, s + 1, T) - seg_start(S, s, T), 0);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) less += __shfl_xor(less, o, 64);
  if (lane == 0) part[wave] = less;
  __syncthreads();
  int64_t at = part[0] + part[1] + part[2] + part[3];
  if (tid == 0) starts[a] = (int)min(at, (int64_t)T);
  for (int s0 = 0; s0 < S.n_seg; s0 += 256) {
    const int s = s0 + tid;
    const bool mine = s < S.n_seg && adapter(s) == a;
    const int f = mine ? seg_start(S, s, T) : 0;
    own[tid] = mine;
    first[tid] = f;
    len[tid] = mine ? max(seg_start(S, s + 1, T) - f, 0) : 0;
    __syncthreads();
    if (tid < 64) {   // prefix sums of 256 lengths, four a lane
      int64_t v[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = sum;
        sum += len[4 * tid + i];
      }
      int64_t inc = sum;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int64_t u = __shfl_up(inc, o, 64);
        if (tid >= o) inc += u;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) before[4 * tid + i] = inc - sum + v[i];
      if (tid == 63) before[256] = inc;
    }
    __syncthreads();
    for (int i = wave; i < 256; i += 4)
      if (own[i])
        for (int j = lane; j < len[i]; j += 64) {
          const int64_t p = at + before[i] + j;
          if (p < T) perm[p] = first[i] + j;
        }
    at += before[256];
    __syncthreads();
  }
}

namespace {

// Sizes of the launches and of the workspace; of the shape alone.
struct Plan {
  int rt, slices, tm_g, tiles_g, tm_x, tiles_x, kp;
  bool wide_g, wide_x, sort, fold, by_tile_g, by_tile_x;   // by_tile: a workgroup a tile
  size_t p, dv, dbp, dap, ad_g, ad_x, perm, starts, total;   // offsets in floats
};

// Columns of a wave in wide slices (narrow ones: 32), as many as its registers
// hold beside the rank. 64 instead of 128 for the g pass of rank 17 to 32: 16384
// tokens of 16 sequences, 8192 -> 28672, 436 us against 403, 4096 tokens, 4096
// -> 11008 76 and 75, 4096 -> 4096 55 and 60.
constexpr int wide_g(int rt) { return rt == 2 ? 128 : rt <= 4 ? 64 : 32; }
constexpr int wide_x(int rt) { return rt <= 4 ? 64 : 32; }
int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Tokens of a workgroup, a multiple of 32: the number of token blocks that fills
// the chip's 256 compute units `rounds` times, never one more. Where the partial
// weight gradients would then pass 16 MB, at least twice the rank: a tile's is
// 4 Rp / tm times as much to write and read as its own 16-bit rows (987 tokens
// of 24 segments, 4480 -> 2792 at rank 64: 81 us with 32 tokens, 69 with 128;
// 698 tokens of 14, 604 -> 1152: 34 and 38).
int tile_tokens(int T, int slices, int rounds, int rp, int width, int n_seg) {
  const int blocks = 256 * rounds / slices, least = 2 * rp;
  const int tm = (cdiv(T, blocks > 0 ? blocks : 1) + 31) / 32 * 32;
  const int64_t partial = ((int64_t)cdiv(T, tm > 0 ? tm : 32) + n_seg) * width * rp * 4;
  return tm < 32 ? 32 : partial > 16 * 1000 * 1000 && tm < least ? least : tm;
}

// A workgroup for every tile, or one for a block of `tm` tokens that walks its
// tiles. Blocks fill the chip evenly, but a block with many short tiles keeps
// the others waiting. 4096 -> 4096, blocks and tiles, segments of even and of
// very uneven lengths: blocks of less than 128 tokens lose (1024 tokens of 12
// segments at rank 32 38 and 34 us, uneven 49 and 34, of 48 55 and 51, 94 and
// 54; 4096 of 24 at rank 16 66 and 64, 75 and 58) but where every segment is a
// block of its own and half the tiles are empty (4096 of 64 at rank 16 62 and
// 73); so do those that leave compute units idle (2048 at rank 64, 128 blocks x
// slices, of 12 segments 79 and 63, 102 and 62). From there on blocks win (4096
// of 3 at rank 32 76 and 85; 8192 uneven of 6 113 and 127; 16384 of 16, 8192 ->
// 28672, 418 and 483) but for many very uneven segments (8192 of 24 126 and 112,
// of 48 142 and 128). Tiles that all run at once need no blocks: 264 workgroups
// at rank 32, a few more than the units, take 75 us against 69, 528 at rank 16,
// where a unit holds two, 69 against 71.
bool one_tile_each(int tiles, int blocks, int slices, int rounds, int tm) {
  return tm < 128 || (int64_t)tiles * slices <= (rounds == 1 ? 256 : 560) || (int64_t)blocks * slices < 192 * rounds;
}

Plan plan_of(int T, int K, int N, int R, int n_adapters, int n_seg) {
  Plan p = {};
  p.rt = rank_tiles(R);
  const int rp = 16 * p.rt;
  // Sorted by adapter there are as many partial sums as adapters instead of
  // segments. The sort takes 13 us, and the rows' indirection slows the passes by
  // some 0.15 us a MB of rows, so up to 64 segments are sorted where that saves
  // more than 100 MB and 1.5 times the rows' own bytes (taken as 16-bit ones) of
  // partial sums, written and read. As they are and sorted, even lengths and
  // very uneven ones: 64 segments of 4096 tokens, 4096 -> 4096, rank 128, 4
  // adapters (495 MB beside 134) 191 and 163 us, 342 and 182; 64 of 1024 tokens,
  // 11008 -> 11008, rank 64, 4 adapters (665 beside 90) 240 and 91, 423 and 97.
  // On the other side 64 of 8192 tokens, 4096 -> 4096, rank 128, 4 adapters (495
  // beside 268) 255 and 281, 397 and 300; 64 of 4096 at rank 32 (124 beside 134)
  // 72 and 88, 131 and 92; 32 of 16384 tokens, 8192 -> 28672, rank 32, 4 adapters
  // (255 beside 1745), uneven, 454 and 754. More than 64 segments are always
  // sorted: 200 of 4096 tokens, 4096 -> 4096, 4 adapters, uneven: 196 and 65 at
  // rank 16, 496 and 129 at rank 64.
  const double partial = 8.0 * ((double)n_seg - n_adapters - 1) * rp * ((double)K + N);
  const double row_bytes = 2.0 * T * (N + 3.0 * K);
  p.sort = n_seg > n_adapters + 1 && (n_seg > 64 || partial > 100e6 + 1.5 * row_bytes);
  const LoraSegs S = {nullptr, nullptr, p.sort ? n_adapters + 1 : n_seg, n_adapters};
  // Wide slices, fewer partial sums of dV, where 64-token tiles of them would
  // fill the chip. bf16, the g pass wide and narrow: 4096 tokens, 4096 -> 11008,
  // rank 64 99 and 112 us, rank 32 73 and 81, rank 16 62 and 62; 16384 tokens,
  // 8192 -> 28672, rank 32 408 and 524. Both passes: 4096 -> 4096, ranks 16, 32
  // and 64, 4096 tokens 52 61 75 and 46 56 72, 16384 tokens 147 153 183 and 136
  // 151 196. Below the bound, 1024 tokens, 29 35 51 and 26 32 43.
  p.wide_g = (int64_t)cdiv(N, 8 * wide_g(p.rt)) * cdiv(T, 64) >= 256;
  p.wide_x = (int64_t)cdiv(K, 8 * wide_x(p.rt)) * cdiv(T, 64) >= 256;
  p.slices = cdiv(N, 8 * (p.wide_g ? wide_g(p.rt) : 32));
  p.slices = p.slices > 0 ? p.slices : 1;
  const int rounds = p.rt == 1 ? 2 : 1;   // rank 16 leaves room for two workgroups a unit
  p.tm_g = tile_tokens(T, p.slices, rounds, rp, N, S.n_seg);
  p.tiles_g = lora_tiles(T, S, p.tm_g);
  const int slices_x = cdiv(K, 8 * (p.wide_x ? wide_x(p.rt) : 32));
  p.tm_x = tile_tokens(T, slices_x > 0 ? slices_x : 1, rounds, rp, K, S.n_seg);
  p.tiles_x = lora_tiles(T, S, p.tm_x);
  // Few slices of a small batch: the x pass adds them up as it reads them, once
  // a slice of its own, instead of a launch for it. With and without: 64 tokens,
  // 1024 -> 1024, rank 16 12.8 and 15.2 us; 1024 tokens, 2048 -> 2048, rank 16
  // (4 MB read) 21.3 and 23.4, rank 64 (17 MB) 60 and 41; 512 tokens, rank 64 (8
  // MB) 31.8 and 30.4. More slices gain little: 16 of 64 tokens, 4096 -> 4096,
  // rank 16 14.8 and 15.4, 43 of 1024 -> 11008 17.8 and 17.1.
  p.fold = !p.wide_x && p.slices > 1 && p.slices <= 8 && (int64_t)p.slices * T * rp * 4 * slices_x <= 4 * 1000 * 1000;
  p.by_tile_g = one_tile_each(p.tiles_g, cdiv(T, p.tm_g), p.slices, rounds, p.tm_g);
  p.by_tile_x = one_tile_each(p.tiles_x, cdiv(T, p.tm_x), slices_x, rounds, p.tm_x);
  p.kp = (K + 15) / 16 * 16;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += (n + 63) / 64 * 64;
    return o;
  };
  p.p = take(p.slices > 1 ? (size_t)p.slices * T * rp : 0);
  p.dv = take((size_t)T * rp);
  p.dbp = take((size_t)p.tiles_g * N * rp);
  p.dap = take((size_t)p.tiles_x * R * p.kp);
  p.ad_g = take(p.tiles_g);
  p.ad_x = take(p.tiles_x);
  p.perm = take(p.sort ? T : 0);
  p.starts = take(p.sort ? n_adapters + 2 : 0);
  p.total = at;
  return p;
}

template <int DT, int RT, int WN, bool BLOCKS>
hipError_t g_pass(const Plan& p, const void* G, const float* V, int T, const void* B, const float* scaling, int R,
                  int N, const LoraSegs& S, const int32_t* perm, float* P, float* dBp, int32_t* ad, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  typedef Tile<DT, WN> TL;
  constexpr int rw = RT < 4 ? 16 * RT : 64;
  constexpr int lds = 8 * TL::BYTES + Small<DT, RT>::VT + 8 * TL::ST * (rw + 4) * 4 + 32;
  auto kern = k_lora_gpass<DT, RT, WN, BLOCKS>;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = lds_limit_once((const void*)kern, lds, done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)p.slices * (BLOCKS ? cdiv(T, p.tm_g) : p.tiles_g)), dim3(512), lds, st, static_cast<const E*>(G), N, T, V,
                     static_cast<const E*>(B), R, scaling, S, perm, p.tm_g, P, dBp, ad, p.slices);
  return hipGetLastError();
}

template <int DT, int RT, int WN, bool BLOCKS>
hipError_t x_pass(const Plan& p, const void* X, int T, int K, const float* dV, int slices, const void* A, int R,
                  const LoraSegs& S, const int32_t* perm, const void* base, void* out, float* dAp, int32_t* ad,
                  hipStream_t st) {
  typedef typename Elem<DT>::T E;
  constexpr int lds = 8 * Tile<DT, WN>::BYTES + Small<DT, RT>::VT + Small<DT, RT>::VR + 32 +
                      (DT == DT_F16 ? (RT <= 4 ? 1 : 2) * Tile<DT, WN>::ST * 4 : 0);
  auto kern = k_lora_xpass<DT, RT, WN, BLOCKS>;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = lds_limit_once((const void*)kern, lds, done);
  if (e != hipSuccess) return e;
  const int slices_x = cdiv(K, 8 * WN);
  hipLaunchKernelGGL(kern, dim3((unsigned)slices_x * (BLOCKS ? cdiv(T, p.tm_x) : p.tiles_x)), dim3(512), lds, st, static_cast<const E*>(X), K, T, dV,
                     slices, static_cast<const E*>(A), R, S, perm, p.tm_x, static_cast<const E*>(base), static_cast<E*>(out),
                     dAp, p.kp, ad, slices_x);
  return hipGetLastError();
}

template <int DT, int RT>
hipError_t backward_t(const Plan& p, const void* G, const void* X, const float* V, int T, int K, const void* A,
                      const void* B, const float* scaling, int R, int N, const LoraSegs& S0, const void* base_grad,
                      void* gX, void* gA, void* gB, float* ws, hipStream_t st) {
  hipError_t e = hipSuccess;
  const int na = S0.n_adapters;
  LoraSegs S = S0;
  const int32_t* perm = nullptr;
  int32_t* ad_g = reinterpret_cast<int32_t*>(ws + p.ad_g);
  int32_t* ad_x = reinterpret_cast<int32_t*>(ws + p.ad_x);
  float* dV = ws + p.dv;
  const bool want_dv = (gX || gA) && na > 0 && T > 0, rows = T > 0;
  if (na == 0) S = LoraSegs{nullptr, nullptr, 1, 0};   // no adapter anywhere: one segment without
  if (rows && p.sort && na > 0) {
    int32_t* to = reinterpret_cast<int32_t*>(ws + p.perm);
    int32_t* starts = reinterpret_cast<int32_t*>(ws + p.starts);
    hipLaunchKernelGGL(k_lora_sort, dim3(na + 1), dim3(256), 0, st, S0, T, to, starts);
    perm = to;
    S = LoraSegs{starts, nullptr, na + 1, na};
  }
  const int rp = 16 * RT;
  SliceSum slices = {};
  if (rows && na > 0 && N > 0 && (want_dv || gB)) {
    float* P = !want_dv ? nullptr : p.slices > 1 ? ws + p.p : dV;
    float* dBp = gB ? ws + p.dbp : nullptr;
    // (at rank 16 batches long enough for blocks of 128 tokens have wide slices)
    auto pass = p.wide_g ? (p.by_tile_g ? g_pass<DT, RT, wide_g(RT), false> : g_pass<DT, RT, wide_g(RT), true>)
                         : (p.by_tile_g ? g_pass<DT, RT, 32, false> : g_pass<DT, RT, 32, (RT > 1)>);
    e = pass(p, G, V, T, B, scaling, R, N, S, perm, P, dBp, ad_g, st);
    if (e != hipSuccess) return e;
    if (want_dv && p.slices > 1 && !p.fold) {
      const int64_t n4 = (int64_t)T * 4 * RT;
      slices = SliceSum{P, dV, n4, p.slices, cdiv(n4, 256)};
    }
  }
  auto sum = [&](const SliceSum& v, const TileSum& a, const TileSum& b) {
    const int64_t blocks = v.blocks + ((int64_t)a.blocks + b.blocks) * na;
    if (blocks > 0) hipLaunchKernelGGL(k_lora_sum<DT>, dim3((unsigned)blocks), dim3(256), 0, st, v, a, b, na);
  };
  TileSum sum_b = {}, sum_a = {};
  if (gB && na > 0 && R > 0 && N > 0)
    sum_b = TileSum{ws + p.dbp, ad_g, gB, rows ? p.tiles_g : 0, N, rp, R, cdiv((int64_t)N * rp, 1024)};
  if (slices.blocks > 0) {   // beside the sum of dV's slices: dB is whole after the g pass
    sum(slices, sum_b, TileSum{});
    sum_b = TileSum{};
  }
  const bool no_dv = N == 0;   // dV = 0: nothing reaches A or X
  if (rows && K > 0 && (gX || (gA && na > 0))) {
    LoraSegs Sx = S;
    if (no_dv) Sx.n_adapters = 0;
    float* dAp = gA && na > 0 ? ws + p.dap : nullptr;
    auto pass = p.wide_x ? (p.by_tile_x ? x_pass<DT, RT, wide_x(RT), false> : x_pass<DT, RT, wide_x(RT), true>)
                         : (p.by_tile_x ? x_pass<DT, RT, 32, false> : x_pass<DT, RT, 32, (RT > 1)>);
    e = pass(p, X, T, K, p.fold ? ws + p.p : dV, p.fold ? p.slices : 1, A, R, Sx, perm, base_grad, gX, dAp, ad_x, st);
    if (e != hipSuccess) return e;
  }
  if (gA && na > 0 && R > 0 && K > 0)
    sum_a = TileSum{ws + p.dap, ad_x, gA, rows ? p.tiles_x : 0, R, p.kp, K, cdiv((int64_t)R * p.kp, 1024)};
  if (((int64_t)sum_a.blocks + sum_b.blocks) * na >= 1 << 24) {   // a launch has fewer than 2^32 threads
    sum(SliceSum{}, sum_a, TileSum{});
    sum_a = TileSum{};
  }
  sum(SliceSum{}, sum_a, sum_b);
  return hipGetLastError();
}

template <int DT>
hipError_t backward_d(const Plan& p, const void* G, const void* X, const float* V, int T, int K, const void* A,
                      const void* B, const float* scaling, int R, int N, const LoraSegs& S, const void* base_grad,
                      void* gX, void* gA, void* gB, float* ws, hipStream_t st) {
  switch (p.rt) {
    case 1: return backward_t<DT, 1>(p, G, X, V, T, K, A, B, scaling, R, N, S, base_grad, gX, gA, gB, ws, st);
    case 2: return backward_t<DT, 2>(p, G, X, V, T, K, A, B, scaling, R, N, S, base_grad, gX, gA, gB, ws, st);
    case 4: return backward_t<DT, 4>(p, G, X, V, T, K, A, B, scaling, R, N, S, base_grad, gX, gA, gB, ws, st);
    default: return backward_t<DT, 8>(p, G, X, V, T, K, A, B, scaling, R, N, S, base_grad, gX, gA, gB, ws, st);
  }
}

}  // namespace

size_t lora_backward_floats(int T, int K, int N, int R, int n_adapters, int n_seg) {
  return plan_of(T, K, N, R, n_adapters, n_seg).total;
}

hipError_t launch_lora_backward(int dt, const void* G, const void* X, const float* V, int T, int K, const void* A,
                                const void* B, const float* scaling, int R, int N, const LoraSegs& S,
                                int n_adapters, const void* base_grad, void* gX, void* gA, void* gB, float* ws,
                                hipStream_t st) {
  const Plan p = plan_of(T, K, N, R, n_adapters, S.n_seg);
  switch (dt) {
    case DT_F32: return backward_d<DT_F32>(p, G, X, V, T, K, A, B, scaling, R, N, S, base_grad, gX, gA, gB, ws, st);
    case DT_F16: return backward_d<DT_F16>(p, G, X, V, T, K, A, B, scaling, R, N, S, base_grad, gX, gA, gB, ws, st);
    default: return backward_d<DT_BF16>(p, G, X, V, T, K, A, B, scaling, R, N, S, base_grad, gX, gA, gB, ws, st);
  }
}

}  // namespace i8l
