// Input gradient of the experts' products on gfx950 matrix cores:
//   gX[r, k] = D(sum_n fp16(G[r, n]) Wdq[e, n, k]),
//   Wdq[e, n, k] = fp16(CB[e, n, k] * fl32(SCB[e, n] * fl32(1/127)))
// for the rows r of a segment with expert e; the weights are frozen. The
// contraction runs along the rows of CB, so each int8 tile is dequantized once
// per workgroup on its way into LDS, transposed to rows of fp16 along n.
#include <type_traits>

#include "expert.hpp"

namespace i8l {

// Any size and alignment: 128 x 128 tiles, 4 waves of 64 x 64, 64 rows of CB a step.
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void k_expert_bwd(const typename Elem<DT>::T* __restrict__ G, int R, ExpertSegs S,
                                                    const int8_t* __restrict__ CBall, const float* __restrict__ SCBall,
                                                    int N, int K, int slots, int64_t total,
                                                    typename Elem<DT>::T* __restrict__ gX) {
  typedef typename Elem<DT>::T T;
  constexpr int BM = 128, BK = 128, BNC = 64, LDN = BNC + 8, TI = 2, TJ = 2;
  __shared__ __attribute__((aligned(16))) _Float16 sW[BK * LDN], sG[BM * LDN];
  const int64_t bid = expert_block();
  if (bid >= total) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 31, lg = lane >> 5;
  const int wk = wave & 1, wm = wave >> 1;
  int ts, tk;
  tile_coords((int)bid, slots, (K + BK - 1) / BK, ts, tk);
  const ExpertTile tile = expert_tile(S, ts, R, BM);
  if (tile.r0 >= tile.r1) return;
  const int r0 = tile.r0, r1 = tile.r1, k0 = tk * BK;
  const int8_t* CB = CBall + (int64_t)max(tile.expert, 0) * N * K;
  const float* SCB = SCBall + (int64_t)max(tile.expert, 0) * N;

  v16f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v16f{};

  const int nend = tile.expert >= 0 ? N : 0;
  for (int nc = 0; nc < nend; nc += BNC) {
    // G: 8 values a thread, rows tid / 8 + 32 i
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (tid >> 3) + 32 * i, n = nc + (tid & 7) * 8, r = r0 + row;
      v8h h = {};
      if (r < r1) {
        const T* p = G + (int64_t)r * N + n;
        if (VEC && n < N) {
          T v[8];
          load8<DT>(p, v);
#pragma unroll
          for (int x = 0; x < 8; ++x) h[x] = to_half<DT>(v[x]);
        } else if (!VEC) {
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (n + x < N) h[x] = to_half<DT>(p[x]);
        }
      }
      *reinterpret_cast<v8h*>(sG + row * LDN + (tid & 7) * 8) = h;
    }
    // W: 8 rows by 4 columns a thread
    {
      const int kq = tid & 31, ng = tid >> 5;
      uint32_t w[8];
      float sig[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int n = nc + 8 * ng + x, k = k0 + 4 * kq;
        w[x] = 0u;
        sig[x] = 0.0f;
        if (n < N) {
          sig[x] = SCB[n] * (1.0f / 127.0f);
          const int8_t* p = CB + (int64_t)n * K + k;
          if (VEC) {
            if (k < K) w[x] = *reinterpret_cast<const uint32_t*>(p);
          } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
              if (k + b < K) w[x] |= ((uint32_t)(uint8_t)p[b]) << (8 * b);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v8h h;
#pragma unroll
        for (int x = 0; x < 8; ++x) h[x] = half_of_f32((float)(int)(int8_t)(w[x] >> (8 * c)) * sig[x]);
        *reinterpret_cast<v8h*>(sW + (4 * kq + c) * LDN + 8 * ng) = h;
      }
    }
    __syncthreads();
    const _Float16* bW = sW + (wk * 64 + lr) * LDN + lg * 8;
    const _Float16* bG = sG + (wm * 64 + lr) * LDN + lg * 8;
#pragma unroll
    for (int ks = 0; ks < BNC / 16; ++ks) {
      v8h P[TI], V[TJ];
#pragma unroll
      for (int i = 0; i < TI; ++i) P[i] = *reinterpret_cast<const v8h*>(bW + i * 32 * LDN + ks * 16);
#pragma unroll
      for (int j = 0; j < TJ; ++j) V[j] = *reinterpret_cast<const v8h*>(bG + j * 32 * LDN + ks * 16);
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(P[i], V[j], acc[i][j], 0, 0, 0);
    }
    __syncthreads();
  }

#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int r = r0 + wm * 64 + j * 32 + lr;
    if (r >= r1) continue;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = k0 + wk * 64 + i * 32 + q * 8 + lg * 4;
        T* p = gX + (int64_t)r * K + k;
        T v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = Elem<DT>::from_f32(acc[i][j][4 * q + x]);
        if (VEC && k + 3 < K) {
          if constexpr (DT == DT_F32)
            *reinterpret_cast<v4f*>(p) = v4f{v[0], v[1], v[2], v[3]};
          else
            *reinterpret_cast<v2u*>(p) =
                v2u{(uint32_t)__builtin_bit_cast(uint16_t, v[0]) | ((uint32_t)__builtin_bit_cast(uint16_t, v[1]) << 16),
                    (uint32_t)__builtin_bit_cast(uint16_t, v[2]) | ((uint32_t)__builtin_bit_cast(uint16_t, v[3]) << 16)};
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (k + x < K) p[x] = v[x];
        }
      }
  }
}

// Large tiles for 16-bit gradients: 256 rows by BK columns (256, or 128 where
// 256-wide tiles would leave compute units idle), 8 waves (two per SIMD) of 64
// rows by BK / 2, the contraction 64 rows of CB at a time through two swizzled
// LDS stages, as in the projection's own kernel: the next stage's weights and
// gradients are loaded two steps ahead, and converted and written between the
// matrix instructions. Waves whose 64 rows all lie past the segment only move
// and convert tiles. Requires N % 8 == 0, K % 4 == 0 and 32-bit offsets within
// an expert's weight.
template <int DT, int BK>
__global__ __launch_bounds__(512, 1) void k_expert_bwd_w8(const typename Elem<DT>::T* __restrict__ G, int R,
                                                          ExpertSegs S, const int8_t* __restrict__ CBall,
                                                          const float* __restrict__ SCBall, int N, int K, int slots,
                                                          int64_t total, typename Elem<DT>::T* __restrict__ gX) {
  static_assert(DT == DT_F16 || DT == DT_BF16, "16-bit gradients only");
  static_assert(BK == 256 || BK == 128, "256- or 128-wide tiles");
  typedef typename Elem<DT>::T T;
  constexpr int BM = 256, BNC = 64, TI = BK / 64, TJ = 2;
  constexpr int WR = BK / 32;                  // weight rows a lane converts in a step
  constexpr int ROW = BNC * 2;
  constexpr int STAGE = (BK + BM) * ROW, GOFF = BK * ROW;
  extern __shared__ __attribute__((aligned(16))) char bsm[];
  const int64_t bid = expert_block();
  if (bid >= total) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 31, lg = lane >> 5;
  const int wk = wave & 1, wm = wave >> 1;
  int ts, tk;
  tile_coords((int)bid, slots, (K + BK - 1) / BK, ts, tk);
  const ExpertTile tile = expert_tile(S, ts, R, BM);
  if (tile.r0 >= tile.r1) return;
  const int r0 = tile.r0, r1 = tile.r1, k0 = tk * BK;
  const bool has = tile.expert >= 0;
  const int8_t* CB = CBall + (int64_t)max(tile.expert, 0) * N * K;
  const float* SCB = SCBall + (int64_t)max(tile.expert, 0) * N;

  const __amdgpu_buffer_rsrc_t rG = make_rsrc(G + (int64_t)r0 * N, has ? (r1 - r0) * N * 2 : 0);
  const __amdgpu_buffer_rsrc_t rW = make_rsrc(CB + k0, has ? max(0, N * K - k0) : 0);
  const __amdgpu_buffer_rsrc_t rS = make_rsrc(SCB, has ? N * 4 : 0);

  // gradient slots: 16-byte chunk gc of rows grow + 64 i (i < 4)
  const int grow = tid >> 3, gc = tid & 7;
  const int gvoff = grow * N * 2 + 16 * gc;
  const int gwoff = GOFF + grow * ROW + 16 * (gc ^ lds_swz(grow));
  // weights: rows nc + 8 wave + wh .. + WR - 1, bytes 4 kq .. 4 kq + 3
  const int kq = BK == 256 ? (tid & 63) : (tid & 31);
  const int wh = BK == 256 ? 0 : 4 * ((tid >> 5) & 1);
  const int wvoff = 4 * kq + wh * K;
  int wwoff[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int r = 4 * kq + c;
    wwoff[c] = r * ROW + 16 * (wave ^ lds_swz(r)) + 2 * wh;
  }
  const int sw = lds_swz(lr);
  int roff[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) roff[ks] = lr * ROW + 16 * ((2 * ks + lg) ^ sw);
  const int pb = wk * (BK / 2) * ROW, qb = GOFF + wm * 64 * ROW;

  v4u RG[4];
  uint32_t RW[WR];
  float SG[WR];
  auto load_w = [&](int nc) {
    const int n8 = nc + 8 * wave;
#pragma unroll
    for (int e = 0; e < WR; ++e) RW[e] = __builtin_amdgcn_raw_buffer_load_b32(rW, wvoff, (n8 + e) * K, 0);
    // N % 8 == 0: the eight rows from n8 are all in the matrix or all past it
    const int so = (n8 < N) ? 4 * (n8 + wh) : OOB_OFFSET;
#pragma unroll
    for (int h = 0; h < WR / 4; ++h) {
      const v4f sv = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rS, so + 16 * h, 0, 0));
#pragma unroll
      for (int e = 0; e < 4; ++e) SG[4 * h + e] = sv[e];
    }
  };
  auto load_g = [&](int nc) {
    const int gv = (nc + 8 * gc < N) ? gvoff : OOB_OFFSET;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      RG[i] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rG, gv, 2 * nc + 128 * i * N, 0));
  };
  auto write_w = [&](int st, int c0) {
    float sg[WR];
#pragma unroll
    for (int e = 0; e < WR; ++e) sg[e] = SG[e] * (1.0f / 127.0f);
#pragma unroll
    for (int c = c0; c < c0 + 2; ++c) {
      uint32_t h[WR / 2];
#pragma unroll
      for (int e = 0; e < WR / 2; ++e) {
        const float w0 = (float)(int)(int8_t)(RW[2 * e] >> (8 * c));
        const float w1 = (float)(int)(int8_t)(RW[2 * e + 1] >> (8 * c));
        h[e] = f32x2_to_f16x2(w0 * sg[2 * e], w1 * sg[2 * e + 1]);
      }
      if constexpr (WR == 8) *reinterpret_cast<v4u*>(bsm + st * STAGE + wwoff[c]) = v4u{h[0], h[1], h[2], h[3]};
      else *reinterpret_cast<v2u*>(bsm + st * STAGE + wwoff[c]) = v2u{h[0], h[1]};
    }
  };
  auto write_g = [&](int st) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v4u v;
      if constexpr (DT == DT_F16) {
        v = RG[i];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = bf16x2_to_f16x2(RG[i][e]);
      }
      *reinterpret_cast<v4u*>(bsm + st * STAGE + gwoff + i * 64 * ROW) = v;
    }
  };

  v16f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v16f{};
  v8h F[2][TI + TJ];
  auto fread = [&](int st, int ks, int b) {
    const char* base = bsm + st * STAGE + roff[ks];
#pragma unroll
    for (int i = 0; i < TI; ++i) F[b][i] = *reinterpret_cast<const v8h*>(base + pb + i * 32 * ROW);
#pragma unroll
    for (int j = 0; j < TJ; ++j) F[b][TI + j] = *reinterpret_cast<const v8h*>(base + qb + j * 32 * ROW);
  };
  auto mma = [&](int b) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(F[b][i], F[b][TI + j], acc[i][j], 0, 0, 0);
  };
  // every matrix instruction of a phase is followed by four conversions, then by its share of the memory work
  auto spread = [&](auto dsr, auto dsw, auto vm) {
    constexpr int Rd = decltype(dsr)::value, Wr = decltype(dsw)::value, Gl = decltype(vm)::value;
#pragma unroll
    for (int q = 0; q < TI * TJ; ++q) {
      I8L_SGB(SG_MFMA, 1);
      I8L_SGB(SG_VALU, 4);
      if (q < Rd) I8L_SGB(SG_DS_R, 1);
      if (q < Wr) I8L_SGB(SG_DS_W, 1);
      if (q < Gl) I8L_SGB(SG_VMEM_R, 1);
    }
  };

  const int nn = has ? (N + BNC - 1) / BNC : 0;
  load_w(0);
  load_g(0);
  write_w(0, 0);
  write_w(0, 2);
  write_g(0);
  load_w(BNC);
  load_g(BNC);
  __syncthreads();
  if (r0 + wm * 64 < r1) {
    fread(0, 0, 0);
    for (int t = 0; t < nn; ++t) {
      const int st = t & 1;
      const int nc2 = (t + 2) * BNC;   // past the end: zeros
      fread(st, 1, 1);
      write_w(st ^ 1, 0);
      mma(0);
      spread(std::integral_constant<int, TI + TJ>{}, std::integral_constant<int, 2>{},
             std::integral_constant<int, 0>{});
      __builtin_amdgcn_sched_barrier(0);
      fread(st, 2, 0);
      write_w(st ^ 1, 2);
      load_w(nc2);
      mma(1);
      spread(std::integral_constant<int, TI + TJ>{}, std::integral_constant<int, 2>{},
             std::integral_constant<int, WR + WR / 4>{});
      __builtin_amdgcn_sched_barrier(0);
      fread(st, 3, 1);
      write_g(st ^ 1);
      load_g(nc2);
      mma(0);
      spread(std::integral_constant<int, TI + TJ>{}, std::integral_constant<int, 4>{},
             std::integral_constant<int, 4>{});
      __builtin_amdgcn_sched_barrier(0);
      mma(1);
      __syncthreads();
      fread(st ^ 1, 0, 0);
    }
  } else {
    for (int t = 0; t < nn; ++t) {
      const int st = t & 1;
      const int nc2 = (t + 2) * BNC;
      write_w(st ^ 1, 0);
      write_w(st ^ 1, 2);
      load_w(nc2);
      write_g(st ^ 1);
      load_g(nc2);
      __syncthreads();
    }
  }

  // lane (lr, lg), register r of tile (i, j): column wk BK / 2 + i 32 + (r / 4) 8 + lg 4 + r % 4, row wm 64 + j 32 + lr;
  // through LDS, stored as whole rows
  __syncthreads();   // every wave is done with the operand stages
#pragma unroll
  for (int j = 0; j < TJ; ++j)
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v2u w;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          w[e] = (uint32_t)__builtin_bit_cast(uint16_t, Elem<DT>::from_f32(acc[i][j][4 * q + 2 * e])) |
                 ((uint32_t)__builtin_bit_cast(uint16_t, Elem<DT>::from_f32(acc[i][j][4 * q + 2 * e + 1])) << 16);
        *reinterpret_cast<v2u*>(bsm + otile_off(wm * 64 + j * 32 + lr, wk * (BK / 16) + i * 4 + q) + 8 * lg) = w;
      }
  __syncthreads();
  otile_store<T>(bsm, gX, K, r0, k0, r1, min(K, k0 + BK), wave, lane);
}

template <int DT, int BK>
static hipError_t launch_bwd_w8(const void* G, int R, const ExpertSegs& S, const int8_t* CB, const float* SCB, int N,
                                int K, void* gX, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  constexpr size_t stages = (size_t)2 * (BK + 256) * 128, otile = (size_t)256 * 512;
  constexpr size_t lds = stages > otile ? stages : otile;
  auto kern = k_expert_bwd_w8<DT, BK>;
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t e = lds_limit_once((const void*)kern, (int)lds, lds_set);
  if (e != hipSuccess) return e;
  const int64_t slots = expert_slots(R, S.n_seg, 256), total = slots * ((K + BK - 1) / BK);
  hipLaunchKernelGGL(kern, expert_grid(total), dim3(512), lds, st, static_cast<const E*>(G), R, S, CB, SCB, N, K,
                     (int)slots, total, static_cast<E*>(gX));
  return hipGetLastError();
}

template <int DT>
static hipError_t launch_bwd_t(const void* G, int R, const ExpertSegs& S, const int8_t* CB, const float* SCB, int N,
                               int K, void* gX, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  const bool vec = N % 8 == 0 && K % 4 == 0 && (uintptr_t)G % 16 == 0 && (uintptr_t)CB % 4 == 0 &&
                   (uintptr_t)gX % (4 * sizeof(E)) == 0;
  if constexpr (DT != DT_F32) {
    const bool fits = (N + (int64_t)128) * K < ((int64_t)1 << 31) - 4096 && (int64_t)N * 512 < ((int64_t)1 << 31) - 4096;
    if (vec && N > 0 && fits && R >= 128 * (int64_t)S.n_seg && R >= 512) {
      // 256-wide tiles, unless they would fill at most half of the chip
      const int64_t tiles = (R + 255) / 256 * (int64_t)((K + 255) / 256);
      if (tiles > 128) return launch_bwd_w8<DT, 256>(G, R, S, CB, SCB, N, K, gX, st);
      if (tiles >= 32) return launch_bwd_w8<DT, 128>(G, R, S, CB, SCB, N, K, gX, st);
    }
  }
  const int64_t slots = expert_slots(R, S.n_seg, 128), total = slots * ((K + 127) / 128);
  auto kern = vec ? k_expert_bwd<DT, true> : k_expert_bwd<DT, false>;
  hipLaunchKernelGGL(kern, expert_grid(total), dim3(256), 0, st, static_cast<const E*>(G), R, S, CB, SCB, N, K,
                     (int)slots, total, static_cast<E*>(gX));
  return hipGetLastError();
}

hipError_t launch_expert_bwd(int dt, const void* G, int R, const ExpertSegs& S, const int8_t* CB, const float* SCB,
                             int N, int K, void* gX, hipStream_t st) {
  if (dt == DT_F32) return launch_bwd_t<DT_F32>(G, R, S, CB, SCB, N, K, gX, st);
  if (dt == DT_F16) return launch_bwd_t<DT_F16>(G, R, S, CB, SCB, N, K, gX, st);
  return launch_bwd_t<DT_BF16>(G, R, S, CB, SCB, N, K, gX, st);
}

}  // namespace i8l
