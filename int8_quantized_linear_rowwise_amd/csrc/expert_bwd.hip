// Input gradient of the experts' products on gfx950 matrix cores:
//   gX[r, k] = D(sum_n fp16(G[r, n]) Wdq[e, n, k]),
//   Wdq[e, n, k] = fp16(CB[e, n, k] * fl32(SCB[e, n] * fl32(1/127)))
// for the rows r of a segment with expert e; the weights are frozen. The
// contraction runs along the rows of CB, so each int8 tile is dequantized once
// per workgroup on its way into LDS, transposed to rows of fp16 along n.
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

template <int DT>
static hipError_t launch_bwd_t(const void* G, int R, const ExpertSegs& S, const int8_t* CB, const float* SCB, int N,
                               int K, void* gX, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  const bool vec = N % 8 == 0 && K % 4 == 0 && (uintptr_t)G % 16 == 0 && (uintptr_t)CB % 4 == 0 &&
                   (uintptr_t)gX % (4 * sizeof(E)) == 0;
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
