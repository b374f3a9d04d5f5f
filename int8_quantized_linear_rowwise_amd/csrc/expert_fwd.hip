// Products of each expert's rows with its int8 weight on gfx950 matrix cores.
//
// The tokens are quantized once (row scales SCA, outlier columns O over all of
// them); row r of a segment with expert e is token t = rows[r]:
//   y[r, n] = C32[r, n] SCA[t] SCB[e, n] / 127^2 + sum_j A16[t, O[j]] Wdq[e, n, O[j]]
//   out = D(y),  C32 = CA[t] . CB[e, n] exact in int32,
//   Wdq[e, n, k] = fp16(CB[e, n, k] * (SCB[e, n] * (1/127)))
// As in the projection's own forward the product is computed transposed (the
// weights on the matrix core's row side), so that a lane owns four
// consecutive features of one row.
#include "expert.hpp"

namespace i8l {

// Any size and alignment: 128 x 128 tiles, 4 waves of 64 x 64, 64 bytes of the
// contraction a step.
template <int DT, bool KV, bool OV>
__global__ __launch_bounds__(256) void k_expert_fwd(ExpertQuantized Q, const typename Elem<DT>::T* __restrict__ X,
                                                    int T, const int32_t* __restrict__ rows, int R, ExpertSegs S,
                                                    const int8_t* __restrict__ CBall, const float* __restrict__ SCBall,
                                                    int N, int K, int slots, int64_t total,
                                                    typename Elem<DT>::T* __restrict__ out) {
  constexpr int BM = 128, BN = 128, BK = 64, LDK = BK + 16, TI = 2, TJ = 2;
  __shared__ __attribute__((aligned(16))) int8_t smem[2 * (BM + BN) * LDK];
  int8_t* sB = smem;
  int8_t* sA = smem + 2 * BN * LDK;
  const int64_t bid = expert_block();
  if (bid >= total) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 31, lg = lane >> 5;
  const int wn = wave & 1, wm = wave >> 1;
  int ts, tn;
  tile_coords((int)bid, slots, (N + BN - 1) / BN, ts, tn);
  const ExpertTile tile = expert_tile(S, ts, R, BM);
  if (tile.r0 >= tile.r1) return;
  const int r0 = tile.r0, r1 = tile.r1, n0 = tn * BN;
  const int e = max(tile.expert, 0);
  const int8_t* CB = CBall + (int64_t)e * N * K;
  const float* SCB = SCBall + (int64_t)e * N;

  // two 16-byte chunks of either tile a thread: rows tid / 4 and tid / 4 + 64
  const int row = tid >> 2, col = (tid & 3) * 16;
  int tok[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + row + 64 * i;
    tok[i] = (r < r1 && tile.expert >= 0) ? row_token(rows, r, T) : -1;
  }
  v4i pre[4];
  auto chunk = [&](const int8_t* p, int k) {
    v4i v = {0, 0, 0, 0};
    if constexpr (KV) {
      if (k < K) v = *reinterpret_cast<const v4i*>(p + k);
    } else {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int b = 0; b < 16; ++b)
        if (k + b < K) w[b >> 2] |= ((uint32_t)(uint8_t)p[k + b]) << (8 * (b & 3));
      v = v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
    }
    return v;
  };
  auto gload = [&](int kt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = n0 + row + 64 * i;
      pre[i] = (n < N && tile.expert >= 0) ? chunk(CB + (int64_t)n * K, kt + col) : v4i{0, 0, 0, 0};
      pre[2 + i] = tok[i] >= 0 ? chunk(Q.CA + (int64_t)tok[i] * K, kt + col) : v4i{0, 0, 0, 0};
    }
  };
  auto sstore = [&](int buf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<v4i*>(sB + (buf * BN + row + 64 * i) * LDK + col) = pre[i];
      *reinterpret_cast<v4i*>(sA + (buf * BM + row + 64 * i) * LDK + col) = pre[2 + i];
    }
  };

  v16i acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v16i{};
  const int nk = (K + BK - 1) / BK;
  if (nk > 0) {
    gload(0);
    sstore(0);
    __syncthreads();
  }
  for (int kt = 0; kt < nk; ++kt) {
    const int cur = kt & 1;
    if (kt + 1 < nk) gload((kt + 1) * BK);
    const int8_t* bB = sB + (cur * BN + wn * 64 + lr) * LDK + lg * 16;
    const int8_t* bA = sA + (cur * BM + wm * 64 + lr) * LDK + lg * 16;
#pragma unroll
    for (int ks = 0; ks < BK / 32; ++ks) {
      v4i P[TI], V[TJ];
#pragma unroll
      for (int i = 0; i < TI; ++i) P[i] = *reinterpret_cast<const v4i*>(bB + i * 32 * LDK + ks * 32);
#pragma unroll
      for (int j = 0; j < TJ; ++j) V[j] = *reinterpret_cast<const v4i*>(bA + j * 32 * LDK + ks * 32);
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(P[i], V[j], acc[i][j], 0, 0, 0);
    }
    if (kt + 1 < nk) sstore(cur ^ 1);
    __syncthreads();
  }

  // lane (lr, lg), register r of tile (i, j): feature n0 + wn 64 + i 32 + (r / 4) 8 + lg 4 + r % 4, row
  // r0 + wm 64 + j 32 + lr
  const int cnt = *Q.count;
  int mt[TJ];
  float sa[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int r = r0 + wm * 64 + j * 32 + lr;
    mt[j] = (r < r1 && tile.expert >= 0) ? row_token(rows, r, T) : -1;
    sa[j] = mt[j] >= 0 ? Q.SCA[mt[j]] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int nb = n0 + wn * 64 + i * 32;
    v16f y[TJ];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int n = nb + (r >> 2) * 8 + lg * 4 + (r & 3);
      const float sb = (n < N && tile.expert >= 0) ? SCB[n] * (1.0f / 16129.0f) : 0.0f;
#pragma unroll
      for (int j = 0; j < TJ; ++j) y[j][r] = (float)acc[i][j][r] * (sa[j] * sb);
    }
    for (int jo = 0; jo < cnt; jo += 16) {
      const int n = nb + lr;
      const v8h P = expert_out_w8(CB, SCB, K, Q.idx, n, n < N && tile.expert >= 0, jo + lg * 8, cnt);
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const v8h V = expert_out_a8<DT>(Q.sub, Q.cap, X, K, Q.idx, mt[j], jo + lg * 8, cnt);
        y[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(P, V, y[j], 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int r = r0 + wm * 64 + j * 32 + lr;
      if (r >= r1) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = nb + q * 8 + lg * 4;
        typename Elem<DT>::T* p = out + (int64_t)r * N + n;
        typename Elem<DT>::T v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = Elem<DT>::from_f32(y[j][4 * q + x]);
        if (OV && n + 3 < N) {
          if constexpr (DT == DT_F32)
            *reinterpret_cast<v4f*>(p) = v4f{v[0], v[1], v[2], v[3]};
          else
            *reinterpret_cast<v2u*>(p) =
                v2u{(uint32_t)__builtin_bit_cast(uint16_t, v[0]) | ((uint32_t)__builtin_bit_cast(uint16_t, v[1]) << 16),
                    (uint32_t)__builtin_bit_cast(uint16_t, v[2]) | ((uint32_t)__builtin_bit_cast(uint16_t, v[3]) << 16)};
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (n + x < N) p[x] = v[x];
        }
      }
    }
  }
}

template <int DT>
static hipError_t launch_fwd_t(const ExpertQuantized& Q, const void* X, int T, const int32_t* rows, int R,
                               const ExpertSegs& S, const int8_t* CB, const float* SCB, int N, int K, void* out,
                               hipStream_t st) {
  typedef typename Elem<DT>::T E;
  const bool kv = K % 16 == 0 && (uintptr_t)CB % 16 == 0;
  const bool ov = N % 4 == 0 && (uintptr_t)out % (4 * sizeof(E)) == 0;
  const int64_t slots = expert_slots(R, S.n_seg, 128), total = slots * ((N + 127) / 128);
  auto kern = kv ? (ov ? k_expert_fwd<DT, true, true> : k_expert_fwd<DT, true, false>)
                 : (ov ? k_expert_fwd<DT, false, true> : k_expert_fwd<DT, false, false>);
  hipLaunchKernelGGL(kern, expert_grid(total), dim3(256), 0, st, Q, static_cast<const E*>(X), T, rows, R, S, CB, SCB, N,
                     K, (int)slots, total, static_cast<E*>(out));
  return hipGetLastError();
}

hipError_t launch_expert_fwd(int dt, const ExpertQuantized& Q, const void* X, int T, const int32_t* rows, int R,
                             const ExpertSegs& S, const int8_t* CB, const float* SCB, int N, int K, void* out,
                             hipStream_t st) {
  if (dt == DT_F32) return launch_fwd_t<DT_F32>(Q, X, T, rows, R, S, CB, SCB, N, K, out, st);
  if (dt == DT_F16) return launch_fwd_t<DT_F16>(Q, X, T, rows, R, S, CB, SCB, N, K, out, st);
  return launch_fwd_t<DT_BF16>(Q, X, T, rows, R, S, CB, SCB, N, K, out, st);
}

}  // namespace i8l
