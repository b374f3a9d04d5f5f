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
#include <stdlib.h>
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
      v = bytes16(p, k, K);
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

// Large tiles: 256 rows by BN features (256, or 128 where 256-wide tiles would
// leave compute units idle), 8 waves (two per SIMD) of 64 rows by BN / 2, the
// contraction 128 bytes at a time through two swizzled LDS stages, as in the
// projection's own kernel; registers hold the next step's tiles. The rows of
// the activation tile are gathered: a lane keeps the offsets of its four
// tokens, so the gather costs nothing in the loop. Waves whose 64 rows all lie
// past the segment only move tiles: a tile of 100 rows takes about half the
// time of a full one. Requires K % 16 == 0 and codes of less than 2^31 bytes.
constexpr int EF_OPAN = 2 * 256 * 32;                 // outlier panels P[n][16], Q[row][16] (fp16)
constexpr int EF_SCALES = (256 + 256) * 4;            // SCB / 127^2, SCA
template <int DT, int BN>
__global__ __launch_bounds__(512, 1) void k_expert_fwd_w8(ExpertQuantized Q, const typename Elem<DT>::T* __restrict__ X,
                                                          int T, const int32_t* __restrict__ rows, int R, ExpertSegs S,
                                                          const int8_t* __restrict__ CBall,
                                                          const float* __restrict__ SCBall, int N, int K, int slots,
                                                          int64_t total, typename Elem<DT>::T* __restrict__ out) {
  static_assert(BN == 256 || BN == 128, "256- or 128-wide tiles");
  constexpr int BM = 256, BK = 128, TI = BN / 64, TJ = 2;
  constexpr int NB = BN / 64;
  constexpr int STAGE = (BM + BN) * BK, AOFF = BN * BK;
  constexpr int OT = 256 * 512;
  constexpr int BASE = 2 * STAGE > OT ? 2 * STAGE : OT;
  extern __shared__ __attribute__((aligned(16))) int8_t smem[];
  const int64_t bid = expert_block();
  if (bid >= total) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 31, lg = lane >> 5;
  const int wn = wave & 1, wm = wave >> 1;
  int ts, tn;
  tile_coords((int)bid, slots, (N + BN - 1) / BN, ts, tn);
  const ExpertTile tile = expert_tile(S, ts, R, BM);
  if (tile.r0 >= tile.r1) return;
  const int r0 = tile.r0, r1 = tile.r1, n0 = tn * BN;
  const bool has = tile.expert >= 0;
  const int8_t* CB = CBall + (int64_t)max(tile.expert, 0) * N * K;
  const float* SCB = SCBall + (int64_t)max(tile.expert, 0) * N;

  const __amdgpu_buffer_rsrc_t rA = make_rsrc(Q.CA, T * K);
  const __amdgpu_buffer_rsrc_t rB = make_rsrc(CB + (int64_t)n0 * K, has ? min(BN, N - n0) * K : 0);
  const int lrow = tid >> 3, lc = tid & 7;
  const int voff = lrow * K + 16 * lc;
  const int woff = lrow * BK + 16 * (lc ^ lds_swz(lrow));
  const int sw = lds_swz(lr);
  int roff[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) roff[ks] = lr * BK + 16 * ((2 * ks + lg) ^ sw);
  const int pb = wn * (BN / 2) * BK, qb = AOFF + wm * 64 * BK;

  v4u RB[NB], RA[4];
  auto load_b = [&](int kt) {
    const int v = (kt + 16 * lc < K) ? voff : OOB_OFFSET;
#pragma unroll
    for (int i = 0; i < NB; ++i)
      RB[i] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rB, v, kt + 64 * i * K, 0));
  };
  load_b(0);
  int aoff[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + lrow + 64 * i;
    const int t = (has && r < r1) ? row_token(rows, r, T) : -1;
    aoff[i] = t >= 0 ? t * K + 16 * lc : OOB_OFFSET;
  }
  auto load_a = [&](int kt) {
    const bool in = kt + 16 * lc < K;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      RA[i] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rA, in ? aoff[i] : OOB_OFFSET, kt, 0));
  };
  auto write_b = [&](int st) {
#pragma unroll
    for (int i = 0; i < NB; ++i) *reinterpret_cast<v4u*>(smem + st * STAGE + woff + i * 64 * BK) = RB[i];
  };
  auto write_a = [&](int st) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<v4u*>(smem + st * STAGE + AOFF + woff + i * 64 * BK) = RA[i];
  };
  load_a(0);

  // the tile's scales and tokens, and the panels of the first 16 outlier
  // columns, while the first operand tiles are in flight
  char* opan = reinterpret_cast<char*>(smem) + BASE;
  float* lsb = reinterpret_cast<float*>(opan + EF_OPAN);
  float* lsa = lsb + 256;
  const int cnt = has ? *Q.count : 0;
  const int orow = tid >> 1, oj = (tid & 1) * 8;
  v8h opP = {}, opQ = {};
  auto panels = [&](int jo) {
    const int n = n0 + orow, r = r0 + orow;
    opP = expert_out_w8(CB, SCB, K, Q.idx, n, orow < BN && n < N, jo + oj, cnt);
    opQ = expert_out_a8<DT>(Q.sub, Q.cap, X, K, Q.idx, (has && r < r1) ? row_token(rows, r, T) : -1, jo + oj, cnt);
  };
  auto put_panels = [&]() {
    *reinterpret_cast<v8h*>(opan + orow * 32 + oj * 2) = opP;
    *reinterpret_cast<v8h*>(opan + EF_OPAN / 2 + orow * 32 + oj * 2) = opQ;
  };
  if (cnt > 0) panels(0);
  if (tid < 256) {
    const int n = n0 + tid;
    lsb[tid] = (has && tid < BN && n < N) ? SCB[n] * (1.0f / 16129.0f) : 0.0f;
  } else {
    const int r = r0 + tid - 256;
    const int t = (has && r < r1) ? row_token(rows, r, T) : -1;
    lsa[tid - 256] = t >= 0 ? Q.SCA[t] : 0.0f;
  }

  v16i acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v16i{};
  v4i F[2][TI + TJ];
  auto fread = [&](int st, int ks, int b) {
    const int8_t* base = smem + st * STAGE + roff[ks];
#pragma unroll
    for (int i = 0; i < TI; ++i) F[b][i] = *reinterpret_cast<const v4i*>(base + pb + i * 32 * BK);
#pragma unroll
    for (int j = 0; j < TJ; ++j) F[b][TI + j] = *reinterpret_cast<const v4i*>(base + qb + j * 32 * BK);
  };
  auto mma = [&](int b) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(F[b][i], F[b][TI + j], acc[i][j], 0, 0, 0);
  };
  const int nk = has ? (K + BK - 1) / BK : 0;
  write_b(0);
  write_a(0);
  load_b(BK);
  load_a(BK);
  if (cnt > 0) put_panels();
  __syncthreads();
  if (r0 + wm * 64 < r1) {
    fread(0, 0, 0);
    for (int kt = 0; kt < nk; ++kt) {
      const int st = kt & 1;
      const int k2 = (kt + 2) * BK;    // past the end: zeros
      fread(st, 1, 1);
      write_b(st ^ 1);
      load_b(k2);
      mma(0);
#pragma unroll
      for (int q = 0; q < TI * TJ; ++q) {
        I8L_SGB(SG_MFMA, 1);
        if (q < TI + TJ) I8L_SGB(SG_DS_R, 1);
        if (q < NB) {
          I8L_SGB(SG_DS_W, 1);
          I8L_SGB(SG_VMEM_R, 1);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      fread(st, 2, 0);
      write_a(st ^ 1);
      load_a(k2);
      mma(1);
#pragma unroll
      for (int q = 0; q < TI * TJ; ++q) {
        I8L_SGB(SG_MFMA, 1);
        if (q < TI + TJ) I8L_SGB(SG_DS_R, 1);
        if (q < 4) {
          I8L_SGB(SG_DS_W, 1);
          I8L_SGB(SG_VMEM_R, 1);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      fread(st, 3, 1);
      mma(0);
#pragma unroll
      for (int q = 0; q < TI * TJ; ++q) {
        I8L_SGB(SG_MFMA, 1);
        if (q < TI + TJ) I8L_SGB(SG_DS_R, 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      mma(1);
      __syncthreads();
      fread(st ^ 1, 0, 0);
    }
  } else {
    for (int kt = 0; kt < nk; ++kt) {
      const int k2 = (kt + 2) * BK;
      write_b((kt & 1) ^ 1);
      load_b(k2);
      write_a((kt & 1) ^ 1);
      load_a(k2);
      __syncthreads();
    }
  }

  // lane (lr, lg), register r of tile (i, j): feature wn BN / 2 + i 32 + (r / 4) 8 + lg 4 + r % 4, row wm 64 + j 32 + lr
  const int nl = wn * (BN / 2), ml = wm * 64;
  // the accumulators become fp32 in place
#pragma unroll
  for (int i = 0; i < TI; ++i) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const v4f sb = *reinterpret_cast<const v4f*>(lsb + nl + i * 32 + q * 8 + lg * 4);
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const float sa = lsa[ml + j * 32 + lr];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          acc[i][j][4 * q + x] = __float_as_int((float)acc[i][j][4 * q + x] * (sa * sb[x]));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int jo = 0; jo < cnt; jo += 16) {
    if (jo > 0) {
      panels(jo);
      __syncthreads();
      put_panels();
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const v8h P = *reinterpret_cast<const v8h*>(opan + (nl + i * 32 + lr) * 32 + lg * 16);
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const v8h V = *reinterpret_cast<const v8h*>(opan + EF_OPAN / 2 + (ml + j * 32 + lr) * 32 + lg * 16);
        acc[i][j] = __builtin_bit_cast(
            v16i, __builtin_amdgcn_mfma_f32_32x32x16_f16(P, V, __builtin_bit_cast(v16f, acc[i][j]), 0, 0, 0));
      }
    }
  }
  if constexpr (DT == DT_F32) {
    const bool ov = N % 4 == 0 && (uintptr_t)out % 16 == 0;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int r = r0 + ml + j * 32 + lr;
      if (r >= r1) continue;
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + nl + i * 32 + q * 8 + lg * 4;
          int* p = reinterpret_cast<int*>(out) + (int64_t)r * N + n;
          if (ov && n + 3 < N) {
            *reinterpret_cast<v4i*>(p) =
                v4i{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          } else {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (n + x < N) p[x] = acc[i][j][4 * q + x];
          }
        }
    }
  } else {
    // through LDS, stored as whole rows of the tile's columns
    char* ot = reinterpret_cast<char*>(smem);
    __syncthreads();   // the operand stages are no longer read
#pragma unroll
    for (int i = 0; i < TI; ++i) {
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v2u w;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float a = __int_as_float(acc[i][j][4 * q + 2 * x]), b = __int_as_float(acc[i][j][4 * q + 2 * x + 1]);
            w[x] = (uint32_t)__builtin_bit_cast(uint16_t, Elem<DT>::from_f32(a)) |
                   ((uint32_t)__builtin_bit_cast(uint16_t, Elem<DT>::from_f32(b)) << 16);
          }
          *reinterpret_cast<v2u*>(ot + otile_off(ml + j * 32 + lr, (nl + i * 32 + q * 8) >> 3) + 8 * lg) = w;
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
    otile_store<typename Elem<DT>::T>(ot, out, N, r0, n0, r1, min(N, n0 + BN), wave, lane);
  }
}

template <int DT, int BN>
static hipError_t launch_fwd_w8(const ExpertQuantized& Q, const void* X, int T, const int32_t* rows, int R,
                                const ExpertSegs& S, const int8_t* CB, const float* SCB, int N, int K, void* out,
                                hipStream_t st) {
  typedef typename Elem<DT>::T E;
  constexpr size_t stages = (size_t)2 * (256 + BN) * 128, otile = (size_t)256 * 512;
  constexpr size_t lds = (stages > otile ? stages : otile) + EF_OPAN + EF_SCALES;
  auto kern = k_expert_fwd_w8<DT, BN>;
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t e = lds_limit_once((const void*)kern, (int)lds, lds_set);
  if (e != hipSuccess) return e;
  const int64_t slots = expert_slots(R, S.n_seg, 256), total = slots * ((N + BN - 1) / BN);
  hipLaunchKernelGGL(kern, expert_grid(total), dim3(512), lds, st, Q, static_cast<const E*>(X), T, rows, R, S, CB, SCB,
                     N, K, (int)slots, total, static_cast<E*>(out));
  return hipGetLastError();
}

// Few rows an expert: tiles of 16 MT rows by 16 features, bound by reading the
// weights once. Four waves share a tile's contraction, 512 bytes of every row
// at a time: a wave brings its 16 weight rows of 512 bytes into LDS with lanes
// side by side on a row (straight from memory into the matrix operands' layout,
// 16 rows a request, a compute unit gets only one request a nanosecond),
// 16-byte pieces p of row r at p ^ r, and reads them as operands; the
// codes, few and shared by all tiles of the expert, come from L2 in the
// operands' layout. No barrier until the waves' int32 sums meet in LDS (exact,
// so their order is nothing to the result).
// Requires K % 16 == 0.
typedef __attribute__((address_space(3))) void* lds_ptr;
constexpr int ET_KC = 512;      // bytes of a row a wave takes at a time
template <int DT, int MT>
__global__ __launch_bounds__(256) void k_expert_fwd_thin(ExpertQuantized Q, const typename Elem<DT>::T* __restrict__ X,
                                                         int T, const int32_t* __restrict__ rows, int R, ExpertSegs S,
                                                         const int8_t* __restrict__ CBall,
                                                         const float* __restrict__ SCBall, int N, int K, int tiles_n,
                                                         int64_t total, typename Elem<DT>::T* __restrict__ out) {
  typedef typename Elem<DT>::T E;
  constexpr int BM = 16 * MT, BN = 16, STEPS = ET_KC / 64;
  __shared__ __attribute__((aligned(1024))) int8_t sw[4][BN * ET_KC];
  const int64_t bid = expert_block();
  if (bid >= total) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int ts = (int)(bid / tiles_n), n0 = (int)(bid - (int64_t)ts * tiles_n) * BN;
  const ExpertTile tile = expert_tile(S, ts, R, BM);
  if (tile.r0 >= tile.r1) return;
  const bool has = tile.expert >= 0;
  const int8_t* CB = CBall + (int64_t)max(tile.expert, 0) * N * K;
  const float* SCB = SCBall + (int64_t)max(tile.expert, 0) * N;
  const __amdgpu_buffer_rsrc_t rB = make_rsrc(CB + (int64_t)n0 * K, has ? min(BN, N - n0) * K : 0);
  const int nc = has ? (K + ET_KC - 1) / ET_KC : 0;

  int8_t* mine = sw[wave];
  auto load_w = [&](int c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 2 * i + (lane >> 5);
      const int k = c * ET_KC + 16 * ((lane & 31) ^ row);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_ptr)(mine + i * 1024), 16,
                                               k < K ? row * K + k : OOB_OFFSET, 0, 0, 0);
    }
  };
  if (wave < nc) load_w(wave);

  int tok[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int r = tile.r0 + 16 * j + lr;
    tok[j] = (has && r < tile.r1) ? row_token(rows, r, T) : -1;
  }
  // wave j finishes tile j: what it needs for that is requested before the contraction
  const int r = tile.r0 + 16 * wave + lr;      // its token's row
  const int nb = n0 + 4 * lg;
  int t = -1, cnt = 0;
  float sa = 0.0f, sb[4] = {};
  v8h P = {}, V = {};
  if (wave < MT && has) {
    t = r < tile.r1 ? row_token(rows, r, T) : -1;
    cnt = *Q.count;
    if (t >= 0) sa = Q.SCA[t];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (nb + x < N) sb[x] = SCB[nb + x];
    if (cnt > 0) {
      P = expert_out_w8(CB, SCB, K, Q.idx, n0 + lr, n0 + lr < N, lg * 8, cnt);
      V = expert_out_a8<DT>(Q.sub, Q.cap, X, K, Q.idx, t, lg * 8, cnt);
    }
  }
  v4i acc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) acc[j] = v4i{0, 0, 0, 0};
  for (int c = wave; c < nc; c += 4) {
    v4i a[STEPS][MT];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int k = c * ET_KC + s * 64 + lg * 16;
        a[s][j] = v4i{0, 0, 0, 0};
        if (tok[j] >= 0 && k < K) a[s][j] = *reinterpret_cast<const v4i*>(Q.CA + (int64_t)tok[j] * K + k);
      }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const v4i w = *reinterpret_cast<const v4i*>(mine + lr * ET_KC + 16 * ((4 * s + lg) ^ lr));
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a[s][j], acc[j], 0, 0, 0);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the next piece lands in the same place
    if (c + 4 < nc) load_w(c + 4);
  }

  // lane (lr, lg): token lr of tile j, features n0 + 4 lg .. + 3
  v4i* part = reinterpret_cast<v4i*>(sw[0]);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < MT; ++j) part[(wave * MT + j) * 64 + lane] = acc[j];
  __syncthreads();
  if (wave >= MT) return;
  v4i sum = part[wave * 64 + lane];
#pragma unroll
  for (int w = 1; w < 4; ++w) sum += part[(w * MT + wave) * 64 + lane];
  v4f y;
#pragma unroll
  for (int x = 0; x < 4; ++x) y[x] = (float)sum[x] * (sa * (sb[x] * (1.0f / 16129.0f)));
  if (cnt > 0) y = __builtin_amdgcn_mfma_f32_16x16x32_f16(P, V, y, 0, 0, 0);
  for (int jo = 32; jo < cnt; jo += 32) {
    P = expert_out_w8(CB, SCB, K, Q.idx, n0 + lr, n0 + lr < N, jo + lg * 8, cnt);
    V = expert_out_a8<DT>(Q.sub, Q.cap, X, K, Q.idx, t, jo + lg * 8, cnt);
    y = __builtin_amdgcn_mfma_f32_16x16x32_f16(P, V, y, 0, 0, 0);
  }
  if (r < tile.r1) {
    E* p = out + (int64_t)r * N + nb;
    const bool ov = N % 4 == 0 && (uintptr_t)out % (4 * sizeof(E)) == 0;
    E v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = Elem<DT>::from_f32(y[x]);
    if (ov && nb + 3 < N) {
      if constexpr (DT == DT_F32)
        *reinterpret_cast<v4f*>(p) = y;
      else
        *reinterpret_cast<v2u*>(p) =
            v2u{(uint32_t)__builtin_bit_cast(uint16_t, v[0]) | ((uint32_t)__builtin_bit_cast(uint16_t, v[1]) << 16),
                (uint32_t)__builtin_bit_cast(uint16_t, v[2]) | ((uint32_t)__builtin_bit_cast(uint16_t, v[3]) << 16)};
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (nb + x < N) p[x] = v[x];
    }
  }
}

template <int DT, int MT>
static hipError_t launch_fwd_thin(const ExpertQuantized& Q, const void* X, int T, const int32_t* rows, int R,
                                  const ExpertSegs& S, const int8_t* CB, const float* SCB, int N, int K, void* out,
                                  hipStream_t st) {
  typedef typename Elem<DT>::T E;
  const int tiles_n = (N + 15) / 16;
  const int64_t total = expert_slots(R, S.n_seg, 16 * MT) * tiles_n;
  hipLaunchKernelGGL((k_expert_fwd_thin<DT, MT>), expert_grid(total), dim3(256), 0, st, Q, static_cast<const E*>(X), T,
                     rows, R, S, CB, SCB, N, K, tiles_n, total, static_cast<E*>(out));
  return hipGetLastError();
}

template <int DT>
static hipError_t launch_fwd_t(const ExpertQuantized& Q, const void* X, int T, const int32_t* rows, int R,
                               const ExpertSegs& S, const int8_t* CB, const float* SCB, int N, int K, void* out,
                               hipStream_t st) {
  typedef typename Elem<DT>::T E;
  const bool kv = K % 16 == 0 && (uintptr_t)CB % 16 == 0;
  const bool ov = N % 4 == 0 && (uintptr_t)out % (4 * sizeof(E)) == 0;
  const char* th = getenv("I8L_THIN");
  const int64_t thin = th ? atoi(th) : 16;
  const char* tm = getenv("I8L_THINMT");
  if (kv && R <= thin * S.n_seg) {
    if (tm && atoi(tm) == 2) return launch_fwd_thin<DT, 2>(Q, X, T, rows, R, S, CB, SCB, N, K, out, st);
    return launch_fwd_thin<DT, 1>(Q, X, T, rows, R, S, CB, SCB, N, K, out, st);
  }
  if (kv && (int64_t)T * K < ((int64_t)1 << 31) && R >= 128 * (int64_t)S.n_seg && R >= 512) {
    // 256-wide tiles, unless they would fill at most half of the chip
    const int64_t tiles = (R + 255) / 256 * ((N + 255) / 256);
    if (tiles > 128) return launch_fwd_w8<DT, 256>(Q, X, T, rows, R, S, CB, SCB, N, K, out, st);
    if (tiles >= 32) return launch_fwd_w8<DT, 128>(Q, X, T, rows, R, S, CB, SCB, N, K, out, st);
  }
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
