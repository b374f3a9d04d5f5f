// Input gradient of the experts' products on gfx950 matrix cores:
//   gX[r, k] = D(sum_n fp16(G[r, n]) Wdq[e, n, k]),
//   Wdq[e, n, k] = fp16(CB[e, n, k] * fl32(SCB[e, n] * fl32(1/127)))
// for the rows r of a segment with expert e; the weights are frozen. The
// contraction runs along the rows of CB, so each int8 tile is dequantized once
// per workgroup on its way into LDS, transposed to rows of fp16 along n.
//
// Tiles of 256 rows by BK columns, 8 waves (two per SIMD) of 64 rows by BK / 2,
// 64 rows of CB a step through two swizzled LDS stages, as in the projection's
// own kernel: the next stage's weights and gradients are loaded two steps
// ahead, and converted and written between the matrix instructions. Waves whose
// 64 rows all lie past the segment only move and convert tiles.
// Bound by the matrix instructions and the conversions beside them (32 weights and
// 32 gradients a lane for 32 matrix instructions): 4096 tokens, two of eight
// 4096 -> 11008 experts, bf16 790 us (0.94 PF/s; the projection's own kernel, with
// no tile cut short by a segment's end, 640 to 670), fp16 780, fp32 874 with the cast;
// 4092 -> 11004 877, 4095 -> 11007 995.
//
// Short contractions (up to 512), and few rows an expert (up to 64 on average)
// where every compute unit gets three tiles: tiles of 128 by 128, 4 waves, one LDS
// stage, three workgroups a compute unit, whose beginnings and ends cover each
// other. Large tiles against these: 4096 tokens, four of 64 experts, fp16, K 2048: N 64
// 42 us against 29, 512 81 against 73, 768 107 against 102, 1408 169 against 171, 4096
// 420 against 454; two of eight, bf16, K 4096, N 1024: 99 against 106. 64 tokens, four of
// 64 experts, K and N 4096: 234 against 193 (the weights alone take 199 at a large
// copy's rate); 16 tokens, two of eight, K 4096, N 11008 (256 tiles): 149 against 224.
//
// fp32 gradients, and those whose rows do not start on 16-byte borders, are cast
// to rows of fp16 first (the same cast that the tiles would do).
#include <type_traits>

#include "expert.hpp"

namespace i8l {

// Bytes of a stage: rows of 64 fp16 values.
constexpr int eb_stage(int bm, int bk) { return (bm + bk) * 128; }

// G is fp16 or bf16 (GT), R rows of ng values (N, or N rounded up to 8 with
// zeros behind it); the result is OT.
// AL: 0, N is a multiple of 8, K of 4, the weights lie on 4-byte borders and an
// expert's weight stays within 32-bit offsets; 1, but for N; 2, none of that:
// loads at any address, a row's last piece loaded so that it ends with the row
// and shifted into place.
template <int GT, int OT, int BM, int BK, int AL>
__device__ __forceinline__ void expert_bwd_tile(const typename Elem<GT>::T* __restrict__ G, int ng,
                                                const ExpertTile& tile, int k0, const int8_t* __restrict__ CBall,
                                                const float* __restrict__ SCBall, int N, int K,
                                                typename Elem<OT>::T* __restrict__ gX, char* bsm) {
  static_assert(GT == DT_F16 || GT == DT_BF16, "16-bit gradients only");
  constexpr int BNC = 64, TI = BK / 64, TJ = 2, THREADS = 2 * BM;
  constexpr int WROWS = BNC / (THREADS / 64);      // weight rows of a wave in a step
  constexpr int WR = BK * BNC / (4 * THREADS);     // and of a lane, which converts four columns of them
  constexpr int NG = BM * BNC / (8 * THREADS);     // gradient pieces of a lane
  constexpr int ROW = BNC * 2;
  constexpr int STAGE = (BK + BM) * ROW, GOFF = BK * ROW;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 31, lg = lane >> 5;
  const int wk = wave & 1, wm = wave >> 1;
  const int r0 = tile.r0, r1 = tile.r1;
  const int8_t* CB = CBall + (int64_t)tile.expert * N * K;
  const float* SCB = SCBall + (int64_t)tile.expert * N;

  const __amdgpu_buffer_rsrc_t rG = make_rsrc(G + (int64_t)r0 * ng, (r1 - r0) * ng * 2);
  const __amdgpu_buffer_rsrc_t rW = make_rsrc(CB + k0, AL == 2 ? 0 : N * K - k0);
  const __amdgpu_buffer_rsrc_t rS = make_rsrc(SCB, AL == 2 ? 0 : N * 4);

  // gradient slots: 16-byte chunk gc of rows grow + THREADS / 8 i (i < NG)
  const int grow = tid >> 3, gc = tid & 7;
  const int gvoff = grow * ng * 2 + 16 * gc;
  const int gwoff = GOFF + grow * ROW + 16 * (gc ^ lds_swz(grow));
  // weights: rows nc + WROWS wave + wh .. + WR - 1, bytes 4 kq .. 4 kq + 3
  constexpr int QUADS = BK / 4;                // lanes side by side on a weight row
  const int kq = lane % QUADS, wh = WR * (lane / QUADS);
  const int wvoff = 4 * kq + wh * K;
  const int ku = min(k0 + 4 * kq, K - 4);      // AL 2: where a lane loads, and what it shifts out
  const int shift = AL == 2 ? min(8 * (k0 + 4 * kq - ku), 31) : 0;
  int wwoff[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int r = 4 * kq + c;
    wwoff[c] = r * ROW + 16 * (((WROWS * wave + wh) >> 3) ^ lds_swz(r)) + 2 * (wh & 7);
  }
  const int sw = lds_swz(lr);
  int roff[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) roff[ks] = lr * ROW + 16 * ((2 * ks + lg) ^ sw);
  const int pb = wk * (BK / 2) * ROW, qb = GOFF + wm * 64 * ROW;

  v4u RG[NG];
  uint32_t RW[WR];
  float SG[WR];
  auto load_w = [&](int nc) {
    const int n8 = nc + WROWS * wave;
    if constexpr (AL == 2) {
#pragma unroll
      for (int e = 0; e < WR; ++e) {
        const int n = n8 + wh + e;
        const int8_t* p = CB + (int64_t)min(n, N - 1) * K;      // past N: its scale is 0
        if (K >= 4) __builtin_memcpy(&RW[e], p + ku, 4);
        else {
          RW[e] = 0u;
          for (int b = k0 + 4 * kq; b < K; ++b) RW[e] |= (uint32_t)(uint8_t)p[b] << (8 * (b & 3));
        }
        SG[e] = n < N ? SCB[n] : 0.0f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < WR; ++e) RW[e] = __builtin_amdgcn_raw_buffer_load_b32(rW, wvoff, (n8 + e) * K, 0);
      // N % 8 == 0: the eight rows from a multiple of 8 are all in the matrix or all past it
      const int so = (n8 + (wh & ~7) < N) ? 4 * (n8 + wh) : OOB_OFFSET;
      if constexpr (AL == 1) {
#pragma unroll
        for (int e = 0; e < WR; ++e)
          SG[e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rS, 4 * (n8 + wh + e), 0, 0));
      } else if constexpr (WR == 2) {
        const v2f sv = __builtin_bit_cast(v2f, __builtin_amdgcn_raw_buffer_load_b64(rS, so, 0, 0));
        SG[0] = sv[0];
        SG[1] = sv[1];
      } else {
#pragma unroll
        for (int h = 0; h < WR / 4; ++h) {
          const v4f sv = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rS, so + 16 * h, 0, 0));
#pragma unroll
          for (int e = 0; e < 4; ++e) SG[4 * h + e] = sv[e];
        }
      }
    }
  };
  auto load_g = [&](int nc) {
    const int gv = (nc + 8 * gc < ng) ? gvoff : OOB_OFFSET;
#pragma unroll
    for (int i = 0; i < NG; ++i)
      RG[i] = __builtin_bit_cast(
          v4u, __builtin_amdgcn_raw_buffer_load_b128(rG, gv, 2 * nc + THREADS / 4 * i * ng, 0));
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
        const uint32_t q0 = AL == 2 && K >= 4 ? RW[2 * e] >> shift : RW[2 * e];
        const uint32_t q1 = AL == 2 && K >= 4 ? RW[2 * e + 1] >> shift : RW[2 * e + 1];
        const float w0 = (float)(int)(int8_t)(q0 >> (8 * c));
        const float w1 = (float)(int)(int8_t)(q1 >> (8 * c));
        h[e] = f32x2_to_f16x2(w0 * sg[2 * e], w1 * sg[2 * e + 1]);
      }
      if constexpr (WR == 8) *reinterpret_cast<v4u*>(bsm + st * STAGE + wwoff[c]) = v4u{h[0], h[1], h[2], h[3]};
      else if constexpr (WR == 4) *reinterpret_cast<v2u*>(bsm + st * STAGE + wwoff[c]) = v2u{h[0], h[1]};
      else *reinterpret_cast<uint32_t*>(bsm + st * STAGE + wwoff[c]) = h[0];
    }
  };
  auto write_g = [&](int st) {
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      v4u v;
      if constexpr (GT == DT_F16) {
        v = RG[i];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = bf16x2_to_f16x2(RG[i][e]);
      }
      *reinterpret_cast<v4u*>(bsm + st * STAGE + gwoff + i * (THREADS / 8) * ROW) = v;
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
  auto spread = [&](auto dsw, auto vm) {
    constexpr int Wr = decltype(dsw)::value, Gl = decltype(vm)::value;
#pragma unroll
    for (int q = 0; q < TI * TJ; ++q) {
      I8L_SGB(SG_MFMA, 1);
      I8L_SGB(SG_VALU, 4);
      if (q < TI + TJ) I8L_SGB(SG_DS_R, 1);
      if (q < Wr) I8L_SGB(SG_DS_W, 1);
      if (q < Gl) I8L_SGB(SG_VMEM_R, 1);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  const int nn = (N + BNC - 1) / BNC;
  load_w(0);
  load_g(0);
  write_w(0, 0);
  write_w(0, 2);
  write_g(0);
  load_w(BNC);
  load_g(BNC);
  __syncthreads();
  const bool busy = r0 + wm * 64 < r1;
  if constexpr (BM == 128) {
    for (int t = 0; t < nn; ++t) {
      if (busy) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          fread(0, ks, ks & 1);
          mma(ks & 1);
        }
      }
      if (t + 1 == nn) break;
      __syncthreads();
      write_w(0, 0);
      write_w(0, 2);
      write_g(0);
      __syncthreads();
      load_w((t + 2) * BNC);
      load_g((t + 2) * BNC);
    }
  } else if (busy) {
    fread(0, 0, 0);
    for (int t = 0; t < nn; ++t) {
      const int st = t & 1;
      const int nc2 = (t + 2) * BNC;   // past the end: zeros
      fread(st, 1, 1);
      write_w(st ^ 1, 0);
      mma(0);
      spread(std::integral_constant<int, 2>{}, std::integral_constant<int, 0>{});
      fread(st, 2, 0);
      write_w(st ^ 1, 2);
      load_w(nc2);
      mma(1);
      spread(std::integral_constant<int, 2>{}, std::integral_constant<int, WR + (WR + 3) / 4>{});
      fread(st, 3, 1);
      write_g(st ^ 1);
      load_g(nc2);
      mma(0);
      spread(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
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

  // lane (lr, lg), register r of tile (i, j): column wk BK / 2 + i 32 + (r / 4) 8 + lg 4 + r % 4, row wm 64 + j 32 + lr
  if constexpr (OT == DT_F32) {
    const bool ov = K % 4 == 0 && (uintptr_t)gX % 16 == 0;
    if (!ov) {
      auto value = [&](int i, int j, int q) {
        return v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
      };
      return etile_f32<BM, BK, THREADS, (BM == 256 ? 2 : 1) * eb_stage(BM, BM)>(bsm, value, nullptr, gX, K, r0, k0, r1,
                                                                              min(K, k0 + BK), wk, wm, lr, lg);
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int r = r0 + wm * 64 + j * 32 + lr;
      if (r >= r1) continue;
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int k = k0 + wk * (BK / 2) + i * 32 + q * 8 + lg * 4;
          const float y[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          expert_store4<OT>(gX + (int64_t)r * K + k, y, K - k, true);
        }
    }
  } else {
    // through LDS, stored as whole rows of the tile's columns
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
            w[e] = (uint32_t)__builtin_bit_cast(uint16_t, Elem<OT>::from_f32(acc[i][j][4 * q + 2 * e])) |
                   ((uint32_t)__builtin_bit_cast(uint16_t, Elem<OT>::from_f32(acc[i][j][4 * q + 2 * e + 1])) << 16);
          *reinterpret_cast<v2u*>(
              bsm + etile_off<2 * BK>(wm * 64 + j * 32 + lr, wk * (BK / 16) + i * 4 + q) + 8 * lg) = w;
        }
    __syncthreads();
    etile_store<BM, BK, THREADS, typename Elem<OT>::T>(bsm, nullptr, gX, K, r0, k0, r1, min(K, k0 + BK));
  }
}

// Tiles 256 wide; the last ones in narrower parts (expert_work).
template <int GT, int OT, int AL>
__global__ __launch_bounds__(512, 1) void k_expert_bwd(const typename Elem<GT>::T* __restrict__ G, int ng, int R,
                                                       ExpertSegs S, const int8_t* __restrict__ CB,
                                                       const float* __restrict__ SCB, int N, int K,
                                                       typename Elem<OT>::T* __restrict__ gX) {
  extern __shared__ __attribute__((aligned(16))) char bsm[];
  const ExpertScan scan = expert_scan(S, R, 256);
  const ExpertWork work = expert_work<true>(expert_block(), scan, (K + 255) / 256);
  if (work.slot < 0) return;
  const ExpertTile tile = expert_tile(S, scan, work.slot, R, 256);
  const int k0 = work.tc * 256 + work.part * (256 / work.parts);
  if (tile.r0 >= tile.r1 || k0 >= K) return;
  if (tile.expert < 0 || N == 0) return expert_zeros(gX, K, tile.r0, tile.r1, k0, min(K, k0 + 256 / work.parts));
  if (work.parts == 1) expert_bwd_tile<GT, OT, 256, 256, AL>(G, ng, tile, k0, CB, SCB, N, K, gX, bsm);
  else if (work.parts == 2) expert_bwd_tile<GT, OT, 256, 128, AL>(G, ng, tile, k0, CB, SCB, N, K, gX, bsm);
  else expert_bwd_tile<GT, OT, 256, 64, AL>(G, ng, tile, k0, CB, SCB, N, K, gX, bsm);
}

// Tiles 128 x 128.
template <int GT, int OT, int AL>
__global__ __launch_bounds__(256, 3) void k_expert_bwd_short(const typename Elem<GT>::T* __restrict__ G, int ng, int R,
                                                             ExpertSegs S, const int8_t* __restrict__ CB,
                                                             const float* __restrict__ SCB, int N, int K,
                                                             typename Elem<OT>::T* __restrict__ gX) {
  __shared__ __attribute__((aligned(16))) char bsm[eb_stage(128, 128)];
  const ExpertScan scan = expert_scan(S, R, 128);
  const ExpertWork work = expert_work<false>(expert_block(), scan, (K + 127) / 128);
  if (work.slot < 0) return;
  const ExpertTile tile = expert_tile(S, scan, work.slot, R, 128);
  const int k0 = work.tc * 128;
  if (tile.r0 >= tile.r1) return;
  if (tile.expert < 0 || N == 0) return expert_zeros(gX, K, tile.r0, tile.r1, k0, min(K, k0 + 128));
  expert_bwd_tile<GT, OT, 128, 128, AL>(G, ng, tile, k0, CB, SCB, N, K, gX, bsm);
}

// Rows of G as fp16, ng values each, zeros behind the N-th.
template <int DT>
__global__ __launch_bounds__(256) void k_expert_cast(const typename Elem<DT>::T* __restrict__ G, int64_t R, int N,
                                                     int ng, _Float16* __restrict__ out) {
  const int chunks = ng / 8;
  const int64_t items = R * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / chunks;
    const int c = (int)(i - r * chunks) * 8;
    const typename Elem<DT>::T* p = G + r * N + c;
    v8h h = {};
    if (c + 8 <= N) {      // at any address
      typename Elem<DT>::T e[8];
      __builtin_memcpy(e, p, sizeof(e));
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = to_half<DT>(e[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < N) h[j] = to_half<DT>(p[j]);
    }
    *reinterpret_cast<v8h*>(out + r * ng + c) = h;
  }
}

static bool rows_as_fp16(const void* G, int dt, int64_t N) {
  return dt == DT_F32 || N % 8 != 0 || (uintptr_t)G % 16 != 0;
}
size_t expert_bwd_bytes(const void* G, int dt, int64_t R, int64_t N) {
  return rows_as_fp16(G, dt, N) ? (size_t)R * (size_t)((N + 7) / 8 * 8) * 2 : 0;
}

template <int GT, int OT>
static hipError_t launch_bwd_t(const void* G, int ng, int R, const ExpertSegs& S, const int8_t* CB, const float* SCB,
                               int N, int K, void* gX, hipStream_t st) {
  constexpr int lds = 2 * eb_stage(256, 256);      // operand stages; the output tile takes their place
  const bool words = K % 4 == 0 && (uintptr_t)CB % 4 == 0 && (N + (int64_t)256) * K < ((int64_t)1 << 31) - 4096;
  const int al = !words ? 2 : N % 8 != 0 ? 1 : 0;
  const int64_t tiles = expert_slots(R, S.n_seg, 128) * ((K + 127) / 128);
  if (N <= 512 || (R <= 64 * (int64_t)S.n_seg && tiles >= 768)) {
    auto kern = al == 2   ? k_expert_bwd_short<GT, OT, 2>
                : al == 1 ? k_expert_bwd_short<GT, OT, 1>
                          : k_expert_bwd_short<GT, OT, 0>;
    hipLaunchKernelGGL(kern, expert_grid(tiles), dim3(256), 0, st, static_cast<const typename Elem<GT>::T*>(G), ng, R,
                       S, CB, SCB, N, K, static_cast<typename Elem<OT>::T*>(gX));
    return hipGetLastError();
  }
  static std::atomic<uint64_t> lds_set[3];
  auto kern = al == 2 ? k_expert_bwd<GT, OT, 2> : al == 1 ? k_expert_bwd<GT, OT, 1> : k_expert_bwd<GT, OT, 0>;
  const hipError_t e = lds_limit_once((const void*)kern, lds, lds_set[al]);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, expert_grid(expert_groups(expert_slots(R, S.n_seg, 256), (K + 255) / 256)), dim3(512), lds,
                     st, static_cast<const typename Elem<GT>::T*>(G), ng, R, S, CB, SCB, N, K,
                     static_cast<typename Elem<OT>::T*>(gX));
  return hipGetLastError();
}

template <int DT>
static hipError_t launch_cast(const void* G, int64_t R, int N, int ng, void* out, hipStream_t st) {
  const int64_t items = R * (ng / 8);
  const int64_t groups = (items + 255) / 256;
  if (groups == 0) return hipSuccess;
  hipLaunchKernelGGL(k_expert_cast<DT>, dim3((unsigned)(groups < 4096 ? groups : 4096)), dim3(256), 0, st,
                     static_cast<const typename Elem<DT>::T*>(G), R, N, ng,
                     static_cast<_Float16*>(out));
  return hipGetLastError();
}

hipError_t launch_expert_bwd(int dt, const void* G, int R, const ExpertSegs& S, const int8_t* CB, const float* SCB,
                             int N, int K, void* gX, void* ws, hipStream_t st) {
  if (rows_as_fp16(G, dt, N)) {
    const int ng = (N + 7) / 8 * 8;
    hipError_t e;
    if (dt == DT_F32) e = launch_cast<DT_F32>(G, R, N, ng, ws, st);
    else if (dt == DT_F16) e = launch_cast<DT_F16>(G, R, N, ng, ws, st);
    else e = launch_cast<DT_BF16>(G, R, N, ng, ws, st);
    if (e != hipSuccess) return e;
    if (dt == DT_F32) return launch_bwd_t<DT_F16, DT_F32>(ws, ng, R, S, CB, SCB, N, K, gX, st);
    if (dt == DT_F16) return launch_bwd_t<DT_F16, DT_F16>(ws, ng, R, S, CB, SCB, N, K, gX, st);
    return launch_bwd_t<DT_F16, DT_BF16>(ws, ng, R, S, CB, SCB, N, K, gX, st);
  }
  if (dt == DT_F16) return launch_bwd_t<DT_F16, DT_F16>(G, N, R, S, CB, SCB, N, K, gX, st);
  return launch_bwd_t<DT_BF16, DT_BF16>(G, N, R, S, CB, SCB, N, K, gX, st);
}

}  // namespace i8l
