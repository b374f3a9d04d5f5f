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
//
// Four forms, taken in this order (the sizes on both sides of each rule are at the
// forms):
//   k_expert_fwd_tiny    up to 4 tokens with few rows an expert, K up to 4096 in whole
//                        words: quantized in the same launch
//   k_expert_fwd_thin    few rows an expert (few_rows), or K below 16: tiles of 16 x 16,
//                        bound by reading the weights once
//   k_expert_fwd_short   K up to 512, or up to 1024 where every compute unit gets a
//                        tile: 128 x 128, three workgroups a compute unit
//   k_expert_fwd         all others: 256 x 256, bound by the matrix cores as the
//                        projection's kernel is, at its rate
#include <type_traits>

#include "expert.hpp"
#include "quantize.hpp"

namespace i8l {

// ---------------------------------------------------------------------------
// Large tiles: 256 rows by BN features, 8 waves (two per SIMD) of 64 rows by
// BN / 2, the contraction 128 bytes at a time through two swizzled LDS stages,
// as in the projection's own kernel; registers hold the next step's tiles. The
// rows of the activation tile are gathered: a lane keeps the places of its four
// tokens, so the gather costs nothing in the loop. Waves whose 64 rows all lie
// past the segment only move tiles: a tile of 100 rows takes about half the
// time of a full one.
// AL, what K and the weights' address are multiples of: 4, buffer loads, whose
// last piece of a weight row may go on into the next row (zeros behind the last
// one) against the zeros that a row of codes ends with; 1, or where the codes pass
// 2^31 bytes, 16-byte loads at any address, for K of 16 at least. 4096 tokens, two
// of eight experts, bf16, 4096 -> 11008 443 us, 4088 -> 11000 476, 4095 -> 11007 561.
//
// Short contractions: 128 rows by 128 features, 4 waves of 64 x 64 and one LDS
// stage, so that three workgroups share a compute unit and their beginnings and
// ends (tile, tokens, outlier panels; the output's way to memory), which are most
// of such a tile's time, cover each other. Up to 512 always, up to 1024 where every
// compute unit gets a tile. bf16, large tiles against these: 4096 tokens, eight of
// 16 experts, 128 -> 2048 80 us against 68, 512 -> 2048 104 against 91; 777 tokens,
// three of five, -> 1530: from 128 28 against 24, 1024 34 against 31, 2048 41 against
// 42; 512 tokens, two of four, -> 1024 (96 tiles): from 512 20.6 against 19.7, 1024
// 22.5 against 23.3.
constexpr int ef_threads(int bm) { return 2 * bm; }
constexpr int ef_stages(int bm) { return bm == 256 ? 2 * (256 + 256) * 128 : (128 + 128) * 128; }
constexpr int ef_opan(int bm) { return 2 * bm * 32; }      // outlier panels P[n][16], Q[row][16] (fp16)
constexpr int ef_lds(int bm) { return ef_stages(bm) + ef_opan(bm) + 2 * bm * 4; }      // and SCB / 127^2, SCA

template <int DT, int BM, int BN, int AL>
__device__ __forceinline__ void expert_fwd_tile(const ExpertQuantized& Q, const typename Elem<DT>::T* __restrict__ X,
                                                int T, const int32_t* __restrict__ rows, const ExpertTile& tile,
                                                int n0, int cnt, OutlierCols cols, const int8_t* __restrict__ CBall,
                                                const float* __restrict__ SCBall, int N, int K,
                                                typename Elem<DT>::T* __restrict__ out, int8_t* smem) {
  constexpr int BK = 128, TI = BN / 64, TJ = 2;
  constexpr int THREADS = ef_threads(BM), RPP = THREADS / 8;      // tile rows a pass loads
  constexpr int NB = BN / RPP, NA = BM / RPP;
  constexpr int STAGE = (BM + BN) * BK, AOFF = BN * BK, STAGES = ef_stages(BM), OPAN = ef_opan(BM);
  static_assert((BM == 256 ? 2 : 1) * STAGE <= STAGES && BM * BN * 2 <= STAGES && BN <= BM,
                "stages and output tile share the same bytes");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 31, lg = lane >> 5;
  const int wn = wave & 1, wm = wave >> 1;
  const int r0 = tile.r0, r1 = tile.r1;
  const int8_t* CB = CBall + (int64_t)tile.expert * N * K;
  const float* SCB = SCBall + (int64_t)tile.expert * N;

  const int lrow = tid >> 3, lc = tid & 7;
  const int woff = lrow * BK + 16 * (lc ^ lds_swz(lrow));
  const int sw = lds_swz(lr);
  int roff[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) roff[ks] = lr * BK + 16 * ((2 * ks + lg) ^ sw);
  const int pb = wn * (BN / 2) * BK, qb = AOFF + wm * 64 * BK;

  v4u RB[NB], RA[NA];
  const __amdgpu_buffer_rsrc_t rB = make_rsrc(CB + (int64_t)n0 * K, AL == 1 ? 0 : min(BN, N - n0) * K);
  const int voff = lrow * K + 16 * lc;
  int boff[NB];
  const int8_t* B0 = CB + (int64_t)n0 * K;
#pragma unroll
  for (int i = 0; i < NB; ++i) boff[i] = (min(n0 + lrow + RPP * i, N - 1) - n0) * K;   // past N: not stored
  auto load_b = [&](int kt) {
    if constexpr (AL == 1) {
      const int at = tail_at(kt + 16 * lc, K);
#pragma unroll
      for (int i = 0; i < NB; ++i) RB[i] = bytes16(B0 + (boff[i] + at));
    } else {
      const int v = (kt + 16 * lc < K) ? voff : OOB_OFFSET;
#pragma unroll
      for (int i = 0; i < NB; ++i)
        RB[i] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rB, v, kt + RPP * i * K, 0));
    }
  };
  load_b(0);
  const __amdgpu_buffer_rsrc_t rA = make_rsrc(Q.CA, AL == 1 ? 0 : T * Q.lda);
  int aoff[NA];
  const int8_t* pA[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int r = r0 + lrow + RPP * i;
    const int t = r < r1 ? row_token(rows, r, T) : -1;
    // no token: the row is stored as zeros, whatever its codes
    if constexpr (AL == 1) pA[i] = Q.CA + (int64_t)max(t, 0) * Q.lda;
    else aoff[i] = t >= 0 ? t * Q.lda + 16 * lc : OOB_OFFSET;
  }
  int ka = 0;      // AL 1: first byte of the codes in RA
  auto load_a = [&](int kt) {
    if constexpr (AL == 1) {
      const int k = kt + 16 * lc, at = tail_at(k, K);
#pragma unroll
      for (int i = 0; i < NA; ++i) RA[i] = bytes16(pA[i] + at);
      ka = k;
    } else {
      const bool in = kt + 16 * lc < K;
#pragma unroll
      for (int i = 0; i < NA; ++i)
        RA[i] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rA, in ? aoff[i] : OOB_OFFSET, kt, 0));
    }
  };
  auto write_b = [&](int st) {
#pragma unroll
    for (int i = 0; i < NB; ++i) *reinterpret_cast<v4u*>(smem + st * STAGE + woff + i * RPP * BK) = RB[i];
  };
  auto write_a = [&](int st) {
#pragma unroll
    for (int i = 0; i < NA; ++i)
      *reinterpret_cast<v4u*>(smem + st * STAGE + AOFF + woff + i * RPP * BK) =
          AL == 4 ? RA[i] : tail_clear(RA[i], ka, K);      // every step: a branch costs the loop more
  };
  load_a(0);

  // the tile's scales, and the panels of the first 16 outlier columns, while
  // the first operand tiles are in flight
  char* opan = reinterpret_cast<char*>(smem) + STAGES;
  float* lsb = reinterpret_cast<float*>(opan + OPAN);
  float* lsa = lsb + BM;
  const int orow = tid >> 1, oj = (tid & 1) * 8;      // cols: those of oj
  v8h opP = {}, opQ = {};
  auto panels = [&](int jo) {
    const int n = n0 + orow, r = r0 + orow;
    opP = expert_out_w8(CB, SCB, K, cols, n, orow < BN && n < N, jo + oj, cnt);
    opQ = expert_out_a8<DT>(Q.sub, Q.cap, X, K, cols, r < r1 ? row_token(rows, r, T) : -1, jo + oj, cnt);
  };
  auto put_panels = [&]() {
    *reinterpret_cast<v8h*>(opan + orow * 32 + oj * 2) = opP;
    *reinterpret_cast<v8h*>(opan + OPAN / 2 + orow * 32 + oj * 2) = opQ;
  };
  if (cnt > 0) panels(0);
  if (tid < BM) {
    const int n = n0 + tid;
    lsb[tid] = (tid < BN && n < N) ? SCB[n] * (1.0f / 16129.0f) : 0.0f;
  } else {
    const int r = r0 + tid - BM;
    const int t = r < r1 ? row_token(rows, r, T) : -1;
    lsa[tid - BM] = t >= 0 ? Q.SCA[t] : NO_TOKEN;
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
  // each matrix instruction of a phase is followed by a fragment read of the next and by its share of the tile traffic
  auto spread = [&](auto writes) {
#pragma unroll
    for (int q = 0; q < TI * TJ; ++q) {
      I8L_SGB(SG_MFMA, 1);
      if (q < TI + TJ) I8L_SGB(SG_DS_R, 1);
      if (q < decltype(writes)::value) {
        I8L_SGB(SG_DS_W, 1);
        I8L_SGB(SG_VMEM_R, 1);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const int nk = (K + BK - 1) / BK;
  write_b(0);
  write_a(0);
  load_b(BK);
  load_a(BK);
  if (cnt > 0) put_panels();
  __syncthreads();
  const bool busy = r0 + wm * 64 < r1;
  if constexpr (BM == 128) {
    for (int kt = 0; kt < nk; ++kt) {
      if (busy) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          fread(0, ks, ks & 1);
          mma(ks & 1);
        }
      }
      if (kt + 1 == nk) break;
      __syncthreads();
      write_b(0);
      write_a(0);
      __syncthreads();
      load_b((kt + 2) * BK);
      load_a((kt + 2) * BK);
    }
  } else if (busy) {
    fread(0, 0, 0);
    for (int kt = 0; kt < nk; ++kt) {
      const int st = kt & 1;
      const int k2 = (kt + 2) * BK;    // past the end: zeros
      fread(st, 1, 1);
      write_b(st ^ 1);
      load_b(k2);
      mma(0);
      spread(std::integral_constant<int, NB>{});
      fread(st, 2, 0);
      write_a(st ^ 1);
      load_a(k2);
      mma(1);
      spread(std::integral_constant<int, 4>{});
      fread(st, 3, 1);
      mma(0);
      spread(std::integral_constant<int, 0>{});
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

  // lane (lr, lg), register r of tile (i, j): feature wn BN / 2 + 32 i + 8 (r / 4) + 4 lg + r % 4, row 64 wm + 32 j
  // + lr
  // (the accumulators become fp32 in place)
  const int nl = wn * (BN / 2), ml = wm * 64;
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
      cols = expert_out_cols(Q.idx, jo + oj, cnt);
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
        const v8h V = *reinterpret_cast<const v8h*>(opan + OPAN / 2 + (ml + j * 32 + lr) * 32 + lg * 16);
        acc[i][j] = __builtin_bit_cast(
            v16i, __builtin_amdgcn_mfma_f32_32x32x16_f16(P, V, __builtin_bit_cast(v16f, acc[i][j]), 0, 0, 0));
      }
    }
  }
  if constexpr (DT == DT_F32) {
    const bool ov = N % 4 == 0 && (uintptr_t)out % 16 == 0;
    if (!ov) {
      auto value = [&](int i, int j, int q) {
        return v4f{__int_as_float(acc[i][j][4 * q]), __int_as_float(acc[i][j][4 * q + 1]),
                   __int_as_float(acc[i][j][4 * q + 2]), __int_as_float(acc[i][j][4 * q + 3])};
      };
      return etile_f32<BM, BN, THREADS, STAGES>(reinterpret_cast<char*>(smem), value, lsa, out, N, r0, n0, r1,
                                                min(N, n0 + BN), wn, wm, lr, lg);
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int r = r0 + ml + j * 32 + lr;
      if (r >= r1) continue;
      const bool none = no_token(lsa[ml + j * 32 + lr]);
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + nl + i * 32 + q * 8 + lg * 4;
          float y[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) y[x] = none ? 0.0f : __int_as_float(acc[i][j][4 * q + x]);
          expert_store4<DT>(out + (int64_t)r * N + n, y, N - n, true);
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
          *reinterpret_cast<v2u*>(ot + etile_off<2 * BN>(ml + j * 32 + lr, (nl + i * 32 + q * 8) >> 3) + 8 * lg) = w;
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
    etile_store<BM, BN, THREADS>(ot, lsa, out, N, r0, n0, r1, min(N, n0 + BN));
  }
}

// Tiles 256 wide; the last ones in narrower parts (expert_work).
template <int DT, int AL>
__global__ __launch_bounds__(512, 1) void k_expert_fwd(ExpertQuantized Q, const typename Elem<DT>::T* __restrict__ X,
                                                       int T, const int32_t* __restrict__ rows, int R, ExpertSegs S,
                                                       const int8_t* __restrict__ CB, const float* __restrict__ SCB,
                                                       int N, int K, typename Elem<DT>::T* __restrict__ out) {
  extern __shared__ __attribute__((aligned(16))) int8_t smem[];
  const int cnt = *Q.count;
  const OutlierCols cols = expert_out_cols(Q.idx, (threadIdx.x & 1) * 8, min(cnt, 16));
  const ExpertScan scan = expert_scan(S, R, 256);
  const ExpertWork work = expert_work<true>(expert_block(), scan, (N + 255) / 256);
  if (work.slot < 0) return;
  const ExpertTile tile = expert_tile(S, scan, work.slot, R, 256);
  const int n0 = work.tc * 256 + work.part * (256 / work.parts);
  if (tile.r0 >= tile.r1 || n0 >= N) return;
  if (tile.expert < 0) return expert_zeros(out, N, tile.r0, tile.r1, n0, min(N, n0 + 256 / work.parts));
  if (work.parts == 1)
    expert_fwd_tile<DT, 256, 256, AL>(Q, X, T, rows, tile, n0, cnt, cols, CB, SCB, N, K, out, smem);
  else if (work.parts == 2)
    expert_fwd_tile<DT, 256, 128, AL>(Q, X, T, rows, tile, n0, cnt, cols, CB, SCB, N, K, out, smem);
  else
    expert_fwd_tile<DT, 256, 64, AL>(Q, X, T, rows, tile, n0, cnt, cols, CB, SCB, N, K, out, smem);
}

// Tiles 128 x 128.
template <int DT, int AL>
__global__ __launch_bounds__(256, 3) void k_expert_fwd_short(ExpertQuantized Q,
                                                             const typename Elem<DT>::T* __restrict__ X, int T,
                                                             const int32_t* __restrict__ rows, int R, ExpertSegs S,
                                                             const int8_t* __restrict__ CB,
                                                             const float* __restrict__ SCB, int N, int K,
                                                             typename Elem<DT>::T* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) int8_t smem[ef_lds(128)];
  const int cnt = *Q.count;
  const OutlierCols cols = expert_out_cols(Q.idx, (threadIdx.x & 1) * 8, min(cnt, 16));
  const ExpertScan scan = expert_scan(S, R, 128);
  const ExpertWork work = expert_work<false>(expert_block(), scan, (N + 127) / 128);
  if (work.slot < 0) return;
  const ExpertTile tile = expert_tile(S, scan, work.slot, R, 128);
  const int n0 = work.tc * 128;
  if (tile.r0 >= tile.r1) return;
  if (tile.expert < 0) return expert_zeros(out, N, tile.r0, tile.r1, n0, min(N, n0 + 128));
  expert_fwd_tile<DT, 128, 128, AL>(Q, X, T, rows, tile, n0, cnt, cols, CB, SCB, N, K, out, smem);
}

// ---------------------------------------------------------------------------
// Few rows an expert: tiles of 16 rows by 16 features, bound by reading the
// weights once. Four waves share a tile's contraction, 256 bytes of every row
// at a time: a wave brings its 16 weight rows of 256 bytes into LDS with lanes
// side by side on a row (straight from memory into the matrix operands' layout,
// 16 rows a request, a compute unit gets only one request a nanosecond),
// 16-byte pieces p of row r at p ^ r, and reads them as operands; the
// codes, few and shared by all tiles of the expert, come from L2 in the
// operands' layout. No barrier until the waves' int32 sums meet in LDS (exact,
// so their order is nothing to the result). 16 KB of LDS and 64 registers, so
// that eight workgroups on a compute unit cover each other's beginnings and
// ends: 512 bytes at a time, five workgroups, took 28 us for one token of two
// 4096 -> 11008 experts instead of 22.
// AL: as above; 1 goes through registers, and takes K below 16.
// KS 1: a wave has a tile of its own and all of its contraction, with no barrier
// at all; for contractions up to 2048 where that fills the chip. 64 tokens, four
// of 64 experts, 512 -> 4096: 27 us against 43 with KS 4, 2048: 80 against 90,
// 4096: 166 against 160; one token, two of eight experts, 2048 -> 11008: 19
// against 17 (too few workgroups).
typedef __attribute__((address_space(3))) void* lds_ptr;
constexpr int ET_KC = 256;      // bytes of a row a wave takes at a time
template <int DT, int AL, int KS>
__global__ __launch_bounds__(256, AL == 1 ? 4 : 8) void k_expert_fwd_thin(ExpertQuantized Q,
                                                            const typename Elem<DT>::T* __restrict__ X, int T,
                                                            const int32_t* __restrict__ rows, int R, ExpertSegs S,
                                                            const int8_t* __restrict__ CBall,
                                                            const float* __restrict__ SCBall, int N, int K,
                                                            int tiles_n, typename Elem<DT>::T* __restrict__ out) {
  typedef typename Elem<DT>::T E;
  constexpr int BM = 16, BN = 16, STEPS = ET_KC / 64, LPR = ET_KC / 16;
  constexpr int WG_N = KS == 1 ? 4 * BN : BN;      // features of a workgroup
  __shared__ __attribute__((aligned(1024))) int8_t sw[4][BN * ET_KC];
  const int64_t bid = expert_block();
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int64_t ts = bid / tiles_n;
  const int n0 = (int)(bid - ts * tiles_n) * WG_N + (KS == 1 ? wave * BN : 0);
  const int cnt = *Q.count;
  const OutlierCols cols = expert_out_cols(Q.idx, lg * 8, cnt);
  const ExpertScan scan = expert_scan(S, R, BM);
  if (ts >= scan.total + scan.zeros) return;
  const ExpertTile tile = expert_tile(S, scan, (int)ts, R, BM);
  if (tile.r0 >= tile.r1) return;
  if (tile.expert < 0) {
    const int c0 = (int)(bid - ts * tiles_n) * WG_N;
    return expert_zeros(out, N, tile.r0, tile.r1, c0, min(N, c0 + WG_N));
  }
  if (n0 >= N) return;      // KS 1: no barrier follows
  const int8_t* CB = CBall + (int64_t)tile.expert * N * K;
  const float* SCB = SCBall + (int64_t)tile.expert * N;
  const __amdgpu_buffer_rsrc_t rB = make_rsrc(CB + (int64_t)n0 * K, AL == 1 ? 0 : min(BN, N - n0) * K);
  const int nc = (K + ET_KC - 1) / ET_KC;

  int8_t* mine = sw[wave];
  v4u W[ET_KC / 64];      // AL 1
  auto load_w = [&](int c) {
#pragma unroll
    for (int i = 0; i < ET_KC / 64; ++i) {
      const int row = (64 / LPR) * i + lane / LPR;
      const int k = c * ET_KC + 16 * ((lane % LPR) ^ row);
      if constexpr (AL == 1) {
        const int8_t* p = CB + (int64_t)min(n0 + row, N - 1) * K;     // past N: not stored
        W[i] = K >= 16 ? bytes16(p + tail_at(k, K)) : short_row(p, k, K);
      } else {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_ptr)(mine + i * 1024), 16, k < K ? row * K + k : OOB_OFFSET,
                                                 0, 0, 0);
      }
    }
  };
  const int first = KS == 1 ? 0 : wave;
  if (first < nc) load_w(first);

  const int r = tile.r0 + lr;
  const int t = r < tile.r1 ? row_token(rows, r, T) : -1;
  // what the wave that finishes the tile needs for that is requested before the contraction
  const int nb = n0 + 4 * lg;
  float sa = 0.0f, sb[4] = {};
  v8h P = {}, V = {};
  if (KS == 1 || wave == 0) {
    if (t >= 0) sa = Q.SCA[t];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (nb + x < N) sb[x] = SCB[nb + x];
    if (cnt > 0) {
      P = expert_out_w8(CB, SCB, K, cols, n0 + lr, n0 + lr < N, lg * 8, cnt);
      V = expert_out_a8<DT>(Q.sub, Q.cap, X, K, cols, t, lg * 8, cnt);
    }
  }
  v4i acc = {0, 0, 0, 0};
  for (int c = first; c < nc; c += KS) {
    v4i a[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int k = c * ET_KC + s * 64 + lg * 16;
      a[s] = v4i{0, 0, 0, 0};
      if (t >= 0) {
        const int8_t* p = Q.CA + (int64_t)t * Q.lda;
        if constexpr (AL == 4) {
          if (k < K) a[s] = *reinterpret_cast<const v4i*>(p + k);
        } else {
          const v4u v = K >= 16 ? bytes16(p + tail_at(k, K)) : short_row(p, k, K);
          a[s] = __builtin_bit_cast(v4i, v);
        }
      }
    }
    if constexpr (AL == 1) {
#pragma unroll
      for (int i = 0; i < ET_KC / 64; ++i) *reinterpret_cast<v4u*>(mine + i * 1024 + lane * 16) = W[i];
    }
    if (AL == 1 && K >= 16 && (c + 1) * ET_KC > K) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int k = c * ET_KC + s * 64 + lg * 16;
        a[s] = __builtin_bit_cast(v4i, tail_clear(__builtin_bit_cast(v4u, a[s]), k, K));
      }
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const v4i w = *reinterpret_cast<const v4i*>(mine + lr * ET_KC + 16 * ((4 * s + lg) ^ lr));
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a[s], acc, 0, 0, 0);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the next piece lands in the same place
    if (c + KS < nc) load_w(c + KS);
  }

  // lane (lr, lg): the token of row lr, features n0 + 4 lg .. + 3
  v4i sum = acc;
  if constexpr (KS > 1) {
    v4i* part = reinterpret_cast<v4i*>(sw[0]);
    __syncthreads();
    part[wave * 64 + lane] = acc;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 1; w < 4; ++w) sum += part[w * 64 + lane];
  }
  v4f y;
#pragma unroll
  for (int x = 0; x < 4; ++x) y[x] = (float)sum[x] * (sa * (sb[x] * (1.0f / 16129.0f)));
  if (cnt > 0) y = __builtin_amdgcn_mfma_f32_16x16x32_f16(P, V, y, 0, 0, 0);
  for (int jo = 32; jo < cnt; jo += 32) {
    const OutlierCols more = expert_out_cols(Q.idx, jo + lg * 8, cnt);
    P = expert_out_w8(CB, SCB, K, more, n0 + lr, n0 + lr < N, jo + lg * 8, cnt);
    V = expert_out_a8<DT>(Q.sub, Q.cap, X, K, more, t, jo + lg * 8, cnt);
    y = __builtin_amdgcn_mfma_f32_16x16x32_f16(P, V, y, 0, 0, 0);
  }
  if (r < tile.r1) {
    float v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = t >= 0 ? y[x] : 0.0f;
    expert_store4<DT>(out + (int64_t)r * N + nb, v, N - nb, N % 4 == 0 && (uintptr_t)out % (4 * sizeof(E)) == 0);
  }
}

// ---------------------------------------------------------------------------
// Up to four tokens: the kernel above (KS 4), with the quantization in it. Every
// workgroup quantizes all of the tokens itself, into LDS, while its first
// weights are on their way: one launch, and nothing to wait for between two. The
// same flags, scales, codes and outlier values as the quantizer's.
// One token of two 4096 -> 11008 experts, bf16: 20 us against 26 in two launches.
// Contractions past 4096 are more than a thread's two pieces of a token: they take
// the launches above (11008 -> 4096: 30 to 37 us for one token, 68 for four; up to 8192
// the quantizer is one launch, past that two).
constexpr int EQ_TOKENS = 4, EQ_COLS = 4096, EQ_LIST = 256;
template <int DT, int TM>      // TM: 1 or EQ_TOKENS, at least T
__global__ __launch_bounds__(256, TM == 1 ? 6 : 4) void k_expert_fwd_tiny(
    const typename Elem<DT>::T* __restrict__ X, int T, bool vec, float tau, const int32_t* __restrict__ rows, int R,
    ExpertSegs S, const int8_t* __restrict__ CBall, const float* __restrict__ SCBall, int N, int K, int tiles_n,
    typename Elem<DT>::T* __restrict__ out) {
#pragma clang fp contract(off)
  typedef typename Elem<DT>::T E;
  constexpr int BN = 16, STEPS = ET_KC / 64, LPR = ET_KC / 16, CH = EQ_COLS / 8 / 256;
  __shared__ __attribute__((aligned(1024))) int8_t sw[4][BN * ET_KC];
  __shared__ uint32_t smask[EQ_COLS / 32];
  __shared__ uint32_t red[TM][4];
  __shared__ uint16_t slist[EQ_LIST];
  extern __shared__ __attribute__((aligned(16))) int8_t codes[];      // TM rows of kp
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int64_t bid = expert_block();
  const int64_t ts = bid / tiles_n;
  const int n0 = (int)(bid - ts * tiles_n) * BN;
  const ExpertScan scan = expert_scan(S, R, 16);
  if (ts >= scan.total + scan.zeros) return;
  const ExpertTile tile = expert_tile(S, scan, (int)ts, R, 16);
  if (tile.r0 >= tile.r1) return;
  if (tile.expert < 0) return expert_zeros(out, N, tile.r0, tile.r1, n0, min(N, n0 + BN));
  const int8_t* CB = CBall + (int64_t)tile.expert * N * K;
  const float* SCB = SCBall + (int64_t)tile.expert * N;
  const __amdgpu_buffer_rsrc_t rB = make_rsrc(CB + (int64_t)n0 * K, min(BN, N - n0) * K);
  const int nc = (K + ET_KC - 1) / ET_KC, kp = nc * ET_KC;
  int8_t* mine = sw[wave];
  auto load_w = [&](int c) {
#pragma unroll
    for (int i = 0; i < ET_KC / 64; ++i) {
      const int row = (64 / LPR) * i + lane / LPR;
      const int k = c * ET_KC + 16 * ((lane % LPR) ^ row);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_ptr)(mine + i * 1024), 16, k < K ? row * K + k : OOB_OFFSET, 0,
                                               0, 0);
    }
  };
  if (wave < nc) load_w(wave);

  // quantization: a thread has chunks tid and tid + 256 of every token
  const int nchunk = (K + 15) / 16 * 2;      // codes up to a border of 16, zeros past K
  v4u ra[TM][CH], rb[TM][CH] = {};
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (t < T && tid + 256 * i < nchunk)
        load_raw8<DT>(X + (int64_t)t * K, (tid + 256 * i) * 8, K, vec, ra[t][i], rb[t][i]);
  const bool tau_on = tau > 0.0f && tau < __builtin_huge_valf();
  uint32_t om[CH], mx[TM] = {};
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    om[i] = 0u;
    if (tid + 256 * i < nchunk) {
      if (tau_on) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint32_t m = 0u;
#pragma unroll
          for (int t = 0; t < TM; ++t)
            if (t < T) m = max(m, chunk_mag<DT>(ra[t][i], rb[t][i], e));
          if (mag_to_half_value<DT>(m) > tau) om[i] |= 1u << e;
        }
      }
#pragma unroll
      for (int t = 0; t < TM; ++t)
        if (t < T) mx[t] = max(mx[t], chunk_absmax<DT, true>(ra[t][i], rb[t][i], om[i], true));
    }
    reinterpret_cast<uint8_t*>(smask)[tid + 256 * i] = (uint8_t)om[i];
  }
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    mx[t] = wave_umax(mx[t]);
    if (lane == 0) red[t][wave] = mx[t];
  }
  __syncthreads();
  auto scale = [&](int t) {
    return mag_to_half_value<DT>(max(max(red[t][0], red[t][1]), max(red[t][2], red[t][3])));
  };
#pragma unroll
  for (int t = 0; t < TM; ++t)
    if (t < T) {
      const float s = scale(t), inv = (s > 0.0f) ? (127.0f / s) : 0.0f;
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (tid + 256 * i < nchunk) {
          uint32_t lo, hi;
          chunk_quant8<DT>(ra[t][i], rb[t][i], inv, lo, hi);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if ((om[i] >> e) & 1u) lo &= ~(0xffu << (8 * e));
            if ((om[i] >> (e + 4)) & 1u) hi &= ~(0xffu << (8 * e));
          }
          *reinterpret_cast<v2u*>(codes + t * kp + (tid + 256 * i) * 8) = v2u{lo, hi};
        }
    }
  __syncthreads();

  const int r = tile.r0 + lr;
  const int t = r < tile.r1 ? row_token(rows, r, T) : -1;
  // the first wave finishes the tile; what it needs for that is requested before the contraction
  const int nb = n0 + 4 * lg;
  int cnt = 0, below = 0;      // outlier columns, and those in the words of the lanes before
  float sa = 0.0f, sb[4] = {};
  v8h P = {}, V = {};
  // columns of rank base .. base + EQ_LIST - 1, ascending
  auto list = [&](int base) {
    int j = below - base;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      for (uint32_t m = smask[2 * lane + h]; m != 0u; m &= m - 1u, ++j)
        if (j >= 0 && j < EQ_LIST) slist[j] = (uint16_t)((2 * lane + h) * 32 + __ffs(m) - 1);
    __builtin_amdgcn_wave_barrier();
  };
  auto operands = [&](int j0, int base) {
    P = v8h{};
    V = v8h{};
    const float sig = n0 + lr < N ? SCB[n0 + lr] * (1.0f / 127.0f) : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = j0 + lg * 8 + e;
      if (j < cnt) {
        const int col = slist[j - base];
        if (n0 + lr < N) P[e] = half_of_f32((float)CB[(int64_t)(n0 + lr) * K + col] * sig);
        if (t >= 0) V[e] = to_half<DT>(X[(int64_t)t * K + col]);
      }
    }
  };
  if (wave == 0) {
    if (t >= 0) sa = scale(t);
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (nb + x < N) sb[x] = SCB[nb + x];
    const int n = __popc(smask[2 * lane]) + __popc(smask[2 * lane + 1]);
    const int incl = lane_scan(n);
    below = incl - n;
    cnt = __builtin_amdgcn_readlane(incl, 63);
    if (cnt > 0) {
      list(0);
      operands(0, 0);
    }
  }
  v4i acc = {0, 0, 0, 0};
  const int8_t* mycodes = codes + max(t, 0) * kp;
  for (int c = wave; c < nc; c += 4) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const v4i w = *reinterpret_cast<const v4i*>(mine + lr * ET_KC + 16 * ((4 * s + lg) ^ lr));
      const v4i a = *reinterpret_cast<const v4i*>(mycodes + c * ET_KC + s * 64 + lg * 16);
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a, acc, 0, 0, 0);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the next piece lands in the same place
    if (c + 4 < nc) load_w(c + 4);
  }
  v4i* part = reinterpret_cast<v4i*>(sw[0]);
  __syncthreads();
  part[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave > 0) return;
  v4i sum = acc;
#pragma unroll
  for (int w = 1; w < 4; ++w) sum += part[w * 64 + lane];
  v4f y;
#pragma unroll
  for (int x = 0; x < 4; ++x) y[x] = (float)sum[x] * (sa * (sb[x] * (1.0f / 16129.0f)));
  if (cnt > 0) y = __builtin_amdgcn_mfma_f32_16x16x32_f16(P, V, y, 0, 0, 0);
  for (int jo = 32; jo < cnt; jo += 32) {
    const int base = jo / EQ_LIST * EQ_LIST;
    if (jo == base) list(base);
    operands(jo, base);
    y = __builtin_amdgcn_mfma_f32_16x16x32_f16(P, V, y, 0, 0, 0);
  }
  if (r < tile.r1) {
    float v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = t >= 0 ? y[x] : 0.0f;
    expert_store4<DT>(out + (int64_t)r * N + nb, v, N - nb, N % 4 == 0 && (uintptr_t)out % (4 * sizeof(E)) == 0);
  }
}

// Few rows: up to 10 a segment on average; or up to 64 where large tiles, cut
// in four, would not fill the chip.
static bool few_rows(int64_t R, int64_t n_seg, int64_t N) {
  if (R <= 10 * n_seg) return true;
  return R <= 64 * n_seg && expert_slots(R, n_seg, 256) * ((N + 255) / 256) <= 32;
}

bool expert_fwd_tiny_fits(int64_t T, int64_t K, const int8_t* CB, int64_t R, int64_t N, int64_t n_seg) {
  return T > 0 && T <= EQ_TOKENS && K > 0 && K <= EQ_COLS && K % 4 == 0 && (uintptr_t)CB % 4 == 0 &&
         few_rows(R, n_seg, N);
}

template <int DT>
static hipError_t launch_tiny_t(const void* X, int T, float tau, const int32_t* rows, int R, const ExpertSegs& S,
                                const int8_t* CB, const float* SCB, int N, int K, void* out, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  const int tiles_n = (N + 15) / 16, tm = T == 1 ? 1 : EQ_TOKENS;
  auto kern = T == 1 ? k_expert_fwd_tiny<DT, 1> : k_expert_fwd_tiny<DT, EQ_TOKENS>;
  const size_t lds = (size_t)tm * ((K + ET_KC - 1) / ET_KC * ET_KC);
  hipLaunchKernelGGL(kern, expert_grid(expert_slots(R, S.n_seg, 16) * tiles_n), dim3(256), lds, st,
                     static_cast<const E*>(X), T, K % 8 == 0 && (uintptr_t)X % 16 == 0, tau, rows, R, S, CB, SCB, N, K,
                     tiles_n, static_cast<E*>(out));
  return hipGetLastError();
}

hipError_t launch_expert_fwd_tiny(int dt, const void* X, int T, float tau, const int32_t* rows, int R,
                                  const ExpertSegs& S, const int8_t* CB, const float* SCB, int N, int K, void* out,
                                  hipStream_t st) {
  if (dt == DT_F32) return launch_tiny_t<DT_F32>(X, T, tau, rows, R, S, CB, SCB, N, K, out, st);
  if (dt == DT_F16) return launch_tiny_t<DT_F16>(X, T, tau, rows, R, S, CB, SCB, N, K, out, st);
  return launch_tiny_t<DT_BF16>(X, T, tau, rows, R, S, CB, SCB, N, K, out, st);
}

template <int DT>
static hipError_t launch_fwd_t(const ExpertQuantized& Q, const void* X, int T, const int32_t* rows, int R,
                               const ExpertSegs& S, const int8_t* CB, const float* SCB, int N, int K, void* out,
                               hipStream_t st) {
  typedef typename Elem<DT>::T E;
  const bool far = (int64_t)T * Q.lda >= ((int64_t)1 << 31);
  const bool words = K % 4 == 0 && (uintptr_t)CB % 4 == 0 && !far;
  if (few_rows(R, S.n_seg, N) || K < 16 || T == 0) {
    const int64_t slots = expert_slots(R, S.n_seg, 16);
    const bool split = K > 2048 || slots * ((N + 63) / 64) < 1024;
    const int tiles_n = split ? (N + 15) / 16 : (N + 63) / 64;
    auto kern = split ? (words ? k_expert_fwd_thin<DT, 4, 4> : k_expert_fwd_thin<DT, 1, 4>)
                      : (words ? k_expert_fwd_thin<DT, 4, 1> : k_expert_fwd_thin<DT, 1, 1>);
    hipLaunchKernelGGL(kern, expert_grid(slots * tiles_n), dim3(256), 0, st, Q,
                       static_cast<const E*>(X), T, rows, R, S, CB, SCB, N, K, tiles_n, static_cast<E*>(out));
    return hipGetLastError();
  }
  const int64_t tiles = expert_slots(R, S.n_seg, 128) * ((N + 127) / 128);
  if (K <= 512 || (K <= 1024 && tiles >= 256)) {
    auto kern = words ? k_expert_fwd_short<DT, 4> : k_expert_fwd_short<DT, 1>;
    hipLaunchKernelGGL(kern, expert_grid(tiles), dim3(256), 0, st, Q,
                       static_cast<const E*>(X), T, rows, R, S, CB, SCB, N, K, static_cast<E*>(out));
    return hipGetLastError();
  }
  static std::atomic<uint64_t> lds_set[2];
  auto kern = words ? k_expert_fwd<DT, 4> : k_expert_fwd<DT, 1>;
  constexpr int lds = ef_lds(256);
  const hipError_t e = lds_limit_once((const void*)kern, lds, lds_set[words]);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, expert_grid(expert_groups(expert_slots(R, S.n_seg, 256), (N + 255) / 256)), dim3(512),
                     lds, st, Q, static_cast<const E*>(X), T, rows, R, S, CB, SCB, N, K, static_cast<E*>(out));
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
