// Tokens to their experts' rows and back: a stable sort by expert, the weighted
// sum of each token's rows, and the gradients of that sum.
#include "expert.hpp"

namespace i8l {

// ---------------------------------------------------------------------------
// Sort. The R choices are cut into blocks and each block's into one run per
// wave. Counting goes through LDS atomics (integers: their order is nothing to
// the result). The place of a choice among those of its expert in the same 64
// is the number of earlier lanes with the same expert, found by one ballot for
// each bit of the number; the wave's own cursor for the expert holds the rest,
// so the sort is stable and the result the same on every run.
//
// Bound by launches and by the chains of dependent LDS accesses. One workgroup
// takes up to 8192 choices in one launch; more take a launch that counts and
// one that places, in which every workgroup adds up the counts of the others
// itself instead of waiting for a third. Two choices of 8 experts 11 us, of which the
// kernel 4.6; 8192 of 64 15 us; 131072 of 128 17 us (3 and 9 in the kernels), where the
// bytes alone would take half a microsecond.
constexpr int SORT_WAVES = 8, SORT_THREADS = 64 * SORT_WAVES;
constexpr int SORT_ALONE = 16 * SORT_THREADS;     // choices that one workgroup takes
constexpr int SORT_BLOCK = 4 * SORT_THREADS;      // of each of several, more where there would be over 256
constexpr int SORT_MAX_BLOCKS = 256;

static int sort_per_block(int64_t R) {
  if (R <= SORT_ALONE) return SORT_ALONE;
  const int64_t most = (R + SORT_MAX_BLOCKS - 1) / SORT_MAX_BLOCKS;
  return (int)((most > SORT_BLOCK ? most : SORT_BLOCK) + SORT_BLOCK - 1) / SORT_BLOCK * SORT_BLOCK;
}
static int sort_blocks(int64_t R) {
  const int pb = sort_per_block(R);
  return (int)((R + pb - 1) / pb);
}
size_t expert_sort_ints(int64_t R, int n_experts) {
  const int b = sort_blocks(R);
  return b > 1 ? (size_t)b * (size_t)n_experts : 0;
}

// f(choice, its expert or -1, whether there is one) for the wave's choices [lo, hi), 64 at a time in order, PER such
// groups loaded at once.
template <int PER, typename ID, typename F>
__device__ __forceinline__ void each_choice(const ID* __restrict__ ids, int lo, int hi, int E, F f) {
  const int lane = threadIdx.x & 63;
  for (int i0 = lo; i0 < hi; i0 += 64 * PER) {
    ID v[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int i = i0 + 64 * u + lane;
      v[u] = i < hi ? ids[i] : (ID)-1;
    }
#pragma unroll
    for (int u = 0; u < PER; ++u)
      if (i0 + 64 * u < hi) {
        const int i = i0 + 64 * u + lane;
        f(i, (v[u] >= 0 && v[u] < (ID)E) ? (int)v[u] : -1, i < hi);
      }
  }
}

// Counts of the block's choices by wave and expert, in LDS.
template <int PER, typename ID>
__device__ __forceinline__ void count_ids(const ID* __restrict__ ids, int lo, int hi, int E, int32_t* hist) {
  const int wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < SORT_WAVES * E; i += SORT_THREADS) hist[i] = 0;
  __syncthreads();
  each_choice<PER>(ids, lo, hi, E, [&](int, int e, bool) {
    if (e >= 0) atomicAdd(&hist[wave * E + e], 1);
  });
  __syncthreads();
}

template <typename ID>
__global__ __launch_bounds__(SORT_THREADS) void k_expert_count(const ID* __restrict__ ids, int R, int E,
                                                               int per_block, int32_t* __restrict__ counts) {
  extern __shared__ int32_t hist[];
  const int run = per_block / SORT_WAVES, wave = threadIdx.x >> 6;
  const int64_t b0 = (int64_t)blockIdx.x * per_block;
  const int lo = (int)min((int64_t)R, b0 + (int64_t)wave * run);
  const int hi = (int)min((int64_t)R, b0 + (int64_t)(wave + 1) * run);
  count_ids<4>(ids, lo, hi, E, hist);
  for (int e = threadIdx.x; e < E; e += SORT_THREADS) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < SORT_WAVES; ++w) n += hist[w * E + e];
    counts[(int64_t)blockIdx.x * E + e] = n;
  }
}

template <int PER, typename ID>
__global__ __launch_bounds__(SORT_THREADS) void k_expert_place(const ID* __restrict__ ids, int R, int k, int E,
                                                               int per_block, const int32_t* __restrict__ counts,
                                                               int32_t* __restrict__ off, int32_t* __restrict__ token,
                                                               int32_t* __restrict__ position) {
  extern __shared__ int32_t hist[];                // [SORT_WAVES][E], then one total a wave
  int32_t* sums = hist + SORT_WAVES * E;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // a block's choices are dealt out evenly, so that a few of them take all waves
  const int64_t b0 = (int64_t)blockIdx.x * per_block;
  const int mine = (int)min((int64_t)per_block, R - b0);
  const int run = ((mine + SORT_WAVES - 1) / SORT_WAVES + 63) / 64 * 64;
  const int lo = (int)b0 + min(mine, wave * run), hi = (int)b0 + min(mine, (wave + 1) * run);
  count_ids<PER>(ids, lo, hi, E, hist);

  // per expert: rows of all blocks, and of the blocks before this one
  int carry = 0;                                   // rows of the experts of earlier passes
  for (int e0 = 0; e0 < E; e0 += SORT_THREADS) {
    const int e = e0 + tid;
    int all = 0, before = 0, own = 0;
    if (e < E) {
#pragma unroll
      for (int w = 0; w < SORT_WAVES; ++w) own += hist[w * E + e];
      if (counts) {
        for (int b1 = 0; b1 < (int)gridDim.x; b1 += 16) {   // 16 loads in flight
          int c[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) c[u] = b1 + u < (int)gridDim.x ? counts[(int64_t)(b1 + u) * E + e] : 0;
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            all += c[u];
            before += b1 + u < (int)blockIdx.x ? c[u] : 0;
          }
        }
      } else {
        all = own;
      }
    }
    const int incl = lane_scan(all);
    if (lane == 63) sums[wave] = incl;
    __syncthreads();
    int first = carry, total = 0;
#pragma unroll
    for (int w = 0; w < SORT_WAVES; ++w) {
      const int v = sums[w];
      first += w < wave ? v : 0;
      total += v;
    }
    first += incl - all;
    if (e < E) {
      if (blockIdx.x == 0) off[e] = first;
      int at = first + before;
#pragma unroll
      for (int w = 0; w < SORT_WAVES; ++w) {       // counts become the waves' cursors
        const int n = hist[w * E + e];
        hist[w * E + e] = at;
        at += n;
      }
    }
    carry += total;
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) off[E] = carry;
  // rows behind the last routed one
  for (int64_t r = (int64_t)carry + blockIdx.x * SORT_THREADS + tid; r < R; r += (int64_t)gridDim.x * SORT_THREADS)
    token[r] = -1;

  const int bits = 32 - __clz(E);                  // of the numbers 0 .. E
  volatile int32_t* cursor = hist + wave * E;
  each_choice<PER>(ids, lo, hi, E, [&](int i, int e, bool in) {
    const int key = e < 0 ? E : e;
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((key >> b) & 1);
      same &= ((key >> b) & 1) ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int row = -1;
    if (e >= 0) row = cursor[e] + rank;
    __builtin_amdgcn_wave_barrier();               // every lane has read before the last one of each expert writes
    if (e >= 0 && rank == __popcll(same) - 1) cursor[e] = row + 1;
    __builtin_amdgcn_wave_barrier();
    if (in) {
      position[i] = row;
      if (row >= 0) token[row] = i / k;
    }
  });
}

template <typename ID>
static hipError_t launch_sort_t(const ID* ids, int R, int k, int E, int32_t* off, int32_t* token, int32_t* position,
                                int32_t* scratch, hipStream_t st) {
  const int blocks = R > 0 ? sort_blocks(R) : 1, pb = sort_per_block(R);
  const size_t lds = ((size_t)SORT_WAVES * E + SORT_WAVES) * sizeof(int32_t);
  if (blocks == 1) {
    hipLaunchKernelGGL((k_expert_place<16, ID>), dim3(1), dim3(SORT_THREADS), lds, st, ids, R, k, E, pb, nullptr, off,
                       token, position);
  } else {
    hipLaunchKernelGGL(k_expert_count<ID>, dim3(blocks), dim3(SORT_THREADS), lds, st, ids, R, E, pb, scratch);
    hipLaunchKernelGGL((k_expert_place<4, ID>), dim3(blocks), dim3(SORT_THREADS), lds, st, ids, R, k, E, pb, scratch,
                       off, token, position);
  }
  return hipGetLastError();
}

hipError_t launch_expert_sort(const void* experts, int id_bytes, int R, int k, int n_experts, int32_t* off,
                              int32_t* token, int32_t* position, int32_t* scratch, hipStream_t st) {
  if (id_bytes == 8)
    return launch_sort_t(static_cast<const int64_t*>(experts), R, k, n_experts, off, token, position, scratch, st);
  return launch_sort_t(static_cast<const int32_t*>(experts), R, k, n_experts, off, token, position, scratch, st);
}

// ---------------------------------------------------------------------------
// Weighted sum. A thread takes 8 columns of one token and adds its k rows in
// order, in fp32, then rounds once. Bound by memory: every row is read once. 4096
// tokens with two rows of 4096 and a base, bf16: 24.6 us, 5.4 TB/s.

template <int DT>
__device__ __forceinline__ void cld(const typename Elem<DT>::T* __restrict__ p, int n, bool vec, float (&f)[8]) {
  typename Elem<DT>::T e[8];
  if (vec) {
    load8<DT>(p, e);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = Elem<DT>::to_f32(e[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < n ? Elem<DT>::to_f32(p[j]) : 0.0f;
  }
}
template <int DT>
__device__ __forceinline__ void cst(typename Elem<DT>::T* __restrict__ p, int n, bool vec, const float (&f)[8]) {
  if (vec) {
    if constexpr (DT == DT_F32) {
      reinterpret_cast<v4f*>(p)[0] = v4f{f[0], f[1], f[2], f[3]};
      reinterpret_cast<v4f*>(p)[1] = v4f{f[4], f[5], f[6], f[7]};
    } else {
      v4u w;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = (uint32_t)__builtin_bit_cast(uint16_t, Elem<DT>::from_f32(f[2 * j])) |
               ((uint32_t)__builtin_bit_cast(uint16_t, Elem<DT>::from_f32(f[2 * j + 1])) << 16);
      *reinterpret_cast<v4u*>(p) = w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = Elem<DT>::from_f32(f[j]);
  }
}

// Workgroups of 256 threads as (256 / tx) tokens by tx chunks of 8 columns.
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void k_expert_combine(const typename Elem<DT>::T* __restrict__ Y, int R, int N,
                                                        const int32_t* __restrict__ position,
                                                        const float* __restrict__ gate,
                                                        const typename Elem<DT>::T* base, int T, int k, int txs,
                                                        typename Elem<DT>::T* out) {
  const int tx = threadIdx.x & ((1 << txs) - 1), ty = threadIdx.x >> txs;
  const int64_t t = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * (256 >> txs) + ty;
  const int c = (blockIdx.y * (1 << txs) + tx) * 8;
  if (t >= T || c >= N) return;
  const int n = min(8, N - c);
  float s[8] = {};
  if (base) cld<DT>(base + t * N + c, n, VEC, s);
  const int32_t* pos = position + t * k;
  const float* gt = gate ? gate + t * k : nullptr;
  for (int j0 = 0; j0 < k; j0 += 4) {
    float f[4][8], w[4];
    bool has[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = j0 + u < k ? pos[j0 + u] : -1;
      has[u] = r >= 0 && r < R;
      w[u] = has[u] ? (gt ? gt[j0 + u] : 1.0f) : 0.0f;
      if (has[u]) cld<DT>(Y + (int64_t)r * N + c, n, VEC, f[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (has[u]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = __builtin_fmaf(w[u], f[u][e], s[e]);
      }
  }
  cst<DT>(out + t * N + c, n, VEC, s);
}

template <int DT>
static hipError_t launch_combine_t(const void* Y, int R, int N, const int32_t* position, const float* gate,
                                   const void* base, int T, int k, void* out, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  const bool vec = N % 8 == 0 && (((uintptr_t)Y | (uintptr_t)base | (uintptr_t)out) % 16 == 0);
  const int chunks = (N + 7) / 8;
  int txs = 3;
  while (txs < 8 && (1 << txs) < chunks) ++txs;
  // workgroups of tokens in x and, over 2^20, in z: a grid axis holds fewer than 2^32 threads
  const dim3 tokens = expert_grid((T + (256 >> txs) - 1) / (256 >> txs));
  const dim3 grid(tokens.x, (unsigned)((chunks + (1 << txs) - 1) >> txs), tokens.y);
  auto kern = vec ? k_expert_combine<DT, true> : k_expert_combine<DT, false>;
  hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, static_cast<const E*>(Y), R, N, position, gate,
                     static_cast<const E*>(base), T, k, txs, static_cast<E*>(out));
  return hipGetLastError();
}

hipError_t launch_expert_combine(int dt, const void* Y, int R, int N, const int32_t* position, const float* gate,
                                 const void* base, int T, int k, void* out, hipStream_t st) {
  if (dt == DT_F32) return launch_combine_t<DT_F32>(Y, R, N, position, gate, base, T, k, out, st);
  if (dt == DT_F16) return launch_combine_t<DT_F16>(Y, R, N, position, gate, base, T, k, out, st);
  return launch_combine_t<DT_BF16>(Y, R, N, position, gate, base, T, k, out, st);
}

// ---------------------------------------------------------------------------
// Its gradients. A wave or a workgroup takes one token: each 8 columns of G are
// read once for four rows at a time, whose products with Y stay in registers
// until the end of the row; the gradient of each row is written as it is
// formed. Sums run in a fixed order. The last ZERO_BLOCKS workgroups write
// zeros into the rows behind the last routed one. 8192 tokens with eight rows of
// 2048, bf16: 119 us, 4.7 TB/s (reads and writes of 2 KB-rows in turn).
//
// ANY, positions of any kind: `named` holds the first and the last choice that
// names each row, by integer atomics, so that their order is nothing to the
// result. The first choice writes the row; where it is not the last one too, it
// looks through the choices between them, 256 at a time, and adds theirs in
// order. The zeros go to rows without a first choice. The same 8192 tokens, no row
// named twice: 148 us, of which 9 for `named`; every row twice 450; all 65536
// choices on one row, which one workgroup adds up, 20 ms.
constexpr int ZERO_BLOCKS = 256;
constexpr int NO_CHOICE = 0x7fffffff;

__global__ __launch_bounds__(256) void k_named_clear(int32_t* __restrict__ named, int R) {
  for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < R; r += (int64_t)gridDim.x * 256) {
    named[r] = NO_CHOICE;
    named[R + r] = -1;
  }
}
__global__ __launch_bounds__(256) void k_named(const int32_t* __restrict__ position, int choices, int R,
                                               int32_t* __restrict__ named) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < choices; i += (int64_t)gridDim.x * 256) {
    const int r = position[i];
    if (r >= 0 && r < R) {
      atomicMin(&named[r], (int)i);
      atomicMax(&named[R + r], (int)i);
    }
  }
}

template <int DT, bool VEC, int TT, bool ANY>   // TT threads a token: 64 or 256
__global__ __launch_bounds__(256) void k_expert_combine_bwd(const typename Elem<DT>::T* __restrict__ G, int T, int N,
                                                            const int32_t* __restrict__ position,
                                                            const float* __restrict__ gate, int k,
                                                            const typename Elem<DT>::T* __restrict__ Y, int R,
                                                            const int32_t* __restrict__ n_rows,   // ANY: named
                                                            typename Elem<DT>::T* __restrict__ gY,
                                                            float* __restrict__ ggate) {
  constexpr int PER = 256 / TT;
  const int blocks = (T + PER - 1) / PER, lane = threadIdx.x & 63;
  const int64_t bid = expert_block();
  if (bid >= blocks) {
    if (!n_rows || bid >= blocks + ZERO_BLOCKS) return;
    const float zero[8] = {};
    if constexpr (ANY) {
      // rows side by side go to different waves: those behind the last routed one lie together
      constexpr int64_t WAVES = ZERO_BLOCKS * 4;
      for (int64_t r0 = (bid - blocks) * 4 + (threadIdx.x >> 6); r0 < R; r0 += 64 * WAVES) {
        const int64_t mine = r0 + lane * WAVES;
        uint64_t none = __ballot(mine < R && n_rows[mine] == NO_CHOICE);
        for (; none != 0; none &= none - 1) {
          const int64_t r = r0 + __builtin_ctzll(none) * WAVES;
          for (int c = lane * 8; c < N; c += 512) cst<DT>(gY + r * N + c, min(8, N - c), VEC, zero);
        }
      }
      return;
    }
    const int64_t from = min(max(n_rows[0], 0), R);
    const int chunks = (N + 7) / 8;
    const int64_t items = (R - from) * (int64_t)chunks;
    for (int64_t i = (bid - blocks) * 256 + threadIdx.x; i < items; i += (int64_t)ZERO_BLOCKS * 256) {
      const int64_t r = i / chunks;
      const int c = (int)(i - r * chunks) * 8;
      cst<DT>(gY + (from + r) * N + c, min(8, N - c), VEC, zero);
    }
    return;
  }
  __shared__ float part[4][4];
  const int tid = threadIdx.x % TT, t = (int)bid * PER + threadIdx.x / TT;
  const bool live = t < T;
  const int32_t* pos = position + (int64_t)(live ? t : 0) * k;
  const float* gt = gate ? gate + (int64_t)(live ? t : 0) * k : nullptr;
  const typename Elem<DT>::T* g = G + (int64_t)(live ? t : 0) * N;
  // ANY: the token's choices (at most 64) that alone name their rows, and those that are the first of several; looked up
  // together, once, so that rows and products wait for nothing (172 us against 148 where every four choices asked)
  uint64_t single = 0, several = 0;
  if constexpr (ANY) {
    if (gY) {
      const int r = live && lane < k ? pos[lane] : -1, i = t * k + lane;
      const bool has = r >= 0 && r < R;
      const int first = has ? n_rows[r] : -1, last = has ? n_rows[R + r] : -1;
      single = __ballot(first == i && last == i);
      several = __ballot(first == i && last > i);
    }
  }
  for (int j0 = 0; j0 < k; j0 += 4) {
    int64_t row[4];
    float w[4], dot[4] = {};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = live && j0 + u < k ? pos[j0 + u] : -1;
      row[u] = (r >= 0 && r < R) ? (int64_t)r * N : -1;
      w[u] = row[u] >= 0 ? (gt ? gt[j0 + u] : 1.0f) : 0.0f;
    }
    for (int c = tid * 8; c < N; c += TT * 8) {
      const int n = min(8, N - c);
      float f[8];
      cld<DT>(g + c, n, VEC, f);
      float y[4][8];
      if (ggate) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (row[u] >= 0) cld<DT>(Y + row[u] + c, n, VEC, y[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (row[u] >= 0) {
          if (gY && (!ANY || (single >> (j0 + u)) & 1)) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = w[u] * f[e];
            cst<DT>(gY + row[u] + c, n, VEC, o);
          }
          if (ggate) {
#pragma unroll
            for (int e = 0; e < 8; ++e) dot[u] = __builtin_fmaf(f[e], y[u][e], dot[u]);
          }
        }
    }
    if constexpr (ANY) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j0 + u < k && (several >> (j0 + u)) & 1) {      // alike in all of the token's threads
          const int r = pos[j0 + u], from = t * k + j0 + u + 1, to = n_rows[R + r];      // below 2^30
          for (int c0 = 0; c0 < N; c0 += TT * 8) {
            const int c = c0 + tid * 8, n = min(8, N - c);
            float s[8] = {}, f[8];
            if (c < N) {
              cld<DT>(g + c, n, VEC, f);
#pragma unroll
              for (int e = 0; e < 8; ++e) s[e] = w[u] * f[e];
            }
            for (int i0 = from; i0 <= to; i0 += 256) {
              int p[4];
#pragma unroll
              for (int b = 0; b < 4; ++b) p[b] = i0 + 64 * b + lane <= to ? position[i0 + 64 * b + lane] : -1;
#pragma unroll
              for (int b = 0; b < 4; ++b)
                for (uint64_t same = __ballot(p[b] == r); same != 0; same &= same - 1) {
                  const int i = i0 + 64 * b + __builtin_ctzll(same);
                  const float wi = gate ? gate[i] : 1.0f;
                  if (c < N) {
                    cld<DT>(G + (int64_t)(i / k) * N + c, n, VEC, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] = __builtin_fmaf(wi, f[e], s[e]);
                  }
                }
            }
            if (c < N) cst<DT>(gY + row[u] + c, n, VEC, s);
          }
        }
    }
    if (ggate) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) dot[u] += __shfl_xor(dot[u], o, 64);
      if constexpr (TT == 256) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
          for (int u = 0; u < 4; ++u) part[threadIdx.x >> 6][u] = dot[u];
        __syncthreads();
        if (tid < 4 && j0 + tid < k)
          ggate[(int64_t)t * k + j0 + tid] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        __syncthreads();
      } else if (live && tid == 0) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (j0 + u < k) ggate[(int64_t)t * k + j0 + u] = dot[u];
      }
    }
  }
}

template <int DT, int TT>
static hipError_t launch_combine_bwd_t(const void* G, int T, int N, const int32_t* position, const float* gate, int k,
                                       const void* Y, int R, const int32_t* n_rows, int32_t* named, void* gY,
                                       float* ggate, hipStream_t st) {
  typedef typename Elem<DT>::T E;
  const bool vec = N % 8 == 0 && (((uintptr_t)G | (uintptr_t)Y | (uintptr_t)gY) % 16 == 0);
  if (!gY || R == 0) n_rows = named = nullptr;
  const int64_t blocks = (T + 256 / TT - 1) / (256 / TT) + (n_rows || named ? ZERO_BLOCKS : 0);
  if (blocks == 0) return hipSuccess;
  auto kern = vec ? k_expert_combine_bwd<DT, true, TT, false> : k_expert_combine_bwd<DT, false, TT, false>;
  if (named) {
    auto grid = [](int64_t n) { return dim3((unsigned)(n < 4096 * 256 ? (n + 255) / 256 : 4096)); };
    hipLaunchKernelGGL(k_named_clear, grid(R), dim3(256), 0, st, named, R);
    if (T > 0) hipLaunchKernelGGL(k_named, grid((int64_t)T * k), dim3(256), 0, st, position, T * k, R, named);
    kern = vec ? k_expert_combine_bwd<DT, true, TT, true> : k_expert_combine_bwd<DT, false, TT, true>;
    n_rows = named;
  }
  hipLaunchKernelGGL(kern, expert_grid(blocks), dim3(256), 0, st, static_cast<const E*>(G), T, N, position, gate, k,
                     static_cast<const E*>(Y), R, n_rows, static_cast<E*>(gY), ggate);
  return hipGetLastError();
}

hipError_t launch_expert_combine_bwd(int dt, const void* G, int T, int N, const int32_t* position, const float* gate,
                                     int k, const void* Y, int R, const int32_t* n_rows, int32_t* named, void* gY,
                                     float* ggate, hipStream_t st) {
#define I8L_CB(D)                                                                                                  \
  return N <= 1024 ? launch_combine_bwd_t<D, 64>(G, T, N, position, gate, k, Y, R, n_rows, named, gY, ggate, st)   \
                   : launch_combine_bwd_t<D, 256>(G, T, N, position, gate, k, Y, R, n_rows, named, gY, ggate, st)
  if (dt == DT_F32) I8L_CB(DT_F32);
  if (dt == DT_F16) I8L_CB(DT_F16);
  I8L_CB(DT_BF16);
#undef I8L_CB
}

}  // namespace i8l
