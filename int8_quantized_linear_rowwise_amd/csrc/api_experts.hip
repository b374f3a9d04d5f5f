// C-ABI host layer of the experts' operators and the gradient norm: argument
// validation before any HIP call, workspace carving and kernel launches on the
// caller's stream.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "../../include/int8lin.h"
#include "kernels.hpp"

namespace {

constexpr size_t ALIGN = 256;
constexpr int64_t MAX_ROWS = (int64_t)1 << 24;
constexpr int64_t MAX_SEGMENTS = 65536;
constexpr int64_t MAX_VALUES = (int64_t)1 << 40;
constexpr int64_t MAX_CHOICES = 64;   // experts of a token in the weighted sum
constexpr int32_t SUB_COLS = 64;      // outlier columns staged by the quantizer; further ones are read from X

size_t align_up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }
bool valid_dtype(int dt) { return dt == I8L_F32 || dt == I8L_F16 || dt == I8L_BF16; }
int hip_status(hipError_t e) { return e == hipSuccess ? I8L_OK : I8L_EHIP; }

// Bytes of a row of codes: rows start on 16-byte borders whatever K is.
int code_row(int64_t K) { return (int)((K + 15) / 16 * 16); }

struct Layout {
  size_t count, idx, scale, codes, sub, scratch, total;
  int32_t cap;
};
Layout forward_layout(int64_t T, int64_t K) {
  Layout L;
  L.cap = K < SUB_COLS ? (int32_t)K : SUB_COLS;
  size_t at = 0;
  L.count = at;
  at += ALIGN;
  L.idx = at;
  at += align_up((size_t)K * 4);
  L.scale = at;
  at += align_up((size_t)T * 4);
  L.codes = at;
  at += align_up((size_t)T * (size_t)code_row(K));
  L.sub = at;
  at += align_up((size_t)T * (size_t)L.cap * 2);
  L.scratch = at;
  at += align_up(i8l::quant_scratch_words(T, K) * 4);
  L.total = at;
  return L;
}

int product_sizes(int64_t R, int64_t N, int64_t K, int64_t n_experts, int64_t n_seg) {
  if (R < 0 || N < 0 || K < 0 || n_experts < 0 || n_seg < 0) return I8L_EINVAL;
  if (R > MAX_ROWS || N > I8L_MAX_COLS || K > I8L_MAX_K || n_experts > MAX_SEGMENTS || n_seg > MAX_SEGMENTS ||
      R * N > MAX_VALUES || R * K > MAX_VALUES || n_experts * N > INT32_MAX || n_experts * N * K > MAX_VALUES)
    return I8L_ESHAPE;
  return I8L_OK;
}

// Lists of at most GRAD_LIST tensors: f(list, its partial sums' start), and for no tensors one empty list. I8L_OK,
// I8L_EINVAL, I8L_EDTYPE or I8L_ESHAPE.
template <typename F>
int grad_lists(const i8l_grad_tensor* t, int64_t count, F f) {
  if (count < 0 || (count > 0 && t == nullptr)) return I8L_EINVAL;
  if (count > ((int64_t)1 << 24)) return I8L_ESHAPE;
  int64_t at = 0, i = 0;
  do {
    i8l::GradList l;
    l.count = 0;
    int64_t chunks = 0;
    for (; i < count && l.count < i8l::GRAD_LIST; ++i) {
      if (t[i].n < 0) return I8L_EINVAL;
      if (!valid_dtype(t[i].dtype)) return I8L_EDTYPE;
      if (t[i].n == 0) continue;
      if (t[i].g == nullptr || (uintptr_t)t[i].g % (t[i].dtype == I8L_F32 ? 4 : 2)) return I8L_EINVAL;
      if (t[i].n > MAX_VALUES) return I8L_ESHAPE;
      l.p[l.count] = t[i].g;
      const int64_t c = (t[i].n + i8l::grad_chunk() - 1) / i8l::grad_chunk();
      l.last[l.count] = (uint16_t)((t[i].n - (c - 1) * i8l::grad_chunk()) << 2 | t[i].dtype);
      l.start[l.count++] = (int32_t)chunks;
      chunks += c;
      if (chunks > (1 << 29)) return I8L_ESHAPE;
    }
    l.start[l.count] = (int32_t)chunks;
    const int rc = f(l, at);
    if (rc != I8L_OK) return rc;
    at += i8l::grad_groups(chunks);
  } while (i < count);
  return I8L_OK;
}
// Partial sums of all lists: *n, 0 where a single list is small enough for one launch.
int grad_partials(const i8l_grad_tensor* t, int64_t count, int64_t* n) {
  *n = 0;
  return grad_lists(t, count, [&](const i8l::GradList& l, int64_t at) {
    const int chunks = l.start[l.count];
    *n = at + (at == 0 && count <= i8l::GRAD_LIST && chunks <= i8l::grad_small_chunks() ? 0 : i8l::grad_groups(chunks));
    return *n > INT32_MAX ? I8L_ESHAPE : I8L_OK;
  });
}

}  // namespace

extern "C" {

size_t int8_expert_sort_workspace_bytes(int64_t T, int64_t k, int64_t n_experts) {
  if (T < 0 || k < 0 || n_experts < 0 || n_experts > I8L_SORT_MAX_EXPERTS || T > MAX_ROWS || k > MAX_ROWS ||
      T * k > MAX_ROWS)
    return 0;
  return align_up(i8l::expert_sort_ints(T * k, (int)n_experts) * sizeof(int32_t));
}

int int8_expert_sort(const void* experts, int id_bytes, int64_t T, int64_t k, int64_t n_experts, int32_t* seg_offsets,
                     int32_t* row_token, int32_t* position, void* ws, size_t ws_bytes, void* stream) {
  if (id_bytes != 4 && id_bytes != 8) return I8L_EDTYPE;
  if (T < 0 || k < 0 || n_experts < 0) return I8L_EINVAL;
  if (n_experts > I8L_SORT_MAX_EXPERTS || T > MAX_ROWS || k > MAX_ROWS || T * k > MAX_ROWS) return I8L_ESHAPE;
  if (seg_offsets == nullptr) return I8L_EINVAL;
  if (T * k > 0 && (experts == nullptr || row_token == nullptr || position == nullptr)) return I8L_EINVAL;
  const size_t need = int8_expert_sort_workspace_bytes(T, k, n_experts);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return I8L_EWORKSPACE;
  if ((uintptr_t)ws % ALIGN) return I8L_EINVAL;
  return hip_status(i8l::launch_expert_sort(experts, id_bytes, (int)(T * k), (int)k, (int)n_experts, seg_offsets,
                                            row_token, position, static_cast<int32_t*>(ws), (hipStream_t)stream));
}

size_t int8_expert_forward_workspace_bytes(int64_t T, int64_t K, const int8_t* CB, int64_t R, int64_t N,
                                           int64_t n_seg) {
  if (T < 0 || T > MAX_ROWS || T * K > MAX_VALUES || product_sizes(R, N, K, 0, n_seg) != I8L_OK) return 0;
  return i8l::expert_fwd_tiny_fits(T, K, CB, R, N, n_seg) ? 0 : forward_layout(T, K).total;
}

int int8_expert_forward(const void* X, int dtype, int64_t T, int64_t K, const int32_t* rows, int64_t R,
                        const int8_t* CB, const float* SCB, int64_t n_experts, int64_t N, const int32_t* seg_offsets,
                        const int32_t* seg_expert, int64_t n_seg, float threshold, void* out, void* ws,
                        size_t ws_bytes, void* stream) {
  if (!valid_dtype(dtype)) return I8L_EDTYPE;
  if (T < 0) return I8L_EINVAL;
  const int rc = product_sizes(R, N, K, n_experts, n_seg);
  if (rc != I8L_OK) return rc;
  if (T > MAX_ROWS || T * K > MAX_VALUES) return I8L_ESHAPE;
  if (rows == nullptr && R != T) return I8L_EINVAL;
  if (n_seg > 0 && seg_offsets == nullptr) return I8L_EINVAL;
  if (R > 0 && N > 0 && out == nullptr) return I8L_EINVAL;
  if (T > 0 && K > 0 && X == nullptr) return I8L_EINVAL;
  if (n_experts > 0 && N > 0 && (SCB == nullptr || (K > 0 && CB == nullptr))) return I8L_EINVAL;
  const Layout L = forward_layout(T, K);
  const bool tiny = i8l::expert_fwd_tiny_fits(T, K, CB, R, N, n_seg);
  if (!tiny && (ws == nullptr || ws_bytes < L.total)) return I8L_EWORKSPACE;
  if ((uintptr_t)ws % ALIGN) return I8L_EINVAL;
  if (R == 0 || N == 0) return I8L_OK;
  const i8l::ExpertSegs S = {seg_offsets, seg_expert, (int)n_seg, (int)n_experts};
  if (tiny)
    return hip_status(i8l::launch_expert_fwd_tiny(dtype, X, (int)T, threshold, rows, (int)R, S, CB, SCB, (int)N, (int)K,
                                                  out, (hipStream_t)stream));
  char* w = static_cast<char*>(ws);
  int32_t* count = reinterpret_cast<int32_t*>(w + L.count);
  int32_t* idx = reinterpret_cast<int32_t*>(w + L.idx);
  float* SCA = reinterpret_cast<float*>(w + L.scale);
  int8_t* CA = reinterpret_cast<int8_t*>(w + L.codes);
  const int lda = code_row(K);
  uint16_t* sub = reinterpret_cast<uint16_t*>(w + L.sub);
  hipStream_t st = (hipStream_t)stream;
  const hipError_t e =
      i8l::quantize_small_fits(T, K, threshold)
          ? i8l::launch_quantize_small(dtype, X, (int)T, (int)K, threshold, CA, lda, SCA, idx, count, sub, L.cap,
                                       st)
          : i8l::launch_quantize(dtype, X, T, (int)K, threshold, CA, SCA, idx, count, sub, L.cap,
                                 reinterpret_cast<uint32_t*>(w + L.scratch), st, nullptr, (int)K, nullptr, lda);
  if (e != hipSuccess) return I8L_EHIP;
  const i8l::ExpertQuantized Q = {CA, lda, SCA, sub, L.cap, idx, count};
  return hip_status(i8l::launch_expert_fwd(dtype, Q, X, (int)T, rows, (int)R, S, CB, SCB, (int)N, (int)K, out, st));
}

size_t int8_expert_backward_workspace_bytes(const void* G, int dtype, int64_t R, int64_t N) {
  if (!valid_dtype(dtype) || R < 0 || N < 0 || R > MAX_ROWS || N > I8L_MAX_COLS || R * N > MAX_VALUES) return 0;
  return align_up(i8l::expert_bwd_bytes(G, dtype, R, N));
}

int int8_expert_backward(const void* G, int dtype, int64_t R, int64_t N, const int8_t* CB, const float* SCB,
                         int64_t n_experts, int64_t K, const int32_t* seg_offsets, const int32_t* seg_expert,
                         int64_t n_seg, void* grad_X, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_dtype(dtype)) return I8L_EDTYPE;
  const int rc = product_sizes(R, N, K, n_experts, n_seg);
  if (rc != I8L_OK) return rc;
  if (n_seg > 0 && seg_offsets == nullptr) return I8L_EINVAL;
  if (R > 0 && K > 0 && grad_X == nullptr) return I8L_EINVAL;
  if (R > 0 && N > 0 && G == nullptr) return I8L_EINVAL;
  if (n_experts > 0 && N > 0 && (SCB == nullptr || (K > 0 && CB == nullptr))) return I8L_EINVAL;
  const size_t need = int8_expert_backward_workspace_bytes(G, dtype, R, N);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return I8L_EWORKSPACE;
  if ((uintptr_t)ws % ALIGN) return I8L_EINVAL;
  if (R == 0 || K == 0) return I8L_OK;
  const i8l::ExpertSegs S = {seg_offsets, seg_expert, (int)n_seg, (int)n_experts};
  return hip_status(
      i8l::launch_expert_bwd(dtype, G, (int)R, S, CB, SCB, (int)N, (int)K, grad_X, ws, (hipStream_t)stream));
}

static int combine_sizes(int dtype, int64_t R, int64_t N, int64_t T, int64_t k) {
  if (!valid_dtype(dtype)) return I8L_EDTYPE;
  if (R < 0 || N < 0 || T < 0 || k < 0) return I8L_EINVAL;
  if (R > MAX_ROWS || T > MAX_ROWS || N > I8L_MAX_COLS || k > MAX_CHOICES || R * N > MAX_VALUES || T * N > MAX_VALUES)
    return I8L_ESHAPE;
  return I8L_OK;
}

int int8_expert_combine(const void* Y, int dtype, int64_t R, int64_t N, const int32_t* position, const float* gate,
                        const void* base, int64_t T, int64_t k, void* out, void* stream) {
  const int rc = combine_sizes(dtype, R, N, T, k);
  if (rc != I8L_OK) return rc;
  if (T == 0 || N == 0) return I8L_OK;
  if (out == nullptr || (k > 0 && position == nullptr) || (k > 0 && R > 0 && Y == nullptr)) return I8L_EINVAL;
  return hip_status(i8l::launch_expert_combine(dtype, Y, (int)R, (int)N, position, gate, base, (int)T, (int)k, out,
                                               (hipStream_t)stream));
}

int int8_expert_combine_backward(const void* G, int dtype, int64_t T, int64_t N, const int32_t* position,
                                 const float* gate, int64_t k, const void* Y, int64_t R, const int32_t* n_rows,
                                 void* grad_Y, float* grad_gate, void* stream) {
  const bool any = dtype >= 0 && (dtype & I8L_ANY_POSITIONS) != 0;
  if (any) dtype &= ~I8L_ANY_POSITIONS;
  const int rc = combine_sizes(dtype, R, N, T, k);
  if (rc != I8L_OK) return rc;
  if (T > 0 && k > 0) {
    if (position == nullptr || (N > 0 && G == nullptr)) return I8L_EINVAL;
    if (grad_gate && N > 0 && R > 0 && Y == nullptr) return I8L_EINVAL;
  }
  if (any && grad_Y && R > 0 && (n_rows == nullptr || (uintptr_t)n_rows % 4)) return I8L_EINVAL;
  if (!grad_Y && !grad_gate) return I8L_OK;
  int32_t* named = any ? const_cast<int32_t*>(n_rows) : nullptr;
  return hip_status(i8l::launch_expert_combine_bwd(dtype, G, k > 0 ? (int)T : 0, (int)N, position, gate, (int)k, Y,
                                                   (int)R, any ? nullptr : n_rows, named, grad_Y, grad_gate,
                                                   (hipStream_t)stream));
}

size_t int8_grad_norm_workspace_bytes(const i8l_grad_tensor* grads, int64_t count) {
  int64_t n = 0;
  if (grad_partials(grads, count, &n) != I8L_OK) return 0;
  return align_up((size_t)n * sizeof(double));
}

int int8_grad_norm(const i8l_grad_tensor* grads, int64_t count, int norm_type, double max_norm,
                   const float* grad_scale, int clip, float* norm, float* factor, float* found_inf, void* ws,
                   size_t ws_bytes, void* stream) {
  int64_t n = 0;
  const int rc = grad_partials(grads, count, &n);
  if (rc != I8L_OK) return rc;
  if (norm_type != 2 && norm_type != I8L_NORM_INF) return I8L_EINVAL;
  if (!(max_norm >= 0.0) || !norm || !factor || !found_inf) return I8L_EINVAL;
  if (n > 0 && (ws == nullptr || ws_bytes < (size_t)n * sizeof(double))) return I8L_EWORKSPACE;
  if ((uintptr_t)ws % ALIGN) return I8L_EINVAL;
  const bool inf = norm_type == I8L_NORM_INF;
  hipStream_t st = (hipStream_t)stream;
  if (n == 0 && count <= i8l::GRAD_LIST)
    return grad_lists(grads, count, [&](const i8l::GradList& l, int64_t) {
      return hip_status(
          i8l::launch_grad_small(l, inf, max_norm, grad_scale, clip, norm, factor, found_inf, st));
    });
  double* partial = static_cast<double*>(ws);
  int e = grad_lists(grads, count, [&](const i8l::GradList& l, int64_t at) {
    return hip_status(i8l::launch_grad_partial(l, inf, partial + at, st));
  });
  if (e != I8L_OK) return e;
  e = hip_status(i8l::launch_grad_final(partial, (int)n, inf, max_norm, grad_scale, norm, factor, found_inf, st));
  if (e != I8L_OK || !clip) return e;
  return grad_lists(grads, count,
                    [&](const i8l::GradList& l, int64_t) { return hip_status(i8l::launch_grad_scale(l, factor, st)); });
}

}  // extern "C"
