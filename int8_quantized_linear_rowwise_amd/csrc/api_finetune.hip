// C-ABI host layer of the operators around the frozen projection (adapters,
// layer norm, AdamW): argument validation before any HIP call, workspace
// carving and kernel launches on the caller's stream.
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/int8lin.h"
#include "kernels.hpp"

namespace {

constexpr size_t ALIGN = 256;
constexpr int64_t MAX_TOKENS = (int64_t)1 << 24;   // rows; tiles of 16 rows and their threads stay within a grid axis
constexpr int64_t MAX_SEGMENTS = (int64_t)1 << 20;
constexpr int64_t MAX_ADAPTERS = 65535;
constexpr int64_t MAX_ADAPTER_VALUES = (int64_t)1 << 33;
constexpr int64_t MAX_VALUES = (int64_t)1 << 40;

size_t align_up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }
bool valid_dtype(int dt) { return dt == I8L_F32 || dt == I8L_F16 || dt == I8L_BF16; }
int hip_status(hipError_t e) { return e == hipSuccess ? I8L_OK : I8L_EHIP; }

// Sizes of an adapter call: I8L_OK, I8L_EINVAL or I8L_ESHAPE.
int lora_sizes(int64_t T, int64_t K, int64_t N, int64_t R, int64_t n_adapters, int64_t n_seg) {
  if (T < 0 || K < 0 || N < 0 || R < 0 || n_adapters < 0 || n_seg < 0) return I8L_EINVAL;
  if (T > MAX_TOKENS || n_seg > MAX_SEGMENTS || K > I8L_MAX_COLS || N > I8L_MAX_COLS ||
      R > I8L_LORA_MAX_RANK || n_adapters > MAX_ADAPTERS || T * K > MAX_VALUES || T * N > MAX_VALUES)
    return I8L_ESHAPE;
  // adapters padded to a rank of 16, 32, 64 or 128: the gradient's sums take a workgroup for 1024 values of them
  const int64_t rp = R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128;
  if (n_adapters * rp * (K > N ? K : N) > MAX_ADAPTER_VALUES) return I8L_ESHAPE;
  return I8L_OK;
}

}  // namespace

extern "C" {

size_t int8_lora_forward_workspace_bytes(int64_t T, int64_t K, int64_t N, int64_t R, int64_t n_seg) {
  if (lora_sizes(T, K, N, R, 0, n_seg) != I8L_OK) return 0;
  return align_up(i8l::lora_forward_floats((int)T, (int)K, (int)N, (int)R, (int)n_seg) * sizeof(float));
}

int int8_lora_forward(const void* X, int dtype, int64_t T, int64_t K, const void* A, const void* B,
                      const float* scaling, int64_t n_adapters, int64_t R, int64_t N, const int32_t* seg_offsets,
                      const int32_t* seg_adapter, int64_t n_seg, const void* base, void* out, float* V, void* ws,
                      size_t ws_bytes, void* stream) {
  if (!valid_dtype(dtype)) return I8L_EDTYPE;
  const int rc = lora_sizes(T, K, N, R, n_adapters, n_seg);
  if (rc != I8L_OK) return rc;
  if (T == 0) return I8L_OK;
  if (N > 0 && out == nullptr) return I8L_EINVAL;
  if (K > 0 && X == nullptr) return I8L_EINVAL;
  if (n_seg > 1 && seg_offsets == nullptr) return I8L_EINVAL;
  const bool any = n_adapters > 0 && R > 0;
  if (any && (scaling == nullptr || (K > 0 && A == nullptr) || (N > 0 && B == nullptr))) return I8L_EINVAL;
  const size_t need = int8_lora_forward_workspace_bytes(T, K, N, R, n_seg);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return I8L_EWORKSPACE;
  if ((uintptr_t)ws % ALIGN) return I8L_EINVAL;
  const i8l::LoraSegs S = {seg_offsets, seg_adapter, (int)n_seg, any ? (int)n_adapters : 0};
  return hip_status(i8l::launch_lora_forward(dtype, X, (int)T, (int)K, A, B, scaling, (int)R, (int)N, S, base, out, V,
                                             static_cast<float*>(ws), (hipStream_t)stream));
}

size_t int8_lora_backward_workspace_bytes(int64_t T, int64_t K, int64_t N, int64_t R, int64_t n_adapters,
                                          int64_t n_seg) {
  if (lora_sizes(T, K, N, R, n_adapters, n_seg) != I8L_OK) return 0;
  return align_up(
      i8l::lora_backward_floats((int)T, (int)K, (int)N, (int)R, (int)n_adapters, (int)n_seg) * sizeof(float));
}

int int8_lora_backward(const void* G, const void* X, const float* V, int dtype, int64_t T, int64_t K, const void* A,
                       const void* B, const float* scaling, int64_t n_adapters, int64_t R, int64_t N,
                       const int32_t* seg_offsets, const int32_t* seg_adapter, int64_t n_seg, const void* base_grad,
                       void* grad_X, void* grad_A, void* grad_B, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_dtype(dtype)) return I8L_EDTYPE;
  const int rc = lora_sizes(T, K, N, R, n_adapters, n_seg);
  if (rc != I8L_OK) return rc;
  const bool any = n_adapters > 0 && R > 0;
  if (T > 0) {
    if (n_seg > 1 && seg_offsets == nullptr) return I8L_EINVAL;
    if (any) {
      if (scaling == nullptr) return I8L_EINVAL;
      if ((grad_X || grad_A) && N > 0 && (G == nullptr || B == nullptr)) return I8L_EINVAL;
      if (grad_X && K > 0 && A == nullptr) return I8L_EINVAL;
      if (grad_A && K > 0 && X == nullptr) return I8L_EINVAL;
      if (grad_B && N > 0 && (G == nullptr || V == nullptr)) return I8L_EINVAL;
    }
  }
  const size_t need = int8_lora_backward_workspace_bytes(T, K, N, R, n_adapters, n_seg);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return I8L_EWORKSPACE;
  if ((uintptr_t)ws % ALIGN) return I8L_EINVAL;
  const i8l::LoraSegs S = {seg_offsets, seg_adapter, (int)n_seg, any ? (int)n_adapters : 0};
  return hip_status(i8l::launch_lora_backward(dtype, G, X, V, (int)T, (int)K, A, B, scaling, (int)R, (int)N, S,
                                              (int)n_adapters, base_grad, grad_X, grad_A, grad_B, static_cast<float*>(ws),
                                              (hipStream_t)stream));
}

static int norm_args(int dtype, int weight_dtype, int64_t T, int64_t C) {
  if (!valid_dtype(dtype) || !valid_dtype(weight_dtype) || (weight_dtype != dtype && weight_dtype != I8L_F32))
    return I8L_EDTYPE;
  if (T < 0 || C < 0) return I8L_EINVAL;
  if (T > MAX_TOKENS || C > I8L_MAX_COLS || T * C > MAX_VALUES) return I8L_ESHAPE;
  return I8L_OK;
}

int int8_layer_norm_forward(const void* X, int dtype, int64_t T, int64_t C, const void* weight, const void* bias,
                            int weight_dtype, float eps, void* out, float* mean, float* rstd, void* stream) {
  const int rc = norm_args(dtype, weight_dtype, T, C);
  if (rc != I8L_OK) return rc;
  if (!(eps >= 0.0f)) return I8L_EINVAL;
  if (T == 0 || C == 0) return I8L_OK;
  if (X == nullptr || weight == nullptr || out == nullptr) return I8L_EINVAL;
  return hip_status(i8l::launch_norm_forward(dtype, weight_dtype, X, (int)T, (int)C, weight, bias, eps, out, mean,
                                             rstd, (hipStream_t)stream));
}

size_t int8_layer_norm_backward_workspace_bytes(int64_t T, int64_t C) {
  if (T < 0 || C < 0 || T > MAX_TOKENS || C > I8L_MAX_COLS) return 0;
  return align_up(i8l::norm_backward_floats((int)T, (int)C) * sizeof(float));
}

int int8_layer_norm_backward(const void* G, const void* X, int dtype, int64_t T, int64_t C, const float* mean,
                             const float* rstd, const void* weight, int weight_dtype, void* grad_X,
                             void* grad_weight, void* grad_bias, void* ws, size_t ws_bytes, void* stream) {
  const int rc = norm_args(dtype, weight_dtype, T, C);
  if (rc != I8L_OK) return rc;
  if (C == 0) return I8L_OK;
  if (T > 0 && (G == nullptr || X == nullptr || mean == nullptr || rstd == nullptr)) return I8L_EINVAL;
  if (T > 0 && grad_X && weight == nullptr) return I8L_EINVAL;
  if (grad_X && grad_X == G && (grad_weight || grad_bias)) return I8L_EINVAL;
  const size_t need = int8_layer_norm_backward_workspace_bytes(T, C);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return I8L_EWORKSPACE;
  if ((uintptr_t)ws % ALIGN) return I8L_EINVAL;
  return hip_status(i8l::launch_norm_backward(dtype, weight_dtype, G, X, mean, rstd, (int)T, (int)C, weight, grad_X,
                                              grad_weight, grad_bias, static_cast<float*>(ws), (hipStream_t)stream));
}

// Table: count AdamWTensor, then one AdamWChunk per workgroup.
static int adamw_chunks(const i8l_adamw_tensor* t, int64_t count, int64_t* chunks) {
  if (count < 0 || count > INT32_MAX || (count > 0 && t == nullptr)) return I8L_EINVAL;
  int64_t c = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n < 0) return I8L_EINVAL;
    if (t[i].n > MAX_VALUES) return I8L_ESHAPE;
    c += (t[i].n + i8l::adamw_chunk() - 1) / i8l::adamw_chunk();
  }
  if (c > ((int64_t)1 << 24) - 1) return I8L_ESHAPE;   // one workgroup of 256 threads each
  *chunks = c;
  return I8L_OK;
}

size_t int8_adamw_table_bytes(const i8l_adamw_tensor* tensors, int64_t count) {
  int64_t c = 0;
  if (adamw_chunks(tensors, count, &c) != I8L_OK) return 0;
  return align_up((size_t)count * sizeof(i8l::AdamWTensor) + (size_t)c * sizeof(i8l::AdamWChunk) + 1);
}

int int8_adamw_table_fill(const i8l_adamw_tensor* tensors, int64_t count, void* table, size_t table_bytes,
                          int64_t* chunks) {
  int64_t c = 0;
  const int rc = adamw_chunks(tensors, count, &c);
  if (rc != I8L_OK) return rc;
  if (chunks == nullptr) return I8L_EINVAL;
  if (table == nullptr || table_bytes < int8_adamw_table_bytes(tensors, count)) return I8L_EWORKSPACE;
  char* at = static_cast<char*>(table);
  char* ch = at + (size_t)count * sizeof(i8l::AdamWTensor);
  for (int64_t i = 0; i < count; ++i) {
    const i8l_adamw_tensor& t = tensors[i];
    if (!valid_dtype(t.dtype)) return I8L_EDTYPE;
    if (t.state_bits != 8 && t.state_bits != 32) return I8L_EINVAL;
    const bool low = t.state_bits == 8;
    if (t.n > 0 && (!t.p || !t.g || !t.m || !t.v || (low && (!t.m_scale || !t.v_scale)))) return I8L_EINVAL;
    const uintptr_t wide = (uintptr_t)t.p | (uintptr_t)t.g | (uintptr_t)t.master;
    const uintptr_t states = (uintptr_t)t.m | (uintptr_t)t.v;
    i8l::AdamWTensor o = {t.p, t.g, t.m, t.v, t.m_scale, t.v_scale, t.master, t.n, t.dtype, t.state_bits, 0, 0};
    o.vec = wide % 16 == 0 && states % (low ? 8 : 16) == 0;
    memcpy(at, &o, sizeof(o));
    at += sizeof(o);
    const int64_t n = (t.n + i8l::adamw_chunk() - 1) / i8l::adamw_chunk();
    for (int64_t j = 0; j < n; ++j) {
      const i8l::AdamWChunk k = {(int32_t)i, (int32_t)j};
      memcpy(ch, &k, sizeof(k));
      ch += sizeof(k);
    }
  }
  *chunks = c;
  return I8L_OK;
}

int int8_adamw_step(const void* table, int64_t count, int64_t chunks, double lr, double beta1, double beta2,
                    double eps, double weight_decay, int64_t step, const float* grad_scale, const float* found_inf,
                    void* stream) {
  if (count < 0 || chunks < 0 || count > INT32_MAX || chunks > INT32_MAX || step < 1) return I8L_EINVAL;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return I8L_EINVAL;
  if (!(lr >= 0.0) || !(eps >= 0.0) || !(weight_decay >= 0.0) || !isfinite(lr) || !isfinite(eps) ||
      !isfinite(weight_decay))
    return I8L_EINVAL;
  if (chunks == 0) return I8L_OK;
  if (table == nullptr || (uintptr_t)table % 16) return I8L_EINVAL;
  i8l::AdamWScalars h;
  h.beta1 = (float)beta1;
  h.one_beta1 = (float)(1.0 - beta1);
  h.beta2 = (float)beta2;
  h.one_beta2 = (float)(1.0 - beta2);
  h.keep = (float)(1.0 - lr * weight_decay);
  h.step_size = (float)(lr / (1.0 - pow(beta1, (double)step)));
  h.inv_root_bc2 = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)step)));
  h.eps = (float)eps;
  const i8l::AdamWTensor* t = static_cast<const i8l::AdamWTensor*>(table);
  return hip_status(i8l::launch_adamw(t, reinterpret_cast<const i8l::AdamWChunk*>(t + count), chunks, h, grad_scale,
                                      found_inf, (hipStream_t)stream));
}

}  // extern "C"
