// C entry points of the training-step operators (routing, weight gradient,
// gradient norm and clipping): argument validation and launch. As in
// fp8gemm_api.hip, every check comes before the first HIP call.

#include <math.h>
#include <stddef.h>

#include "../../include/fp8gemm.h"
#include "internal.h"

using namespace fp8g;

namespace {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
constexpr int64_t kInt31 = 0x7FFFFFFF;
constexpr int64_t kNumelMax = int64_t(1) << 45;     // elements of a tensor of a gradient list

inline bool type_ok(int type) { return type >= FP8G_TYPE_F32 && type <= FP8G_TYPE_F16; }
inline uintptr_t type_size(int type) { return type == FP8G_TYPE_F32 ? 4 : 2; }
inline bool fmt_ok(int fmt) { return fmt == FP8G_FMT_E4M3 || fmt == FP8G_FMT_E5M2; }
inline fp8g_status launched(hipError_t e) { return e == hipSuccess ? FP8G_OK : FP8G_ERR_LAUNCH; }

fp8g_status route_sizes(int type, int64_t T, int E, int64_t ld, int top_k) {
  if (T < 0 || E < 1 || top_k < 1 || top_k > E) return FP8G_ERR_SHAPE;
  if (!type_ok(type) || E > 1024 || top_k > 16 || T > kInt31 / top_k) return FP8G_ERR_UNSUPPORTED;
  if (ld < E) return FP8G_ERR_STRIDE;
  return FP8G_OK;
}

fp8g_status list_ok(const void* const* grads, const int64_t* numels, const int* types, int n) {
  if (n < 0) return FP8G_ERR_SHAPE;
  if (n > 0 && (!grads || !numels || !types)) return FP8G_ERR_NULL_PTR;
  for (int i = 0; i < n; ++i) {
    if (numels[i] < 0) return FP8G_ERR_SHAPE;
    if (!type_ok(types[i]) || numels[i] > kNumelMax) return FP8G_ERR_UNSUPPORTED;
    if (numels[i] == 0) continue;
    if (!grads[i]) return FP8G_ERR_NULL_PTR;
    if (!aligned(grads[i], type_size(types[i]))) return FP8G_ERR_ALIGN;
  }
  return FP8G_OK;
}

}  // namespace

extern "C" {

fp8g_status moe_route_workspace_size(int64_t T, int E, size_t* bytes) {
  if (!bytes) return FP8G_ERR_NULL_PTR;
  *bytes = 0;
  if (T < 0 || E < 1) return FP8G_ERR_SHAPE;
  if (E > 1024 || T > kInt31) return FP8G_ERR_UNSUPPORTED;
  *bytes = route_workspace_bytes(T, E);
  return FP8G_OK;
}

fp8g_status moe_route(const void* logits, int type, int64_t T, int E, int64_t ld,
                      const uint8_t* token_mask, int top_k, int renormalise, float loss_coef,
                      int align, int64_t max_m, int32_t* expert_ids, float* weights,
                      int32_t* counts, int32_t* routed, float* prob_sum, float* loss,
                      int32_t* group_offsets, int32_t* slots, void* workspace,
                      size_t workspace_bytes, hipStream_t stream) {
  const fp8g_status s = route_sizes(type, T, E, ld, top_k);
  if (s != FP8G_OK) return s;
  if (align < 1 || max_m < 0) return FP8G_ERR_SHAPE;
  if (max_m > kInt31 / E || (int64_t)align > kInt31 / E ||
      T * top_k > kInt31 - (int64_t)E * align)
    return FP8G_ERR_UNSUPPORTED;
  if (!counts || !routed || !prob_sum || !loss || !group_offsets) return FP8G_ERR_NULL_PTR;
  if (T > 0 && (!logits || !expert_ids || !weights || !slots)) return FP8G_ERR_NULL_PTR;
  if (!aligned(logits, type_size(type)) || !aligned(expert_ids, 4) || !aligned(weights, 4) ||
      !aligned(counts, 4) || !aligned(routed, 4) || !aligned(prob_sum, 4) || !aligned(loss, 4) ||
      !aligned(group_offsets, 4) || !aligned(slots, 4) || !aligned(workspace, 16))
    return FP8G_ERR_ALIGN;
  if (workspace_bytes < route_workspace_bytes(T, E)) return FP8G_ERR_WORKSPACE;
  if (!workspace && workspace_bytes != 0) return FP8G_ERR_NULL_PTR;
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  RouteCall c;
  c.logits = logits;
  c.type = type;
  c.T = T;
  c.ld = ld;
  c.max_m = max_m;
  c.E = E;
  c.k = top_k;
  c.renorm = renormalise != 0;
  c.align = align;
  c.coef = loss_coef;
  c.mask = token_mask;
  c.ids = expert_ids;
  c.counts = counts;
  c.routed = routed;
  c.offsets = group_offsets;
  c.slots = slots;
  c.weights = weights;
  c.prob_sum = prob_sum;
  c.loss = loss;
  c.workspace = workspace;
  return launched(launch_route(c, stream));
}

fp8g_status moe_route_backward(const void* logits, int type, int64_t T, int E, int64_t ld,
                               const int32_t* expert_ids, int top_k, int renormalise,
                               float loss_coef, const float* d_weights, const float* d_loss,
                               const int32_t* counts, const int32_t* routed, void* d_logits,
                               int64_t ld_d, hipStream_t stream) {
  const fp8g_status s = route_sizes(type, T, E, ld, top_k);
  if (s != FP8G_OK) return s;
  if (ld_d < E) return FP8G_ERR_STRIDE;
  if (T == 0) return FP8G_OK;
  if (!logits || !expert_ids || !counts || !routed || !d_logits) return FP8G_ERR_NULL_PTR;
  if (!aligned(logits, type_size(type)) || !aligned(d_logits, type_size(type)) ||
      !aligned(expert_ids, 4) || !aligned(d_weights, 4) || !aligned(d_loss, 4) ||
      !aligned(counts, 4) || !aligned(routed, 4))
    return FP8G_ERR_ALIGN;
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  RouteBwdCall c;
  c.logits = logits;
  c.type = type;
  c.T = T;
  c.ld = ld;
  c.ldd = ld_d;
  c.E = E;
  c.k = top_k;
  c.renorm = renormalise != 0;
  c.coef = loss_coef;
  c.ids = expert_ids;
  c.counts = counts;
  c.routed = routed;
  c.dw = d_weights;
  c.dloss = d_loss;
  c.d_logits = d_logits;
  return launched(launch_route_backward(c, stream, dev.cu_count));
}

fp8g_status fp8_quantize_transpose(const void* x, int type, int64_t rows, int64_t cols,
                                   int64_t ldx, int fmt, uint8_t* qt, int64_t ldq, uint8_t* st,
                                   hipStream_t stream) {
  if (rows < 0 || cols <= 0 || cols % 16 != 0) return FP8G_ERR_SHAPE;
  if (!type_ok(type) || !fmt_ok(fmt)) return FP8G_ERR_UNSUPPORTED;
  if (rows == 0) return FP8G_OK;
  if (!x || !qt || !st) return FP8G_ERR_NULL_PTR;
  const int64_t nblk = (rows - 1) / 128 + 1;
  // (256 threads for 128 columns, and fewer than 2^32 of them in a launch)
  if (nblk > 65535 || (cols - 1) / 128 + 1 >= (int64_t(1) << 24)) return FP8G_ERR_UNSUPPORTED;
  if (ldx < cols || ldq < nblk * 128) return FP8G_ERR_STRIDE;
  if (!aligned(x, type_size(type)) || !aligned(qt, 16) || ldq % 16 != 0 || !aligned(st, 4))
    return FP8G_ERR_ALIGN;
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  return launched(launch_quantize_transpose(x, type, rows, cols, ldx, fmt, qt, ldq, st, stream));
}

fp8g_status grouped_gemm_fp8_wgrad(const uint8_t* a, int fmt_a, int64_t lda, const uint8_t* sa,
                                   const uint8_t* b, int fmt_b, int64_t ldb, const uint8_t* sb,
                                   uint16_t* d, const int32_t* group_offsets, int G, int64_t T,
                                   int64_t M, int64_t N, hipStream_t stream) {
  if (G < 0 || T < 0 || T % 128 != 0 || M <= 0 || N <= 0 || M % 16 != 0 || N % 16 != 0)
    return FP8G_ERR_SHAPE;
  if (!fmt_ok(fmt_a) || !fmt_ok(fmt_b)) return FP8G_ERR_UNSUPPORTED;
  if (G == 0) return FP8G_OK;
  if (G > 1 && !group_offsets) return FP8G_ERR_NULL_PTR;
  if (!d || (T > 0 && (!a || !sa || !b || !sb))) return FP8G_ERR_NULL_PTR;
  if (lda < T || ldb < T) return FP8G_ERR_STRIDE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(d, 16) || lda % 16 != 0 || ldb % 16 != 0 ||
      !aligned(sa, 4) || !aligned(sb, 4) || !aligned(group_offsets, 4))
    return FP8G_ERR_ALIGN;
  const int64_t mb = (M - 1) / 128 + 1, nb = (N - 1) / 128 + 1;
  if (lda > (int64_t(1) << 24) || ldb > (int64_t(1) << 24) || G > 1024 || mb > kInt31 ||
      nb > kInt31 / mb || (int64_t)G > kInt31 / (mb * nb))
    return FP8G_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  WgradArgs args;
  args.a = a;
  args.sa = sa;
  args.b = b;
  args.sb = sb;
  args.d = d;
  args.group = group_offsets;
  args.lda = lda;
  args.ldb = ldb;
  args.T = T;
  args.M = M;
  args.N = N;
  args.G = G;
  return launched(launch_wgrad(args, fmt_a, fmt_b, dev, stream));
}

fp8g_status grad_norm_sq_workspace_size(const int64_t* numels, int n, size_t* bytes) {
  if (!bytes) return FP8G_ERR_NULL_PTR;
  *bytes = 0;
  if (n < 0) return FP8G_ERR_SHAPE;
  if (n > 0 && !numels) return FP8G_ERR_NULL_PTR;
  for (int i = 0; i < n; ++i) {
    if (numels[i] < 0) return FP8G_ERR_SHAPE;
    if (numels[i] > kNumelMax) return FP8G_ERR_UNSUPPORTED;
  }
  *bytes = grad_norm_workspace_bytes(numels, n);
  return FP8G_OK;
}

fp8g_status grad_norm_sq(const void* const* grads, const int64_t* numels, const int* types, int n,
                         double* sumsq, void* workspace, size_t workspace_bytes,
                         hipStream_t stream) {
  const fp8g_status s = list_ok(grads, numels, types, n);
  if (s != FP8G_OK) return s;
  if (!sumsq || (!workspace && workspace_bytes != 0)) return FP8G_ERR_NULL_PTR;
  if (!aligned(sumsq, 8) || !aligned(workspace, 8)) return FP8G_ERR_ALIGN;
  if (workspace_bytes < grad_norm_workspace_bytes(numels, n)) return FP8G_ERR_WORKSPACE;
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  return launched(launch_grad_norm_sq(grads, numels, types, n, sumsq, workspace, stream));
}

fp8g_status grad_clip(const void* const* grads, void* const* outs, const int64_t* numels,
                      const int* types, int n, const double* sumsq, float max_norm, float* norm,
                      hipStream_t stream) {
  fp8g_status s = list_ok(grads, numels, types, n);
  if (s != FP8G_OK) return s;
  s = list_ok((const void* const*)outs, numels, types, n);
  if (s != FP8G_OK) return s;
  if (!(max_norm > 0.0f)) return FP8G_ERR_SHAPE;
  if (!sumsq || !norm) return FP8G_ERR_NULL_PTR;
  if (!aligned(sumsq, 8) || !aligned(norm, 4)) return FP8G_ERR_ALIGN;
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  return launched(
      launch_grad_clip(grads, outs, numels, types, n, sumsq, max_norm, norm, stream));
}

}  // extern "C"
