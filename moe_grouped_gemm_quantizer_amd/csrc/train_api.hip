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

// The checks that both routings share; fills c.
fp8g_status route_call(const void* logits, int type, int64_t T, int E, int64_t ld, const uint8_t* token_mask,
                       int top_k, int renormalise, float loss_coef, int align, int64_t max_m,
                       int32_t* expert_ids, float* weights, int32_t* counts, int32_t* routed,
                       float* prob_sum, float* loss, int32_t* group_offsets, int32_t* slots, void* workspace,
                       size_t workspace_bytes, RouteCall& c) {
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
  return FP8G_OK;
}

fp8g_status route_bwd_call(const void* logits, int type, int64_t T, int E, int64_t ld, const int32_t* expert_ids,
                           int top_k, int renormalise, float loss_coef, const float* d_weights,
                           const float* d_loss, const int32_t* counts, const int32_t* routed, void* d_logits,
                           int64_t ld_d, RouteBwdCall& c) {
  const fp8g_status s = route_sizes(type, T, E, ld, top_k);
  if (s != FP8G_OK) return s;
  if (ld_d < E) return FP8G_ERR_STRIDE;
  c.T = T;
  if (T == 0) return FP8G_OK;
  if (!logits || !expert_ids || !counts || !routed || !d_logits) return FP8G_ERR_NULL_PTR;
  if (!aligned(logits, type_size(type)) || !aligned(d_logits, type_size(type)) ||
      !aligned(expert_ids, 4) || !aligned(d_weights, 4) || !aligned(d_loss, 4) ||
      !aligned(counts, 4) || !aligned(routed, 4))
    return FP8G_ERR_ALIGN;
  c.logits = logits;
  c.type = type;
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

constexpr int64_t kNumelStepMax = ((int64_t(1) << 24) - 1) * 2048;   // chunks of 2048 in a launch

fp8g_status adamw_list_ok(const AdamwCall& c) {
  const bool eight = c.ms || c.vs;
  if (c.n < 0) return FP8G_ERR_SHAPE;
  if (c.n == 0) return FP8G_OK;
  if (!c.params || !c.param_types || !c.grads || !c.grad_types || !c.m || !c.v || !c.numels ||
      (eight && (!c.ms || !c.vs)) || (c.copies && !c.copy_types))
    return FP8G_ERR_NULL_PTR;
  const uintptr_t state = eight ? 1 : 4;
  for (int i = 0; i < c.n; ++i) {
    if (c.numels[i] < 0) return FP8G_ERR_SHAPE;
    if (!type_ok(c.param_types[i]) || !type_ok(c.grad_types[i]) ||
        c.numels[i] > kNumelStepMax)
      return FP8G_ERR_UNSUPPORTED;
    void* const copy = c.copies ? c.copies[i] : nullptr;
    if (copy && c.copy_types[i] != FP8G_TYPE_BF16 && c.copy_types[i] != FP8G_TYPE_F16)
      return FP8G_ERR_UNSUPPORTED;
    if (c.numels[i] == 0) continue;
    if (!c.params[i] || !c.grads[i] || !c.m[i] || !c.v[i] || (eight && (!c.ms[i] || !c.vs[i])))
      return FP8G_ERR_NULL_PTR;
    if (!aligned(c.params[i], type_size(c.param_types[i])) || !aligned(c.grads[i], type_size(c.grad_types[i])) ||
        !aligned(c.m[i], state) || !aligned(c.v[i], state) || !aligned(copy, 2))
      return FP8G_ERR_ALIGN;
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
  RouteCall c;
  const fp8g_status s =
      route_call(logits, type, T, E, ld, token_mask, top_k, renormalise, loss_coef, align, max_m, expert_ids,
                 weights, counts, routed, prob_sum, loss, group_offsets, slots, workspace, workspace_bytes, c);
  if (s != FP8G_OK) return s;
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  return launched(launch_route(c, stream));
}

fp8g_status moe_route_backward(const void* logits, int type, int64_t T, int E, int64_t ld,
                               const int32_t* expert_ids, int top_k, int renormalise,
                               float loss_coef, const float* d_weights, const float* d_loss,
                               const int32_t* counts, const int32_t* routed, void* d_logits,
                               int64_t ld_d, hipStream_t stream) {
  RouteBwdCall c;
  const fp8g_status s = route_bwd_call(logits, type, T, E, ld, expert_ids, top_k, renormalise, loss_coef, d_weights,
                                       d_loss, counts, routed, d_logits, ld_d, c);
  if (s != FP8G_OK || T == 0) return s;
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  return launched(launch_route_backward(c, stream, dev.cu_count));
}

fp8g_status moe_route_scored(const void* logits, int type, int64_t T, int E, int64_t ld, const float* bias,
                             int score, int groups, int open_groups, int group_best, const uint8_t* token_mask,
                             int top_k, int renormalise, float scale, float loss_coef, int align,
                             int64_t max_m, int32_t* expert_ids, float* weights, int32_t* counts,
                             int32_t* routed, float* prob_sum, float* loss, int32_t* group_offsets,
                             int32_t* slots, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  ScoredCall c;
  const fp8g_status s =
      route_call(logits, type, T, E, ld, token_mask, top_k, renormalise, loss_coef, align, max_m, expert_ids,
                 weights, counts, routed, prob_sum, loss, group_offsets, slots, workspace, workspace_bytes,
                 c.route);
  if (s != FP8G_OK) return s;
  if (groups < 1 || E % groups != 0 || open_groups < 1 || open_groups > groups || group_best < 1 ||
      group_best > E / groups || top_k > open_groups * (E / groups))
    return FP8G_ERR_SHAPE;
  if ((score != FP8G_SCORE_SIGMOID && score != FP8G_SCORE_SOFTMAX) || groups > 32 || group_best > 2)
    return FP8G_ERR_UNSUPPORTED;
  if (!aligned(bias, 4)) return FP8G_ERR_ALIGN;
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  c.bias = bias;
  c.score = score;
  c.groups = groups;
  c.open = open_groups;
  c.best = group_best;
  c.scale = scale;
  return launched(launch_route_scored(c, stream, dev.cu_count));
}

fp8g_status moe_route_scored_backward(const void* logits, int type, int64_t T, int E, int64_t ld, int score,
                                      const int32_t* expert_ids, int top_k, int renormalise, float scale,
                                      float loss_coef, const float* d_weights, const float* d_loss,
                                      const int32_t* counts, const int32_t* routed, void* d_logits,
                                      int64_t ld_d, hipStream_t stream) {
  ScoredBwdCall c;
  const fp8g_status s = route_bwd_call(logits, type, T, E, ld, expert_ids, top_k, renormalise, loss_coef, d_weights,
                                       d_loss, counts, routed, d_logits, ld_d, c.route);
  if (s != FP8G_OK) return s;
  if (score != FP8G_SCORE_SIGMOID && score != FP8G_SCORE_SOFTMAX) return FP8G_ERR_UNSUPPORTED;
  if (T == 0) return FP8G_OK;
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  c.score = score;
  c.scale = scale;
  return launched(launch_route_scored_backward(c, stream, dev.cu_count));
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

fp8g_status adamw_table_size(int n, size_t* bytes) {
  if (!bytes) return FP8G_ERR_NULL_PTR;
  *bytes = 0;
  if (n < 0) return FP8G_ERR_SHAPE;
  *bytes = adamw_table_bytes(n);
  return FP8G_OK;
}

fp8g_status adamw_table(void* const* params, const int* param_types, const void* const* grads,
                        const int* grad_types, void* const* exp_avgs, void* const* exp_avg_sqs,
                        uint8_t* const* avg_scales, uint8_t* const* sq_scales, void* const* copies,
                        const int* copy_types, const int64_t* numels, int n, void* table) {
  AdamwCall c = {};
  c.params = params;
  c.param_types = param_types;
  c.grads = grads;
  c.grad_types = grad_types;
  c.m = exp_avgs;
  c.v = exp_avg_sqs;
  c.ms = avg_scales;
  c.vs = sq_scales;
  c.copies = copies;
  c.copy_types = copy_types;
  c.numels = numels;
  c.n = n;
  const fp8g_status s = adamw_list_ok(c);
  if (s != FP8G_OK || n == 0) return s;
  if (!table) return FP8G_ERR_NULL_PTR;
  if (!aligned(table, 8)) return FP8G_ERR_ALIGN;
  return adamw_table_fill(c, table) ? FP8G_OK : FP8G_ERR_UNSUPPORTED;
}

fp8g_status adamw_step(void* const* params, const int* param_types, const void* const* grads,
                       const int* grad_types, void* const* exp_avgs, void* const* exp_avg_sqs,
                       uint8_t* const* avg_scales, uint8_t* const* sq_scales, void* const* copies,
                       const int* copy_types, const int64_t* numels, int n, const int64_t* step,
                       int64_t step_value, const float* lr, double lr_value, double beta1, double beta2,
                       double eps, double weight_decay, const double* sumsq, float max_norm, float* norm,
                       uint32_t seed, const void* table, hipStream_t stream) {
  AdamwCall c;
  c.params = params;
  c.param_types = param_types;
  c.grads = grads;
  c.grad_types = grad_types;
  c.m = exp_avgs;
  c.v = exp_avg_sqs;
  c.ms = avg_scales;
  c.vs = sq_scales;
  c.copies = copies;
  c.copy_types = copy_types;
  c.numels = numels;
  c.n = n;
  c.step_at = step;
  c.step = step_value;
  c.lr_at = lr;
  c.lr = lr_value;
  c.beta1 = beta1;
  c.beta2 = beta2;
  c.eps = eps;
  c.weight_decay = weight_decay;
  c.sumsq = sumsq;
  c.max_norm = max_norm;
  c.norm = norm;
  c.seed = seed;
  c.table = table;
  const fp8g_status s = adamw_list_ok(c);
  if (s != FP8G_OK) return s;
  if ((!step && step_value < 1) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) ||
      !(eps >= 0.0) || !isfinite(eps) || !isfinite(weight_decay) || (!lr && !isfinite(lr_value)))
    return FP8G_ERR_SHAPE;
  if (sumsq && !(max_norm > 0.0f)) return FP8G_ERR_SHAPE;
  if (norm && !sumsq) return FP8G_ERR_NULL_PTR;
  if (!aligned(step, 8) || !aligned(lr, 4) || !aligned(sumsq, 8) || !aligned(norm, 4) || !aligned(table, 8))
    return FP8G_ERR_ALIGN;
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  return launched(launch_adamw(c, stream));
}

}  // extern "C"
