// The C ABI of mc2_layer8.h: host-side validation, device check and launches.
#include <hip/hip_runtime.h>

#include <string>

#include "api_internal.hpp"
#include "layer8_kernels.hpp"
#include "mc2_layer8.h"
#include "testing.h"
#include "validate_layer8.hpp"

namespace mc2 {
namespace {

mc2_status launched(hipError_t e, const char* where) {
  if (e == hipSuccess) return MC2_OK;
  return fail(MC2_ERR_HIP, std::string(where) + ": " + hipGetErrorString(e));
}

}  // namespace
}  // namespace mc2

using namespace mc2;

extern "C" {

mc2_status mc2_moe_route(const void* logits, const float* bias, int64_t tokens, int64_t experts, int64_t top,
                         mc2_dtype dtype, mc2_score score, int64_t groups, int64_t top_groups, int64_t group_top,
                         int renormalise, float scale, int32_t* expert_ids, float* weights, void* stream) {
  clear_error();
  const bool keep_nan = score == MC2_SCORE_KEEP_NAN + MC2_SCORE_SOFTMAX || score == MC2_SCORE_KEEP_NAN + MC2_SCORE_SIGMOID;
  if (keep_nan) score = (mc2_score)(score - MC2_SCORE_KEEP_NAN);
  mc2_status s = check_moe_route(logits, bias, tokens, experts, top, dtype, score, groups, top_groups, group_top, scale,
                                 expert_ids, weights);
  if (s != MC2_OK || tokens == 0) return s;
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  RouteArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.tokens = tokens;
  a.experts = (int)experts;
  a.top = (int)top;
  a.dtype = dtype;
  a.score = score;
  a.groups = (int)groups;
  a.top_groups = (int)top_groups;
  a.group_top = (int)group_top;
  a.keep_nan = keep_nan;
  a.renormalise = renormalise != 0;
  a.scale = scale;
  a.ids = expert_ids;
  a.weights = weights;
  return launched(launch_moe_route(a, static_cast<hipStream_t>(stream)), "moe_route launch");
}

mc2_status mc2_moe_route_grad(const float* dweights, const void* logits, const int32_t* expert_ids, int64_t tokens,
                              int64_t experts, int64_t top, mc2_dtype dtype, mc2_score score, int renormalise,
                              float scale, void* dlogits, void* stream) {
  clear_error();
  mc2_status s = check_moe_route_grad(dweights, logits, expert_ids, tokens, experts, top, dtype, score, scale, dlogits);
  if (s != MC2_OK || tokens == 0) return s;
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  RouteArgs a{};
  a.logits = logits;
  a.dweights = dweights;
  a.tokens = tokens;
  a.experts = (int)experts;
  a.top = (int)top;
  a.dtype = dtype;
  a.score = score;
  a.renormalise = renormalise != 0;
  a.scale = scale;
  a.ids = const_cast<int32_t*>(expert_ids);
  a.dlogits = dlogits;
  return launched(launch_moe_route_grad(a, static_cast<hipStream_t>(stream)), "moe_route_grad launch");
}

mc2_status mc2_quant_rows(const void* x, int64_t rows, int64_t cols, mc2_dtype dtype, int64_t group, int8_t* codes,
                          float* scale, void* stream) {
  clear_error();
  const bool keep_inf = group == 128 + MC2_KEEP_INF;
  if (keep_inf) group = 128;
  mc2_status s = check_code_rows("quant_rows", x, codes, scale, rows, cols, dtype, group, MC2_ACT_NONE);
  if (s != MC2_OK || rows == 0) return s;
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  CodeArgs a{};
  a.x = x;
  a.codes = codes;
  a.scale = scale;
  a.rows = rows;
  a.cols = cols;
  a.group = group;
  a.dtype = dtype;
  a.keep_inf = keep_inf;
  return launched(launch_quant_rows(a, static_cast<hipStream_t>(stream)), "quant_rows launch");
}

mc2_status mc2_dequant_rows(const int8_t* codes, const float* scale, int64_t rows, int64_t cols, int64_t group,
                            mc2_act act, mc2_dtype dtype, void* out, void* stream) {
  clear_error();
  mc2_status s = check_code_rows("dequant_rows", out, codes, scale, rows, cols, dtype, group, act);
  if (s != MC2_OK || rows == 0) return s;
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  CodeArgs a{};
  a.codes_in = codes;
  a.scale_in = scale;
  a.out = out;
  a.rows = rows;
  a.cols = cols;
  a.group = group;
  a.dtype = dtype;
  a.act = act;
  return launched(launch_dequant_rows(a, static_cast<hipStream_t>(stream)), "dequant_rows launch");
}

mc2_status mc2_linear_i8_workspace_size(int64_t m, int64_t k, int64_t n, int64_t groups, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(MC2_ERR_NULL, "linear_i8_workspace_size: bytes is NULL");
  mc2_status s = check_linear_i8_sizes("linear_i8_workspace_size", m, k, n, groups);
  if (s != MC2_OK) return s;
  *bytes = linear_i8_workspace(m, k, n, groups);
  return MC2_OK;
}

mc2_status mc2_linear_i8(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale,
                         const void* bias, const void* residual, int64_t m, int64_t k, int64_t n,
                         const int32_t* group_offsets, int64_t groups, mc2_dtype dtype, mc2_act act, void* out,
                         void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  mc2_status s = check_linear_i8_sizes("linear_i8", m, k, n, groups);
  if (s != MC2_OK) return s;
  s = check_linear_i8(x, x_scale, w, w_scale, bias, residual, m, k, n, group_offsets, groups, dtype, act, out, workspace,
                      workspace_bytes, linear_i8_workspace(m, k, n, groups));
  if (s != MC2_OK || m == 0) return s;
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  LinearI8Args a{};
  a.x = x;
  a.w = w;
  a.x_scale = x_scale;
  a.w_scale = w_scale;
  a.bias = bias;
  a.residual = residual;
  a.m = m;
  a.k = k;
  a.n = n;
  a.groups = groups;
  a.offsets = group_offsets;
  a.dtype = dtype;
  a.act = act;
  a.out = out;
  a.workspace = workspace;
  return launched(launch_linear_i8(a, static_cast<hipStream_t>(stream)), "linear_i8 launch");
}

mc2_status mc2_linear_act_grad_i8_workspace_size(int64_t m, int64_t k, int64_t n, int64_t groups, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(MC2_ERR_NULL, "linear_act_grad_i8_workspace_size: bytes is NULL");
  mc2_status s = check_linear_sizes("linear_act_grad_i8_workspace_size", m, k, n, groups);
  if (s != MC2_OK) return s;
  *bytes = linear_act_grad_workspace(m, k, n, groups, true);
  return MC2_OK;
}

mc2_status mc2_linear_act_grad_i8(const void* dout, const int8_t* z, const float* z_scale, const int8_t* x,
                                  const float* x_scale, mc2_act x_act, const void* w, int64_t m, int64_t k,
                                  int64_t n, const int32_t* group_offsets, int64_t groups, mc2_dtype dtype,
                                  mc2_act act, void* dx, void* dw, void* dbias, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  clear_error();
  mc2_status s = check_linear_sizes("linear_act_grad_i8", m, k, n, groups);
  if (s != MC2_OK) return s;
  s = check_linear_act_grad_i8(dout, z, z_scale, x, x_scale, x_act, w, m, k, n, group_offsets, groups, dtype, act, dx,
                               dw, dbias, workspace, workspace_bytes, linear_act_grad_workspace(m, k, n, groups, true));
  if (s != MC2_OK) return s;
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  LinearGradArgs a{};
  a.dout = dout;
  a.w = w;
  a.m = m;
  a.k = k;
  a.n = n;
  a.groups = groups;
  a.offsets = group_offsets;
  a.dtype = dtype;
  a.act = act;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.workspace = workspace;
  a.eight = true;
  a.z_codes = z;
  a.z_scale = z_scale;
  a.x_codes = x;
  a.x_scale = x_scale;
  a.x_act = x_act;
  return launched(launch_linear_act_grad(a, static_cast<hipStream_t>(stream)), "linear_act_grad_i8 launch");
}

mc2_status mc2_testing_linear_i8_plan(int64_t m, int64_t k, int64_t n, int64_t groups, int* tile, int* splits) {
  clear_error();
  if (!tile || !splits) return fail(MC2_ERR_NULL, "testing_linear_i8_plan: tile and splits are required");
  mc2_status s = check_linear_i8_sizes("testing_linear_i8_plan", m, k, n, groups);
  if (s != MC2_OK) return s;
  linear_i8_plan(m, k, n, groups, tile, splits);
  return MC2_OK;
}

}  // extern "C"
