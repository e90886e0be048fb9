// The C ABI of mc2_layer.h: host-side validation, device check and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "api_internal.hpp"
#include "layer_kernels.hpp"
#include "mc2_layer.h"
#include "testing.h"
#include "validate_layer.hpp"

namespace mc2 {
namespace {

mc2_status launched(hipError_t e, const char* where) {
  if (e == hipSuccess) return MC2_OK;
  return fail(MC2_ERR_HIP, std::string(where) + ": " + hipGetErrorString(e));
}

size_t norm_grad_workspace(int64_t rows, int64_t h) {
  return (size_t)norm_grad_blocks(rows, h) * (size_t)h * sizeof(float);
}

}  // namespace
}  // namespace mc2

using namespace mc2;

extern "C" {

mc2_status mc2_add_rms_norm(const void* x, const void* residual, const void* weight, int64_t rows, int64_t h,
                            mc2_dtype dtype, float eps, void* out, mc2_dtype out_dtype, float* scale_out,
                            int64_t group, void* sum_out, float* rstd_out, void* stream) {
  clear_error();
  mc2_status s = check_add_rms_norm(x, residual, weight, rows, h, dtype, eps, out, out_dtype, scale_out, group,
                                    sum_out, rstd_out);
  if (s != MC2_OK || rows == 0) return s;
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.rows = rows;
  a.h = h;
  a.group = group;
  a.dtype = dtype;
  a.out_dtype = out_dtype;
  a.eps = eps;
  a.out = out;
  a.scale = scale_out;
  a.sum = sum_out;
  a.rstd = rstd_out;
  return launched(launch_add_rms_norm(a, static_cast<hipStream_t>(stream)), "add_rms_norm launch");
}

mc2_status mc2_add_rms_norm_grad_workspace_size(int64_t rows, int64_t h, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(MC2_ERR_NULL, "add_rms_norm_grad_workspace_size: bytes is NULL");
  mc2_status s = check_norm_sizes("add_rms_norm_grad_workspace_size", rows, h);
  if (s != MC2_OK) return s;
  *bytes = norm_grad_workspace(rows, h);
  return MC2_OK;
}

mc2_status mc2_add_rms_norm_grad(const void* dout, const void* dsum, const void* sum, const void* weight,
                                 const float* rstd, int64_t rows, int64_t h, mc2_dtype dtype, void* dx,
                                 void* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  mc2_status s = check_norm_sizes("add_rms_norm_grad", rows, h);
  if (s != MC2_OK) return s;
  s = check_add_rms_norm_grad(dout, dsum, sum, weight, rstd, rows, h, dtype, dx, dweight, workspace, workspace_bytes,
                              norm_grad_workspace(rows, h));
  if (s != MC2_OK) return s;
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  NormGradArgs a{};
  a.dout = dout;
  a.dsum = dsum;
  a.s = sum;
  a.weight = weight;
  a.rstd = rstd;
  a.rows = rows;
  a.h = h;
  a.dtype = dtype;
  a.dx = dx;
  a.dweight = dweight;
  a.partials = static_cast<float*>(workspace);
  return launched(launch_add_rms_norm_grad(a, static_cast<hipStream_t>(stream)), "add_rms_norm_grad launch");
}

mc2_status mc2_linear_act_workspace_size(int64_t m, int64_t k, int64_t n, int64_t groups, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(MC2_ERR_NULL, "linear_act_workspace_size: bytes is NULL");
  mc2_status s = check_linear_sizes("linear_act_workspace_size", m, k, n, groups);
  if (s != MC2_OK) return s;
  *bytes = linear_act_workspace(m, k, n, groups);
  return MC2_OK;
}

mc2_status mc2_linear_act(const void* x, const void* w, const void* bias, const void* residual, int64_t m,
                          int64_t k, int64_t n, const int32_t* group_offsets, int64_t groups, mc2_dtype dtype,
                          mc2_act act, void* out, void* z_out, void* workspace, size_t workspace_bytes,
                          void* stream) {
  clear_error();
  mc2_status s = check_linear_sizes("linear_act", m, k, n, groups);
  if (s != MC2_OK) return s;
  s = check_linear_act(x, w, bias, residual, m, k, n, group_offsets, groups, dtype, act, out, z_out, workspace,
                       workspace_bytes, linear_act_workspace(m, k, n, groups));
  if (s != MC2_OK || m == 0) return s;
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  LinearArgs a{};
  a.x = x;
  a.w = w;
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
  a.z = z_out;
  a.workspace = workspace;
  return launched(launch_linear_act(a, static_cast<hipStream_t>(stream)), "linear_act launch");
}

mc2_status mc2_linear_act_grad_workspace_size(int64_t m, int64_t k, int64_t n, int64_t groups, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(MC2_ERR_NULL, "linear_act_grad_workspace_size: bytes is NULL");
  mc2_status s = check_linear_sizes("linear_act_grad_workspace_size", m, k, n, groups);
  if (s != MC2_OK) return s;
  *bytes = linear_act_grad_workspace(m, k, n, groups);
  return MC2_OK;
}

mc2_status mc2_linear_act_grad(const void* dout, const void* z, const void* x, const void* w, int64_t m, int64_t k,
                               int64_t n, const int32_t* group_offsets, int64_t groups, mc2_dtype dtype,
                               mc2_act act, void* dx, void* dw, void* dbias, void* workspace,
                               size_t workspace_bytes, void* stream) {
  clear_error();
  mc2_status s = check_linear_sizes("linear_act_grad", m, k, n, groups);
  if (s != MC2_OK) return s;
  s = check_linear_act_grad(dout, z, x, w, m, k, n, group_offsets, groups, dtype, act, dx, dw, dbias, workspace,
                            workspace_bytes, linear_act_grad_workspace(m, k, n, groups));
  if (s != MC2_OK) return s;
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  LinearGradArgs a{};
  a.dout = dout;
  a.z = z;
  a.x = x;
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
  return launched(launch_linear_act_grad(a, static_cast<hipStream_t>(stream)), "linear_act_grad launch");
}

mc2_status mc2_moe_permute_workspace_size(int64_t tokens, int64_t top, int64_t experts, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(MC2_ERR_NULL, "moe_permute_workspace_size: bytes is NULL");
  mc2_status s = check_permute_sizes("moe_permute_workspace_size", tokens, top, experts);
  if (s != MC2_OK) return s;
  *bytes = moe_permute_workspace(tokens * top, experts);
  return MC2_OK;
}

mc2_status mc2_moe_permute(const void* x, const int32_t* expert_ids, int64_t tokens, int64_t top, int64_t h,
                           int64_t experts, mc2_dtype dtype, void* out, int32_t* row_map, int32_t* offsets,
                           void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  mc2_status s = check_permute_sizes("moe_permute", tokens, top, experts);
  if (s != MC2_OK) return s;
  s = check_moe_permute(x, expert_ids, tokens, top, h, experts, dtype, out, row_map, offsets, workspace,
                        workspace_bytes, moe_permute_workspace(tokens * top, experts));
  if (s != MC2_OK) return s;
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  PermuteArgs a{};
  a.x = x;
  a.ids = expert_ids;
  a.tokens = tokens;
  a.top = top;
  a.h = h;
  a.experts = experts;
  a.out = out;
  a.row_map = row_map;
  a.offsets = offsets;
  a.workspace = static_cast<int32_t*>(workspace);
  return launched(launch_moe_permute(a, static_cast<hipStream_t>(stream)), "moe_permute launch");
}

mc2_status mc2_moe_unpermute(const void* y, const int32_t* row_map, const float* weights, int64_t tokens,
                             int64_t top, int64_t h, int64_t rows, mc2_dtype dtype, void* out, void* stream) {
  clear_error();
  mc2_status s = check_moe_unpermute(y, row_map, weights, tokens, top, h, rows, dtype, out);
  if (s != MC2_OK || tokens == 0) return s;
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  UnpermuteArgs a{};
  a.y = y;
  a.row_map = row_map;
  a.weights = weights;
  a.tokens = tokens;
  a.top = top;
  a.h = h;
  a.rows = rows;
  a.dtype = dtype;
  a.out = out;
  return launched(launch_moe_unpermute(a, static_cast<hipStream_t>(stream)), "moe_unpermute launch");
}

mc2_status mc2_moe_unpermute_grad(const void* dout, const void* y, const int32_t* row_map, const float* weights,
                                  int64_t tokens, int64_t top, int64_t h, int64_t rows, mc2_dtype dtype, void* dy,
                                  float* dweights, void* stream) {
  clear_error();
  mc2_status s = check_moe_unpermute_grad(dout, y, row_map, weights, tokens, top, h, rows, dtype, dy, dweights);
  if (s != MC2_OK || ((rows == 0 || !dy) && (tokens == 0 || !dweights))) return s;  // (or nothing to write)
  int dev;
  if ((s = current_device(&dev)) != MC2_OK) return s;
  UnpermuteArgs a{};
  a.dout = dout;
  a.y = y;
  a.row_map = row_map;
  a.weights = weights;
  a.tokens = tokens;
  a.top = top;
  a.h = h;
  a.rows = rows;
  a.dtype = dtype;
  a.dy = dy;
  a.dweights = dweights;
  return launched(launch_moe_unpermute_grad(a, static_cast<hipStream_t>(stream)), "moe_unpermute_grad launch");
}

mc2_status mc2_testing_linear_plan(int product, int64_t m, int64_t k, int64_t n, int64_t groups, int* tile,
                                   int* splits) {
  clear_error();
  if (!tile || !splits) return fail(MC2_ERR_NULL, "testing_linear_plan: tile and splits are required");
  if (product < 0 || product > 2) return fail(MC2_ERR_UNSUPPORTED, "testing_linear_plan: no such product");
  mc2_status s = check_linear_sizes("testing_linear_plan", m, k, n, groups);
  if (s != MC2_OK) return s;
  linear_act_plan(product, m, k, n, groups, tile, splits);
  return MC2_OK;
}

}  // extern "C"
