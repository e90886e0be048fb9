// Host-only argument validation of the router and the 8-bit operators
// (mc2_layer8.h); no HIP calls.
#include "validate_layer8.hpp"

#include <cmath>

#include "validate_util.hpp"

namespace mc2 {

namespace {

constexpr int64_t kTop = 64, kExpertGroups = 64, kCodes = (int64_t)1 << 17;

mc2_status check_route_sizes(const char* who, int64_t tokens, int64_t experts, int64_t top, mc2_dtype dtype,
                             mc2_score score, float scale) {
  if (tokens < 0 || tokens > kTokens) return shape(who, "tokens must lie in [0, 2^23], got " + str(tokens));
  if (experts < 1 || experts > kGroups) return shape(who, "experts must lie in [1, 4096], got " + str(experts));
  if (top < 1 || top > kTop || top > experts)
    return shape(who, "top must lie in [1, min(64, experts)], got " + str(top));
  if (dtype != MC2_F32 && !is_half(dtype)) return fail(MC2_ERR_DTYPE, string(who) + ": dtype must be F32, F16 or BF16");
  if (score != MC2_SCORE_SOFTMAX && score != MC2_SCORE_SIGMOID)
    return fail(MC2_ERR_UNSUPPORTED, string(who) + ": unknown score " + str(score));
  if (!std::isfinite(scale)) return shape(who, "scale must be finite");
  return MC2_OK;
}

mc2_status known_act(const char* who, mc2_act act) {
  if (act < MC2_ACT_NONE || act > MC2_ACT_SILU)
    return fail(MC2_ERR_UNSUPPORTED, string(who) + ": unknown activation " + str(act));
  return MC2_OK;
}

}  // namespace

mc2_status check_moe_route(const void* logits, const void* bias, int64_t tokens, int64_t experts, int64_t top,
                           mc2_dtype dtype, mc2_score score, int64_t groups, int64_t top_groups, int64_t group_top,
                           float scale, const void* expert_ids, const void* weights) {
  const char* who = "moe_route";
  MC2_TRY(check_route_sizes(who, tokens, experts, top, dtype, score, scale));
  if (groups < 1 || groups > kExpertGroups || experts % groups != 0)
    return shape(who, "groups must lie in [1, 64] and divide experts, got " + str(groups));
  if (top_groups < 1 || top_groups > groups) return shape(who, "top_groups must lie in [1, groups], got " + str(top_groups));
  if (group_top < 1 || group_top > 2 || group_top > experts / groups)
    return shape(who, "group_top must be 1 or 2 and at most experts / groups, got " + str(group_top));
  if (top > top_groups * (experts / groups)) return shape(who, "top_groups groups hold fewer than top experts");
  if (tokens == 0) return MC2_OK;
  MC2_TRY(required(who, {logits, expert_ids, weights}, "logits, expert_ids and weights"));
  return aligned(who, {logits, bias, expert_ids, weights});
}

mc2_status check_moe_route_grad(const void* dweights, const void* logits, const void* expert_ids, int64_t tokens,
                                int64_t experts, int64_t top, mc2_dtype dtype, mc2_score score, float scale,
                                const void* dlogits) {
  const char* who = "moe_route_grad";
  MC2_TRY(check_route_sizes(who, tokens, experts, top, dtype, score, scale));
  if (tokens == 0) return MC2_OK;
  MC2_TRY(required(who, {dweights, logits, expert_ids, dlogits}, "dweights, logits, expert_ids and dlogits"));
  return aligned(who, {dweights, logits, expert_ids, dlogits});
}

mc2_status check_code_rows(const char* who, const void* values, const void* codes, const void* scale, int64_t rows,
                           int64_t cols, mc2_dtype dtype, int64_t group, mc2_act act) {
  if (rows < 0 || rows >= kRows) return shape(who, "rows must lie in [0, 2^24), got " + str(rows));
  if (cols < 1 || cols > kWidth) return shape(who, "cols must lie in [1, 2^24], got " + str(cols));
  MC2_TRY(half(who, dtype));
  if (group != 0 && group != 128) return shape(who, "group must be 0 or 128, got " + str(group));
  MC2_TRY(known_act(who, act));
  if (rows == 0) return MC2_OK;
  MC2_TRY(required(who, {values, codes, scale}, "the rows, their codes and their scale"));
  return aligned(who, {values, codes, scale});
}

mc2_status check_linear_i8_sizes(const char* who, int64_t m, int64_t k, int64_t n, int64_t groups) {
  MC2_TRY(check_linear_sizes(who, m, k, n, groups));
  if (k >= kCodes) return shape(who, "k must be below 2^17, got " + str(k));
  return MC2_OK;
}

mc2_status check_linear_i8(const void* x, const void* x_scale, const void* w, const void* w_scale, const void* bias,
                           const void* residual, int64_t m, int64_t k, int64_t n, const void* group_offsets,
                           int64_t groups, mc2_dtype dtype, mc2_act act, const void* out, const void* workspace,
                           size_t workspace_bytes, size_t needed) {
  const char* who = "linear_i8";
  MC2_TRY(check_linear_i8_sizes(who, m, k, n, groups));
  MC2_TRY(check_linear_kind(who, group_offsets, groups, dtype, act));
  if (m == 0) return MC2_OK;
  MC2_TRY(required(who, {x, x_scale, w, w_scale, out}, "x, x_scale, w, w_scale and out"));
  MC2_TRY(aligned(who, {x, x_scale, w, w_scale, bias, residual, out, group_offsets}));
  return workspace_ok(who, workspace, workspace_bytes, needed);
}

mc2_status check_linear_act_grad_i8(const void* dout, const void* z, const void* z_scale, const void* x,
                                    const void* x_scale, mc2_act x_act, const void* w, int64_t m, int64_t k,
                                    int64_t n, const void* group_offsets, int64_t groups, mc2_dtype dtype, mc2_act act,
                                    const void* dx, const void* dw, const void* dbias, const void* workspace,
                                    size_t workspace_bytes, size_t needed) {
  const char* who = "linear_act_grad_i8";
  MC2_TRY(check_linear_sizes(who, m, k, n, groups));
  MC2_TRY(check_linear_kind(who, group_offsets, groups, dtype, act));
  MC2_TRY(known_act(who, x_act));
  if (m > 0) {
    MC2_TRY(required(who, {dout}, "dout"));
    if (act != MC2_ACT_NONE) MC2_TRY(required(who, {z, z_scale}, "z and z_scale (with an activation)"));
    if (dw) MC2_TRY(required(who, {x, x_scale}, "x and x_scale (for dw)"));
    if (dx) MC2_TRY(required(who, {w}, "w (for dx)"));
  }
  MC2_TRY(aligned(who, {dout, z, z_scale, x, x_scale, w, dx, dw, dbias, group_offsets}));
  return workspace_ok(who, workspace, workspace_bytes, needed);
}

}  // namespace mc2
