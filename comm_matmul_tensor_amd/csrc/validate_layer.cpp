// Host-only argument validation of the feed-forward operators (mc2_layer.h);
// no HIP calls.
#include "validate_layer.hpp"

#include <cmath>
#include <initializer_list>

namespace mc2 {

namespace {

using std::string;

constexpr int64_t kRows = (int64_t)1 << 24, kWidth = (int64_t)1 << 24, kDim = (int64_t)1 << 21,
                  kTokens = (int64_t)1 << 23, kGroups = 4096, kGroupWidth = (int64_t)1 << 29;

bool is_half(mc2_dtype d) { return d == MC2_F16 || d == MC2_BF16; }
string str(int64_t v) { return std::to_string(static_cast<long long>(v)); }

mc2_status shape(const char* who, const string& what) { return fail(MC2_ERR_SHAPE, string(who) + ": " + what); }

// Every pointer 16-byte aligned (NULL is).
mc2_status aligned(const char* who, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 15u)
      return fail(MC2_ERR_ALIGN, string(who) + ": tensor not 16-byte aligned");
  return MC2_OK;
}
mc2_status required(const char* who, std::initializer_list<const void*> ps, const char* names) {
  for (const void* p : ps)
    if (!p) return fail(MC2_ERR_NULL, string(who) + ": " + names + " are required");
  return MC2_OK;
}
mc2_status half(const char* who, mc2_dtype d) {
  return is_half(d) ? MC2_OK : fail(MC2_ERR_DTYPE, string(who) + ": dtype must be F16 or BF16");
}
mc2_status workspace_ok(const char* who, const void* ws, size_t bytes, size_t needed) {
  if (needed > 0 && (!ws || bytes < needed))
    return fail(MC2_ERR_WORKSPACE, string(who) + ": workspace needs " + std::to_string(needed) + " bytes");
  return needed > 0 ? aligned(who, {ws}) : MC2_OK;
}

#define MC2_TRY(call)                \
  do {                               \
    mc2_status s_ = (call);          \
    if (s_ != MC2_OK) return s_;     \
  } while (0)

}  // namespace

mc2_status check_norm_sizes(const char* who, int64_t rows, int64_t h) {
  if (rows < 0 || rows >= kRows) return shape(who, "rows must lie in [0, 2^24), got " + str(rows));
  if (h < 1 || h > kWidth) return shape(who, "h must lie in [1, 2^24], got " + str(h));
  return MC2_OK;
}

mc2_status check_add_rms_norm(const void* x, const void* residual, const void* weight, int64_t rows, int64_t h,
                              mc2_dtype dtype, float eps, const void* out, mc2_dtype out_dtype, const void* scale_out,
                              int64_t group, const void* sum_out, const void* rstd_out) {
  const char* who = "add_rms_norm";
  MC2_TRY(check_norm_sizes(who, rows, h));
  MC2_TRY(half(who, dtype));
  const bool eight = out_dtype == MC2_I8 || out_dtype == MC2_F8E4M3FN;
  if (!eight && out_dtype != dtype)
    return fail(MC2_ERR_DTYPE, "add_rms_norm: out_dtype must be dtype, I8 or F8E4M3FN");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return shape(who, "eps must be finite and not negative");
  if (group != 0 && (group != 128 || !eight || h % 128 != 0))
    return shape(who, "group must be 0, or 128 with an 8-bit output and h a multiple of 128, got " + str(group));
  if (rows == 0) return MC2_OK;
  MC2_TRY(required(who, {x, weight, out}, "x, weight and out"));
  if (eight && !scale_out) return fail(MC2_ERR_NULL, "add_rms_norm: an 8-bit output needs scale_out");
  return aligned(who, {x, residual, weight, out, scale_out, sum_out, rstd_out});
}

mc2_status check_add_rms_norm_grad(const void* dout, const void* dsum, const void* s, const void* weight,
                                   const void* rstd, int64_t rows, int64_t h, mc2_dtype dtype, const void* dx,
                                   const void* dweight, const void* workspace, size_t workspace_bytes, size_t needed) {
  const char* who = "add_rms_norm_grad";
  MC2_TRY(check_norm_sizes(who, rows, h));
  MC2_TRY(half(who, dtype));
  MC2_TRY(required(who, {weight, dweight}, "weight and dweight"));
  if (rows > 0) MC2_TRY(required(who, {dout, s, rstd, dx}, "dout, s, rstd and dx"));
  MC2_TRY(aligned(who, {dout, dsum, s, weight, rstd, dx, dweight}));
  return workspace_ok(who, workspace, workspace_bytes, needed);
}

mc2_status check_linear_sizes(const char* who, int64_t m, int64_t k, int64_t n, int64_t groups) {
  if (m < 0 || m >= kRows) return shape(who, "m must lie in [0, 2^24), got " + str(m));
  if (k < 1 || k > kDim) return shape(who, "k must lie in [1, 2^21], got " + str(k));
  if (n < 1 || n > kDim) return shape(who, "n must lie in [1, 2^21], got " + str(n));
  if (groups < 0 || groups > kGroups) return shape(who, "groups must lie in [0, 4096], got " + str(groups));
  // (every group may have a partial tile of rows: bounds the tiles of a launch)
  if (groups * n > kGroupWidth || groups * k > kGroupWidth)
    return shape(who, "groups * n and groups * k must be at most 2^29");
  return MC2_OK;
}

namespace {
mc2_status check_linear_kind(const char* who, const void* group_offsets, int64_t groups, mc2_dtype dtype,
                             mc2_act act) {
  MC2_TRY(half(who, dtype));
  if (act < MC2_ACT_NONE || act > MC2_ACT_SILU)
    return fail(MC2_ERR_UNSUPPORTED, string(who) + ": unknown activation " + str(act));
  if (groups > 0 && !group_offsets) return fail(MC2_ERR_NULL, string(who) + ": groups need group_offsets");
  if (groups == 0 && group_offsets) return shape(who, "group_offsets without groups");
  return MC2_OK;
}
}  // namespace

mc2_status check_linear_act(const void* x, const void* w, const void* bias, const void* residual, int64_t m, int64_t k,
                            int64_t n, const void* group_offsets, int64_t groups, mc2_dtype dtype, mc2_act act,
                            const void* out, const void* z_out, const void* workspace, size_t workspace_bytes,
                            size_t needed) {
  const char* who = "linear_act";
  MC2_TRY(check_linear_sizes(who, m, k, n, groups));
  MC2_TRY(check_linear_kind(who, group_offsets, groups, dtype, act));
  if (m == 0) return MC2_OK;
  MC2_TRY(required(who, {x, w, out}, "x, w and out"));
  MC2_TRY(aligned(who, {x, w, bias, residual, out, z_out, group_offsets}));
  return workspace_ok(who, workspace, workspace_bytes, needed);
}

mc2_status check_linear_act_grad(const void* dout, const void* z, const void* x, const void* w, int64_t m, int64_t k,
                                 int64_t n, const void* group_offsets, int64_t groups, mc2_dtype dtype, mc2_act act,
                                 const void* dx, const void* dw, const void* dbias, const void* workspace,
                                 size_t workspace_bytes, size_t needed) {
  const char* who = "linear_act_grad";
  MC2_TRY(check_linear_sizes(who, m, k, n, groups));
  MC2_TRY(check_linear_kind(who, group_offsets, groups, dtype, act));
  if (m > 0) {
    if (!dout || (act != MC2_ACT_NONE && !z) || (dw && !x) || (dx && !w))
      return fail(MC2_ERR_NULL, "linear_act_grad: dout, z (with an activation), x (for dw) and w (for dx) are required");
  }
  MC2_TRY(aligned(who, {dout, z, x, w, dx, dw, dbias, group_offsets}));
  return workspace_ok(who, workspace, workspace_bytes, needed);
}

mc2_status check_permute_sizes(const char* who, int64_t tokens, int64_t top, int64_t experts) {
  if (tokens < 0 || tokens > kTokens) return shape(who, "tokens must lie in [0, 2^23], got " + str(tokens));
  if (top < 1 || top > INT32_MAX || tokens * top > INT32_MAX)
    return shape(who, "top must be at least 1 and tokens * top below 2^31, got " + str(top));
  if (experts < 1 || experts > kGroups) return shape(who, "experts must lie in [1, 4096], got " + str(experts));
  return MC2_OK;
}

mc2_status check_moe_permute(const void* x, const void* expert_ids, int64_t tokens, int64_t top, int64_t h,
                             int64_t experts, mc2_dtype dtype, const void* out, const void* row_map,
                             const void* offsets, const void* workspace, size_t workspace_bytes, size_t needed) {
  const char* who = "moe_permute";
  MC2_TRY(check_permute_sizes(who, tokens, top, experts));
  if (h < 1 || h > kWidth) return shape(who, "h must lie in [1, 2^24], got " + str(h));
  MC2_TRY(half(who, dtype));
  if (!offsets) return fail(MC2_ERR_NULL, "moe_permute: offsets is required");
  if (tokens > 0) MC2_TRY(required(who, {x, expert_ids, out, row_map}, "x, expert_ids, out and row_map"));
  MC2_TRY(aligned(who, {x, expert_ids, out, row_map, offsets}));
  return workspace_ok(who, workspace, workspace_bytes, needed);
}

namespace {
mc2_status check_unpermute_sizes(const char* who, int64_t tokens, int64_t top, int64_t h, int64_t rows,
                                 mc2_dtype dtype) {
  MC2_TRY(check_permute_sizes(who, tokens, top, 1));
  if (h < 1 || h > kWidth) return shape(who, "h must lie in [1, 2^24], got " + str(h));
  if (rows < 0 || rows > INT32_MAX) return shape(who, "rows must lie in [0, 2^31), got " + str(rows));
  return half(who, dtype);
}
}  // namespace

mc2_status check_moe_unpermute(const void* y, const void* row_map, const void* weights, int64_t tokens, int64_t top,
                               int64_t h, int64_t rows, mc2_dtype dtype, const void* out) {
  const char* who = "moe_unpermute";
  MC2_TRY(check_unpermute_sizes(who, tokens, top, h, rows, dtype));
  if (tokens == 0) return MC2_OK;
  MC2_TRY(required(who, {row_map, out}, "row_map and out"));
  if (rows > 0 && !y) return fail(MC2_ERR_NULL, "moe_unpermute: y is required");
  return aligned(who, {y, row_map, weights, out});
}

mc2_status check_moe_unpermute_grad(const void* dout, const void* y, const void* row_map, const void* weights,
                                    int64_t tokens, int64_t top, int64_t h, int64_t rows, mc2_dtype dtype,
                                    const void* dy, const void* dweights) {
  const char* who = "moe_unpermute_grad";
  MC2_TRY(check_unpermute_sizes(who, tokens, top, h, rows, dtype));
  if (rows > 0 && !dy && !dweights) return fail(MC2_ERR_NULL, "moe_unpermute_grad: dy or dweights is required");
  if (tokens > 0) MC2_TRY(required(who, {dout, row_map}, "dout and row_map"));
  if (dweights && tokens > 0 && rows > 0 && !y)
    return fail(MC2_ERR_NULL, "moe_unpermute_grad: dweights needs y");
  return aligned(who, {dout, y, row_map, weights, dy, dweights});
}

}  // namespace mc2
