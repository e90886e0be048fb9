// Host-only argument validation of the entry points of mc2_layer8.h.
#pragma once
#include "mc2_layer8.h"
#include "validate_layer.hpp"

namespace mc2 {

mc2_status check_moe_route(const void* logits, const void* bias, int64_t tokens, int64_t experts, int64_t top,
                           mc2_dtype dtype, mc2_score score, int64_t groups, int64_t top_groups, int64_t group_top,
                           float scale, const void* expert_ids, const void* weights);
mc2_status check_moe_route_grad(const void* dweights, const void* logits, const void* expert_ids, int64_t tokens,
                                int64_t experts, int64_t top, mc2_dtype dtype, mc2_score score, float scale,
                                const void* dlogits);
mc2_status check_code_rows(const char* who, const void* values, const void* codes, const void* scale, int64_t rows,
                           int64_t cols, mc2_dtype dtype, int64_t group, mc2_act act);
mc2_status check_linear_i8_sizes(const char* who, int64_t m, int64_t k, int64_t n, int64_t groups);
mc2_status check_linear_i8(const void* x, const void* x_scale, const void* w, const void* w_scale, const void* bias,
                           const void* residual, int64_t m, int64_t k, int64_t n, const void* group_offsets,
                           int64_t groups, mc2_dtype dtype, mc2_act act, const void* out, const void* workspace,
                           size_t workspace_bytes, size_t needed);
mc2_status check_linear_act_grad_i8(const void* dout, const void* z, const void* z_scale, const void* x,
                                    const void* x_scale, mc2_act x_act, const void* w, int64_t m, int64_t k,
                                    int64_t n, const void* group_offsets, int64_t groups, mc2_dtype dtype, mc2_act act,
                                    const void* dx, const void* dw, const void* dbias, const void* workspace,
                                    size_t workspace_bytes, size_t needed);

}  // namespace mc2
