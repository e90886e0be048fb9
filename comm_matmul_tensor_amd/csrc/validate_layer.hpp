// Host-only argument validation of the entry points of mc2_layer.h.
#pragma once
#include "mc2_layer.h"
#include "validate.hpp"

namespace mc2 {

mc2_status check_add_rms_norm(const void* x, const void* residual, const void* weight, int64_t rows, int64_t h,
                              mc2_dtype dtype, float eps, const void* out, mc2_dtype out_dtype, const void* scale_out,
                              int64_t group, const void* sum_out, const void* rstd_out);
mc2_status check_norm_sizes(const char* who, int64_t rows, int64_t h);
mc2_status check_add_rms_norm_grad(const void* dout, const void* dsum, const void* s, const void* weight,
                                   const void* rstd, int64_t rows, int64_t h, mc2_dtype dtype, const void* dx,
                                   const void* dweight, const void* workspace, size_t workspace_bytes, size_t needed);
mc2_status check_linear_sizes(const char* who, int64_t m, int64_t k, int64_t n, int64_t groups);
mc2_status check_linear_kind(const char* who, const void* group_offsets, int64_t groups, mc2_dtype dtype,
                             mc2_act act);
mc2_status check_linear_act(const void* x, const void* w, const void* bias, const void* residual, int64_t m, int64_t k,
                            int64_t n, const void* group_offsets, int64_t groups, mc2_dtype dtype, mc2_act act,
                            const void* out, const void* z_out, const void* workspace, size_t workspace_bytes,
                            size_t needed);
mc2_status check_linear_act_grad(const void* dout, const void* z, const void* x, const void* w, int64_t m, int64_t k,
                                 int64_t n, const void* group_offsets, int64_t groups, mc2_dtype dtype, mc2_act act,
                                 const void* dx, const void* dw, const void* dbias, const void* workspace,
                                 size_t workspace_bytes, size_t needed);
mc2_status check_permute_sizes(const char* who, int64_t tokens, int64_t top, int64_t experts);
mc2_status check_moe_permute(const void* x, const void* expert_ids, int64_t tokens, int64_t top, int64_t h,
                             int64_t experts, mc2_dtype dtype, const void* out, const void* row_map,
                             const void* offsets, const void* workspace, size_t workspace_bytes, size_t needed);
mc2_status check_moe_unpermute(const void* y, const void* row_map, const void* weights, int64_t tokens, int64_t top,
                               int64_t h, int64_t rows, mc2_dtype dtype, const void* out);
mc2_status check_moe_unpermute_grad(const void* dout, const void* y, const void* row_map, const void* weights,
                                    int64_t tokens, int64_t top, int64_t h, int64_t rows, mc2_dtype dtype,
                                    const void* dy, const void* dweights);

}  // namespace mc2
