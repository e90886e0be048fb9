/*
 * mc2_layer.h -- the feed-forward operators of a transformer layer around the
 * MC2 matmuls of mc2.h, on one AMD Instinct MI355X (gfx950): the norm before
 * them, a linear with its epilogue (of one matrix or of experts' matrices),
 * and the order of tokens by expert.
 *
 * Conventions are those of mc2.h: caller-owned, contiguous, 16-byte aligned
 * device tensors, work enqueued on `stream`, arguments validated on the host
 * before any device call, an mc2_status from every call, no allocation, the
 * same bits from the same inputs.  Here a call with no rows is a valid call
 * that writes only what does not depend on rows (a rank or an expert may get
 * none); its row tensors may then be NULL.  Values that live on the device
 * (row ranges, expert ids, row maps) cannot be checked on the host: the
 * kernels bound every index they form from them, as each declaration says.
 */
#ifndef MC2_LAYER_H_
#define MC2_LAYER_H_

#include "mc2.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Root-mean-square norm with the residual's addition:
 *   s        = x + residual                       (fp32)
 *   rstd     = 1 / sqrt(mean over h of s^2 + eps) per row (fp32)
 *   y        = s * rstd * weight                  (fp32)
 *   out      = y rounded to 16 bits, or codes of y in 8 bits with scales
 *   sum_out  = s rounded to 16 bits (the residual stream that goes on)
 * 8-bit output: per group of `group` columns (0: per row), a = max |y|,
 *   MC2_I8       scale = a / 127, code = clamp(rint(y / scale), -127, 127)
 *   MC2_F8E4M3FN scale = a / 448, code = y / scale rounded to nearest even
 * in fp32 (ties to even).  A group of zeros has scale 0 and codes 0; a group
 * with a NaN or an infinity has a NaN or infinite scale and codes 0.
 *
 * x, residual  (rows, h) of dtype; residual may be NULL (s = x)
 * weight       (h) of dtype
 * dtype        MC2_F16 or MC2_BF16
 * eps          finite, >= 0
 * rows < 2^24, 1 <= h <= 2^24
 * out          (rows, h) of out_dtype: dtype, MC2_I8 or MC2_F8E4M3FN
 * scale_out    (rows, h / group) fp32 (group 0: (rows, 1)) for 8-bit output, else NULL
 * group        0, or 128 with an 8-bit out_dtype and h a multiple of 128
 * sum_out      (rows, h) of dtype or NULL; may be residual or x themselves
 * rstd_out     (rows) fp32 or NULL
 */
mc2_status mc2_add_rms_norm(const void* x, const void* residual, const void* weight, int64_t rows, int64_t h,
                            mc2_dtype dtype, float eps, void* out, mc2_dtype out_dtype, float* scale_out,
                            int64_t group, void* sum_out, float* rstd_out, void* stream);

/*
 * Gradients of mc2_add_rms_norm with a 16-bit output.  With s the saved sum
 * (x where there was no residual) and g = dout * weight:
 *   dx      = rstd (g - s rstd^2 mean over h of (g s)) + dsum
 *   dweight = sum over rows of dout * s * rstd
 * dx is the gradient of x and of residual alike; dsum (NULL: zero) is the
 * gradient that reached sum_out.  dweight is summed in fp32 in a fixed order.
 * dx may be dout or dsum themselves.  workspace: 16-byte aligned, at least
 * mc2_add_rms_norm_grad_workspace_size bytes.  With no rows dweight is zero.
 */
mc2_status mc2_add_rms_norm_grad_workspace_size(int64_t rows, int64_t h, size_t* bytes);
mc2_status mc2_add_rms_norm_grad(const void* dout, const void* dsum, const void* s, const void* weight,
                                 const float* rstd, int64_t rows, int64_t h, mc2_dtype dtype, void* dx,
                                 void* dweight, void* workspace, size_t workspace_bytes, void* stream);

/* Activations of mc2_linear_act; each maps 0 to 0. */
typedef enum {
  MC2_ACT_NONE = 0,
  MC2_ACT_RELU = 1,
  MC2_ACT_GELU = 2,      /* z Phi(z), Phi the normal distribution function */
  MC2_ACT_GELU_TANH = 3, /* 0.5 z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) */
  MC2_ACT_SILU = 4       /* z / (1 + exp(-z)) */
} mc2_act;

/*
 * Linear with bias, activation and residual in the product's epilogue:
 *   z   = x @ w^T + bias        (fp32 accumulation)
 *   out = residual + act(z)     (z not rounded in between; one rounding)
 * Dense (groups 0): w (n, k), the nn.Linear layout, and bias (n).
 * Grouped (groups G >= 1, the products of experts): w (G, n, k), bias (G, n),
 * and rows [group_offsets[g], group_offsets[g + 1]) of x use matrix g; rows
 * of no group get z = 0 (out = residual, or 0).  group_offsets is (G + 1)
 * int32 on the device, ascending from 0 to at most m: the first is taken as
 * 0, each other as no less than the one before it and no more than m.
 *
 * x         (m, k) of dtype (MC2_F16 or MC2_BF16)
 * bias, residual (m, n)  of dtype, or NULL
 * out       (m, n) of dtype; may be residual itself
 * z_out     (m, n) of dtype or NULL: z rounded, which the gradient needs
 * workspace 16-byte aligned, at least mc2_linear_act_workspace_size bytes
 *           (NULL when that is 0)
 * m < 2^24, 1 <= k, n <= 2^21, G <= 4096, G n and G k <= 2^29.
 */
mc2_status mc2_linear_act_workspace_size(int64_t m, int64_t k, int64_t n, int64_t groups, size_t* bytes);
mc2_status mc2_linear_act(const void* x, const void* w, const void* bias, const void* residual, int64_t m,
                          int64_t k, int64_t n, const int32_t* group_offsets, int64_t groups, mc2_dtype dtype,
                          mc2_act act, void* out, void* z_out, void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * Gradients of mc2_linear_act (residual's is dout itself):
 *   dz    = dout * act'(z)      (z as z_out gave it; NULL with MC2_ACT_NONE)
 *   dx    = dz @ w              rows of no group: 0
 *   dw    = dz^T @ x            per group; a group without rows: 0
 *   dbias = sum over rows of dz per group, from the unrounded dz in fp32
 * The products read dz rounded to dtype (they run on 16-bit operands) and
 * accumulate in fp32.  relu's slope at 0 is 0.  dx, dw and dbias may each be
 * NULL.  workspace: 16-byte aligned, at least
 * mc2_linear_act_grad_workspace_size bytes.
 */
mc2_status mc2_linear_act_grad_workspace_size(int64_t m, int64_t k, int64_t n, int64_t groups, size_t* bytes);
mc2_status mc2_linear_act_grad(const void* dout, const void* z, const void* x, const void* w, int64_t m, int64_t k,
                               int64_t n, const int32_t* group_offsets, int64_t groups, mc2_dtype dtype,
                               mc2_act act, void* dx, void* dw, void* dbias, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * Tokens' rows sorted by expert.  Choice j of token t is expert_ids[t][j]; an
 * id outside [0, experts) drops that choice.  The kept choices are ordered by
 * expert, those of one expert by t * top + j:
 *   out        (tokens * top, h): row i is the row of x of the i-th kept
 *              choice; the rows after the last kept one are 0
 *   row_map    (tokens, top) int32: the row of each choice, -1 if dropped
 *   offsets    (experts + 1) int32: expert e has rows [offsets[e], offsets[e + 1])
 * x (tokens, h) of dtype (MC2_F16 or MC2_BF16); tokens <= 2^23, tokens * top
 * < 2^31, 1 <= h <= 2^24, 1 <= experts <= 4096.  The gradient for x is mc2_moe_unpermute without
 * weights.  workspace: 16-byte aligned, at least
 * mc2_moe_permute_workspace_size bytes.
 */
mc2_status mc2_moe_permute_workspace_size(int64_t tokens, int64_t top, int64_t experts, size_t* bytes);
mc2_status mc2_moe_permute(const void* x, const int32_t* expert_ids, int64_t tokens, int64_t top, int64_t h,
                           int64_t experts, mc2_dtype dtype, void* out, int32_t* row_map, int32_t* offsets,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rows back in token order, weighted:
 *   out[t] = sum over j of weights[t][j] * y[row_map[t][j]]   (fp32, j ascending)
 * y (rows, h) of dtype, row_map (tokens, top) int32 (an entry outside
 * [0, rows) adds nothing), weights (tokens, top) fp32 or NULL (all 1),
 * out (tokens, h) of dtype.
 */
mc2_status mc2_moe_unpermute(const void* y, const int32_t* row_map, const float* weights, int64_t tokens,
                             int64_t top, int64_t h, int64_t rows, mc2_dtype dtype, void* out, void* stream);

/*
 * Gradients of mc2_moe_unpermute:
 *   dy[row_map[t][j]]  = weights[t][j] * dout[t]
 *   dweights[t][j]     = sum over h of y[row_map[t][j]] * dout[t]   (0 if dropped)
 * row_map is one mc2_moe_permute gave: with c kept choices it names each of
 * the rows 0 .. c - 1 once, and dy's rows c .. rows - 1 become 0.  weights
 * NULL: all 1.  dweights (tokens, top) fp32 or NULL, y (rows, h) needed only
 * for it, dy (rows, h) or NULL; with rows one of the two is required.
 */
mc2_status mc2_moe_unpermute_grad(const void* dout, const void* y, const int32_t* row_map, const float* weights,
                                  int64_t tokens, int64_t top, int64_t h, int64_t rows, mc2_dtype dtype, void* dy,
                                  float* dweights, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MC2_LAYER_H_ */
