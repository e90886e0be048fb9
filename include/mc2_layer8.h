/*
 * mc2_layer8.h -- the router of a mixture-of-experts layer, and the 8-bit
 * forms of the feed-forward operators of mc2_layer.h, on one AMD Instinct
 * MI355X (gfx950): int8 codes of rows and back, the linear of int8 codes with
 * its epilogue (serving), and the linear's gradient from activations that
 * were kept as int8 codes (training).
 *
 * Conventions are those of mc2_layer.h: caller-owned, contiguous, 16-byte
 * aligned device tensors, work enqueued on `stream`, arguments validated on
 * the host before any device call, an mc2_status from every call, no
 * allocation, the same bits from the same inputs; a call with no rows is valid
 * and its row tensors may be NULL.  Outputs may not overlap inputs unless a
 * declaration says so.
 */
#ifndef MC2_LAYER8_H_
#define MC2_LAYER8_H_

#include "mc2_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Scores of mc2_moe_route. */
typedef enum {
  MC2_SCORE_SOFTMAX = 0, /* exp(l) / sum over the experts of exp(l) */
  MC2_SCORE_SIGMOID = 1, /* 1 / (1 + exp(-l)) */
  MC2_SCORE_KEEP_NAN = 1 << 16 /* added to one of them in mc2_moe_route: see there */
} mc2_score;

/*
 * Each token's experts and their weights.  With p the scores of a token's
 * logits l, and c = p + bias (the bias takes part in the choice alone):
 *   - an expert is off if its logit is -inf or its c is -inf or NaN;
 *   - groups > 1: the experts stand in `groups` groups of experts / groups
 *     neighbours.  A group's value is the sum of its group_top largest c that
 *     are on; the top_groups groups of the largest values are kept (equal
 *     values: the first), the experts of the others are off for this token;
 *   - the `top` largest c that are on are chosen, in descending order (equal
 *     c: the lowest expert first).  Without a bias c rises with l, and the
 *     order is that of the logits (equal logits: the lowest expert first) also
 *     where their scores round to equal numbers, as sigmoids of 40 and 41 do
 *     in fp64; so is the order of groups with group_top 1;
 *   - weights = scale p of the chosen, with renormalise scale p / sum of the
 *     chosen p.
 *   expert_ids  (tokens, top) int32; -1 where fewer than top experts are on
 *   weights     (tokens, top) fp32; 0 there, and 0 for a sigmoid that is 0 in
 *               fp64 (logits below -709.78; of the scores that fp32 alone would
 *               round to 0 renormalise gives the shares that they have)
 * A token with a NaN among its logits, or with softmax a logit of +inf, has no
 * experts: ids -1, weights NaN.  (mc2_moe_permute drops an id of -1, and
 * mc2_moe_unpermute reads no weight of one: such a token's row is 0.)  With
 * MC2_SCORE_KEEP_NAN added to the score it has the experts 0 .. top - 1, so
 * that its weights make its row NaN.
 * Else c is compared in fp32 where its error there leaves no doubt about the
 * order, and in fp64 otherwise: the choice is that of fp64.
 *
 * logits      (tokens, experts) of dtype: MC2_F32, MC2_F16 or MC2_BF16
 * bias        (experts) fp32 or NULL (0)
 * tokens <= 2^23, 1 <= experts <= 4096, 1 <= top <= 64; groups in [1, 64]
 * divides experts; top_groups in [1, groups]; group_top 1 or 2, at most
 * experts / groups; top <= top_groups * experts / groups; scale finite
 */
mc2_status mc2_moe_route(const void* logits, const float* bias, int64_t tokens, int64_t experts, int64_t top,
                         mc2_dtype dtype, mc2_score score, int64_t groups, int64_t top_groups, int64_t group_top,
                         int renormalise, float scale, int32_t* expert_ids, float* weights, void* stream);

/*
 * Gradient of mc2_moe_route's weights for the logits, at the experts chosen
 * (the choice has no gradient, nor has the bias).  With g_j = scale *
 * dweights_j, and i_j the j-th chosen expert:
 *   softmax                dl_e = p_e (d_e - sum_j g_j p_ij),
 *                          d_e = sum of the g_j with i_j = e
 *   sigmoid                dl_e = d_e p_e (1 - p_e)
 *   softmax, renormalised  a_j = p_ij / sum of the chosen p:
 *                          dl_ij = a_j (g_j - sum_j g_j a_j), 0 elsewhere
 *   sigmoid, renormalised  dl_ij = a_j (1 - p_ij) (g_j - sum_j g_j a_j)
 * Ids outside [0, experts) have no part in it, whatever their dweights hold;
 * a token with no other ids has dl = 0.
 * dweights (tokens, top) fp32; logits, dlogits (tokens, experts) of dtype;
 * dlogits may be logits itself.  Sizes as in mc2_moe_route.
 */
mc2_status mc2_moe_route_grad(const float* dweights, const void* logits, const int32_t* expert_ids, int64_t tokens,
                              int64_t experts, int64_t top, mc2_dtype dtype, mc2_score score, int renormalise,
                              float scale, void* dlogits, void* stream);

/*
 * Rows as int8 codes.  Per row (group 0) or per 128 columns of a row (group
 * 128; a row's last group may be shorter), in fp32:
 *   a = max |x|, scale = a / 127, code = clamp(rint(x / scale), -127, 127)
 * A group of zeros has scale 0 and codes 0; one with a NaN or an infinity has
 * a NaN or infinite scale and codes 0 (its values come back as NaN).
 * x (rows, cols) of dtype (MC2_F16 or MC2_BF16), codes (rows, cols) int8,
 * scale (rows, ceil(cols / group)) fp32 (group 0: (rows, 1)).
 * rows < 2^24, 1 <= cols <= 2^24.
 *
 * group = 128 + MC2_KEEP_INF: as 128, for pre-activations, which their 16 bits
 * may hold as infinities.  a is the largest finite |x| of the group (if that is
 * 0 and an infinity is there, the type's largest number); +inf gets the code
 * of a.  -inf, whose activation and slope are 0, stays one: a group with a -inf
 * has the negative scale -a / 127 (and the codes rint(x / scale) of that), and
 * the code -128 for it.  In mc2_dequant_rows and mc2_linear_act_grad_i8 a code
 * of -128 under a negative scale is -inf.
 */
enum { MC2_KEEP_INF = 1 << 16 };
mc2_status mc2_quant_rows(const void* x, int64_t rows, int64_t cols, mc2_dtype dtype, int64_t group, int8_t* codes,
                          float* scale, void* stream);

/* And back: out = act(code * scale), rounded once to dtype.  Arguments as in mc2_quant_rows (group 0 or 128). */
mc2_status mc2_dequant_rows(const int8_t* codes, const float* scale, int64_t rows, int64_t cols, int64_t group,
                            mc2_act act, mc2_dtype dtype, void* out, void* stream);

/*
 * Linear of int8 codes with bias, activation and residual in its epilogue:
 *   c   = x @ w^T                              (exact in int32)
 *   z   = (c * x_scale) * w_scale + bias       (fp32)
 *   out = residual + act(z)                    (one rounding to dtype)
 * Dense or grouped, and group_offsets read, as in mc2_linear_act; rows of no
 * group get z = 0.
 * x         (m, k) int8, x_scale (m) fp32: one per token
 * w         (n, k) or (G, n, k) int8, w_scale (n) or (G, n) fp32: one per
 *           channel; as mc2_quant_rows or mc2_add_rms_norm with group 0 give
 * bias, residual (m, n)  of dtype (MC2_F16 or MC2_BF16), or NULL
 * out       (m, n) of dtype; may be residual itself
 * workspace 16-byte aligned, at least mc2_linear_i8_workspace_size bytes
 *           (NULL when that is 0)
 * Sizes as in mc2_linear_act, and k < 2^17 (any codes' sums fit int32).
 */
mc2_status mc2_linear_i8_workspace_size(int64_t m, int64_t k, int64_t n, int64_t groups, size_t* bytes);
mc2_status mc2_linear_i8(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale,
                         const void* bias, const void* residual, int64_t m, int64_t k, int64_t n,
                         const int32_t* group_offsets, int64_t groups, mc2_dtype dtype, mc2_act act, void* out,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of mc2_linear_act from what was kept in 8 bits: its input and its
 * pre-activation as codes with a scale per 128 columns (mc2_quant_rows, group
 * 128).  With zv = z * z_scale and xv = x_act(x * x_scale):
 *   dz    = dout * act'(zv)
 *   dx    = dz @ w, dw = dz^T @ xv, dbias = sum over rows of dz
 * as mc2_linear_act_grad gives them, which see; where zv is NaN, so is dz, with
 * relu too.  x_act lets the input be kept as the pre-activation it came from: a
 * feed-forward's second linear takes the codes of its first one's z.  xv is
 * rounded to dtype for its product, as dz is.
 * x (m, k) int8, x_scale (m, ceil(k / 128)) fp32 (needed for dw alone);
 * z (m, n) int8, z_scale (m, ceil(n / 128)) fp32 (NULL with MC2_ACT_NONE);
 * dout, w, dx, dw, dbias of dtype.
 */
mc2_status mc2_linear_act_grad_i8_workspace_size(int64_t m, int64_t k, int64_t n, int64_t groups, size_t* bytes);
mc2_status mc2_linear_act_grad_i8(const void* dout, const int8_t* z, const float* z_scale, const int8_t* x,
                                  const float* x_scale, mc2_act x_act, const void* w, int64_t m, int64_t k,
                                  int64_t n, const int32_t* group_offsets, int64_t groups, mc2_dtype dtype,
                                  mc2_act act, void* dx, void* dw, void* dbias, void* workspace,
                                  size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MC2_LAYER8_H_ */
