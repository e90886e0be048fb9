// Internal launch interface between the C ABI of mc2_layer8.h (layer8_api.cpp)
// and its HIP kernels.
#pragma once
#include "layer_kernels.hpp"

namespace mc2 {

// ---- K13: the router and its gradient
enum : int { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1 };
struct RouteArgs {
  const void* logits;
  const float *bias, *dweights;  // dweights: the gradient's
  int64_t tokens;
  int experts, top, dtype, score;
  int groups, top_groups, group_top, renormalise;
  bool keep_nan;       // a token without a usable logit: its experts are 0 .. top - 1, not -1
  float scale;
  int32_t* ids;        // read by the gradient
  float* weights;
  void* dlogits;
};
hipError_t launch_moe_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_moe_route_grad(const RouteArgs& a, hipStream_t s);

// ---- K14: rows to int8 codes and back
struct CodeArgs {
  const void* x;             // the rows, read
  void* out;                 // the rows, written
  const int8_t* codes_in;
  int8_t* codes;
  const float* scale_in;
  float* scale;
  int64_t rows, cols, group;
  int64_t ld;                // columns between the rows written (dequant): 0 means cols; those past cols become 0
  int dtype, act;
  bool keep_inf;             // quant, group 128: MC2_KEEP_INF
};
hipError_t launch_quant_rows(const CodeArgs& a, hipStream_t s);
hipError_t launch_dequant_rows(const CodeArgs& a, hipStream_t s);

// ---- K15: linear of int8 codes (its gradient's operands in 8 bits: K11)
struct LinearI8Args {
  const int8_t *x, *w;
  const float *x_scale, *w_scale;
  const void *bias, *residual;
  int64_t m, k, n, groups;
  const int32_t* offsets;
  int dtype, act;
  void* out;
  void* workspace;
};
size_t linear_i8_workspace(int64_t m, int64_t k, int64_t n, int64_t groups);
hipError_t launch_linear_i8(const LinearI8Args& a, hipStream_t s);
// The tile and the parts of K of a call's product (testing.h).
void linear_i8_plan(int64_t m, int64_t k, int64_t n, int64_t groups, int* tile, int* splits);

}  // namespace mc2
