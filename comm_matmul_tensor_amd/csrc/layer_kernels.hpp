// Internal launch interface between the C ABI of mc2_layer.h (layer_api.cpp)
// and its HIP kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

namespace mc2 {

// ---- K10: residual addition + RMS norm (+ 8-bit codes with scales), and its gradients
struct NormArgs {
  const void *x, *residual, *weight;
  int64_t rows, h, group;
  int dtype, out_dtype;  // DT_* codes
  float eps;
  void* out;
  float* scale;
  void* sum;
  float* rstd;
};
hipError_t launch_add_rms_norm(const NormArgs& a, hipStream_t s);

struct NormGradArgs {
  const void *dout, *dsum, *s, *weight;
  const float* rstd;
  int64_t rows, h;
  int dtype;
  void *dx, *dweight;
  float* partials;  // norm_grad_blocks(rows, h) rows of h
};
int64_t norm_grad_blocks(int64_t rows, int64_t h);
hipError_t launch_add_rms_norm_grad(const NormGradArgs& a, hipStream_t s);

// ---- K11: linear with bias, activation and residual, dense or by groups of rows
struct LinearArgs {
  const void *x, *w, *bias, *residual;
  int64_t m, k, n, groups;
  const int32_t* offsets;
  int dtype, act;
  void *out, *z;
  void* workspace;
};
size_t linear_act_workspace(int64_t m, int64_t k, int64_t n, int64_t groups);
hipError_t launch_linear_act(const LinearArgs& a, hipStream_t s);

struct LinearGradArgs {
  const void *dout, *z, *x, *w;
  int64_t m, k, n, groups;
  const int32_t* offsets;
  int dtype, act;
  void *dx, *dw, *dbias;
  void* workspace;
  // z and x as int8 codes with a scale per 128 columns (eight: x and z are NULL)
  bool eight;
  const int8_t *z_codes, *x_codes;
  const float *z_scale, *x_scale;
  int x_act;
};
size_t linear_act_grad_workspace(int64_t m, int64_t k, int64_t n, int64_t groups, bool eight = false);
// The tile and the parts of K of a call's product (testing.h).
void linear_act_plan(int product, int64_t m, int64_t k, int64_t n, int64_t groups, int* tile, int* splits);
hipError_t launch_linear_act_grad(const LinearGradArgs& a, hipStream_t s);

// ---- K12: tokens' rows by expert and back
struct PermuteArgs {
  const void* x;
  const int32_t* ids;
  int64_t tokens, top, h, experts;
  void* out;
  int32_t *row_map, *offsets;
  int32_t* workspace;
};
size_t moe_permute_workspace(int64_t choices, int64_t experts);
hipError_t launch_moe_permute(const PermuteArgs& a, hipStream_t s);

struct UnpermuteArgs {
  const void *y, *dout;  // dout: the gradient's
  const int32_t* row_map;
  const float* weights;
  int64_t tokens, top, h, rows;
  int dtype;
  void *out, *dy;
  float* dweights;
};
hipError_t launch_moe_unpermute(const UnpermuteArgs& a, hipStream_t s);
hipError_t launch_moe_unpermute_grad(const UnpermuteArgs& a, hipStream_t s);

}  // namespace mc2
