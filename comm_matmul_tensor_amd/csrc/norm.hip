// K10: residual addition + root-mean-square norm, with a 16-bit output or
// 8-bit codes with scales, and the gradients.
//
//   s = x + residual; rstd = 1 / sqrt(mean(s^2) + eps); y = s rstd weight
//   dx = rstd (g - s rstd^2 mean(g s)) + dsum, g = dout weight
//   dweight = sum over rows of dout s rstd
//
// Bound by HBM: a row is read once, kept in registers across the reduction
// (8 fp32 values per 16-byte chunk) and written once.
//
// Forward: a row is held by TPR threads with NCH chunks each, one row per
// team, as many teams as rows.  Rows of up to 1024 columns take one wavefront
// (no barrier, four rows per workgroup), wider ones a workgroup of 256 to 1024
// threads; rows of more than 32768 columns, which do not fit, are read again
// for every pass (norm_wide).  8192 x 7168 with residual: 79.5 us, 5.9 TB/s (a
// large copy reaches 5.2) with 512 threads per row, 80.4 with 256, 81 with
// 1024; 512 to 2048 workgroups that walk the rows: 85 to 87.
#include <algorithm>

#include "layer_device.hpp"
#include "layer_kernels.hpp"

namespace mc2 {
namespace {

enum : int { OUT_16 = 0, OUT_I8 = 1, OUT_F8 = 2 };

// Codes of eight values; 8 bytes.  `usable`: the scale is positive and finite.
// The division is the IEEE one, so that the codes are those of the formula;
// products with the inverse, divided again only near a rounding boundary, took
// 0.5 us of 16 off 1023 x 7168: the kernel waits for memory.
template <int OUT>
__device__ __forceinline__ u32x2 codes8(const float (&y)[8], float scale, bool usable) {
  constexpr float kTop = OUT == OUT_I8 ? 127.0f : 448.0f;
  u32x2 r = {0u, 0u};
  if (!usable) return r;
#pragma unroll
  for (int w = 0; w < 2; w++) {
    float q[4];
#pragma unroll
    for (int e = 0; e < 4; e++) q[e] = fminf(fmaxf(y[4 * w + e] / scale, -kTop), kTop);
    if constexpr (OUT == OUT_I8) {
#pragma unroll
      for (int e = 0; e < 4; e++) r[w] |= ((uint32_t)(int)__builtin_rintf(q[e]) & 0xFFu) << (8 * e);
    } else {
      int p = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
      r[w] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], p, true);
    }
  }
  return r;
}
// Scale of a group from its largest |y|, compared as an integer, so that a NaN
// or an infinity comes out as the maximum.
template <int OUT>
__device__ __forceinline__ float scale_of(uint32_t top_bits) {
  return __uint_as_float(top_bits) / (OUT == OUT_I8 ? 127.0f : 448.0f);
}
__device__ __forceinline__ bool scale_usable(float scale) { return scale > 0.0f && scale < __builtin_inff(); }

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* row, int64_t c, int64_t h, u32x2 v) {
  if (VEC || c + 8 <= h) {
    __builtin_memcpy(row + c, &v, 8);
  } else {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (c + e < h) row[c + e] = (uint8_t)(v[e / 4] >> (8 * (e & 3)));
  }
}

template <int DT, int TPR, int NCH, int OUT, bool VEC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormArgs a) {
  constexpr int WAVES = TPR / 64;
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[WAVES];
  __shared__ uint32_t redm[WAVES];
  const int t = RPB > 1 ? threadIdx.x % TPR : threadIdx.x;
  const int64_t row = (int64_t)blockIdx.x * RPB + (RPB > 1 ? threadIdx.x / TPR : 0);
  if (RPB > 1 && row >= a.rows) return;  // RPB > 1: no barrier below
  const int64_t h = a.h;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * h;
  const uint16_t* res = a.residual ? static_cast<const uint16_t*>(a.residual) + row * h : nullptr;
  const uint16_t* weight = static_cast<const uint16_t*>(a.weight);
  u32x4 vx[NCH], vr[NCH], vw[NCH];
#pragma unroll
  for (int i = 0; i < NCH; i++) {
    const int64_t c = 8 * (int64_t)(t + i * TPR);
    vx[i] = vr[i] = vw[i] = u32x4{0u, 0u, 0u, 0u};
    if (c < h) {
      vx[i] = load_chunk<VEC>(x, c, h);
      if (res) vr[i] = load_chunk<VEC>(res, c, h);
      vw[i] = load_chunk<VEC>(weight, c, h);
    }
  }
  float s[NCH][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NCH; i++) {
    float r[8];
    unpack8<DT>(vx[i], s[i]);
    unpack8<DT>(vr[i], r);
#pragma unroll
    for (int e = 0; e < 8; e++) {
      s[i][e] = s[i][e] + r[e];
      ss = __builtin_fmaf(s[i][e], s[i][e], ss);
    }
  }
  ss = block_sum<WAVES>(ss, red);
  const float rstd = 1.0f / sqrtf(ss / (float)h + a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd;
  if (a.sum) {
    uint16_t* sum = static_cast<uint16_t*>(a.sum) + row * h;
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const int64_t c = 8 * (int64_t)(t + i * TPR);
      if (c < h) store_chunk<VEC, true>(sum, c, h, pack8<DT>(s[i]));
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NCH; i++) {
    float w[8];
    unpack8<DT>(vw[i], w);
#pragma unroll
    for (int e = 0; e < 8; e++) {
      s[i][e] = s[i][e] * rstd * w[e];
      if constexpr (OUT != OUT_16) top = max(top, __float_as_uint(s[i][e]) & 0x7FFFFFFFu);
    }
  }
  if constexpr (OUT == OUT_16) {
    uint16_t* out = static_cast<uint16_t*>(a.out) + row * h;
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const int64_t c = 8 * (int64_t)(t + i * TPR);
      if (c < h) store_chunk<VEC, true>(out, c, h, pack8<DT>(s[i]));
    }
  } else {
    uint8_t* out = static_cast<uint8_t*>(a.out) + row * h;
    if (a.group == 0) {
      const float scale = scale_of<OUT>(block_max<WAVES>(top, redm));
      const bool usable = scale_usable(scale);
      if (t == 0) a.scale[row] = scale;
#pragma unroll
      for (int i = 0; i < NCH; i++) {
        const int64_t c = 8 * (int64_t)(t + i * TPR);
        if (c < h) store_codes<VEC>(out, c, h, codes8<OUT>(s[i], scale, usable));
      }
    } else {  // 128 columns: the chunks of 16 consecutive lanes (h is a multiple of 128)
#pragma unroll
      for (int i = 0; i < NCH; i++) {
        const int64_t c = 8 * (int64_t)(t + i * TPR);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) m = max(m, __float_as_uint(s[i][e]) & 0x7FFFFFFFu);
        const float scale = scale_of<OUT>(max16(m));
        if (c < h) {
          if (c % 128 == 0) a.scale[row * (h / 128) + c / 128] = scale;
          store_codes<VEC>(out, c, h, codes8<OUT>(s[i], scale, scale_usable(scale)));
        }
      }
    }
  }
}

// Rows wider than the registers of a workgroup: x and residual are read again
// for the maximum and for the output (from the caches, mostly); sum_out is
// written last, by the thread that read those elements, as it may be one of
// the inputs.
constexpr int kWide = 1024;
template <int DT, int OUT, bool VEC>
__global__ __launch_bounds__(kWide) void norm_wide(NormArgs a) {
  __shared__ float red[kWide / 64];
  __shared__ uint32_t redm[kWide / 64];
  const int64_t row = blockIdx.x, h = a.h;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * h;
  const uint16_t* res = a.residual ? static_cast<const uint16_t*>(a.residual) + row * h : nullptr;
  const uint16_t* weight = static_cast<const uint16_t*>(a.weight);
  auto sum_at = [&](int64_t c, float(&s)[8]) {
    unpack8<DT>(load_chunk<VEC>(x, c, h), s);
    if (res) {
      float r[8];
      unpack8<DT>(load_chunk<VEC>(res, c, h), r);
#pragma unroll
      for (int e = 0; e < 8; e++) s[e] = s[e] + r[e];
    }
  };
  float ss = 0.0f;
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < h; c += 8 * kWide) {
    float s[8];
    sum_at(c, s);
#pragma unroll
    for (int e = 0; e < 8; e++) ss = __builtin_fmaf(s[e], s[e], ss);
  }
  ss = block_sum<kWide / 64>(ss, red);
  const float rstd = 1.0f / sqrtf(ss / (float)h + a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  auto y_at = [&](int64_t c, const float(&s)[8], float(&y)[8]) {
    float w[8];
    unpack8<DT>(load_chunk<VEC>(weight, c, h), w);
#pragma unroll
    for (int e = 0; e < 8; e++) y[e] = s[e] * rstd * w[e];
  };
  float scale = 0.0f;
  if constexpr (OUT != OUT_16) {
    if (a.group == 0) {
      uint32_t top = 0;
      for (int64_t c = 8 * (int64_t)threadIdx.x; c < h; c += 8 * kWide) {
        float s[8], y[8];
        sum_at(c, s);
        y_at(c, s, y);
#pragma unroll
        for (int e = 0; e < 8; e++) top = max(top, __float_as_uint(y[e]) & 0x7FFFFFFFu);
      }
      scale = scale_of<OUT>(block_max<kWide / 64>(top, redm));
      if (threadIdx.x == 0) a.scale[row] = scale;
    }
  }
  // whole turns, so that a group's 16 lanes take part in its maximum together
  const int64_t turns = (h + 8 * kWide - 1) / (8 * kWide);
  for (int64_t i = 0; i < turns; i++) {
    const int64_t c = 8 * ((int64_t)threadIdx.x + i * kWide);
    const bool in = c < h;
    float s[8] = {0, 0, 0, 0, 0, 0, 0, 0}, y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (in) {
      sum_at(c, s);
      y_at(c, s, y);
    }
    if constexpr (OUT == OUT_16) {
      if (in) store_chunk<VEC, true>(static_cast<uint16_t*>(a.out) + row * h, c, h, pack8<DT>(y));
    } else {
      float sc = scale;
      if (a.group != 0) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) m = max(m, __float_as_uint(y[e]) & 0x7FFFFFFFu);
        sc = scale_of<OUT>(max16(m));
        if (in && c % 128 == 0) a.scale[row * (h / 128) + c / 128] = sc;
      }
      if (in) store_codes<VEC>(static_cast<uint8_t*>(a.out) + row * h, c, h, codes8<OUT>(y, sc, scale_usable(sc)));
    }
    if (in && a.sum) store_chunk<VEC, true>(static_cast<uint16_t*>(a.sum) + row * h, c, h, pack8<DT>(s));
  }
}

template <int DT, int OUT, bool VEC>
hipError_t norm_launch(const NormArgs& a, hipStream_t st) {
  const int64_t h = a.h;
  auto wave = [&](auto NCH_) {
    norm_kernel<DT, 64, decltype(NCH_)::value, OUT, VEC><<<(unsigned)((a.rows + 3) / 4), 256, 0, st>>>(a);
  };
  using std::integral_constant;
  if (h <= 512) wave(integral_constant<int, 1>());
  else if (h <= 1024) wave(integral_constant<int, 2>());
  else if (h <= 2048) norm_kernel<DT, 256, 1, OUT, VEC><<<(unsigned)a.rows, 256, 0, st>>>(a);
  else if (h <= 4096) norm_kernel<DT, 512, 1, OUT, VEC><<<(unsigned)a.rows, 512, 0, st>>>(a);
  else if (h <= 8192) norm_kernel<DT, 512, 2, OUT, VEC><<<(unsigned)a.rows, 512, 0, st>>>(a);
  else if (h <= 16384) norm_kernel<DT, 1024, 2, OUT, VEC><<<(unsigned)a.rows, 1024, 0, st>>>(a);
  else if (h <= 32768) norm_kernel<DT, 1024, 4, OUT, VEC><<<(unsigned)a.rows, 1024, 0, st>>>(a);
  else norm_wide<DT, OUT, VEC><<<(unsigned)a.rows, kWide, 0, st>>>(a);
  return hipGetLastError();
}

template <int DT>
hipError_t norm_dt(const NormArgs& a, hipStream_t st) {
  const bool vec = a.h % 8 == 0;
  if (a.out_dtype == DT_I8) return vec ? norm_launch<DT, OUT_I8, true>(a, st) : norm_launch<DT, OUT_I8, false>(a, st);
  if (a.out_dtype == DT_E4M3FN)
    return vec ? norm_launch<DT, OUT_F8, true>(a, st) : norm_launch<DT, OUT_F8, false>(a, st);
  return vec ? norm_launch<DT, OUT_16, true>(a, st) : norm_launch<DT, OUT_16, false>(a, st);
}

// ---------------------------------------------------------------- gradients
// A workgroup walks rows blockIdx.x, + gridDim.x, ...; thread t keeps the same
// columns for every row, so dweight's sums stay in its registers until the
// walk ends and go out as one row of fp32 partial sums per workgroup.
// 8192 x 4096 with dsum: 52 us in all, 5.1 TB/s; 4096 x 8192 47.  Rows of more than
// 8192 columns take 1024 threads of 128 registers, which do not hold the row, its
// successor and the sums: 14 to 53 of them live in scratch with two chunks per
// thread (4096 x 16384 167 us, 3.2 TB/s) and 198 to 744 with four (2048 x 32768 509
// us, 1.1 TB/s).
template <int DT, int TPR, int NCH, bool VEC>
__global__ __launch_bounds__(TPR) void norm_grad_kernel(NormGradArgs a) {
  constexpr int WAVES = TPR / 64;
  __shared__ float red[2][WAVES];
  const int t = threadIdx.x;
  const int64_t h = a.h;
  u32x4 vw[NCH];
  float dw[NCH][8];
#pragma unroll
  for (int i = 0; i < NCH; i++) {
    const int64_t c = 8 * (int64_t)(t + i * TPR);
    vw[i] = c < h ? load_chunk<VEC>(static_cast<const uint16_t*>(a.weight), c, h) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; e++) dw[i][e] = 0.0f;
  }
  // the loads of the next row are in flight while this one is reduced
  u32x4 vd[NCH], vs[NCH], vr[NCH], nd[NCH], ns[NCH], nr[NCH];
  float rstd, next_rstd;
  auto load_row = [&](int64_t row) {
    const uint16_t* dout = static_cast<const uint16_t*>(a.dout) + row * h;
    const uint16_t* sp = static_cast<const uint16_t*>(a.s) + row * h;
    const uint16_t* dsum = a.dsum ? static_cast<const uint16_t*>(a.dsum) + row * h : nullptr;
    next_rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const int64_t c = 8 * (int64_t)(t + i * TPR);
      nd[i] = ns[i] = nr[i] = u32x4{0u, 0u, 0u, 0u};
      if (c < h) {
        nd[i] = load_chunk<VEC>(dout, c, h);
        ns[i] = load_chunk<VEC>(sp, c, h);
        if (dsum) nr[i] = load_chunk<VEC>(dsum, c, h);
      }
    }
  };
  load_row(blockIdx.x);  // (no more workgroups than rows)
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      vd[i] = nd[i];
      vs[i] = ns[i];
      vr[i] = nr[i];
    }
    rstd = next_rstd;
    if (row + gridDim.x < a.rows) load_row(row + gridDim.x);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      float d[8], s[8], w[8];
      unpack8<DT>(vd[i], d);
      unpack8<DT>(vs[i], s);
      unpack8<DT>(vw[i], w);
#pragma unroll
      for (int e = 0; e < 8; e++) {
        dot = __builtin_fmaf(d[e] * w[e], s[e], dot);
        dw[i][e] = __builtin_fmaf(d[e], s[e] * rstd, dw[i][e]);
      }
    }
    dot = block_sum<WAVES>(dot, red[turn]);
    const float k = rstd * rstd * (dot / (float)h);
    uint16_t* dx = static_cast<uint16_t*>(a.dx) + row * h;
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const int64_t c = 8 * (int64_t)(t + i * TPR);
      float d[8], s[8], w[8], r[8];
      unpack8<DT>(vd[i], d);
      unpack8<DT>(vs[i], s);
      unpack8<DT>(vw[i], w);
      unpack8<DT>(vr[i], r);
#pragma unroll
      for (int e = 0; e < 8; e++) d[e] = __builtin_fmaf(rstd, d[e] * w[e] - s[e] * k, r[e]);
      if (c < h) store_chunk<VEC, true>(dx, c, h, pack8<DT>(d));
    }
  }
  float* part = a.partials + (int64_t)blockIdx.x * h;
#pragma unroll
  for (int i = 0; i < NCH; i++) {
    const int64_t c = 8 * (int64_t)(t + i * TPR);
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (c + e < h) part[c + e] = dw[i][e];
  }
}

// Rows wider than 32768 columns: the two passes read the row twice, and each
// workgroup keeps its partial sums in memory.
template <int DT, bool VEC>
__global__ __launch_bounds__(kWide) void norm_grad_wide(NormGradArgs a) {
  __shared__ float red[2][kWide / 64];
  const int64_t h = a.h;
  const uint16_t* weight = static_cast<const uint16_t*>(a.weight);
  float* part = a.partials + (int64_t)blockIdx.x * h;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const uint16_t* dout = static_cast<const uint16_t*>(a.dout) + row * h;
    const uint16_t* sp = static_cast<const uint16_t*>(a.s) + row * h;
    const uint16_t* dsum = a.dsum ? static_cast<const uint16_t*>(a.dsum) + row * h : nullptr;
    uint16_t* dx = static_cast<uint16_t*>(a.dx) + row * h;
    const float rstd = a.rstd[row];
    float dot = 0.0f;
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < h; c += 8 * kWide) {
      float d[8], s[8], w[8];
      unpack8<DT>(load_chunk<VEC>(dout, c, h), d);
      unpack8<DT>(load_chunk<VEC>(sp, c, h), s);
      unpack8<DT>(load_chunk<VEC>(weight, c, h), w);
#pragma unroll
      for (int e = 0; e < 8; e++) dot = __builtin_fmaf(d[e] * w[e], s[e], dot);
    }
    dot = block_sum<kWide / 64>(dot, red[turn]);
    const float k = rstd * rstd * (dot / (float)h);
    const bool first = row == blockIdx.x;
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < h; c += 8 * kWide) {
      float d[8], s[8], w[8], r[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      unpack8<DT>(load_chunk<VEC>(dout, c, h), d);
      unpack8<DT>(load_chunk<VEC>(sp, c, h), s);
      unpack8<DT>(load_chunk<VEC>(weight, c, h), w);
      if (dsum) unpack8<DT>(load_chunk<VEC>(dsum, c, h), r);
#pragma unroll
      for (int e = 0; e < 8; e++) {
        if (c + e < h) part[c + e] = __builtin_fmaf(d[e], s[e] * rstd, first ? 0.0f : part[c + e]);
        d[e] = __builtin_fmaf(rstd, d[e] * w[e] - s[e] * k, r[e]);
      }
      store_chunk<VEC, true>(dx, c, h, pack8<DT>(d));
    }
  }
}

// dweight[j] = sum of `blocks` partial sums: 64 columns per workgroup, the
// partial rows shared out over its 16 wavefronts and joined in order.
constexpr int kReduceWaves = 16;
template <int DT>
__global__ __launch_bounds__(64 * kReduceWaves) void norm_grad_reduce(const float* part, int64_t blocks, int64_t h,
                                                                      uint16_t* dweight) {
  __shared__ float red[kReduceWaves][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t j = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (j < h) {
#pragma unroll 8
    for (int64_t b = wave; b < blocks; b += kReduceWaves) s += part[b * h + j];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && j < h) {
    float r = red[0][lane];
#pragma unroll
    for (int w = 1; w < kReduceWaves; w++) r += red[w][lane];
    dweight[j] = enc16<DT>(r);
  }
}

template <int DT, bool VEC>
hipError_t norm_grad_launch(const NormGradArgs& a, hipStream_t st) {
  const int64_t h = a.h, blocks = norm_grad_blocks(a.rows, h);
  if (blocks > 0) {
    const unsigned g = (unsigned)blocks;
    if (h <= 512) norm_grad_kernel<DT, 64, 1, VEC><<<g, 64, 0, st>>>(a);
    else if (h <= 2048) norm_grad_kernel<DT, 256, 1, VEC><<<g, 256, 0, st>>>(a);
    else if (h <= 4096) norm_grad_kernel<DT, 256, 2, VEC><<<g, 256, 0, st>>>(a);
    else if (h <= 8192) norm_grad_kernel<DT, 256, 4, VEC><<<g, 256, 0, st>>>(a);
    else if (h <= 16384) norm_grad_kernel<DT, 1024, 2, VEC><<<g, 1024, 0, st>>>(a);
    else if (h <= 32768) norm_grad_kernel<DT, 1024, 4, VEC><<<g, 1024, 0, st>>>(a);
    else norm_grad_wide<DT, VEC><<<g, kWide, 0, st>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  norm_grad_reduce<DT><<<(unsigned)((h + 63) / 64), 64 * kReduceWaves, 0, st>>>(
      a.partials, blocks, h, static_cast<uint16_t*>(a.dweight));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs& a, hipStream_t s) {
  if (a.rows < 1 || a.h < 1 || (a.dtype != DT_BF16 && a.dtype != DT_F16)) return hipErrorInvalidValue;
  // (a launch's threads are counted in 32 bits: slabs of rows)
  constexpr int64_t kSlab = 1 << 20;
  for (int64_t r0 = 0; r0 < a.rows; r0 += kSlab) {
    NormArgs b = a;
    const int64_t in = r0 * a.h * 2, out_size = a.out_dtype == a.dtype ? 2 : 1;
    b.rows = std::min(kSlab, a.rows - r0);
    b.x = static_cast<const char*>(a.x) + in;
    if (a.residual) b.residual = static_cast<const char*>(a.residual) + in;
    b.out = static_cast<char*>(a.out) + r0 * a.h * out_size;
    if (a.scale) b.scale = a.scale + r0 * (a.group ? a.h / a.group : 1);
    if (a.sum) b.sum = static_cast<char*>(a.sum) + in;
    if (a.rstd) b.rstd = a.rstd + r0;
    const hipError_t e = a.dtype == DT_BF16 ? norm_dt<DT_BF16>(b, s) : norm_dt<DT_F16>(b, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// One workgroup per CU for rows of 4096 columns or more, more for shorter ones
// (as many bytes in flight).  More read and write more rows at a time and
// leave more partial sums: at h = 4096, 256 / 512 / 768 / 1024 workgroups take
// 52 / 55 / 59 / 62 us for 8192 rows.
int64_t norm_grad_blocks(int64_t rows, int64_t h) {
  return std::min<int64_t>(rows, 256 * std::max<int64_t>(1, std::min<int64_t>(8, 4096 / h)));
}

hipError_t launch_add_rms_norm_grad(const NormGradArgs& a, hipStream_t s) {
  if (a.rows < 0 || a.h < 1 || (a.dtype != DT_BF16 && a.dtype != DT_F16)) return hipErrorInvalidValue;
  const bool vec = a.h % 8 == 0;
  if (a.dtype == DT_BF16) return vec ? norm_grad_launch<DT_BF16, true>(a, s) : norm_grad_launch<DT_BF16, false>(a, s);
  return vec ? norm_grad_launch<DT_F16, true>(a, s) : norm_grad_launch<DT_F16, false>(a, s);
}

}  // namespace mc2
