// K14: rows to int8 codes with a scale per row or per 128 columns, and back.
//
//   a = max |x|, scale = a / 127, code = rint(x / scale); out = act(code scale)
//
// Bound by HBM: a row is read once, kept in registers across its maximum and
// its codes written once.
//
// Per 128 columns the 16 lanes that hold a group's chunks of 8 find its
// maximum by DPP; nothing else depends on the row, so threads take chunks of
// rows in any shape: `tpr` of them a row.  Per row a team of TPR threads holds
// it with NCH chunks each; rows that do not fit are read twice (quant_wide).
#include <algorithm>

#include "codes.hpp"

namespace mc2 {
namespace {

__device__ __forceinline__ float scale_of(uint32_t top_bits) { return __uint_as_float(top_bits) / 127.0f; }
__device__ __forceinline__ uint32_t top_of(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; e++) m = max(m, __float_as_uint(x[e]) & 0x7FFFFFFFu);  // (a NaN is the largest)
  return m;
}
// What a group's codes need of its scale.
struct Divisor {
  float scale, inverse;
  bool usable, fast;
  __device__ __forceinline__ explicit Divisor(float s) : scale(s), inverse(1.0f / s) {
    usable = s > 0.0f && s < __builtin_inff();  // a scale that is 0, NaN or infinite gives codes 0
    fast = usable && s > 0x1p-100f;             // the inverse neither overflows nor loses bits
  }
};
// The codes are those of the IEEE quotient, found without dividing: x times the
// inverse is off from it by 127 (2^-24 + 2^-24) at most, so both round to the
// same whole number unless that product lies within 2^-14 of a half; only then
// (one value in 8000) are the eight divided.  Added to 1.5 2^23, the product
// rounds to the whole number in the sum's last bits, its low byte the code.
__device__ __forceinline__ u32x2 codes_of(const float (&x)[8], const Divisor& d) {
  constexpr float kRound = 12582912.0f;
  u32x2 r = {0u, 0u};
  if (!d.usable) return r;
  float t[8], far = 1.0f;
  if (d.fast) {
    far = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      t[e] = __builtin_fmaf(x[e], d.inverse, kRound);
      far = fmaxf(far, __builtin_fabsf(__builtin_fmaf(x[e], d.inverse, -(t[e] - kRound))));
    }
  }
  if (far > 0.5f - 0x1p-14f) {
#pragma unroll
    for (int e = 0; e < 8; e++) t[e] = x[e] / d.scale + kRound;
  }
#pragma unroll
  for (int w = 0; w < 2; w++) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[4 * w + 1]), __float_as_uint(t[4 * w]), 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[4 * w + 3]), __float_as_uint(t[4 * w + 2]), 0x04000C0Cu);
    r[w] = lo | hi;
  }
  return r;
}
template <bool VEC>
__device__ __forceinline__ void store_codes(int8_t* row, int64_t c, int64_t cols, u32x2 v) {
  if (VEC || c + 8 <= cols) {
    __builtin_memcpy(row + c, &v, 8);
  } else {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (c + e < cols) row[c + e] = (int8_t)(v[e / 4] >> (8 * (e & 3)));
  }
}

// ---------------------------------------------------------------- per 128 columns
// INF: infinities do not count for the scale (MC2_KEEP_INF).  A group that has one
// or a NaN, as its largest bits say, takes its maximum again: an infinity is 1
// there, below every number but 0, as 16-bit numbers' last bits are 0 in
// fp32.  (Every group that way, 8191 x 7168: 53 us, 42 without INF.)
constexpr uint32_t kInf = 0x7F800000u;
__device__ __forceinline__ uint32_t finite_top_of(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const uint32_t b = __float_as_uint(x[e]) & 0x7FFFFFFFu;
    m = max(m, b == kInf ? 1u : b);
  }
  return m;
}
template <int DT>
__device__ __forceinline__ float largest() { return DT == DT_BF16 ? 0x1.FEp127f : 65504.0f; }
// The codes and the scale of such a group (its 16 lanes take part).
template <int DT>
__device__ __forceinline__ u32x2 codes_with_inf(float (&x)[8], float& scale) {
  const uint32_t top = max16(finite_top_of(x));
  const float a = top == 1u ? largest<DT>() : __uint_as_float(top);
  const Divisor d(a / 127.0f);
  uint32_t low = 0;
#pragma unroll
  for (int e = 0; e < 8; e++) low |= (uint32_t)(x[e] == -__builtin_inff()) << e;
  const bool has_low = max16(low ? 1u : 0u) != 0 && d.usable;
#pragma unroll
  for (int e = 0; e < 8; e++) {
    x[e] = __builtin_amdgcn_fmed3f(x[e], -a, a);  // (a NaN: no code is used)
    if (has_low) x[e] = -x[e];
  }
  scale = has_low ? -d.scale : d.scale;
  u32x2 r = codes_of(x, d);
  if (has_low && low) {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (low >> e & 1) r[e / 4] = (r[e / 4] & ~(0xFFu << (8 * (e & 3)))) | 0x80u << (8 * (e & 3));
  }
  return r;
}

template <int DT, bool VEC, bool INF>
__global__ __launch_bounds__(256) void quant_groups(CodeArgs a, int tpr) {
  const int64_t row = (int64_t)blockIdx.x * (256 / tpr) + threadIdx.x / tpr;
  if (row >= a.rows) return;  // (whole teams of 16 lanes: tpr is a multiple of 16)
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.cols;
  int8_t* codes = a.codes + row * a.cols;
  float* scales = a.scale + row * scales_of(a.cols, 128);
  const int64_t last = (a.cols + 127) / 128 * 128;  // a group's lanes all take part
  for (int64_t c0 = 8 * (int64_t)(threadIdx.x % tpr); c0 < last; c0 += kFlight * 8 * tpr) {
    u32x4 v[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; u++) {
      const int64_t c = c0 + u * 8 * tpr;
      // (whole rows of chunks: past the end the last one again, so that no load waits for a condition)
      v[u] = load_chunk<VEC>(x, VEC && c >= a.cols ? a.cols - 8 : c, a.cols);
    }
#pragma unroll
    for (int u = 0; u < kFlight; u++) {
      const int64_t c = c0 + u * 8 * tpr;
      float f[8];
      unpack8<DT>(v[u], f);
      const uint32_t top = max16(VEC && c >= a.cols ? 0u : top_of(f));
      if (INF && top >= kInf) {
        if (VEC && c >= a.cols) {
#pragma unroll
          for (int e = 0; e < 8; e++) f[e] = 0.0f;
        }
        float scale;
        const u32x2 r = codes_with_inf<DT>(f, scale);
        if (c >= a.cols) continue;
        if (c % 128 == 0) scales[c / 128] = scale;
        store_codes<VEC>(codes, c, a.cols, r);
        continue;
      }
      const Divisor d(scale_of(top));
      if (c >= a.cols) continue;
      if (c % 128 == 0) scales[c / 128] = d.scale;
      store_codes<VEC>(codes, c, a.cols, codes_of(f, d));
    }
  }
}

// ---------------------------------------------------------------- per row
template <int DT, int TPR, int NCH, bool VEC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void quant_row(CodeArgs a) {
  constexpr int WAVES = TPR / 64;
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  __shared__ uint32_t red[WAVES];
  const int t = RPB > 1 ? threadIdx.x % TPR : threadIdx.x;
  const int64_t row = (int64_t)blockIdx.x * RPB + (RPB > 1 ? threadIdx.x / TPR : 0);
  if (RPB > 1 && row >= a.rows) return;  // RPB > 1: no barrier below
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.cols;
  u32x4 v[NCH];
#pragma unroll
  for (int i = 0; i < NCH; i++) {
    const int64_t c = 8 * (int64_t)(t + i * TPR);
    v[i] = u32x4{0u, 0u, 0u, 0u};
    if (c < a.cols) v[i] = load_chunk<VEC>(x, c, a.cols);
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NCH; i++) {
    float f[8];
    unpack8<DT>(v[i], f);
    top = max(top, top_of(f));
  }
  const Divisor d(scale_of(block_max<WAVES>(top, red)));
  if (t == 0) a.scale[row] = d.scale;
#pragma unroll
  for (int i = 0; i < NCH; i++) {
    const int64_t c = 8 * (int64_t)(t + i * TPR);
    float f[8];
    unpack8<DT>(v[i], f);
    if (c < a.cols) store_codes<VEC>(a.codes + row * a.cols, c, a.cols, codes_of(f, d));
  }
}

constexpr int kWide = 1024;
template <int DT, bool VEC>
__global__ __launch_bounds__(kWide) void quant_wide(CodeArgs a) {
  __shared__ uint32_t red[kWide / 64];
  const int64_t row = blockIdx.x;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.cols;
  uint32_t top = 0;
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < a.cols; c += 8 * kWide) {
    float f[8];
    unpack8<DT>(load_chunk<VEC>(x, c, a.cols), f);
    top = max(top, top_of(f));
  }
  const Divisor d(scale_of(block_max<kWide / 64>(top, red)));
  if (threadIdx.x == 0) a.scale[row] = d.scale;
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < a.cols; c += 8 * kWide) {
    float f[8];
    unpack8<DT>(load_chunk<VEC>(x, c, a.cols), f);
    store_codes<VEC>(a.codes + row * a.cols, c, a.cols, codes_of(f, d));
  }
}

constexpr int64_t kRows = 1 << 21;  // a launch's, so that it has fewer than 2^32 threads

template <int DT, bool VEC>
hipError_t quant_launch(const CodeArgs& given, hipStream_t s) {
  CodeArgs a = given;
  for (; a.rows > kRows; a.rows -= kRows) {
    CodeArgs first = a;
    first.rows = kRows;
    if (const hipError_t e = quant_launch<DT, VEC>(first, s); e != hipSuccess) return e;
    a.x = static_cast<const uint16_t*>(a.x) + kRows * a.cols;
    a.codes += kRows * a.cols;
    a.scale += kRows * scales_of(a.cols, a.group);
  }
  if (a.group) {
    const int tpr = row_threads((a.cols + 127) / 128 * 16, 16), per = 256 / tpr;
    const unsigned blocks = (unsigned)((a.rows + per - 1) / per);
    if (a.keep_inf) quant_groups<DT, VEC, true><<<blocks, 256, 0, s>>>(a, tpr);
    else quant_groups<DT, VEC, false><<<blocks, 256, 0, s>>>(a, tpr);
    return hipGetLastError();
  }
  auto wave = [&](auto NCH_) {
    quant_row<DT, 64, decltype(NCH_)::value, VEC><<<(unsigned)((a.rows + 3) / 4), 256, 0, s>>>(a);
  };
  using std::integral_constant;
  const int64_t h = a.cols;
  if (h <= 512) wave(integral_constant<int, 1>());
  else if (h <= 1024) wave(integral_constant<int, 2>());
  else if (h <= 2048 && a.rows >= 1024) wave(integral_constant<int, 4>());  // 8191 x 1792, there and back: 19.6 us, a workgroup a row 23; 16 x 2048 5.8, 5.3
  else if (h <= 2048) quant_row<DT, 256, 1, VEC><<<(unsigned)a.rows, 256, 0, s>>>(a);
  else if (h <= 4096) quant_row<DT, 256, 2, VEC><<<(unsigned)a.rows, 256, 0, s>>>(a);  // 8192 x 4096, there and back: 512 threads 43 us, 34
  else if (h <= 8192) quant_row<DT, 512, 2, VEC><<<(unsigned)a.rows, 512, 0, s>>>(a);
  else if (h <= 16384) quant_row<DT, 1024, 2, VEC><<<(unsigned)a.rows, 1024, 0, s>>>(a);
  else if (h <= 32768) quant_row<DT, 1024, 4, VEC><<<(unsigned)a.rows, 1024, 0, s>>>(a);
  else quant_wide<DT, VEC><<<(unsigned)a.rows, kWide, 0, s>>>(a);
  return hipGetLastError();
}

// ---------------------------------------------------------------- and back
template <int DT, int ACT, bool VEC>
__global__ __launch_bounds__(256) void dequant_kernel(CodeArgs a, int tpr) {
  dequant_block<DT, ACT, VEC>(a, tpr, blockIdx.x);
}

template <int DT, int ACT>
hipError_t dequant_launch(const CodeArgs& a, hipStream_t s) {
  const int tpr = dequant_threads(a.rows, a.cols), per = 256 / tpr;
  const unsigned blocks = (unsigned)((a.rows + per - 1) / per);
  if (a.cols % 8 == 0) dequant_kernel<DT, ACT, true><<<blocks, 256, 0, s>>>(a, tpr);
  else dequant_kernel<DT, ACT, false><<<blocks, 256, 0, s>>>(a, tpr);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_rows(const CodeArgs& a, hipStream_t s) {
  if (a.rows < 1 || a.cols < 1 || (a.group != 0 && a.group != 128)) return hipErrorInvalidValue;
  const bool vec = a.cols % 8 == 0;
  if (a.dtype == DT_BF16) return vec ? quant_launch<DT_BF16, true>(a, s) : quant_launch<DT_BF16, false>(a, s);
  return vec ? quant_launch<DT_F16, true>(a, s) : quant_launch<DT_F16, false>(a, s);
}

hipError_t launch_dequant_rows(const CodeArgs& given, hipStream_t s) {
  CodeArgs a = given;
  if (a.ld == 0) a.ld = a.cols;
  if (a.rows < 1 || a.cols < 1 || a.ld < a.cols || (a.group != 0 && a.group != 128)) return hipErrorInvalidValue;
  hipError_t e = hipErrorInvalidValue;
  with_act(a.act, [&](auto ACT_) {
    constexpr int ACT = decltype(ACT_)::value;
    e = a.dtype == DT_BF16 ? dequant_launch<DT_BF16, ACT>(a, s) : dequant_launch<DT_F16, ACT>(a, s);
  });
  return e;
}

}  // namespace mc2
