// K15: the linear of int8 codes, around the tiled product (linear_gemm.hpp
// with I8): the plan of a call, the product of few rows, and the copies that
// give rows of a ragged width an aligned one.
#include <algorithm>

#include "layer8_kernels.hpp"
#include "linear_kernels.hpp"

namespace mc2 {
namespace lin {
namespace {

int64_t pad16(int64_t v) { return (v + 15) / 16 * 16; }
// Bytes between padded rows: whole cache lines, so that a step's 128 bytes of a
// row are one of them (4096 x 4001 -> 5000: 128 us, 141 with rows of 4016).
int64_t pad128(int64_t v) { return (v + 127) / 128 * 128; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Sixteen codes of a row of k >= 16 from c (a multiple of 16), the last sixteen
// where they would pass its end, so that no load waits for a condition; trim16
// then puts them in place, with zeros past the end.  VEC: k is a multiple of 16.
template <bool VEC>
__device__ __forceinline__ u32x4 load16(const int8_t* row, int64_t c, int64_t k) {
  const int8_t* p = row + (c + 16 <= k ? c : k - 16);
  if (VEC) return *reinterpret_cast<const u32x4*>(p);
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ u32x4 trim16(u32x4 v, int64_t c, int64_t k) {
  if (c >= k) return u32x4{0u, 0u, 0u, 0u};
  if (c + 16 <= k) return v;
  return __builtin_bit_cast(u32x4, __builtin_bit_cast(unsigned __int128, v) >> (8 * (int)(c + 16 - k)));
}

// ---------------------------------------------------------------- ragged rows
// dst (rows, ld) = src (rows, k) with zeros in columns k .. ld - 1, for x and
// w in one launch; tpr threads per row.
struct PadArgs {
  const int8_t* src[2];
  int8_t* dst[2];
  int64_t rows[2];
  int64_t k, ld;
  int tpr;
};
__global__ __launch_bounds__(256) void pad_codes(PadArgs a) {
  const int per = 256 / a.tpr;
  for (int64_t i = (int64_t)blockIdx.x * per + threadIdx.x / a.tpr; i < a.rows[0] + a.rows[1];
       i += (int64_t)gridDim.x * per) {
    const int which = i >= a.rows[0];
    const int64_t row = which ? i - a.rows[0] : i;
    const int8_t* src = a.src[which] + row * a.k;
    int8_t* dst = a.dst[which] + row * a.ld;
#pragma unroll 4
    for (int64_t c = 16 * (int64_t)(threadIdx.x % a.tpr); c < a.ld; c += 16 * a.tpr) {
      u32x4 v = {0u, 0u, 0u, 0u};
      if (a.k >= 16) {
        v = trim16(load16<false>(src, c, a.k), c, a.k);
      } else {
#pragma unroll
        for (int e = 0; e < 16; e++)
          if (c + e < a.k) v[e / 4] |= (uint32_t)(uint8_t)src[c + e] << (8 * (e & 3));
      }
      *reinterpret_cast<u32x4*>(dst + c) = v;
    }
  }
}

// ---------------------------------------------------------------- few rows
// m <= 16 MF rows (a decoding step): bound by reading w once.  A workgroup
// makes 16 columns of C; its WAVES wavefronts take K in turn, 64 U codes at a
// time, and their int32 sums are added.  An MFMA takes 16 rows of w (its first
// operand) and 16 rows of x (rows past m repeat the last one and are not
// stored); fragments come straight from memory, U of each in flight.
constexpr int kSkinnyU = 4;
template <int DT, int MF, int WAVES, bool VEC>
__global__ __launch_bounds__(64 * WAVES) void skinny_i8_kernel(Product p, int64_t k) {
  __shared__ int red[WAVES][MF * 256];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t wr = n0 + lane % 16 < p.n ? n0 + lane % 16 : p.n - 1;
  const int8_t* w = static_cast<const int8_t*>(p.b) + wr * k;
  const int8_t* x[MF];
  i32x4 acc[MF];
#pragma unroll
  for (int i = 0; i < MF; i++) {
    const int64_t r = 16 * i + lane % 16 < p.m ? 16 * i + lane % 16 : p.m - 1;
    x[i] = static_cast<const int8_t*>(p.a) + r * k;
    acc[i] = i32x4{0, 0, 0, 0};
  }
  for (int64_t kb = (int64_t)wave * 64 * kSkinnyU; kb < k; kb += (int64_t)WAVES * 64 * kSkinnyU) {
    u32x4 fw[kSkinnyU], fx[MF][kSkinnyU];
#pragma unroll
    for (int u = 0; u < kSkinnyU; u++) {
      const int64_t c = kb + 64 * u + 16 * (lane / 16);
      fw[u] = load16<VEC>(w, c, k);
#pragma unroll
      for (int i = 0; i < MF; i++) fx[i][u] = load16<VEC>(x[i], c, k);
    }
    if (kb + 64 * kSkinnyU > k) {
#pragma unroll
      for (int u = 0; u < kSkinnyU; u++) {
        const int64_t c = kb + 64 * u + 16 * (lane / 16);
        fw[u] = trim16(fw[u], c, k);
#pragma unroll
        for (int i = 0; i < MF; i++) fx[i][u] = trim16(fx[i][u], c, k);
      }
    }
#pragma unroll
    for (int u = 0; u < kSkinnyU; u++)
#pragma unroll
      for (int i = 0; i < MF; i++)
        acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, fw[u]),
                                                       __builtin_bit_cast(i32x4, fx[i][u]), acc[i], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < MF; i++)
    *reinterpret_cast<i32x4*>(&red[wave][256 * i + lane % 16 * 16 + 4 * (lane / 16)]) = acc[i];
  __syncthreads();
  for (int t = threadIdx.x; t < MF * 256; t += 64 * WAVES) {
    const int64_t row = t / 16, col = n0 + t % 16;
    if (row >= p.m || col >= p.n) continue;
    int c = red[0][t];
#pragma unroll
    for (int s = 1; s < WAVES; s++) c += red[s][t];
    float v = ((float)c * p.a_scale[row]) * p.b_scale[col];
    if (p.bias) v += dec16<DT>(static_cast<const uint16_t*>(p.bias)[col]);
    const int64_t at = row * p.n + col;
    with_act(p.act, [&](auto ACT_) { v = act_of<decltype(ACT_)::value>(v); });
    if (p.residual) v += dec16<DT>(static_cast<const uint16_t*>(p.residual)[at]);
    static_cast<uint16_t*>(p.out)[at] = enc16<DT>(v);
  }
}

constexpr int64_t kSkinnyRows = 32;

// Wavefronts of a workgroup: 16 while no CU has a second workgroup, and for a
// very long K (one row, in us, 4 / 16: 4096 x 4096 7.6 / 6.7, 7168 x 4096 9.9 /
// 7.8 (k x n); 16384 x 8192 31.2 / 28.1, 16384 x 16384 59.8 / 54.9); else 4, whose
// workgroups start and join sooner (4096 x 28672 25.2 / 27.1, 512 x 20480 5.5 / 6.9,
// 8192 x 8192 14.0 / 14.9).
int skinny_waves(int64_t m, int64_t k, int64_t n) {
  const int64_t blocks = (n + 15) / 16;
  return blocks <= 256 || (k >= 16384 && m <= 16) ? 16 : 4;
}

// Whether up to 32 rows take this product or tiles, whose workgroups share the
// rows of x among 64 columns.  Here a CU reads the 16 rows of w and the m of x of
// each of its workgroups at 30 bytes a ns (16 rows, 16384 x 1024: 17.3 us, tiles
// 11.3; 32 rows 24.3, 12.1), tiles take their plan's time; neither less than
// HBM's (tiles at a lower rate: 16 rows of 4096 x 28672 32.5 us, here 36.0; 8
// rows 32.2, 31.2; 1 row 33.3, 28.1).  16 rows of 4096 x 4096 7.5, tiles 10.1; of 4096 x
// 7168 10.9, 10.3; 24 rows of 1792 x 7168 8.2, 7.6.
bool skinny(int64_t m, int64_t k, int64_t n, int64_t groups, const Plan& tiles) {
  if (groups || m > kSkinnyRows || k < 16) return false;  // (its loads are of 16 codes)
  if (m <= 8) return true;
  const double bytes = (double)n * (double)k, cus = std::max(1.0, (double)n / 16.0 / 256.0);
  const double here = std::max((double)(16 + m) * (double)k * cus / 30e3, bytes / 5e6);
  return here <= std::max(tiles.us, bytes / 4.2e6);
}

template <int DT, int MF>
hipError_t launch_skinny(const Product& p, int64_t k, hipStream_t s) {
  const unsigned blocks = (unsigned)((p.n + 15) / 16);
  const bool vec = k % 16 == 0;
  if (skinny_waves(p.m, k, p.n) == 4) {
    if (vec) skinny_i8_kernel<DT, MF, 4, true><<<blocks, 256, 0, s>>>(p, k);
    else skinny_i8_kernel<DT, MF, 4, false><<<blocks, 256, 0, s>>>(p, k);
  } else {
    if (vec) skinny_i8_kernel<DT, MF, 16, true><<<blocks, 1024, 0, s>>>(p, k);
    else skinny_i8_kernel<DT, MF, 16, false><<<blocks, 1024, 0, s>>>(p, k);
  }
  return hipGetLastError();
}

// Whether the tiles read rows copied to whole cache lines.  Rows of a multiple of
// 4 bytes can be loaded where they stand, in 16-byte chunks that lie across the
// lines: 64 rows for 32 experts of 4008 x 2040 55.7 us (149.5 with the copy), 517
// rows of 1000 x 2000 8.5 (11.7), 8191 of 1000 x 1000 20.8 (25.0).  A step's loads
// then touch twice the lines, and the codes past the last chunk are loaded by
// themselves, which together cost a product bound by its MFMAs about a third of
// their time, and may be more than the copy: 4095 rows of 4008 x 5000 117.6 (100.4
// with the copy), of 1000 x 5000 52.8 (50.1).  Rows of a multiple of 16 bytes that is
// none of 128 have the lines alone against them and are read where they stand at
// all sizes: 4096 x 4000 -> 5000 99 us (95 with the copy), 2048 x 8208 -> 4096 68
// (73), 4095 x 4000 -> 1000 25 (30), 8191 rows for 32 experts of 4000 -> 1792 138
// (201).  Of the largest the copy would be the faster: 8192 x 8176 -> 8192 519 (425).
bool pads(int64_t m, int64_t k, int64_t n, int64_t groups) {
  const double matrices = (double)std::max<int64_t>(groups, 1);
  const double mfma_us = 2.0 * (double)m * (double)n * (double)k / 2.1e9;
  const double copy_us = 3.0 + 2.0 * ((double)m + matrices * (double)n) * (double)k / 5.3e6;
  return k % 4 != 0 || (k % 16 != 0 && 0.35 * mfma_us > copy_us);
}

// Parts of the workspace, each 256-byte aligned.
struct LayoutI8 {
  size_t x, w, partial, total = 0;
  Plan plan{};
  bool few, padded;  // the product of few rows; tiles of rows copied to an aligned width
  LayoutI8(int64_t m, int64_t k, int64_t n, int64_t groups) {
    auto take = [&](size_t bytes) {
      const size_t at = total;
      total += up256(bytes);
      return at;
    };
    if (groups || m > 8 || k < 16) plan = plan_product(m, n, pad16(k) / 2, 0, groups ? BY_ROWS : DENSE, groups, true);
    few = skinny(m, k, n, groups, plan);
    if (few) plan = Plan{};
    padded = !few && pads(m, k, n, groups);
    x = take(padded ? (size_t)m * pad128(k) : 0);
    w = take(padded ? (size_t)std::max<int64_t>(groups, 1) * n * pad128(k) : 0);
    partial = take(plan.partial_bytes);
  }
};

template <int DT>
hipError_t linear_i8_dt(const LinearI8Args& a, hipStream_t s) {
  const LayoutI8 at(a.m, a.k, a.n, a.groups);
  char* ws = static_cast<char*>(a.workspace);
  Product p{};
  p.a = a.x;
  p.b = a.w;
  p.a_scale = a.x_scale;
  p.b_scale = a.w_scale;
  p.m = a.m;
  p.n = a.n;
  p.k = (at.padded ? pad16(a.k) : a.k / 16 * 16) / 2;
  p.tail = at.padded ? 0 : (int)(a.k % 16);
  p.offsets = a.offsets;
  p.groups = a.groups;
  p.bias = a.bias;
  p.residual = a.residual;
  p.out = a.out;
  p.act = a.act;
  p.splits = 1;
  if (at.few) return a.m <= 16 ? launch_skinny<DT, 1>(p, a.k, s) : launch_skinny<DT, 2>(p, a.k, s);
  p.lda = p.ldb = (at.padded ? pad128(a.k) : a.k) / 2;
  p.b_group = a.n * p.ldb;
  if (at.padded) {
    const int64_t matrices = std::max<int64_t>(a.groups, 1);
    PadArgs pad{{a.x, a.w},
                {reinterpret_cast<int8_t*>(ws + at.x), reinterpret_cast<int8_t*>(ws + at.w)},
                {a.m, matrices * a.n},
                a.k,
                pad128(a.k),
                1};
    while (pad.tpr < 256 && 16 * pad.tpr < a.k) pad.tpr *= 2;
    const int64_t per = 256 / pad.tpr, blocks = (a.m + matrices * a.n + per - 1) / per;
    pad_codes<<<(unsigned)std::min<int64_t>(blocks, 256 * 16), 256, 0, s>>>(pad);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.a = ws + at.x;
    p.b = ws + at.w;
  }
  p.partial = reinterpret_cast<float*>(ws + at.partial);
  return launch_product_i8<DT>(p, a.groups ? BY_ROWS : DENSE, at.plan, s);
}

}  // namespace
}  // namespace lin

void linear_i8_plan(int64_t m, int64_t k, int64_t n, int64_t groups, int* tile, int* splits) {
  const lin::LayoutI8 at(m, k, n, groups);
  *tile = at.few ? -lin::skinny_waves(m, k, n) : (int)at.plan.tile;
  *splits = at.few ? 1 : at.plan.splits;
}

size_t linear_i8_workspace(int64_t m, int64_t k, int64_t n, int64_t groups) {
  return m > 0 ? lin::LayoutI8(m, k, n, groups).total : 0;
}

hipError_t launch_linear_i8(const LinearI8Args& a, hipStream_t s) {
  if (a.m < 1 || a.k < 1 || a.n < 1 || a.groups < 0 || a.k > lin::kMaxDim || a.n > lin::kMaxDim)
    return hipErrorInvalidValue;
  return a.dtype == DT_BF16 ? lin::linear_i8_dt<DT_BF16>(a, s) : lin::linear_i8_dt<DT_F16>(a, s);
}

}  // namespace mc2
