// The tiled product's launches for one 16-bit type, and the pass that joins a
// split K.
#pragma once
#include "linear_kernels.hpp"

namespace mc2 {
namespace lin {
namespace {

// out = residual + act(sum of the parts + bias), z likewise; four columns per thread.
template <int DT>
__global__ __launch_bounds__(256) void join_kernel(Product p, int64_t ld, int64_t part) {
  const int64_t quads = (p.n + 3) / 4;
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (q >= quads * p.m) return;
  const int64_t row = q / quads, col = q % quads * 4;
  const float* src = p.partial + row * ld + col;
  f32x4 v = *reinterpret_cast<const f32x4*>(src);
#pragma unroll 4
  for (int s = 1; s < p.splits; s++) v += *reinterpret_cast<const f32x4*>(src + s * part);
  const int n = p.n - col < 4 ? (int)(p.n - col) : 4;
  const uint16_t* bias = static_cast<const uint16_t*>(p.bias);
  const uint16_t* residual = static_cast<const uint16_t*>(p.residual);
  uint16_t* z = static_cast<uint16_t*>(p.z);
  uint16_t* out = static_cast<uint16_t*>(p.out);
  const int64_t at = row * p.n + col;
  if (bias)
    for (int r = 0; r < 4; r++)
      if (r < n) v[r] += dec16<DT>(bias[col + r]);
  auto store = [&](uint16_t* dst, f32x4 f) {
    if (p.n % 4 == 0) {
      *reinterpret_cast<u32x2*>(dst + at) = u32x2{pack2_16<DT>(f[0], f[1]), pack2_16<DT>(f[2], f[3])};
    } else {
      for (int r = 0; r < 4; r++)
        if (r < n) dst[at + r] = enc16<DT>(f[r]);
    }
  };
  if (z) store(z, v);
  with_act(p.act, [&](auto ACT_) {
    for (int r = 0; r < 4; r++) v[r] = act_of<decltype(ACT_)::value>(v[r]);
  });
  if (residual)
    for (int r = 0; r < 4; r++)
      if (r < n) v[r] += dec16<DT>(residual[at + r]);
  store(out, v);
}

template <int DT, int BM, int BN, int WGM, int WGN, int NS, bool AK, bool BK, int GMODE>
hipError_t launch_tile(Product p, const Plan& plan, hipStream_t s) {
  const int64_t tiles_m = (p.m + BM - 1) / BM + (GMODE == BY_ROWS ? p.groups : 0), tiles_n = (p.n + BN - 1) / BN;
  p.splits = plan.splits;
  p.k_part = plan.k_part;
  p.order_cols = GMODE != BY_ROWS && gemm::prefer_column_order(p.m, p.n, p.k, 2) ? 1 : 0;
  p.tile_group = gemm::choose_tile_group(tiles_m * BM, p.n, BM, BN, p.order_cols);
  const dim3 grid((unsigned)(tiles_m * tiles_n), (unsigned)(GMODE == BY_K ? p.groups : plan.splits));
  product_kernel<DT, BM, BN, WGM, WGN, NS, AK, BK, GMODE><<<grid, 64 * WGM * WGN, 0, s>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.splits < 2) return e;
  const int64_t ld = tiles_n * BN;
  const int64_t quads = (p.n + 3) / 4 * p.m;
  join_kernel<DT><<<(unsigned)((quads + 255) / 256), 256, 0, s>>>(p, ld, tiles_m * BM * ld);
  return hipGetLastError();
}

template <int DT, bool AK, bool BK, int GMODE>
hipError_t launch_layout(const Product& p, const Plan& plan, hipStream_t s) {
  if constexpr (AK) {
    if (plan.tile == TILE_96X128) return launch_tile<DT, 96, 128, 2, 2, 4, AK, BK, GMODE>(p, plan, s);
    if (plan.tile == TILE_96X64) return launch_tile<DT, 96, 64, 2, 2, 4, AK, BK, GMODE>(p, plan, s);
  }
  if constexpr (GMODE == DENSE)
    if (plan.tile == TILE_128X64) return launch_tile<DT, 128, 64, 2, 2, 4, AK, BK, GMODE>(p, plan, s);
  if constexpr (GMODE != BY_K)
    if (plan.tile == TILE_64X64) return launch_tile<DT, 64, 64, 2, 2, 4, AK, BK, GMODE>(p, plan, s);
  switch (plan.tile) {
    case TILE_256X256: return launch_tile<DT, 256, 256, 2, 4, 2, AK, BK, GMODE>(p, plan, s);
    case TILE_128X256: return launch_tile<DT, 128, 256, 2, 4, 3, AK, BK, GMODE>(p, plan, s);
    default: return launch_tile<DT, 128, 128, 2, 2, 4, AK, BK, GMODE>(p, plan, s);
  }
}

}  // namespace

template <int DT>
hipError_t launch_product(const Product& p, int layout, int gmode, const Plan& plan, hipStream_t s) {
  if (layout == 0)
    return gmode == BY_ROWS ? launch_layout<DT, true, true, BY_ROWS>(p, plan, s)
                            : launch_layout<DT, true, true, DENSE>(p, plan, s);
  if (layout == 1)
    return gmode == BY_ROWS ? launch_layout<DT, true, false, BY_ROWS>(p, plan, s)
                            : launch_layout<DT, true, false, DENSE>(p, plan, s);
  return gmode == BY_K ? launch_layout<DT, false, false, BY_K>(p, plan, s)
                       : launch_layout<DT, false, false, DENSE>(p, plan, s);
}

}  // namespace lin
}  // namespace mc2
