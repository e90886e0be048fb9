// Device helpers of the feed-forward operators: 8-element chunks of 16-bit
// rows and reductions over a wavefront or a workgroup.
#pragma once
#include "device.hpp"

namespace mc2 {

template <int DT>
__device__ __forceinline__ float dec16(uint32_t bits) {
  if constexpr (DT == DT_BF16) return bf16_bits_to_f32(bits & 0xFFFFu);
  else return f16_bits_to_f32(bits & 0xFFFFu);
}
template <int DT>
__device__ __forceinline__ uint16_t enc16(float f) {
  return DT == DT_BF16 ? f32_to_bf16_bits(f) : f32_to_f16_bits(f);
}

template <int DT>
__device__ __forceinline__ void unpack8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e++) f[e] = dec16<DT>(v[e / 2] >> (16 * (e & 1)));
}
template <int DT>
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  u32x4 v;
#pragma unroll
  for (int w = 0; w < 4; w++) v[w] = pack2_16<DT>(f[2 * w], f[2 * w + 1]);
  return v;
}

// Eight 16-bit elements of a row of h from column c (a multiple of 8), zeros
// past its end.  VEC: h is a multiple of 8, so the chunk is whole and its
// address 16-byte aligned; otherwise a whole chunk is one load of 2-byte
// alignment, and a row's last, partial one is the load of its last 8 elements
// shifted into place (element by element, 8 times a load's latency, only in
// rows shorter than that).
template <bool VEC>
__device__ __forceinline__ u32x4 load_chunk(const uint16_t* row, int64_t c, int64_t h) {
  if constexpr (VEC) {
    return *reinterpret_cast<const u32x4*>(row + c);
  } else {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (c + 8 <= h) {
      __builtin_memcpy(&v, row + c, 16);
    } else if (h >= 8) {
      if (c < h) {
        unsigned __int128 t;
        __builtin_memcpy(&t, row + h - 8, 16);
        v = __builtin_bit_cast(u32x4, t >> (16 * (int)(c + 8 - h)));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (c + e < h) v[e / 2] |= (uint32_t)row[c + e] << (16 * (e & 1));
    }
    return v;
  }
}
// The same for a store; NT: the streaming policy of store_out16.
template <bool VEC, bool NT>
__device__ __forceinline__ void store_chunk(uint16_t* row, int64_t c, int64_t h, u32x4 v) {
  if constexpr (VEC) {
    if constexpr (NT) store_out16(row + c, v);
    else *reinterpret_cast<u32x4*>(row + c) = v;
  } else {
    if (c + 8 <= h) {
      __builtin_memcpy(row + c, &v, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (c + e < h) row[c + e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
    }
  }
}

// Lane permutations within rows of 16 lanes: applied in turn to a reduction,
// each pairs lanes that hold different parts (1, 2, 4, then 8 lanes apart).
template <int STEP>
__device__ __forceinline__ uint32_t dpp16(uint32_t v) {
  constexpr int ctrl[4] = {0xB1, 0x4E, 0x141, 0x140};  // quad_perm 1032, quad_perm 2301, half mirror, mirror
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl[STEP], 0xF, 0xF, true);
}

// Maximum over each row of 16 lanes, in all of its lanes.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, dpp16<0>(v));
  v = max(v, dpp16<1>(v));
  v = max(v, dpp16<2>(v));
  return max(v, dpp16<3>(v));
}
// Sum / maximum over the wavefront, the same bits in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v += __uint_as_float(dpp16<0>(__float_as_uint(v)));
  v += __uint_as_float(dpp16<1>(__float_as_uint(v)));
  v += __uint_as_float(dpp16<2>(__float_as_uint(v)));
  v += __uint_as_float(dpp16<3>(__float_as_uint(v)));
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max16(v);
  v = max(v, (uint32_t)__shfl_xor((int)v, 16));
  return max(v, (uint32_t)__shfl_xor((int)v, 32));
}

// Inclusive scans over the wavefront's lanes (sums; maxima of values >= 0):
// within rows of 16 lanes, then from each row into the next, then from the
// lower 32 lanes into the upper.  Lanes a step does not reach combine with 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or_0(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan_add(int v) {
  v += dpp_or_0<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
  v += dpp_or_0<0x112, 0xF>(v);
  v += dpp_or_0<0x114, 0xF>(v);
  v += dpp_or_0<0x118, 0xF>(v);
  v += dpp_or_0<0x142, 0xA>(v);  // row_bcast 15
  return v + dpp_or_0<0x143, 0xC>(v);  // row_bcast 31
}
__device__ __forceinline__ int wave_scan_max(int v) {
  v = max(v, dpp_or_0<0x111, 0xF>(v));
  v = max(v, dpp_or_0<0x112, 0xF>(v));
  v = max(v, dpp_or_0<0x114, 0xF>(v));
  v = max(v, dpp_or_0<0x118, 0xF>(v));
  v = max(v, dpp_or_0<0x142, 0xA>(v));
  return max(v, dpp_or_0<0x143, 0xC>(v));
}

// Sum / maximum over the WAVES wavefronts of a workgroup in wavefront order.
// `red` (WAVES slots) must not be in use by an earlier call: callers that
// reduce repeatedly alternate between arrays, so that one barrier between
// two uses of the same array is enough.
template <int WAVES>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (WAVES == 1) return v;
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int w = 1; w < WAVES; w++) s += red[w];
  return s;
}
template <int WAVES>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = wave_max(v);
  if constexpr (WAVES == 1) return v;
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
  __syncthreads();
  uint32_t m = red[0];
#pragma unroll
  for (int w = 1; w < WAVES; w++) m = max(m, red[w]);
  return m;
}

}  // namespace mc2
