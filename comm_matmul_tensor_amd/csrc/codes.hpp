// int8 codes of eight values at a time (mc2_quant_rows' definition).
#pragma once
#include "layer_device.hpp"

namespace mc2 {

// Eight codes of a row from column c (a multiple of 8), zeros past its end.
// VEC: rows are a multiple of 8 long, so the eight are one aligned load.
template <bool VEC>
__device__ __forceinline__ u32x2 load_codes(const int8_t* row, int64_t c, int64_t cols) {
  u32x2 v = {0u, 0u};
  if (VEC) {
    v = *reinterpret_cast<const u32x2*>(row + c);
  } else if (c + 8 <= cols) {
    __builtin_memcpy(&v, row + c, 8);
  } else if (cols >= 8) {  // the row's last eight, shifted into place
    if (c < cols) {
      uint64_t t;
      __builtin_memcpy(&t, row + cols - 8, 8);
      v = __builtin_bit_cast(u32x2, t >> (8 * (int)(c + 8 - cols)));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (c + e < cols) v[e / 4] |= (uint32_t)(uint8_t)row[c + e] << (8 * (e & 3));
  }
  return v;
}
__device__ __forceinline__ void code_values(u32x2 v, float scale, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e++) f[e] = (float)(int8_t)(v[e / 4] >> (8 * (e & 3))) * scale;
}
// Which scale of its row column c has (group 0: the only one; 128).
__device__ __forceinline__ int64_t scale_at(int64_t c, int64_t group) { return group ? c / 128 : 0; }
// Scales of a row.
__host__ __device__ __forceinline__ int64_t scales_of(int64_t cols, int64_t group) {
  return group ? (cols + 127) / 128 : 1;
}

}  // namespace mc2
