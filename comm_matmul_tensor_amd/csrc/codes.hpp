// int8 codes of eight values at a time (mc2_quant_rows' definition), and rows of
// them back to 16 bits.
#pragma once
#include "layer8_kernels.hpp"
#include "linear_act.hpp"

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
// -128 under a negative scale is -inf (MC2_KEEP_INF): as fp32's lowest number, of
// which the activations and their slopes are what they tend to (of -inf itself
// a product is -inf * 0), and which rounds to -inf in 16 bits.
__device__ __forceinline__ void code_values(u32x2 v, float scale, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e++) f[e] = (float)(int8_t)(v[e / 4] >> (8 * (e & 3))) * scale;
  if (scale < 0.0f) {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if ((v[e / 4] >> (8 * (e & 3)) & 0xFFu) == 0x80u) f[e] = -3.402823466e38f;
  }
}
// Which scale of its row column c has (group 0: the only one; 128).
__device__ __forceinline__ int64_t scale_at(int64_t c, int64_t group) { return group ? c / 128 : 0; }
// Scales of a row.
__host__ __device__ __forceinline__ int64_t scales_of(int64_t cols, int64_t group) {
  return group ? (cols + 127) / 128 : 1;
}

// Threads of a row of `chunks` chunks: the most, up to 256, that leave no more
// than an eighth of them idle over the row's turns, `least` at least.
inline int row_threads(int64_t chunks, int least) {
  int best = least;
  for (int t = least; t <= 256; t *= 2)
    if ((chunks + t - 1) / t * t - chunks <= chunks / 8) best = t;
  return best;
}
// (A launch has fewer than 2^32 threads: at most 2^22 workgroups here, as the
// gradient's launch has others beside them.)
inline int dequant_threads(int64_t rows, int64_t cols) {
  const int64_t chunks = (cols + 7) / 8;
  int threads = row_threads(chunks, chunks < 8 ? 1 : 8);
  while (threads > 1 && rows > (int64_t)(256 / threads) << 22) threads /= 2;
  return threads;
}

constexpr int kFlight = 4;  // chunks that a thread loads before it uses one

// 256 / tpr rows of codes from row 256 / tpr * block on as act(code scale); out's
// rows are ld apart (a multiple of 8, where the columns past the last one become
// 0, or cols).  VEC: cols is a multiple of 8.
template <int DT, int ACT, bool VEC>
__device__ __forceinline__ void dequant_block(const CodeArgs& a, int tpr, int64_t block) {
  const int64_t row = block * (256 / tpr) + threadIdx.x / tpr;
  if (row >= a.rows) return;
  const int8_t* codes = a.codes_in + row * a.cols;
  const float* scales = a.scale_in + row * scales_of(a.cols, a.group);
  uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.ld;
  for (int64_t c0 = 8 * (int64_t)(threadIdx.x % tpr); c0 < a.ld; c0 += kFlight * 8 * tpr) {
    u32x2 v[kFlight];
    float scale[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; u++) {
      const int64_t c = c0 + u * 8 * tpr, in = c < a.cols ? c : VEC ? a.cols - 8 : 0;
      v[u] = load_codes<VEC>(codes, VEC ? in : c, a.cols);
      scale[u] = scales[scale_at(in, a.group)];
    }
#pragma unroll
    for (int u = 0; u < kFlight; u++) {
      const int64_t c = c0 + u * 8 * tpr;
      if (c >= a.ld) continue;
      float f[8];
      code_values(v[u], scale[u], f);
#pragma unroll
      for (int e = 0; e < 8; e++) f[e] = VEC || c + e < a.cols ? act_of<ACT>(f[e]) : 0.0f;
      store_chunk<VEC, true>(out, c, a.ld, pack8<DT>(f));
    }
  }
}

}  // namespace mc2
