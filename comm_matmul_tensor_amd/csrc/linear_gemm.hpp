// K11: the tiled MFMA product of mc2_linear_act and its gradients (gfx950).
//
//   C (m, n) = A (m, k) @ B (k, n), 16-bit operands, fp32 accumulation, then
//   z = C + bias, out = residual + act(z), rounded once.
//
// Operands: A K-contiguous (AK: stored (m, k)) or M-contiguous ((k, m)); B
// K-contiguous (BK: (n, k)) or N-contiguous ((k, n)).  Their leading
// dimensions are multiples of 8 elements (the launcher copies others), so
// every 16-byte chunk of a row is aligned; m, n and k are arbitrary.
//
// Tile.  A workgroup of WGM x WGN wavefronts makes a BM x BN tile of C in
// 16 x 16 MFMA tiles, 64 of K at a time.  Both operands go from memory to LDS
// with direct-to-LDS buffer loads into two stages; the loads of a step are
// issued at the start of the step before it.
//
// Groups of rows (experts): the tile's rows come from one group's range of
// rows, found from the ranges on the device (find_tile), with that group's
// B, bias; for the weight's gradient the groups are ranges of K.  A tile that
// crosses the end of its rows, columns or K reads zeros or repeats its last
// row, and stores nothing outside.
#pragma once
#include <type_traits>

#include "gemm_mfma.hpp"
#include "layer_kernels.hpp"
#include "linear_act.hpp"

namespace mc2 {
namespace lin {

using gemm::FragReader;
using gemm::lptr_t;
using gemm::make_rsrc;
using gemm::mn_swz;
using gemm::lds_barrier;
using gemm::wait_vmcnt;

constexpr int kStepK = 64;      // K elements per main loop step
constexpr int kMaxDim = 1 << 21;  // n and k: 256 rows of an operand stay below 2 GiB

struct Product {
  const void *a, *b;
  int64_t lda, ldb;                 // elements between rows as stored, multiples of 8
  int64_t m, n, k;
  // groups (0: none).  BY_ROWS: ranges of C's rows, B and bias of group g at
  // g b_group, g n; BY_K: ranges of the contraction (rows of A and B as
  // stored), C of group g at g m n.
  const int32_t* offsets;
  int64_t groups, b_group;
  const void *bias, *residual;
  void *out, *z;
  int act;
  // split K: part s of `splits` covers k_part of K and stores its fp32 sums
  // to partial + s (row tiles BM)(column tiles BN); no epilogue
  int splits;
  int64_t k_part;
  float* partial;
  int tile_group, order_cols;       // order of the tiles (tile_at)
};

enum : int { DENSE = 0, BY_ROWS = 1, BY_K = 2 };

struct RowRange { int64_t group, begin, end, tile; };

// A value below 2^31 that every lane holds, as a scalar (buffer resources and
// loop bounds made from it need no loop over lanes).
__device__ __forceinline__ int64_t uniform(int64_t v) { return __builtin_amdgcn_readfirstlane((int)v); }

// Tile `tile` of the ranges cut into tiles of bm rows, counted group by group
// and then over the rows after the last group (group = groups).  Every
// wavefront finds it for itself, 64 groups at a time: range ends are read as
// ascending and at most m.  tile past them all: begin = end = m.
__device__ __forceinline__ RowRange find_tile(const int32_t* offsets, int64_t groups, int64_t m, int bm,
                                              int64_t tile) {
  const int lane = threadIdx.x % 64;
  int64_t begin = 0, left = tile;  // of the groups still to come
  for (int64_t g0 = 0; g0 < groups; g0 += 64) {
    int64_t end = g0 + lane < groups ? (int64_t)offsets[g0 + lane + 1] : 0;
    end = end < begin ? begin : end > m ? m : end;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int64_t v = __shfl_up(end, d);
      if (lane >= d && v > end) end = v;
    }
    int64_t start = __shfl_up(end, 1);
    if (lane == 0) start = begin;
    const int tiles = (int)((end - start + bm - 1) / bm);
    int64_t incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int64_t v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
    const unsigned long long hit = __ballot(left < incl);
    if (hit) {
      const int l = __ffsll((long long)hit) - 1;
      RowRange r;
      r.group = g0 + l;
      r.begin = uniform(__shfl(start, l));
      r.end = uniform(__shfl(end, l));
      r.tile = uniform(left - __shfl(incl - tiles, l));
      return r;
    }
    left -= __shfl(incl, 63);
    begin = __shfl(end, 63);
  }
  return RowRange{groups, uniform(begin), m, uniform(left)};
}

// Range of group g: the ends as find_tile reads them.
__device__ __forceinline__ void group_range(const int32_t* offsets, int64_t g, int64_t m, int64_t& begin,
                                            int64_t& end) {
  const int lane = threadIdx.x % 64;
  int64_t top = 0;
  for (int64_t i = lane; i < g; i += 64) {
    const int64_t v = offsets[i + 1];
    top = v > top ? v : top;
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t v = __shfl_xor(top, d);
    top = v > top ? v : top;
  }
  begin = uniform(top > m ? m : top);
  const int64_t e = offsets[g + 1];
  end = uniform(e < begin ? begin : e > m ? m : e);
}

// One operand's loads: R rows of MN and 64 of K per step by NT threads.
// Instruction i of wavefront w fills the 1 KB of LDS at 16 (NT i + 64 w) in
// lane order; each lane's address is chosen so that the layout is the
// swizzled one FragReader reads.
template <int R, bool KMAJ, int NT>
struct Loader {
  static constexpr int kN = R * 8 / NT;
  static_assert(kN >= 1 && R * 8 % NT == 0, "whole instructions");
  const uint8_t* base;   // first row (KMAJ) or first K row of the range
  int64_t ld_bytes, k_len;
  int64_t rows;          // KMAJ: rows of the tile that exist
  uint32_t voff[kN];

  // mn0: first row or column of the tile; mn_ext: rows or columns there are
  // (up to the next multiple of 8 for columns: leading dimensions leave room)
  __device__ __forceinline__ void init(const void* p, int64_t ld, int64_t mn0, int64_t mn_ext, int64_t k0,
                                       int64_t k_len_) {
    ld_bytes = ld * 2;
    k_len = k_len_;
    const int t = threadIdx.x;
    if constexpr (KMAJ) {
      rows = mn_ext - mn0 < R ? mn_ext - mn0 : R;
      base = static_cast<const uint8_t*>(p) + mn0 * ld_bytes + k0 * 2;
#pragma unroll
      for (int i = 0; i < kN; i++) {
        const int s = t + NT * i, row = s / 8, c = (s % 8) ^ (row & 7);
        const int64_t r = row < rows ? row : rows - 1;
        voff[i] = (uint32_t)(r * ld_bytes + c * 16);
      }
    } else {
      constexpr int kChunks = R / 8;
      base = static_cast<const uint8_t*>(p) + k0 * ld_bytes;
      const int64_t last = (mn_ext + 7) / 8 * 8 - 8;
#pragma unroll
      for (int i = 0; i < kN; i++) {
        const int s = t + NT * i, k = s / kChunks, c = (s % kChunks) ^ mn_swz<2, R>(k);
        const int64_t col = mn0 + 8 * c < last ? mn0 + 8 * c : last;
        voff[i] = (uint32_t)(k * ld_bytes + col * 2);
      }
    }
  }
  // Loads of step kt.  Elements of K past k_len read as zeros: a buffer load
  // past its resource's size returns zeros, and the resource ends with the
  // range's last K row (MN-contiguous), or the lanes past the end of K get an
  // offset past it (K-contiguous; whole chunks, as the rows are padded to 8).
  __device__ __forceinline__ void issue(uint8_t* tile, int kt) const {
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    const int64_t left = k_len - (int64_t)kt * kStepK;
    if constexpr (KMAJ) {
      const __amdgpu_buffer_rsrc_t rsrc = make_rsrc(base + (int64_t)kt * (kStepK * 2), rows * ld_bytes);
      if (left >= kStepK) {
#pragma unroll
        for (int i = 0; i < kN; i++)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lptr_t)(tile + NT * 16 * i + 1024 * wave), 16, (int)voff[i],
                                                   0, 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < kN; i++) {
          const int s = (int)threadIdx.x + NT * i, row = s / 8, c = (s % 8) ^ (row & 7);
          const uint32_t v = 8 * c < left ? voff[i] : 0x7FFFFFF0u;
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lptr_t)(tile + NT * 16 * i + 1024 * wave), 16, (int)v, 0, 0,
                                                   0);
        }
      }
    } else {
      const int64_t k_rows = left < kStepK ? left : kStepK;
      const __amdgpu_buffer_rsrc_t rsrc = make_rsrc(base + (int64_t)kt * kStepK * ld_bytes, k_rows * ld_bytes);
#pragma unroll
      for (int i = 0; i < kN; i++)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lptr_t)(tile + NT * 16 * i + 1024 * wave), 16, (int)voff[i],
                                                 0, 0, 0);
    }
  }
};

template <int DT>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Tile (tm, tn) of workgroup `block`: blocks are dealt to the 8 XCDs in turn,
// so each XCD gets a contiguous eighth of the tiles, walked in bands of
// `group` tile rows (columns with order_cols), across the band first: the
// tiles an XCD runs at once share bands of A and of B in its L2.
__device__ __forceinline__ void tile_at(int block, int tiles_m, int tiles_n, int order_cols, int group, int& tm,
                                        int& tn) {
  const int tiles = tiles_m * tiles_n;
  const int per = tiles / 8, extra = tiles % 8, xcd = block % 8, at = block / 8;
  const int lin = xcd * per + (xcd < extra ? xcd : extra) + at;
  const int n_major = order_cols ? tiles_n : tiles_m, n_minor = order_cols ? tiles_m : tiles_n;
  const int per_band = group * n_minor;
  const int first = (lin / per_band) * group;
  const int width = n_major - first < group ? n_major - first : group;
  const int r = lin % per_band;
  const int major = first + r % width, minor = r / width;
  tm = order_cols ? minor : major;
  tn = order_cols ? major : minor;
}

template <int BM, int BN>
constexpr int stage_bytes() { return (BM + BN) * kStepK * 2; }
// One LDS array: a stage of both operands, or half of the rounded C tile
// (rows padded by 16 bytes).
template <int BM, int BN>
constexpr int lds_array_bytes() {
  constexpr int c_half = BM / 2 * (BN + 8) * 2;
  return stage_bytes<BM, BN>() > c_half ? stage_bytes<BM, BN>() : c_half;
}

// Stores the BM x BN tile staged in h0 / h1 to rows [m0, m_end) of C (ld n).
template <int BM, int BN, int NT>
__device__ __forceinline__ void store_tile(const uint16_t* h0, const uint16_t* h1, uint16_t* c, int64_t m0,
                                           int64_t m_end, int64_t n0, int64_t n) {
  constexpr int kRow = BN / 8, kPitch = BN + 8;
  static_assert(BM * kRow % NT == 0, "whole turns");
  const bool vec = n % 8 == 0;
#pragma unroll 8
  for (int it = 0; it < BM * kRow / NT; it++) {
    const int s = (int)threadIdx.x + it * NT, row = s / kRow, col = (s % kRow) * 8;
    const uint16_t* src = (row < BM / 2 ? h0 + row * kPitch : h1 + (row - BM / 2) * kPitch) + col;
    const int64_t gr = m0 + row, gc = n0 + col;
    if (gr >= m_end || gc >= n) continue;
    uint16_t* dst = c + gr * n + gc;
    if (vec) {
      store_out16(dst, *reinterpret_cast<const u32x4*>(src));
    } else {
      for (int e = 0; e < 8; e++)
        if (gc + e < n) dst[e] = src[e];
    }
  }
}

// Element r of accumulator (i, j) of lane l is C at row 16 i + l % 16 and
// column 16 j + 4 (l / 16) + r of the wavefront's block (the MFMAs take B's
// fragment first, so they make C transposed).
template <int DT, int BM, int BN, int WGM, int WGN, bool AK, bool BK, int GMODE>
__global__ __launch_bounds__(64 * WGM * WGN) void product_kernel(Product p) {
  constexpr int NT = 64 * WGM * WGN;
  constexpr int WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
  __shared__ __attribute__((aligned(1024))) uint8_t s0[lds_array_bytes<BM, BN>()];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[lds_array_bytes<BM, BN>()];
  constexpr int kATile = BM * kStepK * 2;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, wm = wave / WGN, wn = wave % WGN;

  // the tile, its rows of C, its matrices and its range of K
  const int tiles_n = (int)((p.n + BN - 1) / BN);
  int tiles_m = (int)((p.m + BM - 1) / BM);
  if constexpr (GMODE == BY_ROWS) tiles_m += (int)p.groups;  // each group's last tile may be partial
  int tm, tn;
  tile_at((int)blockIdx.x, tiles_m, tiles_n, p.order_cols, p.tile_group, tm, tn);
  const int64_t n0 = (int64_t)tn * BN;
  int64_t m0 = (int64_t)tm * BM, m_end = p.m, k0 = 0, k_len = p.k;
  const uint16_t* a = static_cast<const uint16_t*>(p.a);
  const uint16_t* b = static_cast<const uint16_t*>(p.b);
  const uint16_t* bias = static_cast<const uint16_t*>(p.bias);
  int64_t c_shift = 0;
  if constexpr (GMODE == BY_ROWS) {
    const RowRange r = find_tile(p.offsets, p.groups, p.m, BM, tm);
    m0 = r.begin + r.tile * BM;
    m_end = r.end;
    if (m0 >= m_end) return;
    if (r.group == p.groups) {  // rows of no group: z = 0
      k_len = 0;
      bias = nullptr;
    } else {
      b += r.group * p.b_group;
      if (bias) bias += r.group * p.n;
    }
  } else if constexpr (GMODE == BY_K) {
    const int64_t g = blockIdx.y;
    int64_t end;
    group_range(p.offsets, g, p.k, k0, end);
    k_len = end - k0;
    c_shift = g * p.m * p.n;
  } else if (BM < 256 && p.splits > 1) {  // (tiles of 256 are not split)
    k0 = (int64_t)blockIdx.y * p.k_part;
    k_len = p.k - k0 < p.k_part ? p.k - k0 : p.k_part;
  }

  Loader<BM, AK, NT> la;
  Loader<BN, BK, NT> lb;
  la.init(a, p.lda, m0, m_end, k0, k_len);
  lb.init(b, p.ldb, n0, p.n, k0, k_len);
  FragReader<2, BM, AK, FM> ra;
  FragReader<2, BN, BK, FN> rb;
  ra.init(wm * WM);
  rb.init(wn * WN);
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int nk = (int)((k_len + kStepK - 1) / kStepK);
  auto step = [&](int kt, uint8_t* cur, uint8_t* nxt) {
    wait_vmcnt<0>();
    lds_barrier();  // step kt has landed; no wavefront reads stage nxt any more
    if (kt + 1 < nk) {
      la.issue(nxt, kt + 1);
      lb.issue(nxt + kATile, kt + 1);
    }
#pragma unroll
    for (int kk = 0; kk < 2; kk++) {
      u32x4 fa[FM], fb[FN];
      ra.read(cur, kk, fa);
      rb.read(cur + kATile, kk, fb);
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++) acc[i][j] = mfma16<DT>(fb[j], fa[i], acc[i][j]);
    }
  };
  if (nk > 0) {
    la.issue(s0, 0);
    lb.issue(s0 + kATile, 0);
  }
  for (int kt = 0; kt < nk; kt += 2) {
    step(kt, s0, s1);
    if (kt + 1 < nk) step(kt + 1, s1, s0);
  }

  if constexpr (GMODE == DENSE && BM < 256) {
    if (p.splits > 1) {  // fp32 sums, tiles whole
      const int64_t ld = (int64_t)tiles_n * BN;
      float* part = p.partial + ((int64_t)blockIdx.y * tiles_m * BM + m0 + wm * WM + lane % 16) * ld + n0 + wn * WN +
                    4 * (lane / 16);
#pragma unroll
      for (int i = 0; i < FM; i++, part += 16 * ld)
#pragma unroll
        for (int j = 0; j < FN; j++) *reinterpret_cast<f32x4*>(part + 16 * j) = acc[i][j];
      return;
    }
  }

  // epilogue: z, then out, each rounded into LDS and stored by rows
  constexpr int kPitch = BN + 8;
  uint16_t* h0 = reinterpret_cast<uint16_t*>(s0);
  uint16_t* h1 = reinterpret_cast<uint16_t*>(s1);
  auto staged = [&](int i, int j) {
    const int row = wm * WM + 16 * i + lane % 16, col = wn * WN + 16 * j + 4 * (lane / 16);
    return reinterpret_cast<u32x2*>((row < BM / 2 ? h0 + row * kPitch : h1 + (row - BM / 2) * kPitch) + col);
  };
  if (bias) {
#pragma unroll
    for (int j = 0; j < FN; j++) {
      const int64_t col = n0 + wn * WN + 16 * j + 4 * (lane / 16);
      float bv[4];
#pragma unroll
      for (int r = 0; r < 4; r++) bv[r] = col + r < p.n ? dec16<DT>(bias[col + r]) : 0.0f;
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int r = 0; r < 4; r++) acc[i][j][r] += bv[r];
    }
  }
  lds_barrier();  // every wavefront has read its last fragments
  if (p.z) {
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
      for (int j = 0; j < FN; j++)
        *staged(i, j) = u32x2{pack2_16<DT>(acc[i][j][0], acc[i][j][1]), pack2_16<DT>(acc[i][j][2], acc[i][j][3])};
    __syncthreads();
    store_tile<BM, BN, NT>(h0, h1, static_cast<uint16_t*>(p.z) + c_shift, m0, m_end, n0, p.n);
    __syncthreads();
  }
  const uint16_t* residual = static_cast<const uint16_t*>(p.residual);
  with_act(p.act, [&](auto ACT_) {
    constexpr int ACT = decltype(ACT_)::value;
#pragma unroll
    for (int i = 0; i < FM; i++) {
      const int64_t row = m0 + wm * WM + 16 * i + lane % 16;
#pragma unroll
      for (int j = 0; j < FN; j++) {
        f32x4 v = acc[i][j];
#pragma unroll
        for (int r = 0; r < 4; r++) v[r] = act_of<ACT>(v[r]);
        if (residual && row < m_end) {
          const int64_t col = n0 + wn * WN + 16 * j + 4 * (lane / 16);
#pragma unroll
          for (int r = 0; r < 4; r++)
            if (col + r < p.n) v[r] += dec16<DT>(residual[row * p.n + col + r]);
        }
        *staged(i, j) = u32x2{pack2_16<DT>(v[0], v[1]), pack2_16<DT>(v[2], v[3])};
      }
    }
  });
  __syncthreads();
  store_tile<BM, BN, NT>(h0, h1, static_cast<uint16_t*>(p.out) + c_shift, m0, m_end, n0, p.n);
}

}  // namespace lin
}  // namespace mc2
