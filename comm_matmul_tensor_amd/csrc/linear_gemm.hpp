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
// with direct-to-LDS buffer loads into a ring of NS stages.  Two wavefronts
// per SIMD (one with the 128 x 128 tile) with interleaved MFMAs, LDS reads and
// loads; the launcher picks the tile (plan_product).
//
// Large products are bound by the MFMAs at the clock the card holds under them: 8192 x 8192 x 8192
// 767 us, 1.43 PFLOP/s (as the vendor library's product on the same card);
// 4096 x 7168 x 4096 with bias, gelu and z 198 to 211 us on different cards (1.14 to
// 1.21); its gradients' two products 174 and 182 us (1.38, 1.32).  In fp16, whose
// 256 x 256 kernels keep 72 to 130 registers per lane in scratch around the
// epilogue (bf16's none), 219 us where bf16 takes 198, and with the gradients'
// dz pass 409 for 378.  Measured and left out: loads ahead of
// time that only bring lines into the L2 (4 bytes per line, 1 to 6 steps
// ahead; by every workgroup or by one per band) 5 to 40 % slower; K walked from
// a step set by the tile, no change or 10 % slower; 256 x 224 tiles, which fill
// the CUs better at n = 7168, within 5 % either way.  Products of one tile per
// CU are bound by the LDS, which a step's loads and fragment reads pass, and by
// their first loads and epilogue, which nothing hides: 517 x 1792 x 4096 13.5 us
// (15.0 in 128 x 128 tiles), 256 x 4096 x 4096 14.8 (22.3), 1024 x 1024 x 1024 8.7
// (10.4).
//
// Groups of rows (experts): the tile's rows come from one group's range of
// rows, found from the ranges on the device (find_tile), with that group's
// B and bias; for the weight's gradient the groups are ranges of K.  A tile
// that crosses the end of its rows, columns or K reads zeros or repeats its
// last column, and stores nothing outside.  32 experts of 4096 x 1792 over
// 16384 rows: 269 us; 231 if all had one matrix, the rest being their 470 MB
// from HBM and the tiles that a group's rows do not fill.
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

struct RowRange { int64_t group, begin, end, tile, tiles; };

// 64 groups from g0 on, one per lane: the rows [start, end) of the lane's
// group, its tiles of bm rows, and the tiles of the 64 groups up to its own.
// Range ends are read as ascending and at most m; `begin`, the end of the
// group before g0, becomes that of the last.
struct GroupTiles {
  int start, end, tiles, incl;
  __device__ __forceinline__ GroupTiles(const int32_t* offsets, int64_t groups, int64_t m, int bm, int64_t g0,
                                        int& begin) {
    const int lane = threadIdx.x % 64;
    const int e = g0 + lane < groups ? offsets[g0 + lane + 1] : 0;
    end = wave_scan_max(max(min(e, (int)m), begin));
    start = __builtin_amdgcn_update_dpp(begin, end, 0x138, 0xF, 0xF, false);  // wave_shr 1; lane 0: begin
    tiles = (end - start + bm - 1) / bm;
    incl = wave_scan_add(tiles);
    begin = __builtin_amdgcn_readlane(end, 63);
  }
  __device__ __forceinline__ int total() const { return __builtin_amdgcn_readlane(incl, 63); }
};

// Tiles of bm rows over all groups (each counts its own) and over the rows
// after the last group, which follow them.
__device__ __forceinline__ int count_tiles(const int32_t* offsets, int64_t groups, int64_t m, int bm) {
  int begin = 0, n = 0;
  for (int64_t g0 = 0; g0 < groups; g0 += 64) n += GroupTiles(offsets, groups, m, bm, g0, begin).total();
  return n + ((int)m - begin + bm - 1) / bm;
}

// Tile `tile` of them, each counted `cols` times: the group (groups: the rows
// after the last one), its rows, its tiles of bm rows, and the tile's place
// among the group's tiles * cols (a place past them all: nothing there).
// Every wavefront finds it for itself.
__device__ __forceinline__ RowRange find_tile(const int32_t* offsets, int64_t groups, int64_t m, int bm, int tile,
                                              int cols = 1) {
  int begin = 0, left = tile;  // left: of the groups still to come
  for (int64_t g0 = 0; g0 < groups; g0 += 64) {
    const GroupTiles t(offsets, groups, m, bm, g0, begin);
    const unsigned long long hit = __ballot(left < t.incl * cols);
    if (hit) {
      const int l = __ffsll((long long)hit) - 1;
      RowRange r;
      r.group = g0 + l;
      r.begin = __builtin_amdgcn_readlane(t.start, l);
      r.end = __builtin_amdgcn_readlane(t.end, l);
      r.tiles = __builtin_amdgcn_readlane(t.tiles, l);
      r.tile = left - (__builtin_amdgcn_readlane(t.incl, l) - (int)r.tiles) * cols;
      return r;
    }
    left -= t.total() * cols;
  }
  return RowRange{groups, begin, m, left, (m - begin + bm - 1) / bm};
}

// Rows [begin, end) of group g, as find_tile reads them, and its tiles of bm
// rows: `count` from number `first` on.
struct GroupAt { int64_t begin, end, first, count; };
__device__ __forceinline__ GroupAt group_at(const int32_t* offsets, int64_t groups, int64_t m, int bm, int64_t g) {
  int begin = 0, first = 0;
  for (int64_t g0 = 0;; g0 += 64) {
    const GroupTiles t(offsets, groups, m, bm, g0, begin);
    if (g < g0 + 64) {
      const int l = (int)(g - g0), count = __builtin_amdgcn_readlane(t.tiles, l);
      return GroupAt{__builtin_amdgcn_readlane(t.start, l), __builtin_amdgcn_readlane(t.end, l),
                     first + __builtin_amdgcn_readlane(t.incl, l) - count, count};
    }
    first += t.total();
  }
}

// One operand's loads: R rows of MN and 64 of K per step by NT threads.
// Instruction i of wavefront w fills the 1 KB of LDS at 16 (NT i + 64 w) in
// lane order; each lane's address is chosen so that the layout is the
// swizzled one FragReader reads.
template <int R, bool KMAJ, int NT>
struct Loader {
  static constexpr int kN = R * 8 / NT;
  static_assert(kN >= 1 && R * 8 % NT == 0, "whole instructions");
  static constexpr int kBytes = kN * NT * 16;  // of LDS
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
        voff[i] = row < rows ? (uint32_t)(row * ld_bytes + c * 16) : 0x7FFFFFF0u;
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
  // Resource and lanes of step kt (any kt: steps past the last one load zeros
  // without touching memory).  Elements of K past k_len read as zeros: a
  // buffer load past its resource's size returns zeros, and the resource ends
  // with the range's last K row (MN-contiguous), or the lanes past the end of
  // K get an offset past it (K-contiguous; whole chunks, as rows are padded to 8).
  struct Step {
    __amdgpu_buffer_rsrc_t rsrc;
    bool off;
  };
  __device__ __forceinline__ Step at(int kt) const {
    const int left = (int)k_len - kt * kStepK;
    if constexpr (KMAJ) {
      // (the lane's chunk is the same in every instruction: 8 rows per 64 lanes)
      return Step{make_rsrc(base + (int64_t)kt * (kStepK * 2), left > 0 ? (int)rows * (int)ld_bytes : 0),
                  8 * (((int)threadIdx.x % 8) ^ ((int)threadIdx.x / 8 & 7)) >= left};
    } else {
      // (a scalar for the resource: the clamp is a vector instruction)
      const int k_rows = __builtin_amdgcn_readfirstlane(max(min(left, kStepK), 0));
      return Step{make_rsrc(base + (int64_t)kt * kStepK * ld_bytes, k_rows * (int)ld_bytes), false};
    }
  }
  // Instruction i of a step.
  __device__ __forceinline__ void issue_one(const Step& s, uint8_t* tile, int wave, int i) const {
    const uint32_t v = KMAJ && s.off ? 0x7FFFFFF0u : voff[i];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(s.rsrc, (lptr_t)(tile + NT * 16 * i + 1024 * wave), 16, (int)v, 0, 0, 0);
  }
};

template <int DT>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Workgroup `block`'s place among the tiles: blocks are dealt to the 8 XCDs in
// turn, so each XCD gets a contiguous eighth of them.
__device__ __forceinline__ int tile_place(int block, int tiles) {
  const int per = tiles / 8, extra = tiles % 8, xcd = block % 8;
  return xcd * per + (xcd < extra ? xcd : extra) + block / 8;
}
// Tile (tm, tn) at that place: bands of `group` tile rows (columns with
// order_cols) one after another, each walked across the band first, so that
// the tiles an XCD runs at once share bands of A and of B in its L2.
__device__ __forceinline__ void tile_at(int lin, int tiles_m, int tiles_n, int order_cols, int group, int& tm,
                                        int& tn) {
  const int n_major = order_cols ? tiles_n : tiles_m, n_minor = order_cols ? tiles_m : tiles_n;
  const int per_band = group * n_minor;
  const int first = (lin / per_band) * group;
  const int width = n_major - first < group ? n_major - first : group;
  const int r = lin % per_band;
  const int major = first + r % width, minor = r / width;
  tm = order_cols ? minor : major;
  tn = order_cols ? major : minor;
}

// One LDS array: a stage of both operands, or half of the rounded C tile
// (rows padded by 16 bytes).
template <int BM, int BN, int NT>
constexpr int lds_array_bytes() {
  constexpr int stage = Loader<BM, true, NT>::kBytes + Loader<BN, true, NT>::kBytes;
  constexpr int c_half = BM / 2 * (BN + 8) * 2;
  return stage > c_half ? stage : c_half;
}

// Stores the BM x BN tile staged in h0 / h1 to rows [m0, m_end) of C (ld n).
template <int BM, int BN, int NT>
__device__ __forceinline__ void store_tile(const uint16_t* h0, const uint16_t* h1, uint16_t* c, int64_t m0,
                                           int64_t m_end, int64_t n0, int64_t n) {
  constexpr int kRow = BN / 8, kPitch = BN + 8;
  constexpr bool kWhole = BM * kRow % NT == 0;
  auto src_of = [&](int row, int col) {
    return (row < BM / 2 ? h0 + row * kPitch : h1 + (row - BM / 2) * kPitch) + col;
  };
  const bool vec = n % 8 == 0;
  if (kWhole && vec && m0 + BM <= m_end && n0 + BN <= n) {  // the tile lies inside C: no tests between the stores
#pragma unroll
    for (int it = 0; it < BM * kRow / NT; it++) {
      const int s = (int)threadIdx.x + it * NT, row = s / kRow, col = (s % kRow) * 8;
      store_out16(c + (m0 + row) * n + n0 + col, *reinterpret_cast<const u32x4*>(src_of(row, col)));
    }
    return;
  }
  for (int s = threadIdx.x; s < BM * kRow; s += NT) {
    const int row = s / kRow, col = (s % kRow) * 8;
    const int64_t gr = m0 + row, gc = n0 + col;
    if (gr >= m_end || gc >= n) continue;
    const u32x4 v = *reinterpret_cast<const u32x4*>(src_of(row, col));
    if (vec) store_chunk<true, true>(c + gr * n, gc, n, v);
    else store_chunk<false, true>(c + gr * n, gc, n, v);
  }
}

// Four 16-bit values from p of which `left` exist (zeros for the others);
// quads: the row length is a multiple of 4, so p is 8-byte aligned and the
// four exist or none.
__device__ __forceinline__ u32x2 load4(const uint16_t* p, int64_t left, bool quads) {
  u32x2 v = {0u, 0u};
  if (quads) {
    if (left > 0) v = *reinterpret_cast<const u32x2*>(p);
  } else if (left >= 4) {
    __builtin_memcpy(&v, p, 8);
  } else {
#pragma unroll
    for (int r = 0; r < 3; r++)
      if (r < left) v[r / 2] |= (uint32_t)p[r] << (16 * (r & 1));
  }
  return v;
}
template <int DT>
__device__ __forceinline__ f32x4 widen4(u32x2 v) {
  return f32x4{dec16<DT>(v[0]), dec16<DT>(v[0] >> 16), dec16<DT>(v[1]), dec16<DT>(v[1] >> 16)};
}

// Element r of accumulator (i, j) of lane l is C at row 16 i + l % 16 and
// column 16 j + 4 (l / 16) + r of the wavefront's block (the MFMAs take B's
// fragment first, so they make C transposed).
template <int DT, int BM, int BN, int WGM, int WGN, int NS, bool AK, bool BK, int GMODE>
__global__ __launch_bounds__(64 * WGM * WGN) void product_kernel(Product p) {
#ifdef __HIP_DEVICE_COMPILE__  // (the host needs only the symbol to launch)
  constexpr int NT = 64 * WGM * WGN;
  constexpr int WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
  __shared__ __attribute__((aligned(1024))) uint8_t s0[lds_array_bytes<BM, BN, NT>()];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[lds_array_bytes<BM, BN, NT>()];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[NS > 2 ? lds_array_bytes<BM, BN, NT>() : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s3[NS > 3 ? lds_array_bytes<BM, BN, NT>() : 16];
  constexpr int kATile = Loader<BM, AK, NT>::kBytes;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, wm = wave / WGN, wn = wave % WGN;

  // the tile, its rows of C, its matrices and its range of K
  const int tiles_n = (int)((p.n + BN - 1) / BN);
  int tiles_m = (int)((p.m + BM - 1) / BM), tm, tn;
  int64_t m0, m_end = p.m, k0 = 0, k_len = p.k, c_shift = 0;
  const uint16_t* a = static_cast<const uint16_t*>(p.a);
  const uint16_t* b = static_cast<const uint16_t*>(p.b);
  const uint16_t* bias = static_cast<const uint16_t*>(p.bias);
  if constexpr (GMODE == BY_ROWS) {
    // The grid has room for a partial tile in every group; the tiles there are
    // go group by group, in bands of rows within each, spread over all XCDs.
    // (Bands across groups had most groups' B read in two turns of the CUs: the
    // 32 experts above took 290 us.)
    tiles_m = count_tiles(p.offsets, p.groups, p.m, BM);
    if ((int)blockIdx.x >= tiles_m * tiles_n) return;
    const RowRange r = find_tile(p.offsets, p.groups, p.m, BM, tile_place((int)blockIdx.x, tiles_m * tiles_n), tiles_n);
    tile_at((int)r.tile, (int)r.tiles, tiles_n, 0, p.tile_group, tm, tn);
    m0 = r.begin + (int64_t)tm * BM;
    m_end = r.end;
    if (r.group == p.groups) {  // rows of no group: z = 0
      k_len = 0;
      bias = nullptr;
    } else {
      b += r.group * p.b_group;
      if (bias) bias += r.group * p.n;
    }
  } else {
    tile_at(tile_place((int)blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, p.order_cols, p.tile_group, tm, tn);
    m0 = (int64_t)tm * BM;
    if constexpr (GMODE == BY_K) {
      const GroupAt g = group_at(p.offsets, p.groups, p.k, 1, blockIdx.y);
      k0 = g.begin;
      k_len = g.end - g.begin;
      c_shift = (int64_t)blockIdx.y * p.m * p.n;
    } else if (BN < 256 && p.splits > 1) {  // (the wider tiles are not split)
      k0 = (int64_t)blockIdx.y * p.k_part;
      k_len = p.k - k0 < p.k_part ? p.k - k0 : p.k_part;
    }
  }
  const int64_t n0 = (int64_t)tn * BN;

  Loader<BM, AK, NT> da;
  Loader<BN, BK, NT> db;
  da.init(a, p.lda, m0, m_end, k0, k_len);
  db.init(b, p.ldb, n0, p.n, k0, k_len);
  FragReader<2, BM, AK, FM> ra;
  FragReader<2, BN, BK, FN> rb;
  ra.init(wm * WM);
  rb.init(wn * WN);
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Main loop, NS stages, in half steps of 32 of K.  Step kt:
  //   MFMAs of half 0, the reads of half 1 between them;
  //   the loads of step kt + 1 have landed; barrier: stage kt is free;
  //   MFMAs of half 1, between them the loads of step kt + NS into stage kt
  //   and the reads of half 0 of step kt + 1.
  // Loads have NS - 1 steps to land and every read nearly a half.  Loads are
  // issued for steps past the last one too (they move nothing), so that no
  // step has a branch in it and the count of loads in flight is constant.
  // The MFMAs go row by row of the wavefront's block, so A's fragment of row i
  // is read for the next half into its own registers once row i is done; only
  // B's fragments and A's last one alternate between two sets.  A wavefront
  // whose rows all lie past the tile's last one only loads.
  const int nk = (int)((k_len + kStepK - 1) / kStepK);
  const int wave_s = __builtin_amdgcn_readfirstlane(wave);
  constexpr int NA = Loader<BM, AK, NT>::kN, ND = NA + Loader<BN, BK, NT>::kN, NM = FM * FN;
  u32x4 fa[FM - 1], la0, la1, fb0[FN], fb1[FN];
  // reads of B: kPerRow in each of rows 1, 2, ..., kGap MFMAs apart; with two
  // rows or columns of MFMAs spread over the rows after the first
  constexpr int kPerRow = (FN + FM - 2) / (FM - 1) < 2 ? 2 : (FN + FM - 2) / (FM - 1), kGap = (FN - 1) / kPerRow;
  static_assert(kGap < 1 || (kPerRow * kGap < FN && kPerRow * (FM - 1) >= FN), "room for B's reads");
  auto read_of_b = [](int q) {  // the fragment read after MFMA q, or FN
    if constexpr (kGap >= 1) {
      const int i = q / FN, j = q % FN;
      return i > 0 && j > 0 && j % kGap == 0 && j / kGap <= kPerRow ? kPerRow * (i - 1) + j / kGap - 1 : FN;
    } else {
      for (int f = 0; f < FN; f++)
        if (FN + f * (NM - FN) / FN == q) return f;
      return FN;
    }
  };
  auto half = [&](const u32x4& last, u32x4& next_last, const u32x4(&fb)[FN], u32x4(&nb)[FN], auto LOAD_, uint8_t* to,
                  int kt_load, const uint8_t* from, int kk) {
    constexpr bool LOAD = decltype(LOAD_)::value;
    const auto sa = da.at(kt_load);
    const auto sb = db.at(kt_load);
#pragma unroll
    for (int i = 0; i < FM; i++) {
#pragma unroll
      for (int j = 0; j < FN; j++) {
        const int q = i * FN + j;
        acc[i][j] = mfma16<DT>(fb[j], i < FM - 1 ? fa[i < FM - 1 ? i : 0] : last, acc[i][j]);
        if (i > 0 && j == 0) fa[i - 1] = ra.read_one(from, kk, i - 1);
        if (i == 0 && j == FN - 1) next_last = ra.read_one(from, kk, FM - 1);
        if (const int f = read_of_b(q); f < FN) nb[f] = rb.read_one(from + kATile, kk, f);
        if constexpr (LOAD) {
#pragma unroll
          for (int d = 0; d < ND; d++)
            if (d * NM / ND == q) {
              if (d < NA) da.issue_one(sa, to, wave_s, d);
              else db.issue_one(sb, to + kATile, wave_s, d - NA);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  auto load_all = [&](uint8_t* to, int kt) {
    const auto sa = da.at(kt);
    const auto sb = db.at(kt);
#pragma unroll
    for (int i = 0; i < NA; i++) da.issue_one(sa, to, wave_s, i);
#pragma unroll
    for (int i = 0; i < ND - NA; i++) db.issue_one(sb, to + kATile, wave_s, i);
  };
  auto step = [&](int kt, uint8_t* cur, uint8_t* nxt) {
    half(la0, la1, fb0, fb1, std::integral_constant<bool, false>(), cur, kt, cur, 1);
    wait_vmcnt<(NS - 2) * ND>();  // this wavefront's loads of step kt + 1
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
    half(la1, la0, fb1, fb0, std::integral_constant<bool, true>(), cur, kt + NS, nxt, 0);
  };
  // The residual's values of this lane.  Where a wavefront has registers for
  // them they are loaded before the main loop (517 x 1792 x 4096 in fp16 by 128 x
  // 128 tiles: 17.4 us, 17.9 from the epilogue).  Their latency is not hidden:
  // load4 tests the lane's place before each of them and its two forms write
  // the same registers, so each waits for the one before, and the operands'
  // first loads for all.  The same product by 96 x 128 tiles: 15.9 us, 13.7
  // without the residual, 12.9 without the bias too, whose loads in the epilogue
  // wait likewise; 4096 x 7168 x 4096: 168 us, 161 without the residual.
  const uint16_t* residual = static_cast<const uint16_t*>(p.residual);
  const bool quads = p.n % 4 == 0;
  const int64_t col0 = n0 + wn * WN + 4 * (lane / 16);  // this lane's first column
  auto load_residual = [&](int i, u32x2(&rv)[FN]) {
    const int64_t row = m0 + wm * WM + 16 * i + lane % 16;
#pragma unroll
    for (int j = 0; j < FN; j++)
      rv[j] = load4(residual + row * p.n + col0 + 16 * j, row < m_end ? p.n - col0 - 16 * j : 0, quads);
  };
  constexpr bool kEarly = FM * FN <= 16;
  u32x2 early[kEarly ? FM : 1][FN];
  if (kEarly && residual && (GMODE != DENSE || p.splits < 2)) {
#pragma unroll
    for (int i = 0; i < (kEarly ? FM : 1); i++) load_residual(i, early[i]);
  }
  if (nk > 0) {
    uint8_t* const st[4] = {s0, s1, s2, s3};
#pragma unroll
    for (int i = 0; i < NS; i++) load_all(st[i], i);
    wait_vmcnt<(NS - 1) * ND>();
    lds_barrier();
    if (GMODE == BY_ROWS && m0 + (int64_t)(wave_s / WGN) * WM >= m_end) {
      const int steps = NS == 2 ? nk + nk % 2 : nk;  // as many barriers as the others
      for (int kt = 0; kt < steps; kt += NS) {
#pragma unroll
        for (int i = 0; i < NS; i++) {
          if (kt + i >= steps) break;
          wait_vmcnt<(NS - 2) * ND>();
          lds_barrier();
          load_all(st[i], kt + i + NS);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < FM - 1; i++) fa[i] = ra.read_one(s0, 0, i);
      la0 = ra.read_one(s0, 0, FM - 1);
      rb.read(s0 + kATile, 0, fb0);
      // two stages: an odd last step is followed by one of zeros (a copy of
      // the step for it costs registers in the loop)
      constexpr int kOver = NS == 2 ? 1 : 0;
      int kt = 0;
      for (; kt + NS <= nk + kOver; kt += NS) {
#pragma unroll
        for (int i = 0; i < NS; i++) step(kt + i, st[i], st[(i + 1) % NS]);
      }
      if constexpr (NS > 2) {
#pragma unroll
        for (int i = 0; i < NS - 1; i++)
          if (kt + i < nk) step(kt + i, st[i], st[i + 1]);
      }
    }
    wait_vmcnt<0>();  // the last loads' zeros are in LDS before the epilogue's values
  }

  if constexpr (GMODE == DENSE && BN < 256) {
    if (p.splits > 1) {  // fp32 sums of the rows there are, whole tiles of columns
      const int64_t ld = (int64_t)tiles_n * BN;
      float* part = p.partial + ((int64_t)blockIdx.y * tiles_m * BM + m0 + wm * WM + lane % 16) * ld + n0 + wn * WN +
                    4 * (lane / 16);
#pragma unroll
      for (int i = 0; i < FM; i++, part += 16 * ld)
        if (m0 + wm * WM + 16 * i + lane % 16 < m_end) {
#pragma unroll
          for (int j = 0; j < FN; j++) *reinterpret_cast<f32x4*>(part + 16 * j) = acc[i][j];
        }
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
      const f32x4 bv = widen4<DT>(load4(bias + col0 + 16 * j, p.n - col0 - 16 * j, quads));
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
  with_act(p.act, [&](auto ACT_) {
    constexpr int ACT = decltype(ACT_)::value;
#pragma unroll
    for (int i = 0; i < FM; i++) {
      u32x2 late[FN];
      if (!kEarly && residual) load_residual(i, late);
#pragma unroll
      for (int j = 0; j < FN; j++) {
        f32x4 v = acc[i][j];
#pragma unroll
        for (int r = 0; r < 4; r++) v[r] = act_of<ACT>(v[r]);
        if (residual) {
          const f32x4 f = widen4<DT>(kEarly ? early[kEarly ? i : 0][j] : late[j]);
#pragma unroll
          for (int r = 0; r < 4; r++) v[r] += f[r];
        }
        *staged(i, j) = u32x2{pack2_16<DT>(v[0], v[1]), pack2_16<DT>(v[2], v[3])};
      }
    }
  });
  __syncthreads();
  store_tile<BM, BN, NT>(h0, h1, static_cast<uint16_t*>(p.out) + c_shift, m0, m_end, n0, p.n);
#endif
}

}  // namespace lin
}  // namespace mc2
