// K11, around the tiled product: the plan of a call (tile, split, workspace),
// the product of few rows, the gradient's dz and bias sums, and the copies
// that give rows of a ragged width an aligned one.
#include <algorithm>
#include <cmath>

#include "codes.hpp"
#include "linear_kernels.hpp"

namespace mc2 {
namespace lin {

// A product runs in turns of one tile per CU; a turn takes a fixed time (first
// loads, epilogue) and a time per step of 64 of K, in us, as fitted to bf16
// products of 256 and more tiles (8192 x 4096, k = 1024: 256 x 256 63, 128 x 256
// 71, 128 x 128 83; one tile per CU, k = 4096: 128 x 128 32.8, 96 x 128 26.6,
// 128 x 64 20.7, 96 x 64 17.5, 64 x 64 15.1; two 64 x 64 per CU 25.4).  The
// small tiles' steps are bound by the LDS: a step's loads and its wavefronts'
// reads of them, 768 / 672 / 576 / 480 / 384 cycles at 128 bytes each where the
// MFMAs take 512 / 384 / 256 / 192 / 128, so fewer rows or columns than a larger
// tile pay only while they fill more CUs.  Groups of rows are taken as equal,
// with half a tile more than their rows fill each, one tile at least (64
// matrices of 4096 x 1792, 8 rows in all: 64 x 64 22.7 us, 128 x 128 32.9; 8
// matrices, 1024 rows: 96 x 128 35.4, 128 x 128 44.3, 128 x 256 60.5).
struct TurnTime { Tile tile; int bm, bn; double fixed, step; };
constexpr TurnTime kTurns[] = {{TILE_256X256, 256, 256, 9.0, 1.39}, {TILE_128X256, 128, 256, 5.5, 0.756},
                               {TILE_128X128, 128, 128, 3.6, 0.43}, {TILE_96X128, 96, 128, 3.0, 0.35},
                               {TILE_128X64, 128, 64, 2.4, 0.27},   {TILE_96X64, 96, 64, 1.2, 0.225},
                               {TILE_64X64, 64, 64, 1.2, 0.18}};

// Of int8 codes, per step of 128 (one turn: 256 x 256 58.0 us at k = 4096, 128 x
// 256 34.0, 128 x 128 21.5, 96 x 128 18.4, 128 x 64 14.6, 96 x 64 12.4, 64 x 64 10.8).
// The steps of 128 x 128 and under are those of many turns, which read 20 TB/s
// from the L2s and miss there: 4096 x 4096 -> 5000 in five turns 103 us, 95 in three
// of 128 x 256; 32 experts of 4096 -> 1792, 8191 rows 126 and 112.
constexpr TurnTime kTurnsI8[] = {{TILE_256X256, 256, 256, 9.5, 1.42}, {TILE_128X256, 128, 256, 5.6, 0.81},
                                 {TILE_128X128, 128, 128, 4.7, 0.50}, {TILE_96X128, 96, 128, 3.7, 0.39},
                                 {TILE_128X64, 128, 64, 2.8, 0.28},   {TILE_96X64, 96, 64, 1.6, 0.245},
                                 {TILE_64X64, 64, 64, 1.2, 0.20}};

Plan plan_product(int64_t m, int64_t n, int64_t k, int layout, int gmode, int64_t groups, bool i8) {
  const double steps = std::ceil((double)k / (gmode == BY_K ? (double)groups : 1.0) / kStepK);
  auto tiles = [&](const TurnTime& t) {
    const double cols = (double)((n + t.bn - 1) / t.bn);
    if (gmode == BY_ROWS) {
      const double some = (double)std::min(m, groups);  // groups with rows, at most
      return std::max(some, (double)m / t.bm + 0.5 * some) * cols;
    }
    return (double)((m + t.bm - 1) / t.bm) * cols * (gmode == BY_K ? (double)groups : 1.0);
  };
  Plan p{TILE_128X128, 1, k, 0, 0.0};
  const TurnTime* chosen = nullptr;
  double best = 0.0;
  int64_t s = 1;
  for (const TurnTime& t : i8 ? kTurnsI8 : kTurns) {
    if (t.tile > TILE_128X128 && gmode == BY_K) break;
    if ((t.bm == 96 && layout == 2) || (t.tile == TILE_128X64 && gmode == BY_ROWS)) continue;
    const double count = tiles(t);
    for (int64_t i = 1; i <= 32; i++) {
      // K in i parts where that leaves no CU a second tile: fewer steps against
      // a second launch (4.5 us) and the partial sums written and read (4 TB/s)
      if (i > 1 && (t.bn > 128 || gmode != DENSE || (double)i * count > 256.0)) break;
      const double join = i > 1 ? 4.5 + (double)i * (double)m * (double)n * 8.0 / 4e6 : 0.0;
      if (i > 1 && t.fixed + join >= best) break;  // nor would more parts
      const double cost =
          std::ceil((double)i * count / 256.0) * (t.fixed + t.step * std::ceil(steps / (double)i)) + join;
      if (!chosen || cost < best) {
        best = cost;
        chosen = &t;
        s = i;
      }
    }
  }
  p.tile = chosen->tile;
  p.us = best;
  if (s > 1) {
    p.k_part = ((k + s - 1) / s + kStepK - 1) / kStepK * kStepK;
    p.splits = (int)((k + p.k_part - 1) / p.k_part);
    if (p.splits > 1) {
      auto whole = [](int64_t v, int64_t by) { return (v + by - 1) / by * by; };
      p.partial_bytes = (size_t)p.splits * whole(m, chosen->bm) * whole(n, chosen->bn) * sizeof(float);
    }
  }
  return p;
}

namespace {

int64_t pad8(int64_t v) { return (v + 7) / 8 * 8; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// ---------------------------------------------------------------- ragged rows
// dst (rows, ld) = src (rows, k) with zeros in columns k .. ld - 1, for up to
// two matrices in one launch; tpr threads per row.
struct PadArgs {
  const uint16_t* src[2];
  uint16_t* dst[2];
  int64_t rows[2];
  int64_t k, ld;
  int tpr;
};
__global__ __launch_bounds__(256) void pad_rows(PadArgs a) {
  const int per = 256 / a.tpr;
  for (int64_t i = (int64_t)blockIdx.x * per + threadIdx.x / a.tpr; i < a.rows[0] + a.rows[1];
       i += (int64_t)gridDim.x * per) {
    const int which = i >= a.rows[0];
    const int64_t row = which ? i - a.rows[0] : i;
    const uint16_t* src = a.src[which] + row * a.k;
    uint16_t* dst = a.dst[which] + row * a.ld;
#pragma unroll 4
    for (int64_t c = 8 * (int64_t)(threadIdx.x % a.tpr); c < a.ld; c += 8 * a.tpr)
      *reinterpret_cast<u32x4*>(dst + c) = load_chunk<false>(src, c, a.k);
  }
}
hipError_t launch_pad_rows(const void* s0, int64_t rows0, void* d0, const void* s1, int64_t rows1, void* d1, int64_t k,
                           hipStream_t s) {
  if (rows0 + rows1 == 0) return hipSuccess;
  int tpr = 1;
  while (tpr < 256 && 8 * tpr < k) tpr *= 2;
  const PadArgs a{{static_cast<const uint16_t*>(s0), static_cast<const uint16_t*>(s1)},
                  {static_cast<uint16_t*>(d0), static_cast<uint16_t*>(d1)},
                  {rows0, rows1},
                  k,
                  pad8(k),
                  tpr};
  const int64_t blocks = (rows0 + rows1 + 256 / tpr - 1) / (256 / tpr);
  pad_rows<<<(unsigned)std::min<int64_t>(blocks, 256 * 16), 256, 0, s>>>(a);
  return hipGetLastError();
}

// ---------------------------------------------------------------- few rows
// m <= 16 MF rows (a decoding step): bound by reading w once.  A workgroup
// makes 16 columns of C; its WAVES wavefronts take K in turn, 32 U at a time,
// and their sums are added in wavefront order.  An MFMA takes 16 rows of w
// (its first operand) and 16 rows of x (rows past m repeat the last one and
// are not stored); fragments come straight from memory, U of each in flight.
constexpr int kSkinnyU = 4;
template <int DT, int MF, int WAVES, bool VEC>
__global__ __launch_bounds__(64 * WAVES) void skinny_kernel(Product p) {
  __shared__ float red[WAVES][MF * 256];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t n0 = (int64_t)blockIdx.x * 16, k = p.k;
  const int64_t wr = n0 + lane % 16 < p.n ? n0 + lane % 16 : p.n - 1;
  const uint16_t* w = static_cast<const uint16_t*>(p.b) + wr * k;
  const uint16_t* x[MF];
  f32x4 acc[MF];
#pragma unroll
  for (int i = 0; i < MF; i++) {
    const int64_t r = 16 * i + lane % 16 < p.m ? 16 * i + lane % 16 : p.m - 1;
    x[i] = static_cast<const uint16_t*>(p.a) + r * k;
    acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  for (int64_t kb = (int64_t)wave * 32 * kSkinnyU; kb < k; kb += (int64_t)WAVES * 32 * kSkinnyU) {
    u32x4 fw[kSkinnyU], fx[MF][kSkinnyU];
#pragma unroll
    for (int u = 0; u < kSkinnyU; u++) {
      const int64_t c = kb + 32 * u + 8 * (lane / 16);
      fw[u] = u32x4{0u, 0u, 0u, 0u};
      if (c < k) fw[u] = load_chunk<VEC>(w, c, k);
#pragma unroll
      for (int i = 0; i < MF; i++) {
        fx[i][u] = u32x4{0u, 0u, 0u, 0u};
        if (c < k) fx[i][u] = load_chunk<VEC>(x[i], c, k);
      }
    }
#pragma unroll
    for (int u = 0; u < kSkinnyU; u++)
#pragma unroll
      for (int i = 0; i < MF; i++) acc[i] = mfma16<DT>(fw[u], fx[i][u], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < MF; i++)
    *reinterpret_cast<f32x4*>(&red[wave][256 * i + lane % 16 * 16 + 4 * (lane / 16)]) = acc[i];
  __syncthreads();
  for (int t = threadIdx.x; t < MF * 256; t += 64 * WAVES) {
    const int64_t row = t / 16, col = n0 + t % 16;
    if (row >= p.m || col >= p.n) continue;
    float v = red[0][t];
#pragma unroll
    for (int s = 1; s < WAVES; s++) v += red[s][t];
    if (p.bias) v += dec16<DT>(static_cast<const uint16_t*>(p.bias)[col]);
    const int64_t at = row * p.n + col;
    if (p.z) static_cast<uint16_t*>(p.z)[at] = enc16<DT>(v);
    with_act(p.act, [&](auto ACT_) { v = act_of<decltype(ACT_)::value>(v); });
    if (p.residual) v += dec16<DT>(static_cast<const uint16_t*>(p.residual)[at]);
    static_cast<uint16_t*>(p.out)[at] = enc16<DT>(v);
  }
}

constexpr int64_t kSkinnyRows = 32;

// Wavefronts of a workgroup: 16 while no CU has a second workgroup, to cover
// HBM's latency (16 / 4, one row, in us: 4096 columns, k = 2048 6.3 / 7.6, 4096
// 9.2 / 12.0, 16384 37.3 / 39.4; with k = 256, or 32 rows of k >= 4096, within 9 %
// either way).  Past that 4, whose workgroups start and join sooner: 4112 columns,
// k = 2048 7.7 / 7.8, 6144 18.3 / 16.7, 16384 51.1 / 41.4; 20480 columns, k = 256 6.8 /
// 4.6, 1024 12.4 / 10.2; 32 rows of 8192 to 28672 columns, k = 4096, 5 to 6 % at any
// width.  Only from a third workgroup per CU on do up to 16 rows of a long K
// gain from 16 again (fewer rows of w read at a time): k = 2048, 8192 columns (two
// per CU) 9.3 / 9.5, 9216 11.2 / 11.9; k = 6144, 8192 columns 22.1 / 22.8, 9216 28.3 /
// 30.7; k = 8192, 28672 columns 86.6 / 92.8 (470 MB, 5.4 TB/s);
// 16 rows, k = 2048 and 6144, 9216 columns 15.2 / 16.5 and 44.3 / 42.5.
int skinny_waves(int64_t m, int64_t k, int64_t n) {
  const int64_t blocks = (n + 15) / 16;
  return blocks <= 256 || (blocks > 512 && k >= 2048 && m <= 16) ? 16 : 4;
}

template <int DT, int MF>
hipError_t launch_skinny(const Product& p, hipStream_t s) {
  const unsigned blocks = (unsigned)((p.n + 15) / 16);
  const bool vec = p.k % 8 == 0;
  if (skinny_waves(p.m, p.k, p.n) == 4) {
    if (vec) skinny_kernel<DT, MF, 4, true><<<blocks, 256, 0, s>>>(p);
    else skinny_kernel<DT, MF, 4, false><<<blocks, 256, 0, s>>>(p);
  } else {
    if (vec) skinny_kernel<DT, MF, 16, true><<<blocks, 1024, 0, s>>>(p);
    else skinny_kernel<DT, MF, 16, false><<<blocks, 1024, 0, s>>>(p);
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------- dz and bias sums
// dz = dout act'(z) for a tile of 64 rows (of one group), and the column sums
// of the unrounded dz over the tile's rows.  dz is stored rounded to 16 bits: the
// two products that read it run on 16-bit operands, as their other factors
// are, at half the bytes and (bf16) 16 times the rate of fp32 ones.  Its rounding
// takes the error of dx and dw against 64 bits from 0.0017 to 0.0023 in the
// 2-norm (bf16, 4096 x 4096 x 7168): two independent roundings instead of one.  A row of the tile is taken by tpr
// threads with 8 columns each (fewer than kDzThreads where n is small), and
// the sums of the 256 / tpr rows in flight are added in order.  Bound by HBM
// and, with gelu, nearly as much by its arithmetic: 4096 x 7168 32 us for the
// sums alone, 38 with dz stored.  Wider tiles (a row's 4 KB at a time) or more
// rows in flight per thread took 35 to 55: they leave fewer wavefronts.
constexpr int kDzRows = 64, kDzThreads = 32;  // rows of a tile, most threads of a row
struct DzArgs {
  const uint16_t *dout, *z;
  uint16_t* dz;    // (m, ld) or NULL
  float* partial;  // (row tiles, n) or NULL
  int64_t m, n, ld;
  const int32_t* offsets;
  int64_t groups;
  int tpr;
  const int8_t* z_codes;  // EIGHT: z as codes, a scale per 128 columns
  const float* z_scale;
  uint16_t* dbias;  // EIGHT, one tile of rows: its sums are the bias's gradient (else NULL)
};
// Tile (bx, by) of it; red: 256 * 8 numbers, [row of threads][column].
template <int DT, int ACT, bool VEC, bool EIGHT>
__device__ __forceinline__ void dz_tile(const DzArgs& a, unsigned bx, unsigned by, float* red) {
  int64_t m0 = (int64_t)bx * kDzRows, m_end = a.m;
  if (a.groups > 0) {
    const RowRange r = find_tile(a.offsets, a.groups, a.m, kDzRows, bx);
    if (r.group == a.groups) return;
    m0 = r.begin + r.tile * kDzRows;
    m_end = r.end;
  }
  if (m0 + kDzRows < m_end) m_end = m0 + kDzRows;
  const int tpr = a.tpr, rows = 256 / tpr, rt = threadIdx.x / tpr, ct = threadIdx.x % tpr;
  const int64_t c0 = (int64_t)by * tpr * 8, c = c0 + 8 * ct;
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (c < a.n) {
#pragma unroll 2
    for (int64_t row = m0 + rt; row < m_end; row += rows) {
      float d[8];
      unpack8<DT>(load_chunk<VEC>(a.dout + row * a.n, c, a.n), d);
      if constexpr (ACT != ACT_NONE) {
        float f[8];
        if constexpr (EIGHT)
          code_values(load_codes<VEC>(a.z_codes + row * a.n, c, a.n), a.z_scale[row * scales_of(a.n, 128) + c / 128], f);
        else
          unpack8<DT>(load_chunk<VEC>(a.z + row * a.n, c, a.n), f);
#pragma unroll
        for (int e = 0; e < 8; e++) {
          // (codes of a group that is NaN: relu's slope of a NaN is 0, which would hide 128 columns)
          const bool lost = EIGHT && ACT == ACT_RELU && f[e] != f[e];
          d[e] *= lost ? f[e] : act_slope<ACT>(f[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; e++) {
        if (!VEC && c + e >= a.n) d[e] = 0.0f;
        sum[e] += d[e];
      }
      if (a.dz) *reinterpret_cast<u32x4*>(a.dz + row * a.ld + c) = pack8<DT>(d);
    }
  }
  if (!a.partial && !(EIGHT && a.dbias)) return;
#pragma unroll
  for (int e = 0; e < 8; e++) red[rt * (8 * tpr) + 8 * ct + e] = sum[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * tpr && c0 + i < a.n; i += 256) {
    float s = red[i];
    for (int r = 1; r < rows; r++) s += red[r * (8 * tpr) + i];
    if (EIGHT && a.dbias) a.dbias[c0 + i] = enc16<DT>(s);
    else a.partial[(int64_t)bx * a.n + c0 + i] = s;
  }
}
template <int DT, int ACT, bool VEC>
__global__ __launch_bounds__(256) void dz_kernel(DzArgs a) {
  __shared__ float red[256 * 8];
  dz_tile<DT, ACT, VEC, false>(a, blockIdx.x, blockIdx.y, red);
}
// The same from z's codes, and x's codes to 16 bits, whose values the product
// for dw reads in many tiles: both in one launch, as a batch of some hundred rows
// is bound by its launches.  The first tiles * cols workgroups are dz's.
template <int DT, bool VECN, bool VECK>
__global__ __launch_bounds__(256) void kept_kernel(DzArgs a, unsigned tiles, unsigned cols, int act, CodeArgs x, int tpr) {
  __shared__ float red[256 * 8];
  if (blockIdx.x < tiles * cols) {
    with_act(act, [&](auto ACT_) {
      dz_tile<DT, decltype(ACT_)::value, VECN, true>(a, blockIdx.x % tiles, blockIdx.x / tiles, red);
    });
  } else {
    with_act(x.act, [&](auto ACT_) {
      dequant_block<DT, decltype(ACT_)::value, VECK>(x, tpr, blockIdx.x - tiles * cols);
    });
  }
}

// dbias[g][j] = sum of the partial sums of group g's row tiles, in order within
// each of 4 wavefronts and over them.
template <int DT>
__global__ __launch_bounds__(256) void dbias_kernel(DzArgs a, int64_t tiles, uint16_t* dbias) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t j = (int64_t)blockIdx.x * 64 + lane;
  int64_t first = 0, count = tiles;
  if (a.groups > 0) {
    const GroupAt g = group_at(a.offsets, a.groups, a.m, kDzRows, blockIdx.y);
    first = g.first;
    count = g.count;
    dbias += blockIdx.y * a.n;
  }
  float s = 0.0f;
  if (j < a.n) {
#pragma unroll 4
    for (int64_t t = first + wave; t < first + count; t += 4) s += a.partial[t * a.n + j];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && j < a.n) dbias[j] = enc16<DT>(((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane]);
}

int64_t dz_tiles(int64_t m, int64_t groups) { return (m + kDzRows - 1) / kDzRows + groups; }

// wide: x's codes to be widened on the way (z is codes then too), or NULL.
template <int DT>
hipError_t launch_dz(DzArgs a, int act, void* dbias, const CodeArgs* wide, hipStream_t s) {
  a.tpr = 8;
  while (a.tpr < kDzThreads && 8 * a.tpr < a.n) a.tpr *= 2;
  const int64_t tiles = dz_tiles(a.m, a.groups);
  const bool vec = a.n % 8 == 0;
  const bool sums = a.dz || dbias;
  if (a.m > 0 && (wide || (a.z_codes && sums))) {
    if (tiles == 1 && dbias) a.dbias = static_cast<uint16_t*>(dbias);
    const unsigned cols = sums ? (unsigned)((a.n + 8 * a.tpr - 1) / (8 * a.tpr)) : 0;
    const CodeArgs x = wide ? *wide : CodeArgs{};
    const int tpr = wide ? dequant_threads(x.rows, x.cols) : 1;
    const unsigned blocks = (unsigned)tiles * cols + (wide ? (unsigned)((x.rows + 256 / tpr - 1) / (256 / tpr)) : 0);
    auto kept = [&](auto VECN_, auto VECK_) {
      kept_kernel<DT, decltype(VECN_)::value, decltype(VECK_)::value>
          <<<blocks, 256, 0, s>>>(a, (unsigned)tiles, cols, act, x, tpr);
    };
    const std::true_type yes;
    const std::false_type no;
    if (vec) x.cols % 8 == 0 ? kept(yes, yes) : kept(yes, no);
    else x.cols % 8 == 0 ? kept(no, yes) : kept(no, no);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  } else if (a.m > 0 && sums) {
    const dim3 grid((unsigned)tiles, (unsigned)((a.n + 8 * a.tpr - 1) / (8 * a.tpr)));
    with_act(act, [&](auto ACT_) {
      constexpr int ACT = decltype(ACT_)::value;
      if (vec) dz_kernel<DT, ACT, true><<<grid, 256, 0, s>>>(a);
      else dz_kernel<DT, ACT, false><<<grid, 256, 0, s>>>(a);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dbias && !a.dbias) {
    const dim3 grid((unsigned)((a.n + 63) / 64), (unsigned)std::max<int64_t>(a.groups, 1));
    dbias_kernel<DT><<<grid, 256, 0, s>>>(a, tiles, static_cast<uint16_t*>(dbias));
    return hipGetLastError();
  }
  return hipSuccess;
}

// Parts of a workspace, in order, each 256-byte aligned.
struct Parts {
  size_t used = 0;
  size_t take(size_t bytes) {
    const size_t at = used;
    used += up256(bytes);
    return at;
  }
};

struct ForwardLayout {
  size_t x8, w8, partial, total;
  Plan plan;
  ForwardLayout(int64_t m, int64_t k, int64_t n, int64_t groups) {
    Parts p;
    const bool skinny = !groups && m <= kSkinnyRows;
    plan = skinny ? Plan{} : plan_product(m, n, k, 0, groups ? BY_ROWS : DENSE, groups);
    const bool ragged = k % 8 != 0 && !skinny;
    x8 = p.take(ragged ? (size_t)m * pad8(k) * 2 : 0);
    w8 = p.take(ragged ? (size_t)std::max<int64_t>(groups, 1) * n * pad8(k) * 2 : 0);
    partial = p.take(plan.partial_bytes);
    total = p.used;
  }
};

struct GradLayout {
  size_t dz, sums, x8, w8, partial, total;
  Plan dx, dw;
  GradLayout(int64_t m, int64_t k, int64_t n, int64_t groups, bool eight = false) {
    Parts p;
    dx = plan_product(m, k, n, 1, groups ? BY_ROWS : DENSE, groups);
    dw = plan_product(n, k, m, 2, groups ? BY_K : DENSE, groups);
    dz = p.take((size_t)m * pad8(n) * 2);
    sums = p.take((size_t)dz_tiles(m, groups) * n * sizeof(float));
    x8 = p.take(k % 8 || eight ? (size_t)m * pad8(k) * 2 : 0);  // x padded, or widened from its codes
    w8 = p.take(k % 8 ? (size_t)std::max<int64_t>(groups, 1) * n * pad8(k) * 2 : 0);
    partial = p.take(std::max(dx.partial_bytes, dw.partial_bytes));
    total = p.used;
  }
};

template <int DT>
hipError_t forward_dt(const LinearArgs& a, hipStream_t s) {
  const ForwardLayout at(a.m, a.k, a.n, a.groups);
  char* ws = static_cast<char*>(a.workspace);
  Product p{};
  p.a = a.x;
  p.b = a.w;
  p.m = a.m;
  p.n = a.n;
  p.k = a.k;
  p.offsets = a.offsets;
  p.groups = a.groups;
  p.bias = a.bias;
  p.residual = a.residual;
  p.out = a.out;
  p.z = a.z;
  p.act = a.act;
  p.splits = 1;
  if (!a.groups && a.m <= kSkinnyRows)
    return a.m <= 16 ? launch_skinny<DT, 1>(p, s) : launch_skinny<DT, 2>(p, s);
  p.lda = p.ldb = pad8(a.k);
  p.b_group = a.n * p.ldb;
  if (a.k % 8) {
    const hipError_t e = launch_pad_rows(a.x, a.m, ws + at.x8, a.w, std::max<int64_t>(a.groups, 1) * a.n, ws + at.w8,
                                         a.k, s);
    if (e != hipSuccess) return e;
    p.a = ws + at.x8;
    p.b = ws + at.w8;
  }
  p.partial = reinterpret_cast<float*>(ws + at.partial);
  return launch_product<DT>(p, 0, a.groups ? BY_ROWS : DENSE, at.plan, s);
}

template <int DT>
hipError_t grad_dt(const LinearGradArgs& a, hipStream_t s) {
  const GradLayout at(a.m, a.k, a.n, a.groups, a.eight);
  char* ws = static_cast<char*>(a.workspace);
  const int64_t matrices = std::max<int64_t>(a.groups, 1);
  // dz: dout itself without an activation, where its rows are aligned
  const bool products = a.dx || a.dw, copy = a.act != ACT_NONE || a.n % 8 != 0;
  DzArgs d{};
  d.dout = static_cast<const uint16_t*>(a.dout);
  d.z = static_cast<const uint16_t*>(a.z);
  d.z_codes = a.z_codes;
  d.z_scale = a.z_scale;
  d.dz = products && copy ? reinterpret_cast<uint16_t*>(ws + at.dz) : nullptr;
  d.partial = a.dbias ? reinterpret_cast<float*>(ws + at.sums) : nullptr;
  d.m = a.m;
  d.n = a.n;
  d.ld = pad8(a.n);
  d.offsets = a.offsets;
  d.groups = a.groups;
  CodeArgs codes{};
  const bool wide = a.eight && a.dw;
  if (wide) {
    codes.codes_in = a.x_codes;
    codes.scale_in = a.x_scale;
    codes.out = ws + at.x8;
    codes.rows = a.m;
    codes.cols = a.k;
    codes.ld = pad8(a.k);
    codes.group = 128;
    codes.act = a.x_act;
  }
  hipError_t e = launch_dz<DT>(d, a.act, a.dbias, wide ? &codes : nullptr, s);
  if (e != hipSuccess || !products) return e;
  const void *x = a.x, *w = a.w, *dz = copy ? d.dz : a.dout;
  if (a.k % 8) {
    // x for dw, w for dx
    e = launch_pad_rows(a.x, a.dw && !a.eight ? a.m : 0, ws + at.x8, a.w, a.dx ? matrices * a.n : 0, ws + at.w8, a.k, s);
    if (e != hipSuccess) return e;
    x = ws + at.x8;
    w = ws + at.w8;
  }
  if (wide) x = ws + at.x8;
  Product p{};
  p.offsets = a.offsets;
  p.groups = a.groups;
  p.act = ACT_NONE;
  p.partial = reinterpret_cast<float*>(ws + at.partial);
  if (a.dx && a.m > 0) {  // (m, k) = dz (m, n) @ w (n, k)
    p.a = dz;
    p.lda = pad8(a.n);
    p.b = w;
    p.ldb = pad8(a.k);
    p.b_group = a.n * p.ldb;
    p.m = a.m;
    p.n = a.k;
    p.k = a.n;
    p.out = a.dx;
    e = launch_product<DT>(p, 1, a.groups ? BY_ROWS : DENSE, at.dx, s);
    if (e != hipSuccess) return e;
  }
  if (a.dw) {  // (n, k) = dz (m, n)^T @ x (m, k)
    p.a = dz;
    p.lda = pad8(a.n);
    p.b = x;
    p.ldb = pad8(a.k);
    p.b_group = 0;
    p.m = a.n;
    p.n = a.k;
    p.k = a.m;
    p.out = a.dw;
    e = launch_product<DT>(p, 2, a.groups ? BY_K : DENSE, at.dw, s);
  }
  return e;
}

}  // namespace
}  // namespace lin

void linear_act_plan(int product, int64_t m, int64_t k, int64_t n, int64_t groups, int* tile, int* splits) {
  lin::Plan p{};
  if (product == 0) {
    if (!groups && m <= lin::kSkinnyRows) {
      *tile = -lin::skinny_waves(m, k, n);
      *splits = 1;
      return;
    }
    p = lin::ForwardLayout(m, k, n, groups).plan;
  } else {
    const lin::GradLayout at(m, k, n, groups);
    p = product == 1 ? at.dx : at.dw;
  }
  *tile = p.tile;
  *splits = p.splits;
}

size_t linear_act_workspace(int64_t m, int64_t k, int64_t n, int64_t groups) {
  return m > 0 ? lin::ForwardLayout(m, k, n, groups).total : 0;
}
size_t linear_act_grad_workspace(int64_t m, int64_t k, int64_t n, int64_t groups, bool eight) {
  return lin::GradLayout(m, k, n, groups, eight).total;
}

hipError_t launch_linear_act(const LinearArgs& a, hipStream_t s) {
  if (a.m < 1 || a.k < 1 || a.n < 1 || a.groups < 0 || a.k > lin::kMaxDim || a.n > lin::kMaxDim)
    return hipErrorInvalidValue;
  return a.dtype == DT_BF16 ? lin::forward_dt<DT_BF16>(a, s) : lin::forward_dt<DT_F16>(a, s);
}
hipError_t launch_linear_act_grad(const LinearGradArgs& a, hipStream_t s) {
  if (a.m < 0 || a.k < 1 || a.n < 1 || a.groups < 0 || a.k > lin::kMaxDim || a.n > lin::kMaxDim)
    return hipErrorInvalidValue;
  return a.dtype == DT_BF16 ? lin::grad_dt<DT_BF16>(a, s) : lin::grad_dt<DT_F16>(a, s);
}

}  // namespace mc2
