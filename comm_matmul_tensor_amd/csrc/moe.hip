// K12: tokens' rows by expert and back.
//
// Sort.  A stable counting sort of the choices i = t top + j by expert.  The
// choices are split into contiguous segments, one per wavefront; with
// count[w][e] the choices of expert e in segment w,
//   row(i) = offsets[e] + sum of count[w'][e] over earlier segments w'
//            + the choices of e before i in i's own segment,
// the last by a ballot per bit of the expert id (lanes with equal ids) and a
// running count in LDS.  No step depends on the order of atomics (counts
// only).  Up to kAlone choices take one workgroup and one launch; more take a
// count, a scan over the workgroups' counts (one wavefront per expert) and a
// ranking launch.  Up to kFew choices (a decoding batch, bound by launches) are
// not sorted at all: the workgroups that move the rows count for themselves
// the keys, expert then choice, below each of their own (permute_few).
//
// Rows.  All three row kernels go token by token, so that a token's row of x
// or dout is read once for all its choices; HBM bound (8192 tokens, 4 choices, h =
// 4096: unpermute 52 us, 6.4 TB/s), but for the gradient of narrow rows.
#include <algorithm>

#include "layer_device.hpp"
#include "layer_kernels.hpp"

namespace mc2 {
namespace {

// Choices that one workgroup sorts alone, and choices per workgroup where there
// are more.  32768 choices with their rows (h = 4096): chunks of 8192 / 4096 /
// 2048 / 1024 take 68 / 64 / 62 / 61 us; 524288 choices (h = 64) 46 / 43 / 46 /
// 56.  2048 or 8192 choices alone: 13 us a call, 20 in three launches.
constexpr int kAlone = 8192, kChunk = 2048;
// Workgroups that walk the tokens of the gradient: enough to fill the CUs
// once.  More in flight only scatter the rows read and written at a time:
// 8192 tokens, 4 choices, h = 4096: 1024 workgroups 125 us, 2048 130, 4096
// 139, one per token 142; 256 are too few (181).
constexpr int kGradBlocks = 1024;
constexpr int kZeroBlocks = 64;  // workgroups that clear the rows of no choice

__device__ __forceinline__ int expert_of(const int32_t* ids, int64_t i, int64_t end, int experts) {
  if (i >= end) return -1;
  const int e = ids[i];
  return e >= 0 && e < experts ? e : -1;
}

// Segment of this wavefront within the workgroup's choices [begin, end).
struct Segment {
  int64_t first, last;
  __device__ __forceinline__ Segment(int64_t begin, int64_t end) {
    const int waves = blockDim.x / 64, w = threadIdx.x / 64;
    const int64_t per = ((end - begin + waves - 1) / waves + 63) / 64 * 64;
    first = begin + w * per;
    last = first + per < end ? first + per : end;
  }
};

// count[w][e] of every wavefront (zeroed here); ends with a barrier.
__device__ __forceinline__ void count_segments(const int32_t* ids, int64_t begin, int64_t end, int experts,
                                               unsigned* count) {
  const int waves = blockDim.x / 64, w = threadIdx.x / 64, lane = threadIdx.x % 64;
  for (int i = threadIdx.x; i < waves * experts; i += blockDim.x) count[i] = 0;
  __syncthreads();
  const Segment seg(begin, end);
  for (int64_t i = seg.first + lane; i < seg.last; i += 64) {
    const int e = expert_of(ids, i, end, experts);
    if (e >= 0) atomicAdd(&count[w * experts + e], 1u);
  }
  __syncthreads();
}

// Rows of this wavefront's choices; base = its row of count, holding the row
// of the segment's first choice of each expert.
__device__ __forceinline__ void rank_segment(const int32_t* ids, int64_t begin, int64_t end, int experts,
                                             volatile unsigned* base, int32_t* row_map) {
  const int lane = threadIdx.x % 64;
  const Segment seg(begin, end);
  int bits = 0;
  while ((1 << bits) < experts) bits++;
  for (int64_t i0 = seg.first; i0 < seg.last; i0 += 64) {
    const int64_t i = i0 + lane;
    const int e = expert_of(ids, i, end, experts);
    unsigned long long same = __ballot(e >= 0);
    for (int b = 0; b < bits; b++) {
      const unsigned long long m = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? m : ~m;
    }
    if (e >= 0) {
      const int before = __popcll(same & ((1ull << lane) - 1));
      const unsigned first = base[e];
      __builtin_amdgcn_wave_barrier();
      if (before == 0) base[e] = first + (unsigned)__popcll(same);
      row_map[i] = (int32_t)(first + before);
    } else if (i < end) {
      row_map[i] = -1;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Exclusive sums of total[0 .. experts) by the first wavefront, in place;
// also written to offsets with the grand total.  Starts and ends with a barrier.
__device__ __forceinline__ void scan_experts(unsigned* total, int experts, int32_t* offsets) {
  __syncthreads();
  if (threadIdx.x < 64) {
    unsigned run = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
      const int e = e0 + threadIdx.x;
      const unsigned own = e < experts ? total[e] : 0u;
      unsigned incl = own;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const unsigned v = __shfl_up(incl, d);
        if ((int)threadIdx.x >= d) incl += v;
      }
      if (e < experts) {
        total[e] = run + incl - own;
        offsets[e] = (int32_t)(run + incl - own);
      }
      run += __shfl(incl, 63);
    }
    if (threadIdx.x == 0) offsets[experts] = (int32_t)run;
  }
  __syncthreads();
}

// One workgroup: the whole sort.  LDS: count[waves][experts], total[experts].
__global__ __launch_bounds__(1024) void sort_one(const int32_t* ids, int64_t n, int experts, int32_t* row_map,
                                                 int32_t* offsets) {
  extern __shared__ unsigned lds[];
  const int waves = blockDim.x / 64;
  unsigned* count = lds;
  unsigned* total = lds + waves * experts;
  count_segments(ids, 0, n, experts, count);
  for (int e = threadIdx.x; e < experts; e += blockDim.x) {
    unsigned s = 0;
    for (int w = 0; w < waves; w++) s += count[w * experts + e];
    total[e] = s;
  }
  scan_experts(total, experts, offsets);
  for (int e = threadIdx.x; e < experts; e += blockDim.x) {
    unsigned run = total[e];
    for (int w = 0; w < waves; w++) {
      const unsigned c = count[w * experts + e];
      count[w * experts + e] = run;
      run += c;
    }
  }
  __syncthreads();
  rank_segment(ids, 0, n, experts, count + (threadIdx.x / 64) * experts, row_map);
}

// Several workgroups: hist[e][b] = choices of expert e in workgroup b.
__global__ __launch_bounds__(1024) void sort_count(const int32_t* ids, int64_t n, int experts, int32_t* hist) {
  extern __shared__ unsigned lds[];
  const int waves = blockDim.x / 64;
  const int64_t begin = (int64_t)blockIdx.x * kChunk, end = begin + kChunk < n ? begin + kChunk : n;
  count_segments(ids, begin, end, experts, lds);
  for (int e = threadIdx.x; e < experts; e += blockDim.x) {
    unsigned s = 0;
    for (int w = 0; w < waves; w++) s += lds[w * experts + e];
    hist[(int64_t)e * gridDim.x + blockIdx.x] = (int32_t)s;
  }
}

// hist[e][b] becomes the choices of e in workgroups before b; offsets.
__global__ __launch_bounds__(1024) void sort_scan(int32_t* hist, int64_t blocks, int experts, int32_t* offsets) {
  extern __shared__ unsigned lds[];
  const int waves = blockDim.x / 64, w = threadIdx.x / 64, lane = threadIdx.x % 64;
  for (int e = w; e < experts; e += waves) {
    int32_t* h = hist + (int64_t)e * blocks;
    unsigned run = 0;
    for (int64_t b0 = 0; b0 < blocks; b0 += 64) {
      const int64_t b = b0 + lane;
      const unsigned own = b < blocks ? (unsigned)h[b] : 0u;
      unsigned incl = own;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const unsigned v = __shfl_up(incl, d);
        if (lane >= d) incl += v;
      }
      if (b < blocks) h[b] = (int32_t)(run + incl - own);
      run += __shfl(incl, 63);
    }
    if (lane == 0) lds[e] = run;
  }
  scan_experts(lds, experts, offsets);
}

__global__ __launch_bounds__(1024) void sort_rank(const int32_t* ids, int64_t n, int experts, const int32_t* hist,
                                                  const int32_t* offsets, int32_t* row_map) {
  extern __shared__ unsigned lds[];
  const int waves = blockDim.x / 64;
  const int64_t begin = (int64_t)blockIdx.x * kChunk, end = begin + kChunk < n ? begin + kChunk : n;
  count_segments(ids, begin, end, experts, lds);
  for (int e = threadIdx.x; e < experts; e += blockDim.x) {
    unsigned run = (unsigned)(offsets[e] + hist[(int64_t)e * gridDim.x + blockIdx.x]);
    for (int w = 0; w < waves; w++) {
      const unsigned c = lds[w * experts + e];
      lds[w * experts + e] = run;
      run += c;
    }
  }
  __syncthreads();
  rank_segment(ids, begin, end, experts, lds + (threadIdx.x / 64) * experts, row_map);
}

// Clears rows [first, rows) of a (rows, h) matrix; workgroup b of `blocks`.
template <bool VEC>
__device__ __forceinline__ void zero_rows(uint16_t* p, int64_t first, int64_t rows, int64_t h, int64_t b,
                                          int64_t blocks) {
  for (int64_t r = first + b; r < rows; r += blocks)
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < h; c += 8 * (int64_t)blockDim.x)
      store_chunk<VEC, false>(p + r * h, c, h, u32x4{0u, 0u, 0u, 0u});
}

// Threads that share a row: a power of two up to the workgroup of 256.
int row_threads(int64_t h) {
  const int64_t chunks = (h + 7) / 8;
  int t = 8;
  while (t < 256 && t < chunks) t *= 2;
  return t;
}

// The whole of a small permute: no counting sort, no second launch.  Every
// wavefront holds the keys e kFew + i of all choices, 64 R at most, in
// registers; row(i) is the number of keys below i's, by R ballots, and
// offsets[e] that below e kFew.  Threads, rows and clearing as permute_rows,
// with a wavefront or more per row.  16 tokens, 4 choices, 64 experts, h =
// 4096: 3.7 us, 7.9 with a sort before; a call 10.6 us, 13.3.  1024 choices of
// 1024 tokens, h = 7168, where every workgroup reads all ids for little work,
// 14.7 us a call, 13.5.
constexpr int kFew = 1024;
template <bool VEC, int R>
__global__ __launch_bounds__(256) void permute_few(PermuteArgs a, int tpr, int token_blocks) {
  __shared__ int rows[kFew];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int n = (int)(a.tokens * a.top), experts = (int)a.experts, top = (int)a.top;
  const int64_t h = a.h;
  uint16_t* out = static_cast<uint16_t*>(a.out);
  auto key_of = [&](int i) {
    const int e = expert_of(a.ids, i, n, experts);
    return e < 0 ? 0x7FFFFFFF : e * kFew + i;
  };
  int key[R];
#pragma unroll
  for (int r = 0; r < R; r++) key[r] = key_of(64 * r + lane);
  auto below = [&](int k) {
    int c = 0;
#pragma unroll
    for (int r = 0; r < R; r++) c += __popcll(__ballot(key[r] < k));
    return c;
  };
  if ((int)blockIdx.x >= token_blocks) {
    if (blockIdx.y > 0) return;
    const int b = (int)blockIdx.x - token_blocks;
    for (int e = 4 * b + wave; e <= experts; e += 4 * kZeroBlocks) {
      const int c = below(e * kFew);
      if (lane == 0) a.offsets[e] = c;
    }
    zero_rows<VEC>(out, below(0x7FFFFFFF), n, h, b, kZeroBlocks);
    return;
  }
  const int per = 256 / tpr, t0 = (int)blockIdx.x * per, own = threadIdx.x / tpr;
  const int64_t c = 8 * ((int64_t)blockIdx.y * tpr + threadIdx.x % tpr);
  const bool on = t0 + own < a.tokens && c < h;
  u32x4 v = {0u, 0u, 0u, 0u};
  if (on) v = load_chunk<VEC>(static_cast<const uint16_t*>(a.x) + (t0 + own) * h, c, h);
  const int first = t0 * top, count = min(per * top, n - first);
  for (int q = threadIdx.x; q < count; q += 256) rows[q] = key_of(first + q);
  __syncthreads();
  for (int q = wave; q < count; q += 4) {
    const int k = __builtin_amdgcn_readfirstlane(rows[q]), r = k == 0x7FFFFFFF ? -1 : below(k);
    if (lane == 0) {
      rows[q] = r;
      if (blockIdx.y == 0) a.row_map[first + q] = r;
    }
  }
  __syncthreads();
  if (!on) return;
  for (int j = 0; j < top; j++) {
    const int64_t r = rows[own * top + j];
    if (r >= 0) store_chunk<VEC, true>(out + r * h, c, h, v);
  }
}

// out row row_map[t][j] = x row t.  TPR threads per row, one chunk each; grid
// (tokens / (256 / TPR) + kZeroBlocks, chunks / TPR).
template <bool VEC>
__global__ __launch_bounds__(256) void permute_rows(PermuteArgs a, int tpr, int64_t token_blocks) {
  uint16_t* out = static_cast<uint16_t*>(a.out);
  const int64_t h = a.h;
  if (blockIdx.x >= token_blocks) {
    if (blockIdx.y == 0)
      zero_rows<VEC>(out, a.offsets[a.experts], a.tokens * a.top, h, blockIdx.x - token_blocks, kZeroBlocks);
    return;
  }
  const int64_t t = (int64_t)blockIdx.x * (256 / tpr) + threadIdx.x / tpr;
  const int64_t c = 8 * ((int64_t)blockIdx.y * tpr + threadIdx.x % tpr);
  if (t >= a.tokens || c >= h) return;
  const u32x4 v = load_chunk<VEC>(static_cast<const uint16_t*>(a.x) + t * h, c, h);
  const int32_t* map = a.row_map + t * a.top;
  for (int64_t j = 0; j < a.top; j++) {
    const int64_t r = map[j];
    if (r >= 0) store_chunk<VEC, true>(out + r * h, c, h, v);
  }
}

// out[t] = sum over j of weights[t][j] y[row_map[t][j]]; grid as permute_rows
// without the clearing workgroups.  The loads of JB choices are in flight
// together.
template <int DT, bool VEC, int JB>
__global__ __launch_bounds__(256) void unpermute_rows(UnpermuteArgs a, int tpr) {
  const int64_t h = a.h;
  const int64_t t = (int64_t)blockIdx.x * (256 / tpr) + threadIdx.x / tpr;
  const int64_t c = 8 * ((int64_t)blockIdx.y * tpr + threadIdx.x % tpr);
  if (t >= a.tokens || c >= h) return;
  const int32_t* map = a.row_map + t * a.top;
  const float* weights = a.weights ? a.weights + t * a.top : nullptr;
  const uint16_t* y = static_cast<const uint16_t*>(a.y);
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t j0 = 0; j0 < a.top; j0 += JB) {
    u32x4 v[JB];
    float w[JB];
    bool on[JB];
#pragma unroll
    for (int j = 0; j < JB; j++) {
      const int64_t r = j0 + j < a.top ? map[j0 + j] : -1;
      on[j] = r >= 0 && r < a.rows;
      w[j] = on[j] ? (weights ? weights[j0 + j] : 1.0f) : 0.0f;
      v[j] = u32x4{0u, 0u, 0u, 0u};
      if (on[j]) v[j] = load_chunk<VEC>(y + r * h, c, h);
    }
#pragma unroll
    for (int j = 0; j < JB; j++) {
      float f[8];
      unpack8<DT>(v[j], f);
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (on[j]) s[e] = __builtin_fmaf(w[j], f[e], s[e]);
    }
  }
  store_chunk<VEC, true>(static_cast<uint16_t*>(a.out) + t * h, c, h, pack8<DT>(s));
}

// Gradients: a token's dout row goes to its choices' rows of dy, scaled, and
// its products with their rows of y are summed over the row.  TPR threads per
// token (64: a wavefront, no barrier; 256: the workgroup), JB choices at a
// time.  The last kZeroBlocks workgroups count the kept choices and clear the
// rows of dy past them.  Each counts the whole map, 128 loads a thread for 8192
// tokens of 4 choices with few in flight: h = 64 takes 20 us, 256 23, where the
// rows alone are 2 to 7; 512 40, 1024 49, 2048 58 (5.2 TB/s), 4096 124.
template <int DT, bool VEC, int TPR, int JB>
__global__ __launch_bounds__(256) void unpermute_grad(UnpermuteArgs a, int64_t token_blocks) {
  constexpr int WAVES = TPR / 64;
  __shared__ float red[2][JB][WAVES];
  __shared__ unsigned kept[4];
  const int64_t h = a.h;
  uint16_t* dy = static_cast<uint16_t*>(a.dy);
  if (blockIdx.x >= token_blocks) {
    if (!dy) return;
    unsigned n = 0;
    for (int64_t i = threadIdx.x; i < a.tokens * a.top; i += 256) {
      const int64_t r = a.row_map[i];
      n += r >= 0 && r < a.rows;
    }
    for (int d = 1; d < 64; d *= 2) n += __shfl_xor(n, d);
    if (threadIdx.x % 64 == 0) kept[threadIdx.x / 64] = n;
    __syncthreads();
    zero_rows<VEC>(dy, (int64_t)kept[0] + kept[1] + kept[2] + kept[3], a.rows, h, blockIdx.x - token_blocks,
                   kZeroBlocks);
    return;
  }
  const int lane = threadIdx.x % TPR;
  const uint16_t* y = static_cast<const uint16_t*>(a.y);
  int turn = 0;
  const int64_t step = token_blocks * (256 / TPR);
  for (int64_t t = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR; t < a.tokens; t += step) {
    const int32_t* map = a.row_map + t * a.top;
    const uint16_t* dout = static_cast<const uint16_t*>(a.dout) + t * h;
    for (int64_t j0 = 0; j0 < a.top; j0 += JB, turn ^= 1) {
      int64_t r[JB];
      float w[JB], dot[JB];
#pragma unroll
      for (int j = 0; j < JB; j++) {
        r[j] = j0 + j < a.top ? map[j0 + j] : -1;
        if (r[j] >= a.rows) r[j] = -1;
        w[j] = r[j] >= 0 ? (a.weights ? a.weights[t * a.top + j0 + j] : 1.0f) : 0.0f;
        dot[j] = 0.0f;
      }
      for (int64_t c = 8 * lane; c < h; c += 8 * TPR) {
        const u32x4 vd = load_chunk<VEC>(dout, c, h);
        u32x4 vy[JB];
#pragma unroll
        for (int j = 0; j < JB; j++) {
          vy[j] = u32x4{0u, 0u, 0u, 0u};
          if (a.dweights && r[j] >= 0) vy[j] = load_chunk<VEC>(y + r[j] * h, c, h);
        }
        float d[8];
        unpack8<DT>(vd, d);
#pragma unroll
        for (int j = 0; j < JB; j++) {
          float f[8], g[8];
          unpack8<DT>(vy[j], f);
#pragma unroll
          for (int e = 0; e < 8; e++) {
            dot[j] = __builtin_fmaf(f[e], d[e], dot[j]);
            g[e] = w[j] * d[e];
          }
          if (dy && r[j] >= 0) store_chunk<VEC, true>(dy + r[j] * h, c, h, pack8<DT>(g));
        }
      }
      if (a.dweights) {
#pragma unroll
        for (int j = 0; j < JB; j++) {
          dot[j] = wave_sum(dot[j]);
          if (WAVES > 1 && threadIdx.x % 64 == 0) red[turn][j][threadIdx.x / 64] = dot[j];
        }
        if constexpr (WAVES > 1) {
          __syncthreads();
#pragma unroll
          for (int j = 0; j < JB; j++) {
            dot[j] = red[turn][j][0];
#pragma unroll
            for (int v = 1; v < WAVES; v++) dot[j] += red[turn][j][v];
          }
        }
        if (lane == 0) {
#pragma unroll
          for (int j = 0; j < JB; j++)
            if (j0 + j < a.top) a.dweights[t * a.top + j0 + j] = r[j] >= 0 ? dot[j] : 0.0f;
        }
      }
    }
  }
}

int64_t sort_blocks(int64_t n) { return n <= kAlone ? 1 : (n + kChunk - 1) / kChunk; }

template <int DT, bool VEC>
hipError_t unpermute_launch(const UnpermuteArgs& a, hipStream_t s) {
  const int tpr = row_threads(a.h);
  const dim3 grid((unsigned)((a.tokens + 256 / tpr - 1) / (256 / tpr)), (unsigned)(((a.h + 7) / 8 + tpr - 1) / tpr));
  if (a.top == 1) unpermute_rows<DT, VEC, 1><<<grid, 256, 0, s>>>(a, tpr);
  else if (a.top == 2) unpermute_rows<DT, VEC, 2><<<grid, 256, 0, s>>>(a, tpr);
  else unpermute_rows<DT, VEC, 4><<<grid, 256, 0, s>>>(a, tpr);
  return hipGetLastError();
}

template <int DT, bool VEC, int TPR>
hipError_t unpermute_grad_launch(const UnpermuteArgs& a, hipStream_t s) {
  const int64_t blocks = std::min<int64_t>((a.tokens + 256 / TPR - 1) / (256 / TPR), kGradBlocks);
  const unsigned grid = (unsigned)(blocks + kZeroBlocks);
  if (a.top == 1) unpermute_grad<DT, VEC, TPR, 1><<<grid, 256, 0, s>>>(a, blocks);
  else if (a.top == 2) unpermute_grad<DT, VEC, TPR, 2><<<grid, 256, 0, s>>>(a, blocks);
  else unpermute_grad<DT, VEC, TPR, 4><<<grid, 256, 0, s>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace

size_t moe_permute_workspace(int64_t choices, int64_t experts) {
  const int64_t blocks = sort_blocks(choices);
  return blocks > 1 ? (size_t)(blocks * experts) * sizeof(int32_t) : 0;
}

hipError_t launch_moe_permute(const PermuteArgs& a, hipStream_t s) {
  const int64_t n = a.tokens * a.top, blocks = sort_blocks(n);
  const int experts = (int)a.experts;
  if (n <= kFew) {
    const int tpr = std::max(row_threads(a.h), 64), per = 256 / tpr;
    const int token_blocks = n == 0 ? 0 : (int)((a.tokens + per - 1) / per);
    const dim3 grid((unsigned)(token_blocks + kZeroBlocks), (unsigned)(((a.h + 7) / 8 + tpr - 1) / tpr));
    const bool vec = a.h % 8 == 0;
    if (n <= 256) {
      if (vec) permute_few<true, 4><<<grid, 256, 0, s>>>(a, tpr, token_blocks);
      else permute_few<false, 4><<<grid, 256, 0, s>>>(a, tpr, token_blocks);
    } else {
      if (vec) permute_few<true, kFew / 64><<<grid, 256, 0, s>>>(a, tpr, token_blocks);
      else permute_few<false, kFew / 64><<<grid, 256, 0, s>>>(a, tpr, token_blocks);
    }
    return hipGetLastError();
  }
  // counts of each wavefront's segment per expert, and the totals, in 64 KB of
  // LDS: 16 wavefronts up to 963 experts, 3 with 4096
  const int threads = 64 * std::min(16, 16384 / experts - 1);
  const size_t lds = (size_t)(threads / 64 + 1) * experts * sizeof(unsigned);
  if (blocks <= 1) {
    sort_one<<<1, threads, lds, s>>>(a.ids, n, experts, a.row_map, a.offsets);
  } else {
    sort_count<<<(unsigned)blocks, threads, lds, s>>>(a.ids, n, experts, a.workspace);
    sort_scan<<<1, 1024, (size_t)experts * sizeof(unsigned), s>>>(a.workspace, blocks, experts, a.offsets);
    sort_rank<<<(unsigned)blocks, threads, lds, s>>>(a.ids, n, experts, a.workspace, a.offsets, a.row_map);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int tpr = row_threads(a.h);
  const int64_t token_blocks = (a.tokens + 256 / tpr - 1) / (256 / tpr);
  const dim3 grid((unsigned)(token_blocks + kZeroBlocks), (unsigned)(((a.h + 7) / 8 + tpr - 1) / tpr));
  if (a.h % 8 == 0) permute_rows<true><<<grid, 256, 0, s>>>(a, tpr, token_blocks);
  else permute_rows<false><<<grid, 256, 0, s>>>(a, tpr, token_blocks);
  return hipGetLastError();
}

hipError_t launch_moe_unpermute(const UnpermuteArgs& a, hipStream_t s) {
  if (a.tokens < 1 || a.top < 1 || a.h < 1 || (a.dtype != DT_BF16 && a.dtype != DT_F16)) return hipErrorInvalidValue;
  const bool vec = a.h % 8 == 0;
  if (a.dtype == DT_BF16)
    return vec ? unpermute_launch<DT_BF16, true>(a, s) : unpermute_launch<DT_BF16, false>(a, s);
  return vec ? unpermute_launch<DT_F16, true>(a, s) : unpermute_launch<DT_F16, false>(a, s);
}

template <int DT, bool VEC>
static hipError_t unpermute_grad_dt(const UnpermuteArgs& a, hipStream_t s) {
  return a.h <= 1024 ? unpermute_grad_launch<DT, VEC, 64>(a, s) : unpermute_grad_launch<DT, VEC, 256>(a, s);
}
hipError_t launch_moe_unpermute_grad(const UnpermuteArgs& a, hipStream_t s) {
  if (a.tokens < 0 || a.top < 1 || a.h < 1 || (a.dtype != DT_BF16 && a.dtype != DT_F16)) return hipErrorInvalidValue;
  const bool vec = a.h % 8 == 0;
  if (a.dtype == DT_BF16) return vec ? unpermute_grad_dt<DT_BF16, true>(a, s) : unpermute_grad_dt<DT_BF16, false>(a, s);
  return vec ? unpermute_grad_dt<DT_F16, true>(a, s) : unpermute_grad_dt<DT_F16, false>(a, s);
}

}  // namespace mc2
