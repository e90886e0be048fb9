// K13: the router of a mixture-of-experts layer and its gradient.
//
//   p = softmax(l) or sigmoid(l), c = p + bias; the top largest c of the kept
//   groups; weights = scale p (/ the sum of the chosen p)
//
// A team of TEAM lanes takes a token: lane i of it holds the logits i, i +
// TEAM, ... in SLOTS registers.  The choice goes by rounds (pick): the team's
// largest key, the lowest expert that has it, on to those below.  Teams of 16
// lanes (up to 256 experts and 16 choices) reduce by DPP alone, four tokens at a
// time; larger ones take a wavefront.  Bound by these instructions and their
// latency, not by memory (8.4 MB at the copy's rate would take 2 us): 8191
// tokens x 256 fp32 logits, top 8: 6.6 us in a graph of such calls, where an
// empty kernel takes 3; with bias 8.9, with 16 groups of which 6 are kept too
// 12.4.  (A wavefront a token, its rounds by ballots: 8.6 and 19; loads each
// under a condition, which are waited for one by one: 11 and 22.)
//
// Order.  Without a bias the keys are the logits themselves: p rises with l,
// so no score is formed but those of the chosen.  Otherwise c is formed in
// fp32 with an error bound (Doubt).  Where two neighbours of the order lie
// within it, a tie among them, fp64 decides: on the chosen and the next few
// alone where that is enough (order64), else on the whole row (choose64), 3
// us for the few rows of a batch that need it (8191 rows of equal logits: 23).  So
// the experts chosen are those of fp64, at fp32's cost; bf16 logits under a
// bias of zeros, which tie in many rows, take 10 us.
#include "layer8_kernels.hpp"
#include "layer_device.hpp"

namespace mc2 {
namespace {

constexpr float kLog2eHi = 1.44269504088896340736f;
constexpr float kLog2eLo = 1.925963033500e-8f;  // log2(e) - kLog2eHi
constexpr float kLn2 = 0.693147180559945309417f;
constexpr uint32_t kOff = 0;                    // key of an expert that is off; all others are larger

// exp(x) within 2^-22: the argument in base 2 to twice fp32's precision (x log2(e)
// rounded alone is off by |x| 2^-24).  Past +-200 it is 0 or infinite in fp32.
// The instruction gives no subnormal numbers: below 2^-126 e is 0, or with LOW
// formed at 2^64 times its size and scaled down (t + 64 is exact).
template <bool LOW = false>
__device__ __forceinline__ float exp_near(float x) {
  x = __builtin_amdgcn_fmed3f(x, -200.0f, 200.0f);
  const float t = x * kLog2eHi;
  const float lo = __builtin_fmaf(x, kLog2eLo, __builtin_fmaf(x, kLog2eHi, -t));
  const bool low = LOW && t < -125.0f;
  float e = __builtin_amdgcn_exp2f(low ? t + 64.0f : t);
  e = e < __builtin_inff() ? __builtin_fmaf(e * kLn2, lo, e) : e;
  return low ? e * 0x1p-64f : e;
}

// sigmoid(v) = 1 / (1 + exp(-v)) from the exponential of the sign that keeps it
// exact: for v < 0 exp(v) / (1 + exp(v)).  `base`, 0 or less, scales it by
// exp(-base): the largest of a token's chosen logits where all of them lie below
// 0, so that their shares of each other are those of numbers of ordinary size,
// whatever is left of the sigmoids themselves in fp32 (for v > 0 base is 0).
// rest: 1 - sigmoid(v), not scaled.
struct Sigmoid {
  float p, rest;
  static __device__ __forceinline__ Sigmoid of(float v, float base) {
    const float e = exp_near(-__builtin_fabsf(v)), big = 1.0f / (1.0f + e);
    return v < 0.0f ? Sigmoid{exp_near<true>(v - base) * big, big} : Sigmoid{big, e * big};
  }
};
constexpr float kNoSigmoid = -709.7827f;  // below it 1 / (1 + exp(-v)) is 0 in fp64 too, and so is the share

template <int DT>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
  if constexpr (DT == DT_F32) return static_cast<const float*>(p)[i];
  else return dec16<DT>(static_cast<const uint16_t*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void store_logit(void* p, int64_t i, float f) {
  if constexpr (DT == DT_F32) static_cast<float*>(p)[i] = f;
  else static_cast<uint16_t*>(p)[i] = enc16<DT>(f);
}

// Floats in an order of unsigned integers (no NaN; -0 has been added to 0).
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }

// Maximum over the team, in all of its lanes.
template <int TEAM>
__device__ __forceinline__ uint32_t team_max(uint32_t v) {
  v = max16(v);
  if constexpr (TEAM == 64) {
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16),
                   c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    v = max(max(a, b), max(c, d));
  }
  return v;
}
// The team's first lane that says `is` (some lane does).
template <int TEAM>
__device__ __forceinline__ int first_lane(bool is) {
  const unsigned long long at = __ballot(is);
  if constexpr (TEAM == 64) return __ffsll((long long)at) - 1;
  const int wlane = threadIdx.x % 64;
  const uint32_t half = wlane & 32 ? (uint32_t)(at >> 32) : (uint32_t)at;
  return __ffs((int)(half >> (wlane & 16) & 0xFFFFu)) - 1;
}
template <int TEAM>
__device__ __forceinline__ float team_sum(float v) {
  if constexpr (TEAM == 64) return wave_sum(v);
  v += __uint_as_float(dpp16<0>(__float_as_uint(v)));
  v += __uint_as_float(dpp16<1>(__float_as_uint(v)));
  v += __uint_as_float(dpp16<2>(__float_as_uint(v)));
  return v + __uint_as_float(dpp16<3>(__float_as_uint(v)));
}
template <int STEP>
__device__ __forceinline__ double dpp16d(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{dpp16<STEP>(b[0]), dpp16<STEP>(b[1])});
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_readlane((int)b[0], lane),
                                          (uint32_t)__builtin_amdgcn_readlane((int)b[1], lane)});
}
// f over the wavefront's doubles, as a scalar.
template <typename F>
__device__ __forceinline__ double wave_fold(double v, F f) {
  v = f(v, dpp16d<0>(v));
  v = f(v, dpp16d<1>(v));
  v = f(v, dpp16d<2>(v));
  v = f(v, dpp16d<3>(v));
  return f(f(lane_value(v, 0), lane_value(v, 16)), f(lane_value(v, 32), lane_value(v, 48)));
}

// What rounding can move between two values that are compared.  p of a
// softmax: its exponential, the sum's additions (SLOTS and 6 in a row) and a
// product, relative to p, of which 1 / sum is the largest; of a sigmoid:
// 2^-22 at most.  Twice that for two values, twice more for sums of two; and
// the additions' own roundings, relative to the values (of sums: Two::slack).
struct Doubt {
  float abs, rel;
  __device__ __forceinline__ bool operator()(float a, float b) const {  // a >= b: not surely a > b
    return !(a - b > abs + rel * fmaxf(__builtin_fabsf(a), __builtin_fabsf(b)));
  }
};

// The top largest keys, equal ones from the lowest expert on: lane j < top of
// the team gets the j-th's expert (-1: none left); so do lanes up to count where
// the set of the first top is not sure but that of the first count is.
//
// A key's last bits (as many as number the registers) give way to its
// register's number, counted down.  So the keys of a lane differ, and what a lane
// has left are those below the last one taken from it: its largest is found
// by a subtraction and half a minimum each, nothing is marked as taken, and the
// round's key names its register.  For keys that then agree in the bits above
// (CHECK: that doubt says may be either way round) the order is not known.
// exact: those bits said nothing, so keys that agree are equal.
template <int SLOTS>
constexpr uint32_t slot_bits() {
  uint32_t n = 0;
  while ((1 << n) < SLOTS) n++;
  return n;
}
enum : int { SURE = 0, ORDER = 1, CHOICE = 2 };  // pick's doubt: none, the order of the first count alone, which they are
template <int TEAM, int SLOTS, bool CHECK>
__device__ __forceinline__ int pick(const uint32_t (&given)[SLOTS], int top, Doubt doubt, bool exact, int& id, int& count) {
  constexpr uint32_t kMask = (1u << slot_bits<SLOTS>()) - 1;
  const int lane = threadIdx.x % TEAM;
  uint32_t key[SLOTS], below = 0xFFFFFFFFu, best, m = kOff, mine = kOff;
#pragma unroll
  for (int s = 0; s < SLOTS; s++) key[s] = given[s] == kOff ? kOff : (given[s] & ~kMask) | (kMask - s);
  id = -1;
  count = top;
  auto largest = [&] {
    // distance from `below` down to the nearest key under it; one that is not under it is further than any that is
    uint32_t near = below - 1;
#pragma unroll
    for (int s = 0; s < SLOTS; s++) near = min(near, below - 1 - key[s]);
    best = below - 1 - near;
    return team_max<TEAM>(best);
  };
  auto take = [&](int j) {
    const int l = first_lane<TEAM>(best == m);
    if (lane == l && m != kOff) below = m;
    if (lane == j) {
      mine = m;
      id = m == kOff ? -1 : l + TEAM * (int)(kMask - (m & kMask));
    }
  };
  for (int j = 0; j < top; j++) {
    m = largest();
    take(j);
  }
  if (!CHECK && exact) return SURE;
  auto open = [&](uint32_t a, uint32_t b) {  // a the larger
    if (b == kOff) return false;
    return CHECK ? doubt(of_key(a & ~kMask), of_key(b & ~kMask)) : ((a ^ b) & ~kMask) == 0;
  };
  uint32_t next = largest();
  bool edge = open(m, next);
  // where the last and the next are in doubt, up to four more, until two are not
  for (; __ballot(edge) && count < TEAM && count < top + 4; count++) {
    m = next;
    take(count);
    next = largest();
    edge = edge && open(m, next);
  }
  // each lane's key against the one before it (wave_shr 1, or within rows of 16)
  const uint32_t before = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mine, TEAM == 64 ? 0x138 : 0x111, 0xF, 0xF, false);
  const bool here = lane > 0 && lane < count && open(before, mine);
  return edge ? CHOICE : team_max<TEAM>(here ? 1 : 0) ? ORDER : SURE;
}

// Two largest of the values seen.
template <typename T>
struct Two {
  T a, b;
  __device__ __forceinline__ void add(T v) {
    b = fmax(b, fmin(a, v));
    a = fmax(a, v);
  }
  __device__ __forceinline__ void join(T c, T d) {
    b = fmax(fmax(b, d), fmin(a, c));
    a = fmax(a, c);
  }
  // What fp32's roundings of the two and of their sum can be at most: relative to
  // the terms, which may cancel (2^-23 of both, and half of that for the compared
  // numbers' own).
  __device__ __forceinline__ T slack(int group_top) const {
    const T one = (T)0x1p-22 * fabs(a);
    return group_top != 2 || !(b > -__builtin_inf()) ? one : one + (T)0x1p-22 * fabs(b);
  }
  // (a sum past fp32's lowest number is that number, a group still; equal ones are in doubt)
  __device__ __forceinline__ T value(int group_top) const {
    if (group_top != 2 || !(b > -__builtin_inf())) return a;
    return sizeof(T) == 4 ? fmax(a + b, (T)-3.402823466e38f) : a + b;
  }
};

// The groups of a lane's experts: (e + 0.5) / per in fp32 is off by less than
// 2^-10 / per, and no nearer to a whole number than 0.5 / per.
template <int TEAM, int SLOTS>
__device__ __forceinline__ void groups_of(float inv_per, int (&group)[SLOTS]) {
  const float first = ((float)(int)(threadIdx.x % TEAM) + 0.5f) * inv_per;
#pragma unroll
  for (int s = 0; s < SLOTS; s++) group[s] = (int)__builtin_fmaf((float)(TEAM * s), inv_per, first);
}

// How groups are spread: 2^shift lanes of the team share one (one where there
// are more than half as many as lanes); a lane's i-th group is i TEAM / 2^shift
// past its first.  In LDS a token has its groups' values, `quads` of four, their
// slack, as many, then its scores, a row of per or per + 1 for each group: odd,
// so that the rows start in different banks (odd_mask: -1 where one is added);
// then a place that is written only.
struct Spread {
  int per, odd_mask, quads, shift, size;  // size: numbers that a token takes, a multiple of four
  float inv_per;
};
// Scores into their places.
template <int TEAM, int SLOTS, typename T, typename F>
__device__ __forceinline__ void lay_out(const RouteArgs& a, const Spread& sp, const int (&group)[SLOTS], T* mine, F score) {
  const int lane = threadIdx.x % TEAM;
#pragma unroll
  for (int s = 0; s < SLOTS; s++) {
    const int e = lane + TEAM * s, at = 8 * sp.quads + e + (group[s] & sp.odd_mask);
    mine[e < a.experts ? at : sp.size - 1] = score(s);
  }
}

// The groups kept, as a mask (bit g, the same in the team's lanes), from the
// team's scores at[s] in `mine`, which no other team touches.  For the lane's
// own groups `least` and `most` become the smallest value kept and the largest
// dropped; in fp32 what they may be at least and at most.
template <int TEAM, typename T>
__device__ __forceinline__ unsigned long long keep_groups(const RouteArgs& a, const Spread& sp, T* mine, T& least,
                                                          T& most) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  const int wlane = threadIdx.x % 64, lane = wlane % TEAM;
  const T off = -__builtin_inf();
  constexpr bool kSlack = sizeof(T) == 4;
  const T* scores = mine + 8 * sp.quads;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const int step = 1 << sp.shift, stride = TEAM >> sp.shift, rows = 4 * sp.quads, pitch = sp.per - sp.odd_mask;
  const int part = lane & (step - 1);
  for (int g0 = 0; g0 < rows; g0 += stride) {
    const int g = g0 + (lane >> sp.shift);
    const T* row = scores + min(g, a.groups - 1) * pitch;
    Two<T> t{off, off};
    for (int i = part; i - part < sp.per; i += 8 * step) {  // eight in flight
      T v[8];
#pragma unroll
      for (int u = 0; u < 8; u++) v[u] = row[min(i + u * step, sp.per - 1)];
#pragma unroll
      for (int u = 0; u < 8; u++) t.add(i + u * step < sp.per ? v[u] : off);
    }
    for (int o = 1; o < step; o *= 2) t.join(__shfl_xor(t.a, o), __shfl_xor(t.b, o));
    if (g < rows && part == 0) {
      mine[g] = g < a.groups ? t.value(a.group_top) : off;
      if (kSlack) mine[rows + g] = t.slack(a.group_top);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  unsigned long long kept = 0;
  least = __builtin_inf();
  most = off;
  for (int g0 = 0; g0 < a.groups; g0 += TEAM) {
    const int g = g0 + lane;
    const T v = g < a.groups ? mine[g] : off;
    int rank = 0;
#pragma unroll 4
    for (int o = 0; o < rows; o += 4) {
      const T4 u = *reinterpret_cast<const T4*>(mine + o);
#pragma unroll
      for (int i = 0; i < 4; i++) rank += o + i < g ? u[i] >= v : u[i] > v;
    }
    const bool is = v > off && rank < a.top_groups;
    const T slack = kSlack && g < a.groups ? mine[rows + g] : (T)0;
    if (is) least = fmin(least, v - slack);
    else most = fmax(most, v + slack);  // (of a group that is off NaN, which fmax drops)
    unsigned long long bits = __ballot(is);
    if constexpr (TEAM < 64) bits = bits >> (wlane - lane) & ((1ull << TEAM) - 1);
    kept |= bits << g0;
  }
  return kept;
}
__device__ __forceinline__ bool is_kept(unsigned long long kept, int g) {
  return (g & 32 ? (uint32_t)(kept >> 32) : (uint32_t)kept) >> (g & 31) & 1;
}

template <int TEAM>
__device__ __forceinline__ uint32_t send(uint32_t v, int to) {  // to lane `to` of the team
  const int lane = threadIdx.x % TEAM;
  return (uint32_t)__builtin_amdgcn_ds_permute(4 * (int)(threadIdx.x % 64 - lane + to), (int)v);
}
// The first count of a team in the order of fp64 (their set is right): each
// lane's logit, or its c in fp64, and its place among them.  A softmax's p is
// then that of the fp32 sum, whose error of 2^-17 at most all p share: it moves
// the difference of two c by that part of the difference of their p.  Returns
// whether two neighbours are still in doubt.
template <int TEAM, int DT>
__device__ __forceinline__ bool order64(const RouteArgs& a, int64_t row, int count, float m, float sum, int& id) {
  const int lane = threadIdx.x % TEAM;
  const bool softmax = a.score == SCORE_SOFTMAX;
  float l = 0.0f, b = 0.0f;
  double c = -__builtin_inf(), p = 0.0;
  if (id >= 0) {
    l = logit_at<DT>(a.logits, row + id) + 0.0f;
    c = (double)l;
    if (a.bias) {
      b = a.bias[id];
      p = softmax ? exp(c - (double)m) / (double)sum : 1.0 / (1.0 + exp(-c));
      c = p + (double)b;
    }
  }
  int place = 0;
  for (int j = 0; j < count; j++) {
    const double u = __shfl(c, j, TEAM);
    const int other = __shfl(id, j, TEAM);
    place += u > c || (u == c && other < id);
  }
  const int to = id < 0 ? lane : place;  // (those without an expert come last already)
  id = (int)send<TEAM>((uint32_t)id, to);
  if (!softmax || !a.bias) return false;
  const u32x2 pb = __builtin_bit_cast(u32x2, p), cb = __builtin_bit_cast(u32x2, c);
  p = __builtin_bit_cast(double, u32x2{send<TEAM>(pb[0], to), send<TEAM>(pb[1], to)});
  c = __builtin_bit_cast(double, u32x2{send<TEAM>(cb[0], to), send<TEAM>(cb[1], to)});
  l = __uint_as_float(send<TEAM>(__float_as_uint(l), to));
  b = __uint_as_float(send<TEAM>(__float_as_uint(b), to));
  const int from = lane > 0 ? lane - 1 : 0;
  const double gap = __shfl(c, from, TEAM) - c, apart = fabs(__shfl(p, from, TEAM) - p);
  const bool alike = __shfl(l, from, TEAM) == l && __shfl(b, from, TEAM) == b;  // equal c whatever the sum
  const bool open = lane > 0 && lane < count && id >= 0 && !alike && !(gap > apart * 0x1p-17 + fabs(c) * 0x1p-50);
  return team_max<TEAM>(open ? 1 : 0) != 0;
}

// Whether the choice goes by the logits alone: without a bias, and with one score
// of each group the groups' order is that of the logits too.
__device__ __forceinline__ bool goes_by_logit(const RouteArgs& a) {
  return !a.bias && (a.groups == 1 || a.group_top == 1);
}

// The choice for one token with all scores in fp64, by the whole wavefront;
// `mine` has room for a token's scores.
template <int DT, int SLOTS>
__device__ __forceinline__ int choose64(const RouteArgs& a, int64_t row, const Spread& sp, double* mine) {
  const int lane = threadIdx.x % 64;
  const double off = -__builtin_inf();
  const bool softmax = a.score == SCORE_SOFTMAX;
  auto larger = [](double x, double y) { return fmax(x, y); };
  double c[SLOTS], m = off, sum = 1.0, part = 0.0;
  float l[SLOTS];
#pragma unroll
  for (int s = 0; s < SLOTS; s++) l[s] = logit_at<DT>(a.logits, row + min(lane + 64 * s, a.experts - 1));
#pragma unroll
  for (int s = 0; s < SLOTS; s++) l[s] = lane + 64 * s < a.experts ? l[s] : -__builtin_inff();
  const bool by_logit = goes_by_logit(a);
  if (softmax) {
#pragma unroll
    for (int s = 0; s < SLOTS; s++) m = fmax(m, (double)l[s]);
    m = wave_fold(m, larger);
  }
#pragma unroll
  for (int s = 0; s < SLOTS; s++) {
    c[s] = exp(softmax ? (double)l[s] - m : -(double)l[s]);
    part += c[s];
  }
  if (softmax) sum = wave_fold(part, [](double x, double y) { return x + y; });
#pragma unroll
  for (int s = 0; s < SLOTS; s++) {
    const double v = by_logit ? (double)l[s] :
                     (softmax ? c[s] / sum : 1.0 / (1.0 + c[s])) +
                     (a.bias ? (double)a.bias[min(lane + 64 * s, a.experts - 1)] : 0.0);
    c[s] = l[s] > -__builtin_inff() && v > off ? v : off;  // (a NaN is off)
  }
  if (a.groups > 1) {
    int group[SLOTS];
    groups_of<64>(sp.inv_per, group);
    lay_out<64>(a, sp, group, mine, [&](int s) { return c[s]; });
    double least, most;
    Spread wide = sp;
    wide.shift = 0;
    while ((2 << wide.shift) * a.groups <= 64) wide.shift++;
    const unsigned long long kept = keep_groups<64>(a, wide, mine, least, most);
#pragma unroll
    for (int s = 0; s < SLOTS; s++)
      if (!is_kept(kept, group[s])) c[s] = off;
  }
  if (!a.bias) {
#pragma unroll
    for (int s = 0; s < SLOTS; s++)
      if (c[s] > off) c[s] = (double)l[s];
  }
  int id = -1;
  for (int j = 0; j < a.top; j++) {
    double best = c[0];
#pragma unroll
    for (int s = 1; s < SLOTS; s++) best = fmax(best, c[s]);
    best = wave_fold(best, larger);
    if (best == off) break;
    uint32_t last = 0;  // 4096 less the lowest expert with it
#pragma unroll
    for (int s = SLOTS - 1; s >= 0; s--) last = c[s] == best ? 4096 - 64 * s - lane : last;
    const int won = 4096 - (int)team_max<64>(last);
#pragma unroll
    for (int s = 0; s < SLOTS; s++) c[s] = won - lane == 64 * s ? off : c[s];
    if (lane == j) id = won;
  }
  return id;
}

constexpr int kWaves = 4;  // wavefronts of a workgroup (fewer where the groups' scores would not fit)
constexpr size_t kMostLds = 64 << 10;

template <int DT, int TEAM, int SLOTS>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs a, Spread sp) {
  extern __shared__ __attribute__((aligned(32))) double shared_scores[];
  constexpr int kTeams = 64 / TEAM;  // tokens of a wavefront
  const int wlane = threadIdx.x % 64, wave = threadIdx.x / 64, lane = wlane % TEAM, team = wlane / TEAM;
  const int64_t first = ((int64_t)blockIdx.x * (blockDim.x / 64) + wave) * kTeams, token = first + team;
  if (first >= a.tokens) return;  // (no barrier below)
  const bool there = token < a.tokens, softmax = a.score == SCORE_SOFTMAX;
  const int64_t row = token * a.experts;
  const float ninf = -__builtin_inff();
  float l[SLOTS], b[SLOTS];
  bool wrong = false;
  uint32_t top_key = kOff;
  // Every lane loads, those past the row's end its last logit: a load under a
  // condition would be waited for before the next.
  const int64_t at = (there ? token : a.tokens - 1) * a.experts;
#pragma unroll
  for (int s = 0; s < SLOTS; s++) l[s] = logit_at<DT>(a.logits, at + min(lane + TEAM * s, a.experts - 1));
#pragma unroll
  for (int s = 0; s < SLOTS; s++) b[s] = 0.0f;
  if (a.bias) {
#pragma unroll
    for (int s = 0; s < SLOTS; s++) b[s] = a.bias[min(lane + TEAM * s, a.experts - 1)];
  }
#pragma unroll
  for (int s = 0; s < SLOTS; s++) {
    l[s] = there && lane + TEAM * s < a.experts ? l[s] + 0.0f : ninf;
    wrong |= l[s] != l[s] || (softmax && l[s] == __builtin_inff());
    top_key = max(top_key, l[s] > ninf ? key_of(l[s]) : kOff);
  }
  wrong = team_max<TEAM>(wrong ? 1 : 0) != 0;
  const bool by_logit = goes_by_logit(a);
  float m = 0.0f, sum = 1.0f;  // softmax: the largest logit, the sum of exp(l - m)
  if (softmax) m = of_key(team_max<TEAM>(top_key));
  uint32_t key[SLOTS];
  Doubt doubt{0.0f, 0.0f}, keys_doubt = doubt;
  if (by_logit) {
#pragma unroll
    for (int s = 0; s < SLOTS; s++) key[s] = l[s] > ninf ? key_of(l[s]) : kOff;
  }
  if (!by_logit || (softmax && !a.renormalise)) {
    float p[SLOTS], part = 0.0f;
#pragma unroll
    for (int s = 0; s < SLOTS; s++) {
      p[s] = __builtin_amdgcn_exp2f((softmax ? l[s] - m : -l[s]) * kLog2eHi);  // (-inf - m: 0; no expert on: NaN, not used)
      part += p[s];
    }
    if (softmax) sum = team_sum<TEAM>(part);
    if (!by_logit) {
      const float inv = softmax ? 1.0f / sum : 1.0f;
      doubt = Doubt{softmax ? (SLOTS > 16 ? 0x1p-15f : 0x1p-17f) * inv : 0x1p-20f, 0x1p-22f};
      keys_doubt = Doubt{doubt.abs, 0x1p-22f + (1 << slot_bits<SLOTS>()) * 0x1p-23f};
#pragma unroll
      for (int s = 0; s < SLOTS; s++) {
        const float c = (softmax ? p[s] * inv : __builtin_amdgcn_rcpf(1.0f + p[s])) + b[s];
        key[s] = l[s] > ninf && c > ninf ? key_of(c) : kOff;
      }
    }
  }
  // the wavefront's LDS: kTeams tokens in fp32, or one in fp64
  double* const wave_scores = shared_scores + wave * sp.size * (kTeams > 2 ? kTeams / 2 : 1);
  int open = SURE;
  if (a.groups > 1) {
    float* const mine = reinterpret_cast<float*>(wave_scores) + team * sp.size;
    int group[SLOTS];
    groups_of<TEAM>(sp.inv_per, group);
    lay_out<TEAM>(a, sp, group, mine, [&](int s) { return key[s] == kOff ? ninf : of_key(key[s]); });
    float least, most;
    const unsigned long long kept = keep_groups<TEAM>(a, sp, mine, least, most);
    if (!by_logit) {
      least = -of_key(team_max<TEAM>(key_of(-least)));
      most = of_key(team_max<TEAM>(key_of(most)));
      if (most != ninf && !(least - most > doubt.abs)) open = CHOICE;
    }
#pragma unroll
    for (int s = 0; s < SLOTS; s++) {
      const uint32_t k = a.bias ? key[s] : key_of(l[s]);
      key[s] = key[s] != kOff && is_kept(kept, group[s]) ? k : kOff;
    }
  }
  int id, count;
  // (16-bit logits end in zeros: 13 of fp16's, for up to 64 registers)
  open = max(open, a.bias ? pick<TEAM, SLOTS, true>(key, a.top, keys_doubt, false, id, count)
                          : pick<TEAM, SLOTS, false>(key, a.top, keys_doubt, DT != DT_F32, id, count));
  if (wrong) open = SURE;
  if (__ballot(open == ORDER)) {
    int ordered = id;
    const bool still = order64<TEAM, DT>(a, row, count, m, sum, ordered);
    if (open == ORDER) {
      id = ordered;
      open = still ? CHOICE : SURE;
    }
  }
  for (unsigned long long again = __ballot(open != SURE); again;) {
    const int t = (__ffsll((long long)again) - 1) / TEAM;
    const int of = choose64<DT, (SLOTS * TEAM + 63) / 64>(a, (first + t) * a.experts, sp, wave_scores);
    const int moved = __shfl(of, lane);
    if (team == t) id = moved;
    again &= ~(((TEAM < 64 ? 1ull << TEAM : 0ull) - 1) << (t * TEAM));
  }
  const bool chosen = there && lane < a.top && id >= 0;
  float w = 0.0f, v = ninf;
  if (chosen) v = logit_at<DT>(a.logits, row + id) + 0.0f;
  if (a.renormalise) {  // shares of the chosen alone, however far below the others or below 0
    const uint32_t k = team_max<TEAM>(chosen ? key_of(v) : kOff);
    m = k == kOff ? 0.0f : of_key(k);
    if (!softmax) m = fminf(m, 0.0f);
  }
  if (chosen) w = softmax ? exp_near<true>(v - m) : v < kNoSigmoid ? 0.0f : Sigmoid::of(v, m).p;
  if (a.renormalise) sum = team_sum<TEAM>(w);
  if (there && lane < a.top) {
    a.ids[token * a.top + lane] = !wrong ? id : a.keep_nan ? lane : -1;
    a.weights[token * a.top + lane] = wrong ? __builtin_nanf("") : w > 0.0f ? a.scale * (w / sum) : 0.0f;
  }
}

// ---------------------------------------------------------------- gradient
// One wavefront a token: every expert's slope from the softmax's sum, then the chosen
// ones' terms added in the order of the choices.
template <int DT, int SLOTS>
__global__ __launch_bounds__(64 * kWaves) void route_grad_kernel(RouteArgs a) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t token = (int64_t)blockIdx.x * kWaves + wave;
  if (token >= a.tokens) return;
  const int64_t row = token * a.experts;
  const bool softmax = a.score == SCORE_SOFTMAX;
  int id = lane < a.top ? a.ids[token * a.top + lane] : -1;
  if (id < 0 || id >= a.experts) id = -1;
  float g = 0.0f, v = -__builtin_inff();
  if (id >= 0) {
    g = a.scale * a.dweights[token * a.top + lane];
    v = logit_at<DT>(a.logits, row + id);
  }
  float d[SLOTS];  // the row's gradient
#pragma unroll
  for (int s = 0; s < SLOTS; s++) d[s] = 0.0f;
  float term = 0.0f;  // what the lane's choice adds to its expert's
  if (__ballot(id >= 0)) {
    if (softmax && !a.renormalise) {
      uint32_t top_key = kOff;
#pragma unroll
      for (int s = 0; s < SLOTS; s++) d[s] = logit_at<DT>(a.logits, row + min(lane + 64 * s, a.experts - 1));
#pragma unroll
      for (int s = 0; s < SLOTS; s++) {
        d[s] = lane + 64 * s < a.experts ? d[s] + 0.0f : -__builtin_inff();
        top_key = max(top_key, d[s] > -__builtin_inff() ? key_of(d[s]) : kOff);
      }
      const float m = of_key(team_max<64>(top_key));
      float part = 0.0f;
#pragma unroll
      for (int s = 0; s < SLOTS; s++) {
        d[s] = d[s] > -__builtin_inff() ? exp_near(d[s] - m) : 0.0f;
        part += d[s];
      }
      const float inv = 1.0f / wave_sum(part);
      const float p = id >= 0 && v > -__builtin_inff() ? exp_near(v - m) * inv : 0.0f;
      term = p * g;
      const float mean = wave_sum(term);
#pragma unroll
      for (int s = 0; s < SLOTS; s++) d[s] = d[s] * inv * -mean;
    } else if (softmax) {
      const float m = of_key(team_max<64>(id >= 0 && v > -__builtin_inff() ? key_of(v + 0.0f) : kOff));
      const float e = id >= 0 && v > -__builtin_inff() ? exp_near(v - m) : 0.0f;
      const float sum = wave_sum(e), share = sum > 0.0f ? e / sum : 0.0f;
      term = share * (g - wave_sum(share * g));
    } else {
      float m = 0.0f;
      if (a.renormalise) {
        const uint32_t k = team_max<64>(id >= 0 && v > -__builtin_inff() ? key_of(v + 0.0f) : kOff);
        if (k != kOff) m = fminf(of_key(k), 0.0f);
      }
      const Sigmoid s = Sigmoid::of(v, m);
      const float p = id < 0 || v < kNoSigmoid ? 0.0f : s.p;
      if (a.renormalise) {
        const float sum = wave_sum(p), share = sum > 0.0f ? p / sum : 0.0f;
        term = share * s.rest * (g - wave_sum(share * g));
      } else {
        term = p * s.rest * g;
      }
    }
    for (int j = 0; j < a.top; j++) {
      const int e = __builtin_amdgcn_readlane(id, j);
      const float t = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(term), j));
      if (e < 0) continue;
#pragma unroll
      for (int s = 0; s < SLOTS; s++)
        if (e / 64 == s && lane == e % 64) d[s] += t;
    }
  }
#pragma unroll
  for (int s = 0; s < SLOTS; s++) {
    const int e = lane + 64 * s;
    if (e < a.experts) store_logit<DT>(a.dlogits, row + e, d[s]);
  }
}

template <int TEAM>
struct Slots {
  // f(SLOTS) for the fewest of a few sizes that hold the experts
  template <int FIRST, int... REST, typename F>
  static hipError_t call(int experts, F f) {
    if (sizeof...(REST) == 0 || experts <= FIRST * TEAM) return f(std::integral_constant<int, FIRST>());
    if constexpr (sizeof...(REST) > 0) return call<REST...>(experts, f);
  }
};
template <typename F>
hipError_t with_logits(int dtype, F f) {
  using std::integral_constant;
  if (dtype == DT_F32) return f(integral_constant<int, DT_F32>());
  if (dtype == DT_BF16) return f(integral_constant<int, DT_BF16>());
  return f(integral_constant<int, DT_F16>());
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t s) {
  if (a.tokens < 1 || a.experts < 1 || a.experts > 4096 || a.top < 1 || a.top > 64 || a.groups < 1 || a.groups > 64 ||
      a.experts % a.groups != 0)
    return hipErrorInvalidValue;
  const int per = a.experts / a.groups;
  const bool small = a.experts <= 256 && a.top <= 16;
  const int team = small ? 16 : 64, teams = 64 / team;
  Spread sp{per, per % 2 ? 0 : -1, (a.groups + 3) / 4, 0, 0, 1.0f / (float)per};
  sp.size = (8 * sp.quads + a.groups * (per - sp.odd_mask) + 4) / 4 * 4;
  while ((2 << sp.shift) * a.groups <= team) sp.shift++;
  int waves = kWaves;
  size_t lds = 0;
  if (a.groups > 1) {
    const size_t each = (size_t)sp.size * sizeof(double) * (teams > 2 ? teams / 2 : 1);
    while (waves > 1 && waves * each > kMostLds) waves /= 2;
    lds = waves * each;
  }
  const int64_t tokens = (int64_t)waves * teams;
  const unsigned blocks = (unsigned)((a.tokens + tokens - 1) / tokens);
  return with_logits(a.dtype, [&](auto DT_) {
    constexpr int DT = decltype(DT_)::value;
    if (small)
      return Slots<16>::call<1, 2, 4, 6, 8, 10, 12, 16>(a.experts, [&](auto SLOTS_) {
        route_kernel<DT, 16, decltype(SLOTS_)::value><<<blocks, 64 * waves, lds, s>>>(a, sp);
        return hipGetLastError();
      });
    return Slots<64>::call<1, 4, 8, 16, 64>(a.experts, [&](auto SLOTS_) {
      route_kernel<DT, 64, decltype(SLOTS_)::value><<<blocks, 64 * waves, lds, s>>>(a, sp);
      return hipGetLastError();
    });
  });
}

hipError_t launch_moe_route_grad(const RouteArgs& a, hipStream_t s) {
  if (a.tokens < 1 || a.experts < 1 || a.experts > 4096 || a.top < 1 || a.top > 64) return hipErrorInvalidValue;
  return with_logits(a.dtype, [&](auto DT_) {
    return Slots<64>::call<1, 2, 3, 4, 8, 16, 64>(a.experts, [&](auto SLOTS_) {
      route_grad_kernel<decltype(DT_)::value, decltype(SLOTS_)::value>
          <<<(unsigned)((a.tokens + kWaves - 1) / kWaves), 64 * kWaves, 0, s>>>(a);
      return hipGetLastError();
    });
  });
}

}  // namespace mc2
