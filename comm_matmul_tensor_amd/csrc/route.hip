// K13: the router of a mixture-of-experts layer and its gradient.
//
//   p = softmax(l) or sigmoid(l), c = p + bias; the top largest c of the kept
//   groups; weights = scale p (/ the sum of the chosen p)
//
// One wavefront takes a token: lane i holds the logits i, i + 64, ... in SLOTS
// registers, so that a row is read once in whole lines and every reduction is
// one of DPP steps.  The choice goes by rounds: the wavefront's largest key,
// then the lowest register and lane that hold it.
//
// Order.  Without a bias the keys are the logits themselves: p rises with l,
// so no score is formed but those of the chosen.  Otherwise c is formed in
// fp32 with an error bound (below), and a row in which two neighbours of the
// order lie within it, a tie among them, is done again in fp64 (choose64): the
// experts chosen are those of fp64, at fp32's cost.
#include "layer8_kernels.hpp"
#include "layer_device.hpp"

namespace mc2 {
namespace {

constexpr float kLog2eHi = 1.44269504088896340736f;
constexpr float kLog2eLo = 1.925963033500e-8f;  // log2(e) - kLog2eHi
constexpr float kLn2 = 0.693147180559945309417f;
constexpr int kOff = INT32_MIN;                 // key of an expert that is off

// exp(x) within 2^-22: the argument in base 2 to twice fp32's precision (x log2(e)
// rounded alone is off by |x| 2^-24).  Past +-200 it is 0 or infinite in fp32.
__device__ __forceinline__ float exp_near(float x) {
  x = __builtin_amdgcn_fmed3f(x, -200.0f, 200.0f);
  const float t = x * kLog2eHi;
  const float lo = __builtin_fmaf(x, kLog2eLo, __builtin_fmaf(x, kLog2eHi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return e < __builtin_inff() ? __builtin_fmaf(e * kLn2, lo, e) : e;
}

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

// Floats in an order of signed integers (no NaN; -0 has been added to 0).
__device__ __forceinline__ int key_of(float f) {
  const int b = __float_as_int(f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float of_key(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }

// Maximum over the wavefront, as a scalar.
__device__ __forceinline__ int wave_max_key(int v) {
  v = max(v, (int)dpp16<0>((uint32_t)v));
  v = max(v, (int)dpp16<1>((uint32_t)v));
  v = max(v, (int)dpp16<2>((uint32_t)v));
  v = max(v, (int)dpp16<3>((uint32_t)v));
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x142, 0xA, 0xF, false));  // row_bcast 15
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x143, 0xC, 0xF, false));  // row_bcast 31
  return __builtin_amdgcn_readlane(v, 63);
}

// What rounding can move between two values that are compared.  p of a
// softmax: its exponential, the sum's additions (SLOTS and 6 in a row) and a
// product, relative to p, of which 1 / sum is the largest; of a sigmoid:
// 2^-22 at most.  Twice that for two values, twice more for sums of two; and
// the additions' own roundings, relative to the values.
struct Doubt {
  float abs, rel;
  __device__ __forceinline__ bool operator()(float a, float b) const {  // a >= b: not surely a > b
    return !(a - b > abs + rel * fmaxf(__builtin_fabsf(a), __builtin_fabsf(b)));
  }
};

// The top largest keys: lane j < top gets the j-th's expert (-1: none left).
// CHECK: false where the order of two of them, or of the last and the next, is
// in doubt.
template <int SLOTS, bool CHECK>
__device__ __forceinline__ bool pick(int (&key)[SLOTS], int top, Doubt doubt, int& id) {
  const int lane = threadIdx.x % 64;
  float prev = __builtin_inff();
  id = -1;
  for (int j = 0; j < top + (CHECK ? 1 : 0); j++) {
    int best = key[0];
#pragma unroll
    for (int s = 1; s < SLOTS; s++) best = max(best, key[s]);
    const int m = wave_max_key(best);
    if (m == kOff) return true;
    if constexpr (CHECK) {
      const float f = of_key(m);
      if (j > 0 && doubt(prev, f)) return false;
      prev = f;
      if (j == top) return true;
    }
    int won = -1;
#pragma unroll
    for (int s = 0; s < SLOTS; s++) {
      if (won < 0) {
        const unsigned long long at = __ballot(key[s] == m);
        if (at) {
          const int l = __ffsll((long long)at) - 1;
          won = 64 * s + l;
          if (lane == l) key[s] = kOff;
        }
      }
    }
    if (lane == j) id = won;
  }
  return true;
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
  __device__ __forceinline__ T value(int group_top) const { return group_top == 2 && b > -__builtin_inf() ? a + b : a; }
};

// Lane g step's value of group g, for g < groups: those kept, as a mask of lanes.
template <typename T>
__device__ __forceinline__ unsigned long long kept_groups(T v, int groups, int step, int top_groups) {
  const int lane = threadIdx.x % 64, g = lane / step;
  int rank = 0;
  for (int o = 0; o < groups; o++) {
    const T u = __shfl(v, o * step);
    rank += u > v || (u == v && o < g);
  }
  return __ballot(g < groups && v > -__builtin_inf() && rank < top_groups);
}

// Expert e's group; `magic` is 2^32 / per rounded up (e and per are at most 4096).
__device__ __forceinline__ int group_of(int e, unsigned long long magic) { return (int)((unsigned)e * magic >> 32); }

// The choice with all scores in fp64.
template <int DT, int SLOTS>
__device__ __attribute__((noinline)) int choose64(const RouteArgs& a, int64_t row, unsigned long long magic) {
  const int lane = threadIdx.x % 64;
  const double off = -__builtin_inf();
  double c[SLOTS];
  double m = off, sum = 0.0;
  if (a.score == SCORE_SOFTMAX) {
#pragma unroll 1
    for (int e = lane; e < a.experts; e += 64) m = fmax(m, (double)logit_at<DT>(a.logits, row + e));
    for (int o = 1; o < 64; o *= 2) m = fmax(m, __shfl_xor(m, o));
#pragma unroll 1
    for (int e = lane; e < a.experts; e += 64) sum += exp((double)logit_at<DT>(a.logits, row + e) - m);
    for (int o = 1; o < 64; o *= 2) sum += __shfl_xor(sum, o);
  }
#pragma unroll
  for (int s = 0; s < SLOTS; s++) {
    const int e = lane + 64 * s;
    c[s] = off;
    if (e < a.experts) {
      const double l = (double)logit_at<DT>(a.logits, row + e);
      const double p = a.score == SCORE_SOFTMAX ? exp(l - m) / sum : 1.0 / (1.0 + exp(-l));
      const double v = p + (a.bias ? (double)a.bias[e] : 0.0);
      if (l > off && v > off) c[s] = v;
    }
  }
  if (a.groups > 1) {
    double value = off;
    for (int g = 0; g < a.groups; g++) {
      Two<double> t{off, off};
#pragma unroll
      for (int s = 0; s < SLOTS; s++)
        if (group_of(lane + 64 * s, magic) == g) t.add(c[s]);
      for (int o = 1; o < 64; o *= 2) t.join(__shfl_xor(t.a, o), __shfl_xor(t.b, o));
      if (lane == g) value = t.value(a.group_top);
    }
    const unsigned long long kept = kept_groups(value, a.groups, 1, a.top_groups);
#pragma unroll
    for (int s = 0; s < SLOTS; s++) {
      const int e = lane + 64 * s;
      if (e < a.experts && !(kept >> group_of(e, magic) & 1)) c[s] = off;
    }
  }
  if (!a.bias) {
#pragma unroll
    for (int s = 0; s < SLOTS; s++)
      if (c[s] > off) c[s] = (double)logit_at<DT>(a.logits, row + lane + 64 * s);
  }
  int id = -1;
  for (int j = 0; j < a.top; j++) {
    double best = c[0];
#pragma unroll
    for (int s = 1; s < SLOTS; s++) best = fmax(best, c[s]);
    for (int o = 1; o < 64; o *= 2) best = fmax(best, __shfl_xor(best, o));
    if (best == off) break;
    int won = -1;
#pragma unroll
    for (int s = 0; s < SLOTS; s++) {
      const unsigned long long at = __ballot(c[s] == best);
      if (won < 0 && at) {
        const int l = __ffsll((long long)at) - 1;
        won = 64 * s + l;
        if (lane == l) c[s] = off;
      }
    }
    if (lane == j) id = won;
  }
  return id;
}

constexpr int kWaves = 4;  // tokens of a workgroup (two where the groups' scores would not fit 64 KB of LDS)

template <int DT, int SLOTS>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs a, int pitch, int step, unsigned long long magic) {
  extern __shared__ float shared_scores[];  // groups rows of `pitch` for each wavefront
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t token = (int64_t)blockIdx.x * (blockDim.x / 64) + wave;
  if (token >= a.tokens) return;  // (no barrier below)
  const int64_t row = token * a.experts;
  const float ninf = -__builtin_inff();
  float l[SLOTS];
  bool wrong = false;
  int top_key = kOff;
#pragma unroll
  for (int s = 0; s < SLOTS; s++) {
    const int e = lane + 64 * s;
    l[s] = e < a.experts ? logit_at<DT>(a.logits, row + e) + 0.0f : ninf;
    wrong |= l[s] != l[s] || (a.score == SCORE_SOFTMAX && l[s] == __builtin_inff());
    top_key = max(top_key, l[s] > ninf ? key_of(l[s]) : kOff);
  }
  if (__ballot(wrong)) {
    if (lane < a.top) {
      a.ids[token * a.top + lane] = -1;
      a.weights[token * a.top + lane] = __builtin_nanf("");
    }
    return;
  }
  const bool softmax = a.score == SCORE_SOFTMAX;
  // with one key a group the group's order is its logit's
  const bool by_logit = !a.bias && (a.groups == 1 || a.group_top == 1);
  float m = 0.0f, sum = 1.0f;  // softmax: the largest logit, the sum of exp(l - m)
  if (softmax) m = of_key(wave_max_key(top_key));
  int key[SLOTS];
  Doubt doubt{0.0f, 0.0f};
  if (by_logit) {
#pragma unroll
    for (int s = 0; s < SLOTS; s++) key[s] = l[s] > ninf ? key_of(l[s]) : kOff;
  }
  if (!by_logit || (softmax && !a.renormalise)) {
    float p[SLOTS], part = 0.0f;
#pragma unroll
    for (int s = 0; s < SLOTS; s++) {
      p[s] = l[s] > ninf ? exp_near(softmax ? l[s] - m : -l[s]) : 0.0f;
      part += p[s];
    }
    if (softmax) sum = wave_sum(part);
    if (!by_logit) {
      const float inv = 1.0f / sum;
      doubt = Doubt{softmax ? (SLOTS > 16 ? 0x1p-15f : 0x1p-17f) * inv : 0x1p-20f, 0x1p-22f};
#pragma unroll
      for (int s = 0; s < SLOTS; s++) {
        const int e = lane + 64 * s;
        float c = softmax ? p[s] * inv : __builtin_amdgcn_rcpf(1.0f + p[s]);
        if (a.bias && e < a.experts) c += a.bias[e];
        key[s] = l[s] > ninf && c > ninf ? key_of(c) : kOff;
      }
    }
  }
  bool sure = true;
  if (a.groups > 1) {
    float* mine = shared_scores + wave * a.groups * pitch;
    const int per = a.experts / a.groups;
    int at[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; s++) {
      const int e = lane + 64 * s, g = group_of(e, magic);
      at[s] = g;
      if (e < a.experts) mine[g * pitch + e - g * per] = key[s] == kOff ? ninf : of_key(key[s]);
    }
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int g = lane / step;
    Two<float> t{ninf, ninf};
    if (g < a.groups)
      for (int i = lane % step; i < per; i += step) t.add(mine[g * pitch + i]);
    for (int o = 1; o < step; o *= 2) t.join(__shfl_xor(t.a, o), __shfl_xor(t.b, o));
    const float value = t.value(a.group_top);
    const unsigned long long kept = kept_groups(value, a.groups, step, a.top_groups);
    if (!by_logit && a.top_groups < a.groups) {
      const bool is = kept >> lane & 1;
      const int least = wave_max_key(is ? ~key_of(value) : kOff);  // ~: the order turned round
      const int most = wave_max_key(!is && g < a.groups && value > ninf ? key_of(value) : kOff);
      if (least != kOff && most != kOff) sure = !doubt(of_key(~least), of_key(most));
    }
#pragma unroll
    for (int s = 0; s < SLOTS; s++) {
      if (!(kept >> (at[s] * step & 63) & 1)) key[s] = kOff;
      else if (!a.bias && key[s] != kOff) key[s] = key_of(l[s]);
    }
  }
  int id = -1;
  if (sure) sure = a.bias ? pick<SLOTS, true>(key, a.top, doubt, id) : pick<SLOTS, false>(key, a.top, doubt, id);
  if (!sure) id = choose64<DT, SLOTS>(a, row, magic);

  float w = 0.0f;
  if (lane < a.top && id >= 0) {
    const float v = logit_at<DT>(a.logits, row + id);
    w = softmax ? exp_near(v - m) : 1.0f / (1.0f + exp_near(-v));
  }
  if (a.renormalise) sum = wave_sum(w);
  if (lane < a.top) {
    a.ids[token * a.top + lane] = id;
    a.weights[token * a.top + lane] = w > 0.0f ? a.scale * (w / sum) : 0.0f;
  }
}

// ---------------------------------------------------------------- gradient
// The same rows: every expert's slope from the softmax's sum, then the chosen
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
      int top_key = kOff;
#pragma unroll
      for (int s = 0; s < SLOTS; s++) {
        const int e = lane + 64 * s;
        d[s] = e < a.experts ? logit_at<DT>(a.logits, row + e) + 0.0f : -__builtin_inff();
        top_key = max(top_key, d[s] > -__builtin_inff() ? key_of(d[s]) : kOff);
      }
      const float m = of_key(wave_max_key(top_key));
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
      const float m = of_key(wave_max_key(id >= 0 && v > -__builtin_inff() ? key_of(v + 0.0f) : kOff));
      const float e = id >= 0 && v > -__builtin_inff() ? exp_near(v - m) : 0.0f;
      const float sum = wave_sum(e), share = sum > 0.0f ? e / sum : 0.0f;
      term = share * (g - wave_sum(share * g));
    } else {
      // p and 1 - p, each from the exponential of the sign that keeps it exact
      const float e = exp_near(-__builtin_fabsf(v)), big = 1.0f / (1.0f + e), small = e * big;
      const float p = id < 0 ? 0.0f : v < 0.0f ? small : big, q = v < 0.0f ? big : small;
      if (a.renormalise) {
        const float sum = wave_sum(p), share = sum > 0.0f ? p / sum : 0.0f;
        term = share * q * (g - wave_sum(share * g));
      } else {
        term = p * q * g;
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

template <typename F>
hipError_t with_slots(int experts, F f) {
  using std::integral_constant;
  if (experts <= 64) return f(integral_constant<int, 1>());
  if (experts <= 128) return f(integral_constant<int, 2>());
  if (experts <= 256) return f(integral_constant<int, 4>());
  if (experts <= 512) return f(integral_constant<int, 8>());
  if (experts <= 1024) return f(integral_constant<int, 16>());
  if (experts <= 2048) return f(integral_constant<int, 32>());
  return f(integral_constant<int, 64>());
}
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
  const int per = a.experts / a.groups, pitch = per | 1;  // odd: the lanes' rows start in different banks
  int step = 1;  // lanes of a group
  while (2 * step * a.groups <= 64) step *= 2;
  const int waves = a.groups > 1 && a.experts > 2048 ? 2 : kWaves;
  const size_t lds = a.groups > 1 ? (size_t)waves * a.groups * pitch * sizeof(float) : 0;
  const unsigned long long magic = ((1ull << 32) + per - 1) / per;
  return with_logits(a.dtype, [&](auto DT_) {
    return with_slots(a.experts, [&](auto SLOTS_) {
      route_kernel<decltype(DT_)::value, decltype(SLOTS_)::value>
          <<<(unsigned)((a.tokens + waves - 1) / waves), 64 * waves, lds, s>>>(a, pitch, step, magic);
      return hipGetLastError();
    });
  });
}

hipError_t launch_moe_route_grad(const RouteArgs& a, hipStream_t s) {
  if (a.tokens < 1 || a.experts < 1 || a.experts > 4096 || a.top < 1 || a.top > 64) return hipErrorInvalidValue;
  return with_logits(a.dtype, [&](auto DT_) {
    return with_slots(a.experts, [&](auto SLOTS_) {
      route_grad_kernel<decltype(DT_)::value, decltype(SLOTS_)::value>
          <<<(unsigned)((a.tokens + kWaves - 1) / kWaves), 64 * kWaves, 0, s>>>(a);
      return hipGetLastError();
    });
  });
}

}  // namespace mc2
