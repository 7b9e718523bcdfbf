// route.cu -- the router: a token's top-k experts and their weights.
//
//   s[e] = softmax_e(logits) or 1 / (1 + exp(-logit[e]))
//   c[e] = s[e] + bias[e]                                    the choice
//   worth of a group of experts = sum of its `best` largest c; topk_groups groups stay
//   ids  = the topk largest c of their experts, the lowest index among equals
//   w[k] = s[ids[k]] (/ sum_k s[ids[k]]) * scale
//
// One warp a token, VPL neighbouring experts a lane, so that the lowest lane
// among equals holds the lowest index.  The topk-th largest of the lanes' maxima
// is a bound that all chosen experts reach; those that do are few (topk to 2
// topk, mostly): a lane takes each and counts the ones before it, which is its
// place (route_fast).  What that form leaves (numbers that are none, more than 32
// experts that reach the bound, fewer candidates than places) takes the largest
// topk times (route_general).  Bound by latency for a few tokens, by instructions
// for many: 16384 tokens of 256 experts take about 420 a token by their logits
// (9.6 us; the bytes, 2.6) and 870 under a bias in groups (20.7 us), and one token
// 1.7 us.  Taking the largest eight times for all of them took 21.6 and 48 us.
//
// Which experts are chosen is what arithmetic in 64 bits says.  Without a bias
// the logits decide, which needs no arithmetic, but for sums of a group's scores.
// With one, c is computed in fp32 with a bound of its error, and where two
// neighbours of the order lie within that bound it is done again in fp64: for
// few tokens, as the bound is 1e-6 of the scores.  A bias adds half an ulp of the choice, which moves no
// choice past another (rounding keeps the order); in a group's sum of two, where biases may cancel,
// it moves sums past one another, so that each group's doubt counts both of its choices (sum_error).
#include <cuda_runtime.h>

#include <cfloat>

#include <algorithm>

#include "device_utils.cuh"
#include "launch.cuh"
#include "route.h"

namespace moe_lora {

namespace {

constexpr int kThreads = 128;
constexpr unsigned kAll = 0xFFFFFFFFu;

// Keys: unsigned numbers in the order of the values.  0 stands for an expert
// that is taken or does not exist, below -inf's key.
__device__ __forceinline__ uint32_t to_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);   // (-0 as +0: equal values have equal keys)
  return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t to_key(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return u ^ (uint64_t(int64_t(u) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double from_key(uint64_t k) {
  return __longlong_as_double((long long)(k ^ (k >> 63 ? 0x8000000000000000ull : 0xFFFFFFFFFFFFFFFFull)));
}
template <typename T>
struct KeyOf {
  typedef uint32_t type;
};
template <>
struct KeyOf<double> {
  typedef uint64_t type;
};

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = max(v, (uint64_t)__shfl_xor_sync(kAll, v, d));
  return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// The two largest of (a1 >= a2) and (b1 >= b2).
template <typename T>
__device__ __forceinline__ void merge2(T &a1, T &a2, T b1, T b2) {
  const T lo = a1 < b1 ? a1 : b1;
  a1 = a1 < b1 ? b1 : a1;
  a2 = a2 < b2 ? b2 : a2;
  a2 = a2 < lo ? lo : a2;
}

template <typename T>
__device__ __forceinline__ T sigmoid(T x) {
  const T e = exp(-fabs(x));
  return (x < 0 ? e : T(1)) / (1 + e);
}

__device__ __forceinline__ float logit_at(const RouteArgs &p, long long i) {
  return p.logits_f32 ? load_global(static_cast<const float *>(p.logits) + i)
                      : bf16_bits_to_float(load_global(static_cast<const uint16_t *>(p.logits) + i));
}

// exp(a - b) for numbers whose difference is at most zero, to two ulp: what the difference
// loses to rounding (2^-18 of the result from -64 on) is multiplied in again.
__device__ __forceinline__ float exp_diff(float a, float b) {
  const float d = a - b, t = d - a, lost = (a - (d - t)) - (b + t), e = expf(d);
  return d > -128.f ? fmaf(e, lost, e) : 0.f;
}
__device__ __forceinline__ double exp_diff(double a, double b) { return exp(a - b); }

// How far the fp32 sum `worth` of two choices a1 and a2 may be off (a2 of zero: of one choice): the scores' errors (slack
// is twice that of one), half an ulp of each choice, whose biases may be far larger than their sum, and of the sum.
__device__ __forceinline__ float sum_error(float slack, float a1, float a2, float worth) {
  return slack + 6e-8f * fabsf(a1) + 6e-8f * fabsf(a2) + 6e-8f * fabsf(worth);
}

struct Routed {
  int id;         // of place `lane`, in lanes below topk
  float weight;
  bool unsure;    // the fp32 scores cannot tell the order (T = float)
};

// One token, whatever its logits.  Apart, so that the fast form keeps its
// registers.  Errors of fp32 scores: expf, its argument and the quotient within
// 2^-21 of s (an ulp, half an ulp of 1 + e and of the quotient, and for the
// softmax |x| exp(-|x|) half ulps of x); a sum of VPL + 5 steps, (VPL + 5) half ulps.  The
// biases' roundings are counted where choices are compared (close) or added up (sum_error).
template <typename T, int VPL>
__device__ __noinline__ Routed route_general(const RouteArgs &p, long long row) {
  const int lane = threadIdx.x & 31;
  Routed r = {0, 0.f, false};
  float l[VPL], b[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    l[i] = e < p.E ? logit_at(p, row + e) : -INFINITY;
    b[i] = e < p.E && p.bias ? load_global(p.bias + e) : 0.f;
  }
  typedef typename KeyOf<T>::type Key;
  const T kLow = -INFINITY;
  const int E = p.E, e0 = lane * VPL;
  const bool sums = p.groups > p.topk_groups && p.best == 2;   // of scores, for the groups
  const bool scores = p.bias != nullptr || sums;
  // a row whose scores are not numbers has weights that are none either
  bool bad = false;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    bad |= l[i] != l[i] || b[i] != b[i] || (!p.sigmoid && l[i] == INFINITY);
    top = fmaxf(top, l[i]);
  }
  bad = __any_sync(kAll, bad);
  T sum = 1;
  if (!p.sigmoid) {
    top = from_key(warp_max(to_key(top)));
    if (scores || !p.renormalize) {
      T part = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) part += exp(T(l[i]) - T(top));
      sum = warp_sum(part);
    }
  }
  auto score = [&](float x) { return p.sigmoid ? sigmoid(T(x)) : exp(T(x) - T(top)) / sum; };
  T c[VPL], largest = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    c[i] = T(l[i]);
    if (scores) {
      const T s = score(l[i]);
      largest = s > largest ? s : largest;
      c[i] = s + T(b[i]);
    }
    if (!(l[i] > -INFINITY) || c[i] != c[i]) c[i] = kLow;   // no candidate
  }
  // what the order of two choices can be wrong by: twice the error of the
  // scores, and of the addition of the bias (`of`: the larger of the two)
  float slack = 0.f;
  if (sizeof(T) == 4 && scores)
    slack = (p.sigmoid ? 1.f : from_key(warp_max(to_key((float)largest)))) * ((VPL + 16) * 2 * 5.9604645e-8f);
  auto close = [&](T hi, T lo) {
    return sizeof(T) == 4 && scores && hi < INFINITY && lo > -INFINITY &&
           hi - lo <= slack + 2.3841858e-7f * fmaxf(fabsf((float)hi), fabsf((float)lo));
  };
  bool unsure = false;

  if (p.groups > p.topk_groups) {
    const int size = E / p.groups;
    T worth = kLow, error = 0;   // of group `lane`; error: how far its worth may be off (T = float)
    auto sum2 = [&](T a1, T a2) {
      const bool two = p.best == 2 && a2 > kLow;
      worth = two ? a1 + a2 : a1;
      if (sizeof(T) == 4 && scores && a1 > kLow && a1 < INFINITY) {
        if (two) worth = worth > FLT_MAX ? FLT_MAX : worth < -FLT_MAX ? -FLT_MAX : worth;
        error = sum_error(slack, (float)a1, two ? (float)a2 : 0.f, (float)worth);
      }
    };
    const int span = size / VPL;   // lanes of a group
    if (size % VPL == 0 && (span & (span - 1)) == 0) {
      T a1 = kLow, a2 = kLow;
#pragma unroll
      for (int i = 0; i < VPL; ++i) merge2(a1, a2, c[i], kLow);
      for (int d = 1; d < span; d <<= 1) merge2(a1, a2, __shfl_xor_sync(kAll, a1, d), __shfl_xor_sync(kAll, a2, d));
      a1 = __shfl_sync(kAll, a1, lane * span & 31);
      a2 = __shfl_sync(kAll, a2, lane * span & 31);
      if (lane < p.groups) sum2(a1, a2);
    } else {
      for (int g = 0; g < p.groups; ++g) {
        T a1 = kLow, a2 = kLow;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if ((unsigned)(e0 + i - g * size) < (unsigned)size) merge2(a1, a2, c[i], kLow);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) merge2(a1, a2, __shfl_xor_sync(kAll, a1, d), __shfl_xor_sync(kAll, a2, d));
        if (lane == g) sum2(a1, a2);
      }
    }
    int before = 0;   // groups that come before group `lane`
    for (int g = 0; g < p.groups; ++g) {
      const T o = __shfl_sync(kAll, worth, g);
      before += o > worth || (o == worth && g < lane);
    }
    const bool stays = lane < p.groups && before < p.topk_groups;
    const uint32_t open = __ballot_sync(kAll, stays);
    // the least that one which stays may be worth, against the most that one which does not may be
    if (sizeof(T) == 4 && scores) {
      const float least = -from_key(warp_max(to_key(stays ? __fadd_ru((float)error, -(float)worth) : -INFINITY)));
      const float most = from_key(warp_max(to_key(lane < p.groups && !stays && worth > kLow ? __fadd_ru((float)worth, (float)error) : -INFINITY)));
      unsure |= most > -INFINITY && !(least > most);
    }
    const int g0 = size % VPL == 0 ? e0 / size : -1;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int g = g0 >= 0 ? g0 : (e0 + i) / size;
      if (g < p.groups && !(open >> g & 1)) c[i] = kLow;
    }
    // (the scores were for the groups: without a bias the logits decide)
    if (!p.bias) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (c[i] > kLow) c[i] = T(l[i]);
    }
  }

  Key key[VPL], best = 0;
  int at = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    key[i] = e0 + i < E ? to_key(c[i]) : Key(0);
    if (key[i] > best) best = key[i], at = i;
  }
  T mine = kLow, before = INFINITY;
  int last = -1;
  for (int k = 0; k < p.topk; ++k) {
    const Key m = warp_max(best);
    const int from = __ffs(__ballot_sync(kAll, best == m)) - 1;
    const int e = __shfl_sync(kAll, e0 + at, from);
    const T v = from_key(m);
    if (p.bias && close(before, v)) {
      // equal inputs are equal: the lowest index is first, whatever the scores' errors
      const bool same = logit_at(p, row + last) == logit_at(p, row + e) &&
                        load_global(p.bias + last) == load_global(p.bias + e);
      unsure |= !same;
    }
    before = v;
    last = e;
    if (lane == k) {
      r.id = e;
      mine = v;
    }
    if (lane == from) {
      best = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (i == at) key[i] = 0;
      }
      at = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (key[i] > best) best = key[i], at = i;
    }
  }
  if (sizeof(T) == 4 && p.bias) unsure |= close(before, from_key(warp_max(best)));
  r.unsure = unsure;
  if (unsure) return r;

  // s = exp(a - ref) / under: under a renormalisation by the largest of the chosen, as
  // their sum may be out of range otherwise
  const bool have = lane < p.topk && mine > kLow;
  const float x = !have ? -INFINITY : scores ? logit_at(p, row + r.id) : (float)mine;
  const float a = p.sigmoid ? fminf(x, 0.f) : x;
  const float ref = p.renormalize ? from_key(warp_max(to_key(a))) : p.sigmoid ? 0.f : top;
  T s = 0;
  if (have) s = exp_diff(T(a), T(ref)) / (p.sigmoid ? 1 + exp(-fabs(T(x))) : p.renormalize ? T(1) : sum);
  if (p.renormalize) {
    const T total = warp_sum(s);
    if (total > 0) s = s / total;
  }
  r.weight = bad ? __int_as_float(0x7FC00000) : (float)(s * T(p.scale));
  return r;
}

// ------------------------------------------------------------------ fast

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

constexpr float kLog2e = 1.44269504f;
// Scores that only order experts.  x log2(e) is rounded twice, so that exp(x) is
// within 2^-22 + |x| 2^-23 of itself, and zero below 2^-126.  A sigmoid, whose
// slope is s (1 - s) <= 1/4, with s (1 - s) |x| < 0.23, and whose quotient adds 2^-23 +
// 2^-24, is within 2^-22; a softmax's numerator (|x| exp(-|x|) < 0.37) within 2^-21 of
// the largest, and a sum of them in VPL + 5 steps within 2^-21 + (VPL + 5) 2^-24 of itself.
__device__ __forceinline__ float order_sigmoid(float x) {
  const float e = exp2_unit(-kLog2e * fabsf(x)), r = rcp_unit(1.f + e);
  return x < 0.f ? e * r : r;
}

// What does not depend on the token.
struct Lane {
  int lane, span, group;   // span: lanes of a group, a power of two, or 0; group: of this lane's experts
  int size;                // experts of a group
  uint32_t inv;            // e / size is e * inv >> 20
  bool ok;                 // the biases are ordinary numbers
};

// Experts of a token that reach the bound: expert and choice, then a key (the
// larger choice first, then the lower index), then in order.  Unused entries
// are zero, as all are between tokens.
struct __align__(16) Picks {
  unsigned long long entry[32];
  int count;
};
__device__ __forceinline__ unsigned long long pack(uint32_t lo, uint32_t hi) { return lo | (unsigned long long)hi << 32; }

// The choice, in fp64, of the expert that each lane has (negative: none).
template <int VPL>
__device__ __noinline__ double exact_choice(const RouteArgs &p, long long row, int expert) {
  double sum = 1.0;
  float top = -INFINITY;
  if (!p.sigmoid) {
    const int e0 = (threadIdx.x & 31) * VPL;
    for (int i = 0; i < VPL && e0 + i < p.E; ++i) top = fmaxf(top, logit_at(p, row + e0 + i));
    __syncwarp();
    top = warp_max(top);
    sum = 0.0;
    for (int i = 0; i < VPL && e0 + i < p.E; ++i) sum += exp((double)logit_at(p, row + e0 + i) - top);
    sum = warp_sum(sum);
  }
  if (expert < 0) return 0.0;
  const double x = logit_at(p, row + expert);
  return (p.sigmoid ? sigmoid(x) : exp(x - top) / sum) + (p.bias ? (double)load_global(p.bias + expert) : 0.0);
}

// What orders the experts: the logits; the logits, and sums of scores their groups; scores
// and the bias.
enum { kByLogits, kByLogitsInGroups, kByChoice };

// One token without NaN or +inf; false where it is left to the general form.
template <int VPL, int ORDER, bool FULL>
__device__ __forceinline__ bool route_fast(const RouteArgs &p, const float (&l)[VPL], const float (&b)[VPL], const Lane &at,
                                           long long row, Picks &picks, Routed *out) {
  constexpr bool SCORES = ORDER != kByLogits, CHOICE = ORDER == kByChoice;
  const int lane = at.lane, e0 = lane * VPL;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool exists = FULL || e0 + i < p.E;
    odd |= exists && !(l[i] < INFINITY);
  }
  if (__any_sync(kAll, odd)) return false;

  float c[VPL], top = 0.f, sum = 1.f, slack = 0.f;
  if (!p.sigmoid && (SCORES || !p.renormalize)) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    top = warp_max(m);
    float part = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      c[i] = exp2_unit((l[i] - top) * kLog2e);
      part += c[i];
    }
    sum = warp_sum(part);
  }
  if constexpr (SCORES) {
    // twice the scores' error
    if (p.sigmoid) {
      slack = 4.7683716e-7f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = order_sigmoid(l[i]) + (CHOICE ? b[i] : 0.f);
    } else {
      const float inv = rcp_unit(sum);
      slack = inv * ((VPL + 32) * 2 * 5.9604645e-8f);
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = c[i] * inv + (CHOICE ? b[i] : 0.f);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = l[i] > -INFINITY ? c[i] : -INFINITY;   // (of experts that do not exist, too)
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = l[i];
  }
  // by how much a choice near v may be wrong, twice: the scores' errors, and half an ulp of its sum
  auto doubt = [&](float v) { return slack + 1.1920929e-7f * fabsf(v); };

  if (p.groups > p.topk_groups) {
    auto merge = [](float &a1, float &a2, float b1, float b2) {
      a2 = fmaxf(fmaxf(a2, b2), fminf(a1, b1));
      a1 = fmaxf(a1, b1);
    };
    float a1 = -INFINITY, a2 = -INFINITY, g1 = -INFINITY, g2 = -INFINITY;   // the two largest of this lane's group, and of group `lane`
    if (at.span) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) merge(a1, a2, c[i], -INFINITY);
      for (int d = 1; d < at.span; d <<= 1) merge(a1, a2, __shfl_xor_sync(kAll, a1, d), __shfl_xor_sync(kAll, a2, d));
      g1 = __shfl_sync(kAll, a1, lane * at.span & 31);
      g2 = __shfl_sync(kAll, a2, lane * at.span & 31);
      if (lane >= p.groups) g1 = g2 = -INFINITY;
    } else {
#pragma unroll 1
      for (int g = 0; g < p.groups; ++g) {
        float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) merge(b1, b2, (unsigned)(e0 + i - g * at.size) < (unsigned)at.size ? c[i] : -INFINITY, -INFINITY);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) merge(b1, b2, __shfl_xor_sync(kAll, b1, d), __shfl_xor_sync(kAll, b2, d));
        if (lane == g) g1 = b1, g2 = b2;
      }
    }
    // (finite choices have a finite sum here: near ties of such are done again in 64 bits)
    const bool two = p.best == 2 && g2 > -INFINITY;
    const float worth = two ? fminf(fmaxf(g1 + g2, -FLT_MAX), FLT_MAX) : g1;
    uint32_t open = 0;
    float rest = worth, last = 0.f;   // last: what the last one that stays is worth
    for (int k = 0; k < p.topk_groups; ++k) {
      last = warp_max(rest);
      const int from = __ffs(__ballot_sync(kAll, rest == last)) - 1;
      open |= 1u << from;
      if (lane == from) rest = -INFINITY;
    }
    if (SCORES) {
      // The least that one which stays may be worth, against the most that one which does not may be; both in relation to
      // `last`, from which near ones differ exactly.
      const bool stays = open >> lane & 1;
      const float error = sum_error(slack, g1, two ? g2 : 0.f, worth);
      const float edge = stays ? __fadd_ru(error, __fadd_ru(last, -worth)) : __fadd_ru(error, __fadd_ru(worth, -last));
      const float least = -warp_max(stays ? edge : -INFINITY);
      const float most = warp_max(!stays && worth > -INFINITY ? edge : -INFINITY);
      if (last > -INFINITY && !(least > most)) {   // (with no candidates in the last, the others have none)
        if (!at.span) return false;
        // The groups that may belong on the other side again, from exact choices of those experts that may be their best.
        const bool again = worth > -INFINITY && (stays ? -edge <= most : edge >= least);
        const bool close = __ballot_sync(kAll, again) >> at.group & 1;
        const float least_c = p.best == 2 && a2 > -INFINITY ? a2 : a1, need_from = fmaxf(least_c - 2.f * doubt(least_c), -FLT_MAX);
        double exact = again ? -INFINITY : worth;
        double second = -INFINITY;
        for (int i = 0; i < VPL; ++i) {   // (one expert a lane at a time, where any has one)
          float ci = 0.f;
#pragma unroll
          for (int k = 0; k < VPL; ++k)
            if (k == i) ci = c[k];
          const bool need = close && ci >= need_from;
          uint32_t who = __ballot_sync(kAll, need);
          if (!who) continue;
          const double x = exact_choice<VPL>(p, row, need ? e0 + i : -1);
          for (; who; who &= who - 1) {
            const int from = __ffs(who) - 1;
            const double v = __shfl_sync(kAll, x, from);
            if (__shfl_sync(kAll, at.group, from) == lane) merge2(exact, second, v, (double)-INFINITY);
          }
        }
        if (p.best == 2 && second > -INFINITY) exact += second;
        int before = 0;
        for (int o = 0; o < p.groups; ++o) {
          const double w = __shfl_sync(kAll, exact, o);
          before += w > exact || (w == exact && o < lane);
        }
        open = __ballot_sync(kAll, lane < p.groups && before < p.topk_groups);
      }
    }
    if (!at.span) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (!(open >> ((e0 + i) * at.inv >> 20 & 31) & 1)) c[i] = -INFINITY;
    } else if (!(open >> at.group & 1)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = -INFINITY;
    }
    // (the scores were for the groups: without a bias the logits decide)
    if (ORDER == kByLogitsInGroups) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = c[i] > -INFINITY ? l[i] : -INFINITY;
    }
  }

  // the bound: at least topk lanes reach it (every finite choice does where fewer have one)
  float best = c[0], bound = -INFINITY;
#pragma unroll
  for (int i = 1; i < VPL; ++i) best = fmaxf(best, c[i]);
#pragma unroll 2
  for (int k = 0; k < p.topk; ++k) {
    bound = warp_max(best);
    if (best == bound) best = -INFINITY;
  }
  if (CHOICE) bound -= doubt(bound);   // and what is as large but for errors
  bound = fmaxf(bound, -FLT_MAX);      // (-inf: experts of closed groups, and those that do not exist)
  int mine = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) mine += c[i] >= bound;
  int to = 0;
  if (mine) to = atomicAdd(&picks.count, mine);
  __syncwarp();
  const int count = picks.count;
  __syncwarp();
  picks.count = 0;
  if (count > 32 || count < p.topk) return false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (c[i] >= bound) picks.entry[to++] = pack(e0 + i, __float_as_uint(c[i]));
  }
  __syncwarp();
  const bool have = lane < count;
  const unsigned long long own = picks.entry[lane];
  int expert = have ? (int)(uint32_t)own : -1;
  const float choice = __uint_as_float((uint32_t)(own >> 32));
  const unsigned long long key = have ? pack(~(uint32_t)expert, to_key(choice)) : 0;
  __syncwarp();
  picks.entry[lane] = key;
  __syncwarp();
  int place = 0;
#pragma unroll 1
  for (int j = 0; j < count; j += 4) {
    const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(&picks.entry[j]);
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&picks.entry[j + 2]);
    place += (u.x > key) + (u.y > key) + (v.x > key) + (v.y > key);
  }
  __syncwarp();
  if (have) picks.entry[place] = pack(expert, __float_as_uint(choice));
  __syncwarp();
  const unsigned long long first = picks.entry[lane], after = picks.entry[min(lane + 1, 31)];
  expert = have ? (int)(uint32_t)first : -1;
  float mine_c = __uint_as_float((uint32_t)(first >> 32));
  if constexpr (CHOICE) {
    const float next = __uint_as_float((uint32_t)(after >> 32));
    if (__any_sync(kAll, lane < p.topk && lane + 1 < count && mine_c - next <= doubt(fmaxf(fabsf(mine_c), fabsf(next))))) {
      // again in 64 bits, which tell equal inputs from others
      const double exact = exact_choice<VPL>(p, row, expert);
      place = 0;
      for (int j = 0; j < count; ++j) {
        const double o = __shfl_sync(kAll, exact, j);
        const int e = __shfl_sync(kAll, expert, j);
        place += o > exact || (o == exact && e < expert);
      }
      if (have) picks.entry[place] = (uint32_t)expert;
      __syncwarp();
      expert = have ? (int)(uint32_t)picks.entry[lane] : -1;
    }
  }
  __syncwarp();
  picks.entry[lane] = 0;   // (for the next token)

  // s = exp(a - ref) / under, all chosen being finite: under a renormalisation by the
  // largest of them, as their sum may be out of range otherwise
  const float logit = !CHOICE ? mine_c : (lane < p.topk ? logit_at(p, row + expert) : -INFINITY);
  const float a = p.sigmoid ? fminf(logit, 0.f) : logit;
  float ref = p.sigmoid ? 0.f : top;
  if (p.renormalize) ref = CHOICE ? warp_max(a) : __shfl_sync(kAll, a, 0);
  float s = 0.f;
  if (lane < p.topk) {
    if (p.sigmoid) {
      const float e = expf(-fabsf(logit));
      s = __fdividef(ref < 0.f ? exp_diff(a, ref) : logit < 0.f ? e : 1.f, 1.f + e);
    } else {
      s = exp_diff(a, ref);
    }
  }
  float scale = p.scale;
  if (p.renormalize) {
    const float total = warp_sum(s);
    if (total > 0.f) scale = __fdividef(scale, total);
  } else if (!p.sigmoid) {
    scale = __fdividef(scale, sum);
  }
  out->id = expert;
  out->weight = s * scale;
  return true;
}

// VPL values of a row, n of which exist.
template <int VPL, typename V>
__device__ __forceinline__ void load_row(const V *src, int n, bool vec, float missing, float (&v)[VPL]) {
  constexpr int kBytes = VPL * (int)sizeof(V), kUnit = kBytes < 16 ? kBytes : 16, kPer = kUnit / (int)sizeof(V);
  uint32_t raw[(kBytes + 3) / 4];
  if (kUnit >= 4 && vec) {
#pragma unroll
    for (int u = 0; u < kBytes / kUnit; ++u) {
      if (u * kPer >= n) break;
      if constexpr (kUnit == 16) {
        const uint4 q = load_global(reinterpret_cast<const uint4 *>(src) + u);
        raw[4 * u] = q.x, raw[4 * u + 1] = q.y, raw[4 * u + 2] = q.z, raw[4 * u + 3] = q.w;
      } else if constexpr (kUnit == 8) {
        const uint2 q = load_global(reinterpret_cast<const uint2 *>(src));
        raw[0] = q.x, raw[1] = q.y;
      } else {
        raw[0] = load_global(reinterpret_cast<const uint32_t *>(src));
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float x;
      if constexpr (sizeof(V) == 4) x = __uint_as_float(raw[i]);
      else x = __uint_as_float(i & 1 ? raw[i >> 1] & 0xFFFF0000u : raw[i >> 1] << 16);
      v[i] = i < n ? x : missing;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = missing;
      if (i < n) {
        if constexpr (sizeof(V) == 4) v[i] = load_global(src + i);
        else v[i] = bf16_bits_to_float(load_global(src + i));
      }
    }
  }
}

template <int VPL>
__device__ __forceinline__ void load_logits(const RouteArgs &p, long long at, int n, bool vec, float (&v)[VPL]) {
  if (p.logits_f32) load_row<VPL, float>(static_cast<const float *>(p.logits) + at, n, vec, -INFINITY, v);
  else load_row<VPL, uint16_t>(static_cast<const uint16_t *>(p.logits) + at, n, vec, -INFINITY, v);
}

template <int VPL, int ORDER, bool FULL>
__global__ void __launch_bounds__(kThreads, VPL <= 8 ? 8 : VPL <= 16 ? 5 : 3)
    route_kernel(const __grid_constant__ RouteArgs p, bool vec) {
  __shared__ Picks picks[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = gridDim.x * (kThreads / 32);
  const int n = FULL ? VPL : p.E - lane * VPL;   // (VPL at least, or none where rows are read as vectors)
  picks[warp].entry[lane] = 0;
  picks[warp].count = 0;
  __syncwarp();
  wait_for_prior_grid();
  Lane at = {lane, 1, 0, 1, 0, true};
  if (p.groups > p.topk_groups) {
    at.size = p.E / p.groups;
    at.inv = ((1u << 20) + at.size - 1) / at.size;   // (exact: e < 1024, so that e * (inv - 2^20 / size) < 2^10 <= 2^20 / size)
    at.span = at.size % VPL == 0 && (at.size / VPL & (at.size / VPL - 1)) == 0 ? at.size / VPL : 0;
    at.group = at.span ? lane / at.span : 0;
  }
  float b[VPL], l[VPL];
  if (ORDER == kByChoice) {
    load_row<VPL, float>(p.bias + lane * VPL, n, vec, 0.f, b);
    bool odd = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) odd |= !(fabsf(b[i]) < INFINITY);
    at.ok &= !__any_sync(kAll, odd);
  }
  long long m = (long long)blockIdx.x * (kThreads / 32) + warp;
  if (m < p.M) load_logits<VPL>(p, m * p.ld + lane * VPL, n, vec, l);
  for (; m < p.M; m += warps) {
    float next[VPL];   // on its way meanwhile
    if (m + warps < p.M) load_logits<VPL>(p, (m + warps) * p.ld + lane * VPL, n, vec, next);
    const long long row = m * p.ld;
    Routed r;
    if (!at.ok || !route_fast<VPL, ORDER, FULL>(p, l, b, at, row, picks[warp], &r)) {
      r = route_general<float, VPL>(p, row);
      if (r.unsure) r = route_general<double, VPL>(p, row);
    }
    if (lane < p.topk) {
      p.ids[m * p.topk + lane] = r.id;
      p.weights[m * p.topk + lane] = r.weight;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = next[i];
  }
}

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int VPL>
int launch_vpl(const RouteArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
  const bool vec = a.E % VPL == 0 && on16(a.logits) && on16(a.bias) && a.ld % (a.logits_f32 ? 4 : 8) == 0;
  const unsigned grid = (unsigned)std::min<long long>(((long long)a.M + kThreads / 32 - 1) / (kThreads / 32), dev.sm_count * 8ll);
  const bool full = a.E == 32 * VPL;
  const auto kernel = a.bias ? (full ? route_kernel<VPL, kByChoice, true> : route_kernel<VPL, kByChoice, false>)
                      : a.groups > a.topk_groups && a.best == 2
                          ? (full ? route_kernel<VPL, kByLogitsInGroups, true> : route_kernel<VPL, kByLogitsInGroups, false>)
                          : (full ? route_kernel<VPL, kByLogits, true> : route_kernel<VPL, kByLogits, false>);
  return launch_dependent(kernel, grid, kThreads, 1, 0, stream, a, vec);
}

}  // namespace

int launch_route(const RouteArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
  if (a.E <= 32) return launch_vpl<1>(a, dev, stream);
  if (a.E <= 64) return launch_vpl<2>(a, dev, stream);
  if (a.E <= 128) return launch_vpl<4>(a, dev, stream);
  if (a.E <= 256) return launch_vpl<8>(a, dev, stream);
  if (a.E <= 512) return launch_vpl<16>(a, dev, stream);
  return launch_vpl<32>(a, dev, stream);
}

}  // namespace moe_lora
