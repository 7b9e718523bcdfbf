// route.cu -- the router: a token's top-k experts and their weights.
//
//   s[e] = softmax_e(logits) or 1 / (1 + exp(-logit[e]))
//   c[e] = s[e] + bias[e]                                    the choice
//   worth of a group of experts = sum of its `best` largest c; topk_groups groups stay
//   ids  = the topk largest c of their experts, the lowest index among equals
//   w[k] = s[ids[k]] (/ sum_k s[ids[k]]) * scale
//
// One warp a token, VPL neighbouring experts a lane, so that the lowest lane
// among equals holds the lowest index.  Bound by latency for a few tokens, by
// instructions for many (the logits' bytes are less).
//
// Which experts are chosen is what arithmetic in 64 bits says.  Without a bias
// (and sums of a group's scores) the logits decide, which needs no arithmetic.
// With one, c is computed in fp32 with a bound of its error, and a token for
// which two neighbours of the order lie within that bound is done again in
// fp64: few tokens, as the bound is 1e-6 of the scores.
#include <cuda_runtime.h>

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

// Numerators and scores.  expf, its argument and the quotient: within 2^-21 of s
// each (an ulp, half an ulp of 1 + e and of the quotient, and for the softmax
// |x| exp(-|x|) half ulps of x); a sum of VPL + 5 steps, (VPL + 5) half ulps.
template <typename T>
__device__ __forceinline__ T sigmoid(T x) {
  const T e = exp(-fabs(x));
  return (x < 0 ? e : T(1)) / (1 + e);
}

__device__ __forceinline__ float logit_at(const RouteArgs &p, long long i) {
  return p.logits_f32 ? load_global(static_cast<const float *>(p.logits) + i)
                      : bf16_bits_to_float(load_global(static_cast<const uint16_t *>(p.logits) + i));
}

// Experts of one token: id of place `lane` (lanes below topk), and its weight.
// Returns whether the fp32 scores cannot tell the order (T = float).
template <typename T, int VPL>
__device__ __forceinline__ bool route_token(const RouteArgs &p, const float (&l)[VPL], const float (&b)[VPL], int lane,
                                            long long row, int *id, float *weight) {
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
  auto close = [&](T hi, T lo, float times) {
    return sizeof(T) == 4 && scores && hi < INFINITY && lo > -INFINITY &&
           hi - lo <= times * (slack + 2.3841858e-7f * fmaxf(fabsf((float)hi), fabsf((float)lo)));
  };
  bool unsure = false;

  if (p.groups > p.topk_groups) {
    const int size = E / p.groups;
    T worth = kLow;   // of group `lane`
    auto sum2 = [&](T a1, T a2) { return p.best == 2 && a2 > kLow ? a1 + a2 : a1; };
    const int span = size / VPL;   // lanes of a group
    if (size % VPL == 0 && (span & (span - 1)) == 0) {
      T a1 = kLow, a2 = kLow;
#pragma unroll
      for (int i = 0; i < VPL; ++i) merge2(a1, a2, c[i], kLow);
      for (int d = 1; d < span; d <<= 1) merge2(a1, a2, __shfl_xor_sync(kAll, a1, d), __shfl_xor_sync(kAll, a2, d));
      worth = __shfl_sync(kAll, sum2(a1, a2), lane * span & 31);
      if (lane >= p.groups) worth = kLow;
    } else {
      for (int g = 0; g < p.groups; ++g) {
        T a1 = kLow, a2 = kLow;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if ((unsigned)(e0 + i - g * size) < (unsigned)size) merge2(a1, a2, c[i], kLow);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) merge2(a1, a2, __shfl_xor_sync(kAll, a1, d), __shfl_xor_sync(kAll, a2, d));
        if (lane == g) worth = sum2(a1, a2);
      }
    }
    int before = 0;   // groups that come before group `lane`
    for (int g = 0; g < p.groups; ++g) {
      const T o = __shfl_sync(kAll, worth, g);
      before += o > worth || (o == worth && g < lane);
    }
    const bool stays = lane < p.groups && before < p.topk_groups;
    const uint32_t open = __ballot_sync(kAll, stays);
    // the last that stays against the first that does not
    const int last = __ffs(__ballot_sync(kAll, lane < p.groups && before == p.topk_groups - 1)) - 1;
    const int next = __ffs(__ballot_sync(kAll, lane < p.groups && before == p.topk_groups)) - 1;
    const T hi = __shfl_sync(kAll, worth, last), lo = __shfl_sync(kAll, worth, next);
    unsure |= close(hi, lo, (float)p.best);
    const int g0 = size % VPL == 0 ? e0 / size : -1;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int g = g0 >= 0 ? g0 : (e0 + i) / size;
      if (g < p.groups && !(open >> g & 1)) c[i] = kLow;
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
  *id = 0;
  int last = -1;
  for (int k = 0; k < p.topk; ++k) {
    const Key m = warp_max(best);
    const int from = __ffs(__ballot_sync(kAll, best == m)) - 1;
    const int e = __shfl_sync(kAll, e0 + at, from);
    const T v = from_key(m);
    if (close(before, v, 1.f)) {
      // equal inputs are equal: the lowest index is first, whatever the scores' errors
      const bool same = logit_at(p, row + last) == logit_at(p, row + e) &&
                        (!p.bias || load_global(p.bias + last) == load_global(p.bias + e));
      unsure |= !same;
    }
    before = v;
    last = e;
    if (lane == k) {
      *id = e;
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
  if (sizeof(T) == 4 && scores) unsure |= close(before, from_key(warp_max(best)), 1.f);
  if (unsure) return true;

  T s = 0;
  if (lane < p.topk && mine > kLow) {
    float x = (float)mine;   // without scores, the logit itself
    if (scores) x = logit_at(p, row + *id);
    s = score(x);
  }
  if (p.renormalize) {
    const T total = warp_sum(s);
    if (total > 0) s = s / total;
  }
  *weight = bad ? __int_as_float(0x7FC00000) : (float)(s * T(p.scale));
  return false;
}

// VPL values of a row from element e0 on, n of which exist.
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

// The same in fp64; apart, so that the fp32 form keeps its registers.
struct Routed {
  int id;
  float weight;
};
template <int VPL>
__device__ __noinline__ Routed route_token_64(const RouteArgs &p, int lane, long long row) {
  float l[VPL], b[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    l[i] = e < p.E ? logit_at(p, row + e) : -INFINITY;
    b[i] = e < p.E && p.bias ? load_global(p.bias + e) : 0.f;
  }
  Routed r;
  route_token<double, VPL>(p, l, b, lane, row, &r.id, &r.weight);
  return r;
}

template <int VPL, typename V>
__global__ void __launch_bounds__(kThreads, VPL <= 8 ? 8 : 4) route_kernel(const __grid_constant__ RouteArgs p, bool vec) {
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * (kThreads / 32);
  const int n = p.E - lane * VPL;   // (VPL at least, or none where rows are read as vectors)
  wait_for_prior_grid();
  float b[VPL];
  load_row<VPL, float>(p.bias + lane * VPL, p.bias ? n : 0, vec, 0.f, b);
  for (long long m = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); m < p.M; m += warps) {
    const long long row = m * p.ld;
    float l[VPL];
    load_row<VPL, V>(static_cast<const V *>(p.logits) + row + lane * VPL, n, vec, -INFINITY, l);
    Routed r;
    if (route_token<float, VPL>(p, l, b, lane, row, &r.id, &r.weight)) r = route_token_64<VPL>(p, lane, row);
    if (lane < p.topk) {
      p.ids[m * p.topk + lane] = r.id;
      p.weights[m * p.topk + lane] = r.weight;
    }
  }
}

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int VPL>
int launch_vpl(const RouteArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
  const bool vec = a.E % VPL == 0 && on16(a.logits) && on16(a.bias) && a.ld % (a.logits_f32 ? 4 : 8) == 0;
  const unsigned grid = (unsigned)std::min<long long>((a.M + kThreads / 32 - 1) / (kThreads / 32), dev.sm_count * 8ll);
  return a.logits_f32 ? launch_dependent(route_kernel<VPL, float>, grid, kThreads, 1, 0, stream, a, vec)
                      : launch_dependent(route_kernel<VPL, uint16_t>, grid, kThreads, 1, 0, stream, a, vec);
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
