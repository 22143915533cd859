// route.cu - a mixture-of-experts router on the device: logits to expert numbers and weights, the gradient of
// the logits, and the routed rows grouped by expert without padding.
//
//   s = softmax(l) or 1 / (1 + e^-l)             scores of a token's E logits; l = -inf: 0
//   c = s + bias                                 what experts are chosen by (l = -inf: -inf)
//   a group's value = its two largest c added;   the top_groups largest groups are taken
//   ids = the k largest c of the groups taken, larger ones first, equal ones by number
//   w = scale s / (sum of the k s + 1e-20)       renormalised, or scale s
//
// The order is that of c in double precision: an expert that a rounding of fp32 puts ahead of another would
// make the result depend on how the scores are computed.  It is found from fp32 scores whose errors are
// bounded.  Where two neighbours among the k largest are closer than the bounds of both allow, and not equal by their
// inputs, these k are ordered again by scores of 44 bits (pairs of fp32 values), with the one behind them where that one alone
// is as close to the k-th as any error allows; where that holds for groups at the border, the experts of these groups are
// (groups_closely), for the k-th and more than one behind it (and not all so close are equal by their inputs, those before
// it among them), those of all groups taken (route_closely), and where 44 bits leave it open too, all in double precision
// (route_exactly; its fp64 instructions take a warp some 15 us).  Without a bias and groups the logits themselves are the order and there is nothing to bound.
//
// Bounds of fp32 scores.  expf is off by two steps of its last place, as CUDA documents it, 2^-22 of itself at most (over all
// x from -87 to 88 it is 2.56 2^-24 on a GB300).  Sigmoid: that moves s by 2^-22 s (1 - s), 1 + t and the reciprocal by
// 2^-24 s each: 2^-23 s (3 - 2 s) together.  Softmax: expf and the product 5 2^-24 of s, and l - max is rounded by 2^-24
// |l - max|, at most 2^-24 (-ln s) of s; a sum of E terms, with the terms' own errors (4 2^-24, and of the differences 4.5 at
// most), is off by (V + 14) 2^-24: that scales all scores of a token alike, so it moves the difference of two by that much of
// itself.  c is rounded by 2^-24.  Underflow ends at 2^-126, and e^-x overflows where s is below 2^-127.
//
// A warp has a token and a lane V neighbouring experts.  What bounds the kernels is a launch's and a few loads' latency
// and, from some thousand tokens on, instructions: about 20 for each of the k rounds that find the next largest c (eight
// lanes a token and four tokens a warp take as many, and the first build of either took 2.8 against 2.0 us for 8 tokens).
// On a GB300 (back to back in a graph; a launch that does nothing takes 1.5 us): 8 tokens of 64 experts, top 8, 2.4 us, their
// grouping 3.0, backward 1.9; 16384 tokens 7.7 us (sigmoid) and 8.6 (softmax), with a bias 11.8 and 13.5, with 8 groups besides
// 13.7 to 16.5 (256 experts: 29 to 36), of which tokens in doubt take 2 to 5; grouping their rows 6.9; backward 4.6 (sigmoid)
// and 5.7 (softmax).  Their bytes are 2.4 us.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "swiglu_math.cuh"

namespace mx {

namespace {

constexpr uint32_t FULL = 0xFFFFFFFFu;
// 16384 tokens of 64 experts with two, four and eight: 10.3, 8.6, 9.1 us (softmax), 8.8, 7.7, 7.8 (sigmoid); backward 8.7, 4.6 to
// 5.7, 4.1 to 4.9.
constexpr int ROUTE_WARPS = 4;

MX_DEVINL float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

MX_DEVINL float logit(const void* row, bool wide, int e) {
  // + 0: -0 and 0 are one value
  return wide ? reinterpret_cast<const float*>(row)[e] + 0.0f : bf16_value(reinterpret_cast<const uint16_t*>(row)[e]) + 0.0f;
}

// V neighbouring values from the first on: in vectors of up to 16 bytes where rows lie on them.
template <int V>
MX_DEVINL void load_values(const void* row, bool wide, bool vec, int first, int E, float none, float (&l)[V]) {
  if (vec && first < E) {  // E is a multiple of V
    if (wide) {
      const float* p = reinterpret_cast<const float*>(row) + first;
      if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
          l[4 * i] = v.x, l[4 * i + 1] = v.y, l[4 * i + 2] = v.z, l[4 * i + 3] = v.w;
        }
      } else if constexpr (V == 2) {
        const float2 v = __ldg(reinterpret_cast<const float2*>(p));
        l[0] = v.x, l[1] = v.y;
      } else {
        l[0] = __ldg(p);
      }
    } else {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + first;
      if constexpr (V >= 8) {
#pragma unroll
        for (int i = 0; i < V / 8; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) l[8 * i + 2 * j] = bf16_value(w[j]), l[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
      } else if constexpr (V >= 2) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
          l[2 * i] = bf16_value(w), l[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
        }
      } else {
        l[0] = bf16_value(__ldg(p));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      l[i] = first + i >= E ? none : wide ? __ldg(reinterpret_cast<const float*>(row) + first + i) : bf16_value(__ldg(reinterpret_cast<const uint16_t*>(row) + first + i));
  }
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] += 0.0f;
}

// Larger floats have larger keys; 0 is below all of them (NaN does not occur).
MX_DEVINL uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
MX_DEVINL float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

MX_DEVINL float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}
template <class T>
MX_DEVINL T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

struct RouteParams {
  const void* logits;     // [T, E] bf16 or fp32
  const float* bias;      // [E] or NULL
  int64_t T;
  int32_t E, k, groups, top_groups;
  int wide, sigmoid, renorm;
  int vec, vec_bias;      // rows of logits, and bias, can be read in vectors
  float scale;
  int32_t* ids;           // [T, k]
  float* weights;         // [T, k]
};

// Half the sum of the two largest of a group's values (the sum of two fp32 values may be none), or the only one.
template <class T>
MX_DEVINL T group_value(const T* c, int size, int first) {
  T a = (T)-INFINITY, b = (T)-INFINITY;
  for (int i = 0; i < size; ++i) {
    int j = i + first;  // lanes start apart: another bank each
    j = j >= size ? j - size : j;
    const T v = c[j];
    b = v > a ? a : v > b ? v : b;
    a = v > a ? v : a;
  }
  return size > 1 ? (T)0.5 * a + (T)0.5 * b : a;
}

// Rank of `value` among the values that lanes 0, step, ... of the warp have; `mine` is its own place there.
template <class T>
MX_DEVINL int rank_of(T value, int mine, int n, int step) {
  int rank = 0;
  for (int g = 0; g < n; ++g) {
    const T v = __shfl_sync(FULL, value, g * step);
    if (v > value || (v == value && g < mine)) ++rank;
  }
  return rank;
}

// A token's experts in double precision, by one warp: lane j returns the j-th.  flat: all logits are equal, so there is one
// score to be worked out, by its formula (2029 tokens of 256 experts, some of them flat and in doubt: 21 against 51 us).
__device__ __noinline__ int route_exactly(const RouteParams& p, const void* row, bool flat, double* c) {
  const int lane = threadIdx.x & 31;
  const int E = p.E, n = (E + 31) / 32;
  const bool wide = p.wide;
  __syncwarp();
  double most = 0, z = 0, one = 0;
  if (flat) {
    one = p.sigmoid ? 1 / (1 + exp(-(double)logit(row, wide, 0))) : 1.0 / E;
  } else {
    most = -INFINITY;
    for (int i = 0; i < n; ++i) {
      const int e = lane + 32 * i;
      if (e < E) most = fmax(most, (double)logit(row, wide, e));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) most = fmax(most, __shfl_xor_sync(FULL, most, o));
    if (most == -INFINITY) most = 0;
    for (int i = 0; i < n; ++i) {
      const int e = lane + 32 * i;
      if (e >= E) continue;
      const double l = logit(row, wide, e);
      const double v = exp(p.sigmoid ? -l : l - most);
      c[e] = p.sigmoid ? 1 / (1 + v) : v;
      z += v;
    }
    z = warp_sum(z);
  }
  for (int i = 0; i < n; ++i) {
    const int e = lane + 32 * i;
    if (e >= E) continue;
    double v = flat ? one : p.sigmoid ? c[e] : z > 0 ? c[e] / z : 0.0;
    if (p.bias) v += (double)p.bias[e];
    if (logit(row, wide, e) == -INFINITY) v = -INFINITY;
    c[e] = v;
  }
  __syncwarp();
  uint32_t taken = 0;  // bit i: expert lane + 32 i is chosen, or of no group that is
  if (p.groups > 1) {
    const int size = E / p.groups;
    const double v = lane < p.groups ? group_value(c + lane * size, size, lane % size) : 0.0;
    const int rank = rank_of(v, lane, p.groups, 1);  // by all lanes: they exchange values
    const uint32_t in = __ballot_sync(FULL, lane < p.groups && rank < p.top_groups);
    for (int i = 0; i < n; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !(in >> (e / size) & 1)) taken |= 1u << i;
    }
  }
  if (!p.bias) {  // the logits' own order
    __syncwarp();
    for (int i = 0; i < n; ++i) {
      const int e = lane + 32 * i;
      if (e < E) c[e] = logit(row, wide, e);
    }
  }
  int mine = 0;
  for (int j = 0; j < p.k; ++j) {
    double v = -INFINITY;
    int at = INT32_MAX;
    for (int i = 0; i < n; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !(taken >> i & 1) && (at == INT32_MAX || c[e] > v)) { v = c[e]; at = e; }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double w = __shfl_xor_sync(FULL, v, o);
      const int b = __shfl_xor_sync(FULL, at, o);
      if (b != INT32_MAX && (at == INT32_MAX || w > v || (w == v && b < at))) { v = w; at = b; }
    }
    if (lane == j) mine = at;
    if ((at & 31) == lane) taken |= 1u << (at >> 5);
  }
  __syncwarp();
  return mine;
}

// ---- scores of 44 bits
using swiglu_math::ff;

MX_DEVINL bool ff_more(ff a, ff b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
MX_DEVINL float ff_minus(ff a, ff b) { return (a.hi - b.hi) + (a.lo - b.lo); }  // a little off: bounds have room
MX_DEVINL ff ff_shfl(ff v, int lane) { return ff{__shfl_sync(FULL, v.hi, lane), __shfl_sync(FULL, v.lo, lane)}; }
MX_DEVINL ff ff_shfl_xor(ff v, int o) { return ff{__shfl_xor_sync(FULL, v.hi, o), __shfl_xor_sync(FULL, v.lo, o)}; }

// swiglu_math::ff_exp and ff_rcp (|x| <= 64; relative error below 2^-43) in few instructions: a warp that comes here finds
// none of them in its instruction cache, and fetching them is what it waits for.
__constant__ float2 kFfTaylor[7] = {{1.0f, 0.0f}, {1.0f, 0.0f}, {0.5f, 0.0f}, {0x1.555556p-3f, -0x1.555556p-28f},
                                    {0x1.555556p-5f, -0x1.555556p-30f}, {0x1.111112p-7f, -0x1.dddddep-32f},
                                    {0x1.6c16c2p-10f, -0x1.27d27ep-35f}};
__device__ __noinline__ ff ff_exp_small(float x) {
  using namespace swiglu_math;
  constexpr float L1 = 0x1.62e4p-1f, L2 = 0x1.7f7d1cp-20f, L3 = 0x1.ef357ap-45f;
  const float n = rintf(__fmul_rn(x, 0x1.715476p+0f));
  ff r = two_sum(x, -__fmul_rn(n, L1));  // exact
  const float p2 = __fmul_rn(n, L2);
  r = ff_add(r, ff{-p2, -__fmaf_rn(n, L2, -p2)});
  r = ff_add_f(r, -__fmul_rn(n, L3));
  float tail = 0x1.ae6456p-26f;
  tail = __fmaf_rn(tail, r.hi, 0x1.27e4fcp-22f);
  tail = __fmaf_rn(tail, r.hi, 0x1.71de3ap-19f);
  tail = __fmaf_rn(tail, r.hi, 0x1.a01a02p-16f);
  tail = __fmaf_rn(tail, r.hi, 0x1.a01a02p-13f);
  ff acc{tail, 0.0f};
#pragma unroll 1
  for (int k = 6; k >= 0; --k) acc = ff_add(ff_mul(acc, r), ff{kFfTaylor[k].x, kFfTaylor[k].y});
  const float two_n = __uint_as_float((uint32_t)((int)n + 127) << 23);
  return {__fmul_rn(acc.hi, two_n), __fmul_rn(acc.lo, two_n)};
}
MX_DEVINL ff ff_rcp_small(ff x) {  // one Newton step on an approximate reciprocal
  const float q = swiglu_math::rcp_approx(x.hi);
  return swiglu_math::fast_two_sum(q, __fmul_rn(q, __fmaf_rn(-x.lo, q, __fmaf_rn(-x.hi, q, 1.0f))));
}

// e^(l - most) for |l - most| <= 64: of the difference's nearest fp32 value and the rest
MX_DEVINL ff ff_exp_difference(float l, float most) {
  const ff d = swiglu_math::two_sum(l, -most);
  return swiglu_math::ff_mul(ff_exp_small(d.hi), ff{1.0f, fmaf(0.5f * d.lo, d.lo, d.lo)});
}
// Scores within 2^-42 of themselves; |l| (sigmoid) or |l - most| up to 64.  inv: 1 / sum (softmax).
MX_DEVINL ff ff_score(bool sigmoid, float l, float most, ff inv) {
  if (sigmoid) return ff_rcp_small(swiglu_math::ff_add_f(ff_exp_small(-l), 1.0f));
  return swiglu_math::ff_mul(ff_exp_difference(l, most), inv);
}
MX_DEVINL bool ff_in_range(bool sigmoid, float l, float most) { return fabsf(sigmoid ? l : l - most) <= 64.0f; }
// 1 / sum of a token's e^(l - most), by the warp; terms beyond the range are less than 2^-92 of it.
__device__ __noinline__ ff ff_inverse_sum(const void* row, bool wide, int E, float most) {
  ff z{0.0f, 0.0f};
#pragma unroll 1
  for (int e = threadIdx.x & 31; e < E; e += 32) {
    const float l = logit(row, wide, e);
    if (l - most >= -64.0f) z = swiglu_math::ff_add(z, ff_exp_difference(l, most));
  }
#pragma unroll 1
  for (int o = 16; o; o >>= 1) z = swiglu_math::ff_add(z, ff_shfl_xor(z, o));
  return ff_rcp_small(z);
}

// A token's experts (with a bias) by scores of 44 bits, by one warp: lane j returns the j-th.  Bit g of groups_in: group g
// is taken.  *sure: no difference that decides is
// within what they are off by (2^-40 with room), or the inputs are equal.
__device__ __noinline__ int route_closely(const RouteParams& p, const void* row, float most, uint32_t groups_in, double* buf,
                                          bool* sure) {
  const int lane = threadIdx.x & 31;
  const int E = p.E, n = (E + 31) / 32, group_size = E / p.groups;
  const bool wide = p.wide, sigmoid = p.sigmoid;
  float2* c = reinterpret_cast<float2*>(buf);
  ff inv{1.0f, 0.0f};
  if (!sigmoid) inv = ff_inverse_sum(row, wide, E, most);
  bool ok = true;
  __syncwarp();
  float size_of_c = 0.0f;
  uint32_t taken = 0;  // bit i: expert lane + 32 i is chosen, or of no group that is
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int e = lane + 32 * i;
    if (e >= E) continue;
    if (!(groups_in >> (e / group_size) & 1)) {
      taken |= 1u << i;
      continue;
    }
    const float l = logit(row, wide, e), b = p.bias[e];
    ff v{-INFINITY, 0.0f};
    if (l != -INFINITY) {
      ok = ok && ff_in_range(sigmoid, l, most);
      v = ff_score(sigmoid, l, most, inv);
      v = isinf(b) ? ff{b, 0.0f} : swiglu_math::ff_add_f(v, b);
      if (!isinf(v.hi)) size_of_c = fmaxf(size_of_c, fabsf(v.hi));
    }
    c[e] = make_float2(v.hi, v.lo);
  }
  if (!__all_sync(FULL, ok)) {
    // A logit that these scores are not made for: its score may be NaN, of which lanes that exchange values find no common
    // largest; each would cross out its own until there is none left.
    *sure = false;
    return 0;
  }
  const float off = 0x1p-39f * (1.0f + warp_max(size_of_c));
  __syncwarp();
  int mine = 0;
  ff last{0.0f, 0.0f};
  float last_l = 0.0f, last_b = 0.0f;
#pragma unroll 1
  for (int j = 0; j < p.k; ++j) {
    ff v{-INFINITY, 0.0f};
    int at = INT32_MAX;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int e = lane + 32 * i;
      if (e >= E || (taken >> i & 1)) continue;
      const ff w{c[e].x, c[e].y};
      if (at == INT32_MAX || ff_more(w, v)) { v = w; at = e; }
    }
#pragma unroll 1
    for (int o = 16; o; o >>= 1) {
      const ff w = ff_shfl_xor(v, o);
      const int b = __shfl_xor_sync(FULL, at, o);
      if (b != INT32_MAX && (at == INT32_MAX || ff_more(w, v) || (w.hi == v.hi && w.lo == v.lo && b < at))) { v = w; at = b; }
    }
    if (lane == j) mine = at;
    if ((at & 31) == lane) taken |= 1u << (at >> 5);
    const float l = logit(row, wide, at), b = p.bias[at];
    if (j && !(ff_minus(last, v) > off) && !(l == last_l && b == last_b) && !(isinf(v.hi) && v.hi == last.hi)) ok = false;
    last = v, last_l = l, last_b = b;
  }
#pragma unroll 1
  for (int i = 0; i < n; ++i) {  // against all that are left
    const int e = lane + 32 * i;
    if (e >= E || (taken >> i & 1)) continue;
    const ff w{c[e].x, c[e].y};
    if (!(ff_minus(last, w) > off) && !(logit(row, wide, e) == last_l && p.bias[e] == last_b) && !(isinf(w.hi) && w.hi == last.hi))
      ok = false;
  }
  *sure = __all_sync(FULL, ok);
  __syncwarp();
  return mine;
}

// The `slots` most valuable of the groups in `open` (lane g has group g), by scores of 44 bits.  *sure as in route_closely.
__device__ __noinline__ uint32_t groups_closely(const RouteParams& p, const void* row, float most, uint32_t open, int slots, double* buf,
                                                bool* sure) {
  const int lane = threadIdx.x & 31, size = p.E / p.groups, n = __popc(open) * size;
  const bool wide = p.wide, sigmoid = p.sigmoid;
  float2* c = reinterpret_cast<float2*>(buf);
  ff inv{1.0f, 0.0f};
  if (!sigmoid) inv = ff_inverse_sum(row, wide, p.E, most);
  bool ok = true;
  float size_of_c = 0.0f;
  __syncwarp();
#pragma unroll 1
  for (int i = lane; i < n; i += 32) {
    uint32_t rest = open;
#pragma unroll 1
    for (int g = i / size; g; --g) rest &= rest - 1;
    const int e = (__ffs(rest) - 1) * size + i % size;
    const float l = logit(row, wide, e), b = p.bias ? p.bias[e] : 0.0f;
    ff v{-INFINITY, 0.0f};
    if (l != -INFINITY) {
      ok = ok && ff_in_range(sigmoid, l, most);
      v = ff_score(sigmoid, l, most, inv);
      v = isinf(b) ? ff{b, 0.0f} : p.bias ? swiglu_math::ff_add_f(v, b) : v;
      if (!isinf(v.hi)) size_of_c = fmaxf(size_of_c, fabsf(v.hi));
    }
    c[e] = make_float2(v.hi, v.lo);
  }
  const float off = 0x1p-39f * (1.0f + warp_max(size_of_c));
  __syncwarp();
  const bool mine = open >> lane & 1;
  ff a{-INFINITY, 0.0f}, b{-INFINITY, 0.0f};
  int ea = lane * size, eb = ea;
  if (mine)
#pragma unroll 1
    for (int i = 0; i < size; ++i) {
      const float2 f = c[lane * size + i];
      const ff v{f.x, f.y};
      if (ff_more(v, a)) { b = a; eb = ea; a = v; ea = lane * size + i; }
      else if (i && ff_more(v, b)) { b = v; eb = lane * size + i; }
    }
  const ff value = size == 1 || isinf(a.hi) ? a : isinf(b.hi) ? b : swiglu_math::ff_add(ff{0.5f * a.hi, 0.5f * a.lo}, ff{0.5f * b.hi, 0.5f * b.lo});
  int rank = 0;
#pragma unroll 1
  for (uint32_t rest = open; rest; rest &= rest - 1) {
    const int g = __ffs(rest) - 1;
    const ff v = ff_shfl(value, g);
    if (ff_more(v, value) || (v.hi == value.hi && v.lo == value.lo && g < lane)) ++rank;
  }
  const uint32_t in = __ballot_sync(FULL, mine && rank < slots);
  // the last group taken and the first that is not: apart, or both of the same two values
  const int last = __ffs(__ballot_sync(FULL, mine && rank == slots - 1)) - 1;
  const int next = __ffs(__ballot_sync(FULL, mine && rank == slots)) - 1;
  if (last >= 0 && next >= 0) {
    const ff va = ff_shfl(value, last), vb = ff_shfl(value, next);
    if (!(ff_minus(va, vb) > off) && !(va.hi == vb.hi && isinf(va.hi))) {
      // Open, unless all that are as near have the same two experts' inputs, which no third comes near to.
      const int a1 = __shfl_sync(FULL, ea, last), a2 = __shfl_sync(FULL, eb, last);
      auto alike = [&](int x, int y) { return logit(row, wide, x) == logit(row, wide, y) && (!p.bias || p.bias[x] == p.bias[y]); };
      if (mine && !(fabsf(ff_minus(value, va)) > off)) {
        ok = ok && alike(ea, a1) && (size == 1 || alike(eb, a2));
#pragma unroll 1
        for (int i = 0; i < size; ++i) {
          const int e = lane * size + i;
          if (e != ea && e != eb && !(ff_minus(b, ff{c[e].x, c[e].y}) > off) && !alike(e, eb)) ok = false;
        }
      }
    }
  }
  *sure = __all_sync(FULL, ok);
  __syncwarp();
  return in;
}

// The n experts that lanes 0 to n - 1 have (numbers and logits) in order by scores of 44 bits: each lane's place.  *sure as
// in route_closely.
__device__ __noinline__ int order_closely(const RouteParams& p, const void* row, float most, int n, int id, float x, bool* sure) {
  const bool has = (int)(threadIdx.x & 31) < n, sigmoid = p.sigmoid;
  ff inv{1.0f, 0.0f}, c{-INFINITY, 0.0f};
  if (!sigmoid) inv = ff_inverse_sum(row, p.wide, p.E, most);
  bool fine = true;
  const float b = has ? p.bias[id] : 0.0f;
  if (has && x != -INFINITY) {
    fine = ff_in_range(sigmoid, x, most);
    c = ff_score(sigmoid, x, most, inv);
    c = isinf(b) ? ff{b, 0.0f} : swiglu_math::ff_add_f(c, b);
  }
  int place = 0;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const ff v = ff_shfl(c, j);
    const int e = __shfl_sync(FULL, id, j);
    const float xj = __shfl_sync(FULL, x, j), bj = __shfl_sync(FULL, b, j);
    const bool same = (xj == x && bj == b) || (v.hi == c.hi && isinf(v.hi));
    if (same ? e < id : ff_more(v, c)) ++place;
    if (has && !same && !(fabsf(ff_minus(v, c)) > 0x1p-39f * (1.0f + fabsf(c.hi)))) fine = false;
  }
  *sure = __all_sync(FULL, fine);
  return place;
}

// Lane i has experts i V to i V + V - 1.
template <int V, bool WIDE, bool SIGMOID>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) moe_route_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ double s_c[];
  pdl_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp;
  if (t >= p.T) return;
  double* const buf = s_c + (size_t)warp * p.E;
  const int E = p.E, k = p.k, first = lane * V;
  constexpr bool sigmoid = SIGMOID, wide = WIDE;
  const void* row = reinterpret_cast<const uint8_t*>(p.logits) + (size_t)t * E * (wide ? 4 : 2);
  float l[V];
  load_values<V>(row, wide, p.vec, first, E, -INFINITY, l);
  bool bad = false;
  float most = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bad |= l[i] != l[i] || (!sigmoid && l[i] == INFINITY);
    most = fmaxf(most, l[i]);
  }
  float inv = 1.0f;
  if (!sigmoid) {
    most = warp_max(most);
    if (most == -INFINITY) most = 0.0f;
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) z += expf(l[i] - most);
    z = warp_sum(z);
    inv = z > 0.0f ? 1.0f / z : 0.0f;
  }
  // what choosing needs: its bounds have room for the difference's rounding and for underflow
  auto score = [&](float x) { return sigmoid ? __frcp_rn(1.0f + expf(-x)) : expf(x - most) * inv; };
  uint32_t key[V];
  bool sure_groups = true, sure = true;   // of the groups, of the set of k
  auto all_equal = [&](const float (&x)[V]) {
    float least = INFINITY, high = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (first + i < E) least = fminf(least, x[i]), high = fmaxf(high, x[i]);
    return warp_max(high) == -warp_max(-least);
  };
  if (p.bias || p.groups > 1) {
    float c[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.0f;
    if (p.bias) load_values<V>(p.bias, true, p.vec_bias, first, E, 0.0f, b);
    float largest = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = l[i] == -INFINITY ? -INFINITY : score(l[i]) + b[i];
      bad |= c[i] != c[i];  // a NaN among biases, but not of an expert that is masked
      if (c[i] != -INFINITY) largest = fmaxf(largest, fabsf(c[i]));
      key[i] = first + i >= E ? 0 : key_of(p.bias ? c[i] : l[i]);
    }
    if (p.groups > 1) {
      // a score is off by 1.13 2^-23 (sigmoid: s = 3/4), or by (V + 22) 2^-24 of the largest there is (softmax), and half a sum of two by no
      // more; c and that are rounded
      const float off = (sigmoid ? 0x1.3p-22f : (V + 22) * 0x1p-23f * inv) + 0x1p-22f * warp_max(largest);
      const int size = E / p.groups, step = size / V;
      float value;
      int mine, rank, width = 1;  // width: lanes from one group to the next
      bool have = true;
      if (size % V == 0 && (step & (step - 1)) == 0) {  // a group has lanes of its own, a power of two of them
        float a = -INFINITY, d = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          d = fmaxf(d, fminf(a, c[i]));
          a = fmaxf(a, c[i]);
        }
        for (int o = 1; o < step; o <<= 1) {
          const float a2 = __shfl_xor_sync(FULL, a, o), d2 = __shfl_xor_sync(FULL, d, o);
          d = fmaxf(fmaxf(d, d2), fminf(a, a2));
          a = fmaxf(a, a2);
        }
        value = size > 1 ? 0.5f * a + 0.5f * d : a;
        mine = lane / step;
        width = step;
        have = mine < p.groups;
        rank = rank_of(value, mine, p.groups, step);
        if (have && rank >= p.top_groups) {
#pragma unroll
          for (int i = 0; i < V; ++i) key[i] = 0;
        }
      } else {  // through shared memory: lane g has group g
        float* cf = reinterpret_cast<float*>(buf);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (first + i < E) cf[first + i] = c[i];
        __syncwarp();
        have = lane < p.groups;
        mine = lane;
        value = have ? group_value(cf + lane * size, size, lane % size) : 0.0f;
        rank = rank_of(value, mine, p.groups, 1);
        const uint32_t in = __ballot_sync(FULL, have && rank < p.top_groups);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (first + i < E && !(in >> ((first + i) / size) & 1)) key[i] = 0;
      }
      bad |= have && value != value;
      // the last group taken and the first that is not
      const uint32_t at_last = __ballot_sync(FULL, have && rank == p.top_groups - 1);
      const uint32_t at_next = __ballot_sync(FULL, have && rank == p.top_groups);
      if (at_next) {
        const float a = __shfl_sync(FULL, value, __ffs(at_last) - 1), d = __shfl_sync(FULL, value, __ffs(at_next) - 1);
        sure_groups = a - d > off || (a == d && isinf(a));
        if (!sure_groups && !__any_sync(FULL, bad)) {
          if (!all_equal(l)) {
            // those well above the first that is not taken are in, those well below the last that is are out
            const float v = __shfl_sync(FULL, value, lane < p.groups ? lane * width : 0);
            const uint32_t in = __ballot_sync(FULL, lane < p.groups && v - d > off);
            const uint32_t open = __ballot_sync(FULL, lane < p.groups && !(v - d > off) && !(a - v > off));
            const uint32_t taken = in | groups_closely(p, row, most, open, p.top_groups - __popc(in), buf, &sure_groups);
#pragma unroll
            for (int i = 0; i < V; ++i)
              key[i] = first + i < E && (taken >> ((first + i) / size) & 1) ? key_of(p.bias ? c[i] : l[i]) : 0;
          } else if (!p.bias) {
            sure_groups = true;  // numbers decide, as they did
          }
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = first + i >= E ? 0 : key_of(l[i]);
  }
  // the k largest, and with a bias the one behind them
  uint32_t best = 0;
  int at = 0;
  auto find = [&] {
    best = key[0];
    at = first;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (key[i] > best) { best = key[i]; at = first + i; }
  };
  find();
  uint32_t mine = 0, behind = 0;  // key of the lane's expert; of the one behind the last
  int id = 0, behind_e = 0;
  auto round = [&](int& e) {
    const uint32_t top = __reduce_max_sync(FULL, best);
    e = __shfl_sync(FULL, at, __ffs(__ballot_sync(FULL, best == top)) - 1);  // of equal ones the lowest lane has the lowest numbers
    return top;
  };
  for (int j = 0; j < k; ++j) {
    int e;
    const uint32_t top = round(e);
    if (lane == j) { mine = top; id = e; }
    if (V <= 2 || e == at) {  // numbers are one lane's each
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (first + i == e) key[i] = 0;
      find();
    }
  }
  // A score for its weight: e^-x does not overflow (below -88 it is e^x to within 2^-126 of itself), and what rounding
  // l - max leaves off, up to 2^-18 where they are 64 apart, is made up for (the rest is a number while the difference is).
  auto score_of = [&](float x) {
    if (sigmoid) return x < -88.0f ? expf(x) : __frcp_rn(1.0f + expf(-x));
    const swiglu_math::ff d = swiglu_math::two_sum(x, -most);
    const float e = expf(d.hi);
    return d.hi > -120.0f ? fmaf(e, d.lo, e) * inv : 0.0f;
  };
  const bool has = lane < k;
  float x = has ? logit(row, wide, id) : 0.0f;
  float s = has ? score_of(x) : 0.0f;
  bool ordered = true;  // within the k
  float border = 0.0f;  // how far off the difference of one of the k and another may be
  if (p.bias) {
    behind = round(behind_e);
    const float b = has ? p.bias[id] : 0.0f, c1 = of_key(mine);
    const float x2 = __shfl_down_sync(FULL, x, 1), s2 = __shfl_down_sync(FULL, s, 1), b2 = __shfl_down_sync(FULL, b, 1);
    const uint32_t next = __shfl_down_sync(FULL, mine, 1);
    const float u1 = fmaxf(s, 0x1p-126f), own = sigmoid ? 0x1p-22f * u1 * (1.51f - u1) : 0x1.7p-22f * u1 - 0x1p-23f * u1 * __logf(u1);
    const float own2 = __shfl_down_sync(FULL, own, 1);
    // the least of the k may be another than the k-th, and off by more than it
    const float own_most = __uint_as_float(__reduce_max_sync(FULL, has ? __float_as_uint(own) : 0u));
    if (lane < k - 1) {
      const float c2 = of_key(next), rounding = 0x1.01p-24f * (fabsf(c1) + fabsf(c2)) + 0x1p-125f;
      const bool equal = (x == x2 && b == b2) || (c1 == c2 && isinf(c1));
      const float off = own + own2 + rounding + (sigmoid ? 0.0f : (V + 14) * 0x1p-24f * fabsf(s - s2));
      ordered = equal || c1 - c2 > off || c1 - c2 == INFINITY;  // (off is infinite with either)
    } else if (lane == k - 1 && behind) {  // against any that was not chosen: a score of the largest there is
      const float c2 = of_key(behind);
      border = own_most + (sigmoid ? 0x1.3p-23f : (V + 22) * 0x1p-24f * inv) + 0x1p-22f * fabsf(c1) + 0x1p-23f * fabsf(c2) + 0x1p-125f;
      sure = c1 - c2 > border || c1 - c2 == INFINITY || (c1 == c2 && isinf(c1));  // else border is finite
    }
  }
  int place = lane;
  const bool spoilt = __any_sync(FULL, bad);
  bool again = __any_sync(FULL, !sure || !sure_groups);
  bool contest = false;
  if (again && !spoilt && sure_groups) {
    // Equal by their inputs, all experts as near to the k-th as their scores are off, chosen or not?  Then numbers decide, as
    // they did: the others of the k are above these, those that are left below.
    const float xk = __shfl_sync(FULL, x, k - 1), ck = of_key(__shfl_sync(FULL, mine, k - 1));
    const float bk = p.bias[__shfl_sync(FULL, id, k - 1)], off = __shfl_sync(FULL, border, k - 1);
    bool equal = !has || of_key(mine) - ck > off || (x == xk && p.bias[id] == bk);
    int near = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] && !(ck - of_key(key[i]) > off)) {
        equal = equal && l[i] == xk && p.bias[first + i] == bk;
        ++near;
      }
    again = !__all_sync(FULL, equal);
    // one expert alone behind the k-th is put in order with the k (any other is below all of them)
    contest = again && k < 32 && warp_sum(near) == 1;
  }
  bool chosen = has;
  if (!spoilt && (contest || (!again && !__all_sync(FULL, ordered)))) {
    if (contest && lane == k) {
      id = behind_e;
      x = logit(row, wide, id);
      s = score_of(x);
    }
    bool fine;
    place = order_closely(p, row, most, contest ? k + 1 : k, id, x, &fine);
    chosen = lane < (contest ? k + 1 : k) && place < k;
    again = !fine;
    contest = false;
  }
  if (again && !spoilt) {
    // a token of equal logits (padding) is in doubt by its biases alone: sums that are alike to the last of 44 bits as well
    const bool flat = all_equal(l);
    bool fine = false;
    if (!flat && sure_groups) {
      const int size = E / p.groups;   // a group was taken if an expert of it is chosen or could have been
      uint32_t in = has ? 1u << id / size : 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i]) in |= 1u << (first + i) / size;
      id = route_closely(p, row, most, __reduce_or_sync(FULL, in), buf, &fine);
    }
    if (!fine) id = route_exactly(p, row, flat, buf);
    chosen = has;
    place = lane;
    x = has ? logit(row, wide, id) : 0.0f;
    s = has ? score_of(x) : 0.0f;
  }
  const float total = p.renorm ? warp_sum(chosen ? s : 0.0f) + 1e-20f : 1.0f;
  if (!chosen) return;
  float w = p.scale * (s / total);
  if (spoilt) {  // no order: the first k, and weights that say so
    id = place = lane;
    w = __uint_as_float(0x7FC00000u);
  }
  p.ids[t * k + place] = id;
  p.weights[t * k + place] = w;
}

struct RouteBwdParams {
  const float* dweights;  // [T, k]
  const void* logits;     // [T, E]
  const int32_t* ids;     // [T, k]
  int64_t T;
  int32_t E, k;
  int wide, sigmoid, renorm;
  int vec;                // rows of logits and dlogits can be read and written in vectors
  float scale;
  void* dlogits;          // [T, E], the logits' type
  int32_t* err;
};

// ds_j = scale (dw_j - (sum dw s) / t) / t with t = sum s + 1e-20 (scale dw_j without renormalisation);
// softmax: dl = s (ds - sum ds s), where sum ds s = scale (sum dw s) 1e-20 / t^2 with renormalisation;
// sigmoid: dl = ds s (1 - s), which lane j has for its expert and puts into the token's row in shared memory (a look at
// each of the k by all lanes took 16.0 against 8.4 us for 16384 tokens, 256 experts).  An expert that is named twice gets
// both gradients, added in their order.
template <int V, bool WIDE, bool SIGMOID>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) moe_route_bwd_kernel(RouteBwdParams p) {
  __shared__ __align__(16) float s_row[ROUTE_WARPS][32 * V];
  pdl_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp;
  if (t >= p.T) return;
  const int E = p.E, k = p.k, first = lane * V;
  constexpr bool sigmoid = SIGMOID, wide = WIDE;
  const void* row = reinterpret_cast<const uint8_t*>(p.logits) + (size_t)t * E * (wide ? 4 : 2);
  float* const buf = s_row[warp];
  int id = lane < k ? p.ids[t * k + lane] : -1;
  float dw = lane < k ? p.dweights[t * k + lane] : 0.0f;
  float l[V];
  float most = -INFINITY, inv = 1.0f;
  if (!sigmoid) load_values<V>(row, wide, p.vec, first, E, -INFINITY, l);
#pragma unroll
  for (int i = 0; i < V; ++i) buf[first + i] = 0.0f;
  if (!sigmoid) {
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) most = fmaxf(most, l[i]);
    most = warp_max(most);
    if (most == -INFINITY) most = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] = expf(l[i] - most);
      z += l[i];
    }
    z = warp_sum(z);
    inv = z != 0.0f ? 1.0f / z : 0.0f;
  }
  if (lane < k && (id < 0 || id >= E)) {
    record_error(p.err, MX_ERR_BAD_OFFSETS);
    id = -1;
    dw = 0.0f;
  }
  const float x = id >= 0 ? logit(row, wide, id) : 0.0f;
  const float q = expf(sigmoid ? -fabsf(x) : x - most), r = sigmoid ? 1.0f / (1.0f + q) : 0.0f;
  const float s = id < 0 ? 0.0f : !sigmoid ? q * inv : x >= 0.0f ? r : q * r;
  float ds = p.scale * dw, back = 0.0f;  // back: sum ds s
  if (p.renorm) {
    // From dw less that of the largest score, so that gradients which are alike leave nothing (k = 1: an exact 0):
    // dw - dot / t = d - (sum d s) / t + top (t - sum s) / t
    const uint32_t bits = __float_as_uint(s);  // s >= 0
    const float top = __shfl_sync(FULL, dw, __ffs(__ballot_sync(FULL, bits == __reduce_max_sync(FULL, bits))) - 1);
    const float d = dw - top, dot = warp_sum(d * s), sum = warp_sum(s);
    const float t = sum + 1e-20f, over = 1.0f / t, rest = (t - sum) * over;
    ds = p.scale * ((d - dot * over) + top * rest) * over;
    back = p.scale * ((dot + top * sum) * over) * rest;
  } else {
    back = p.scale * warp_sum(dw * s);
  }
  float mine = sigmoid ? ds * (q * r) * r : ds;   // s (1 - s) = q r r
  if (sigmoid && q == 0.0f) mine = 0.0f;          // a score of 0 or 1 (a logit of -inf: whatever ds is)
  // an expert named twice: one of the two finds the other's number in its place
  __syncwarp();
  if (id >= 0) buf[id] = (float)lane;
  __syncwarp();
  bool first_of = id >= 0;
  if (__any_sync(FULL, id >= 0 && buf[id] != (float)lane)) {
    const unsigned same = __match_any_sync(FULL, id >= 0 ? id : -1 - lane);
    first_of = first_of && lane == __ffs(same) - 1;
    float sum = 0.0f;
    for (int j = 0; j < k; ++j) {
      const float v = __shfl_sync(FULL, mine, j);
      if (same >> j & 1) sum += v;
    }
    mine = sum;
  }
  __syncwarp();
  if (first_of) buf[id] = mine;
  __syncwarp();
  float out[V];
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = sigmoid ? buf[first + i] : l[i] * inv * (buf[first + i] - back);
  if (first >= E) return;
  uint8_t* dst = reinterpret_cast<uint8_t*>(p.dlogits) + (size_t)t * E * (wide ? 4 : 2);
  if (p.vec && wide && V >= 4) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      reinterpret_cast<float4*>(dst)[first / 4 + i] = make_float4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
  } else if (p.vec && !wide && V >= 8) {
#pragma unroll
    for (int i = 0; i < V / 8; ++i)
      reinterpret_cast<uint4*>(dst)[first / 8 + i] =
          make_uint4(f2_to_bf16x2(f2_pack(out[8 * i], out[8 * i + 1])), f2_to_bf16x2(f2_pack(out[8 * i + 2], out[8 * i + 3])),
                     f2_to_bf16x2(f2_pack(out[8 * i + 4], out[8 * i + 5])), f2_to_bf16x2(f2_pack(out[8 * i + 6], out[8 * i + 7])));
  } else if (p.vec && wide && V == 2) {
    reinterpret_cast<float2*>(dst)[lane] = make_float2(out[0], out[V - 1]);
  } else if (p.vec && !wide && V > 1) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      reinterpret_cast<uint32_t*>(dst)[first / 2 + i] = f2_to_bf16x2(f2_pack(out[2 * i], out[2 * i + (V > 1)]));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (first + i >= E) break;
      if (wide) reinterpret_cast<float*>(dst)[first + i] = out[i];
      else reinterpret_cast<uint16_t*>(dst)[first + i] = (uint16_t)f32_to_bf16_bits(out[i]);
    }
  }
}

// f(width, wide, sigmoid) for the kernel of these.
template <class F>
cudaError_t for_kernel(int v, bool wide, bool sigmoid, F&& f) {
  auto kinds = [&](auto w) {
    using Yes = std::true_type;
    using No = std::false_type;
    return wide ? (sigmoid ? f(w, Yes{}, Yes{}) : f(w, Yes{}, No{})) : (sigmoid ? f(w, No{}, Yes{}) : f(w, No{}, No{}));
  };
  switch (v) {
    case 1: return kinds(std::integral_constant<int, 1>{});
    case 2: return kinds(std::integral_constant<int, 2>{});
    case 4: return kinds(std::integral_constant<int, 4>{});
    case 8: return kinds(std::integral_constant<int, 8>{});
    case 16: return kinds(std::integral_constant<int, 16>{});
    default: return kinds(std::integral_constant<int, 32>{});
  }
}
int route_width(int E) {
  int v = 1;
  while (32 * v < E) v *= 2;
  return v;
}

// Rows of E values of `size` bytes can be read V at a time, in vectors of 16 bytes at most.
bool in_vectors(const void* p, int E, int size, int v) {
  const int bytes = std::min(16, v * size);
  return E % v == 0 && (int64_t)E * size % bytes == 0 && reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

// ---------------------------------------------------------------- grouping

constexpr int TG_WARPS = 8;

// The lanes that have the same expert (below 2^bits; -1: none), bit by bit: a match instruction of 32 numbers takes longer
// (grouping 131072 rows over 64 experts 8.3 against 7.3 us).
MX_DEVINL unsigned lanes_like(int32_t e, int bits) {
  unsigned peers = __ballot_sync(FULL, e >= 0);
  if (e < 0) peers = ~peers;
  for (int b = 0; b < bits; ++b) {
    const unsigned one = __ballot_sync(FULL, e >> b & 1);
    peers &= e >> b & 1 ? one : ~one;
  }
  return peers;
}

// Rows r0 to r1 of a warp, 32 at a time in order: f(row, expert or -1, lanes of the same expert).
template <class F>
MX_DEVINL void walk(const int32_t* expert_of, int64_t r0, int64_t r1, int32_t E, F&& f) {
  const int lane = threadIdx.x & 31, bits = 32 - __clz(E - 1);
  for (int64_t rb = r0; rb < r1; rb += 32) {
    const int64_t r = rb + lane;
    int32_t e = r < r1 ? expert_of[r] : -1;
    if (e < 0 || e >= E) e = -1;
    f(r, e, lanes_like(e, bits));
  }
}

// Each CTA counts the experts of its chunk of rows.
__global__ void __launch_bounds__(TG_WARPS * 32)
    token_group_count_kernel(const int32_t* __restrict__ expert_of, int64_t R, int32_t E, int64_t chunk,
                             int32_t* __restrict__ counts) {
  extern __shared__ int32_t hist[];  // [E]
  pdl_begin();
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t c0 = blockIdx.x * chunk, c1 = min(R, c0 + chunk);
  for (int64_t r = c0 + threadIdx.x; r < c1; r += blockDim.x) {
    const int32_t e = expert_of[r];
    if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) counts[(int64_t)blockIdx.x * E + e] = hist[e];
}

// A row's place is its group's start, plus the group's rows in chunks before, in warps before, in earlier steps of the
// warp and in lower lanes.  Each CTA adds up the counts of the chunks before its own and of all; alone it needs none.
// ITER: steps of a warp's 32 rows, kept in registers; 0: any number, walked twice.
template <int WARPS, int ITER>
__global__ void __launch_bounds__(WARPS * 32)
    token_group_place_kernel(const int32_t* __restrict__ expert_of, int64_t R, int32_t E, int64_t chunk,
                             const int32_t* __restrict__ counts, int32_t* __restrict__ offs,
                             int32_t* __restrict__ row_dst, int32_t* __restrict__ row_src, int32_t* err) {
  extern __shared__ int32_t sm[];
  int32_t* next = sm;                  // [WARPS][E]
  int32_t* total = sm + WARPS * E;     // [E], then the groups' ends
  int32_t* before = total + E;         // [E]
  __shared__ int32_t warp_total[WARPS];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_chunks = gridDim.x, mine = blockIdx.x;
  const int64_t c0 = mine * chunk, c1 = min(R, c0 + chunk), share = chunk / WARPS;
  const int64_t w0 = min(c1, c0 + warp * share), w1 = min(c1, w0 + share);
  int32_t* h = next + warp * E;
  int32_t ex[ITER + 1], pos[ITER + 1];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int64_t r = w0 + i * 32 + lane;
    ex[i] = r < w1 ? expert_of[r] : -1;
  }
  for (int e = tid; e < (WARPS + 2) * E; e += WARPS * 32) sm[e] = 0;
  __syncthreads();
  if (n_chunks > 1) {
    // threads side by side take experts, and as many threads as there are for each share the chunks
    if (E % 4 == 0) {  // four at a time
      const int e4 = E / 4, parts4 = max(1, WARPS * 32 / e4);
      for (int i = tid; i < parts4 * e4; i += WARPS * 32) {
        const int q = i % e4;
        int4 all = make_int4(0, 0, 0, 0), b = all;
#pragma unroll 8
        for (int c = i / e4; c < n_chunks; c += parts4) {
          const int4 n = __ldg(reinterpret_cast<const int4*>(counts + (int64_t)c * E) + q);
          all.x += n.x, all.y += n.y, all.z += n.z, all.w += n.w;
          if (c < mine) b.x += n.x, b.y += n.y, b.z += n.z, b.w += n.w;
        }
        atomicAdd(&total[4 * q], all.x), atomicAdd(&total[4 * q + 1], all.y), atomicAdd(&total[4 * q + 2], all.z);
        atomicAdd(&total[4 * q + 3], all.w);
        atomicAdd(&before[4 * q], b.x), atomicAdd(&before[4 * q + 1], b.y), atomicAdd(&before[4 * q + 2], b.z);
        atomicAdd(&before[4 * q + 3], b.w);
      }
    }
    const int parts = E % 4 ? max(1, WARPS * 32 / E) : 0;
    for (int i = tid; i < parts * E; i += WARPS * 32) {
      const int e = i % E;
      int32_t all = 0, b = 0;
#pragma unroll 8
      for (int c = i / E; c < n_chunks; c += parts) {
        const int32_t n = counts[(int64_t)c * E + e];
        all += n;
        b += c < mine ? n : 0;
      }
      atomicAdd(&total[e], all);
      atomicAdd(&before[e], b);
    }
  }
  if (ITER) {
    const int bits = 32 - __clz(E - 1);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      if (ex[i] < 0 || ex[i] >= E) ex[i] = -1;
      const unsigned peers = lanes_like(ex[i], bits);
      pos[i] = ex[i] >= 0 ? h[ex[i]] + __popc(peers & ((1u << lane) - 1u)) : 0;
      __syncwarp();
      if (ex[i] >= 0 && lane == __ffs(peers) - 1) h[ex[i]] += __popc(peers);
      __syncwarp();
    }
  } else {
    walk(expert_of, w0, w1, E, [&](int64_t, int32_t e, unsigned peers) {
      if (e >= 0 && lane == __ffs(peers) - 1) h[e] += __popc(peers);
      __syncwarp();
    });
  }
  __syncthreads();
  for (int e = tid; e < E; e += WARPS * 32) {
    int32_t run = before[e];
#pragma unroll 8
    for (int w = 0; w < WARPS; ++w) {
      const int32_t n = next[w * E + e];
      next[w * E + e] = run;
      run += n;
    }
    if (n_chunks == 1) total[e] = run;
  }
  __syncthreads();
  // ends of the groups: each thread adds up neighbours, then the threads before it
  const int per = (E + WARPS * 32 - 1) / (WARPS * 32), e0 = tid * per;
  int32_t sum = 0;
  for (int i = 0; i < per && e0 + i < E; ++i) sum += total[e0 + i];
  int32_t run = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t v = __shfl_up_sync(FULL, run, o);
    if (lane >= o) run += v;
  }
  if (lane == 31) warp_total[warp] = run;
  __syncthreads();
  run -= sum;
  for (int w = 0; w < warp; ++w) run += warp_total[w];
  for (int i = 0; i < per && e0 + i < E; ++i) {
    const int32_t n = total[e0 + i];
    before[e0 + i] = run;   // now the group's start
    run += n;
    total[e0 + i] = run;
    if (mine == 0) offs[e0 + i] = run;
  }
  __syncthreads();
  const int32_t placed = total[E - 1];
  bool bad = false;
  auto put = [&](int64_t r, int32_t e, int32_t at) {
    row_dst[r] = at;
    if (e >= 0) row_src[at] = (int32_t)r;
    else bad = true;
    if (r >= placed) row_src[r] = -1;
  };
  if (ITER) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int64_t r = w0 + i * 32 + lane;
      if (r < w1) put(r, ex[i], ex[i] >= 0 ? before[ex[i]] + h[ex[i]] + pos[i] : -1);
    }
  } else {
    walk(expert_of, w0, w1, E, [&](int64_t r, int32_t e, unsigned peers) {
      const int32_t at = e >= 0 ? before[e] + h[e] + __popc(peers & ((1u << lane) - 1u)) : -1;
      __syncwarp();
      if (e >= 0 && lane == __ffs(peers) - 1) h[e] += __popc(peers);
      __syncwarp();
      if (r < w1) put(r, e, at);
    });
  }
  if (__any_sync(FULL, bad) && lane == 0) record_error(err, MX_ERR_BAD_OFFSETS);
}

}  // namespace

int launch_moe_route(const RouteLaunch& a, cudaStream_t stream) {
  const int v = route_width(a.E);
  RouteParams p{};
  p.logits = a.logits; p.bias = a.bias; p.T = a.T; p.E = a.E; p.k = a.k; p.groups = a.groups; p.top_groups = a.top_groups;
  p.wide = a.wide; p.sigmoid = a.score == MX_SCORE_SIGMOID; p.renorm = a.renorm; p.scale = a.scale; p.ids = a.ids;
  p.weights = a.weights;
  p.vec = in_vectors(a.logits, a.E, a.wide ? 4 : 2, v);
  p.vec_bias = in_vectors(a.bias, a.E, 4, v);
  count_launch(MX_KERNEL_ROUTE);
  return cuda_status(for_kernel(v, a.wide, p.sigmoid, [&](auto w, auto wide, auto sigmoid) {
    return launch_overlapped(moe_route_kernel<decltype(w)::value, decltype(wide)::value, decltype(sigmoid)::value>, (unsigned)((a.T + ROUTE_WARPS - 1) / ROUTE_WARPS),
                             ROUTE_WARPS * 32, (size_t)ROUTE_WARPS * a.E * 8, stream, 1, p);
  }), "moe_route_kernel launch");
}

int launch_moe_route_bwd(const RouteBwdLaunch& a, cudaStream_t stream) {
  const int v = route_width(a.E);
  RouteBwdParams p{};
  p.dweights = a.dweights; p.logits = a.logits; p.ids = a.ids; p.T = a.T; p.E = a.E; p.k = a.k; p.wide = a.wide;
  p.sigmoid = a.score == MX_SCORE_SIGMOID; p.renorm = a.renorm; p.scale = a.scale; p.dlogits = a.dlogits; p.err = a.err;
  p.vec = in_vectors(a.logits, a.E, a.wide ? 4 : 2, v) && in_vectors(a.dlogits, a.E, a.wide ? 4 : 2, v);
  count_launch(MX_KERNEL_ROUTE);
  return cuda_status(for_kernel(v, a.wide, p.sigmoid, [&](auto w, auto wide, auto sigmoid) {
    return launch_overlapped(moe_route_bwd_kernel<decltype(w)::value, decltype(wide)::value, decltype(sigmoid)::value>, (unsigned)((a.T + ROUTE_WARPS - 1) / ROUTE_WARPS),
                             ROUTE_WARPS * 32, 0, stream, 1, p);
  }), "moe_route_bwd_kernel launch");
}

namespace {
// Up to 8192 rows one large CTA does it all, if its warps' counts fit 48 KB; 1024 rows one small one.
bool one_cta(int64_t R, int32_t E) { return R <= 1024 || (R <= 8192 && E <= 352); }
constexpr int64_t TG_MOST_CHUNKS = 512;  // on a device of any size: two for each SM of 256
}  // namespace

size_t token_group_workspace(int64_t R, int32_t E) {
  // for any number of SMs: a chunk has 1024 rows at least
  return one_cta(R, E) ? 0 : (size_t)std::min<int64_t>((R + 1023) / 1024, TG_MOST_CHUNKS) * (size_t)E * 4;
}

int launch_token_group(const int32_t* expert_of, int64_t R, int32_t E, int32_t* offs, int32_t* row_dst, int32_t* row_src,
                       void* workspace, int32_t* err, cudaStream_t stream) {
  int32_t* counts = reinterpret_cast<int32_t*>(workspace);
  auto place = [&](auto k, unsigned grid, int warps, int64_t chunk) {
    count_launch(MX_KERNEL_DISPATCH);
    return cuda_status(launch_overlapped(k, grid, warps * 32, (size_t)(warps + 2) * E * 4, stream, 1, expert_of, R, E, chunk,
                                         (const int32_t*)counts, offs, row_dst, row_src, err),
                       "token_group_place_kernel launch");
  };
  if (one_cta(R, E) && E <= 352) {
    if (R <= 1024) return place(token_group_place_kernel<32, 1>, 1, 32, 1024);
    if (R <= 2048) return place(token_group_place_kernel<32, 2>, 1, 32, 2048);
    if (R <= 4096) return place(token_group_place_kernel<32, 4>, 1, 32, 4096);
    return place(token_group_place_kernel<32, 8>, 1, 32, 8192);
  }
  // chunks of 1024 rows while each SM has two of them at most, larger ones else: a CTA reads every chunk's counts
  const int64_t most = std::min<int64_t>(2 * (int64_t)num_sms(), TG_MOST_CHUNKS);
  const int64_t chunk = std::max<int64_t>(1024, ((R + most - 1) / most + 255) / 256 * 256);
  const unsigned grid = (unsigned)((R + chunk - 1) / chunk);
  if (grid > 1) {  // the chunks are counted first
    count_launch(MX_KERNEL_DISPATCH);
    const cudaError_t e = launch_overlapped(token_group_count_kernel, grid, TG_WARPS * 32, (size_t)E * 4, stream, 1, expert_of, R, E,
                                            chunk, counts);
    if (e != cudaSuccess) return cuda_status(e, "token_group_count_kernel launch");
  }
  return chunk == 1024 ? place(token_group_place_kernel<TG_WARPS, 4>, grid, TG_WARPS, chunk)
                       : place(token_group_place_kernel<TG_WARPS, 0>, grid, TG_WARPS, chunk);
}

}  // namespace mx
