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
// bounded: a warp has a token, finds the k + 1 largest c, and where two neighbours among them (or the
// groups at the border) are closer than the bounds of both allow, and are not equal by their inputs, it
// orders the token's experts again in double precision.  Without a bias and groups the logits themselves
// are the order and there is nothing to bound.
//
// Bounds of fp32 scores.  expf is off by 1 ulp (2^-23), l - max is rounded by 2^-24 |l - max|, which is at
// most 2^-24 (-ln s); sums of E terms in a tree of V + 5 levels by 2^-24 each, and with the exponentials'
// own errors (their mean |l - max| is at most ln E) by less than 2^-18; it scales all scores of a token
// alike, so two scores' difference by that much of itself.  Underflow ends at 2^-126.
#include "common.cuh"
#include "kernels.h"

namespace mx {

namespace {

constexpr uint32_t FULL = 0xFFFFFFFFu;
constexpr int ROUTE_WARPS = 4;

template <bool WIDE>
MX_DEVINL float logit(const void* row, int e) {
  // + 0: -0 and 0 are one value
  return WIDE ? reinterpret_cast<const float*>(row)[e] + 0.0f
              : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[e] << 16) + 0.0f;
}

// Larger floats have larger keys; 0 is below all of them (NaN does not occur).
MX_DEVINL uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
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
  int renorm;
  float scale;
  int32_t* ids;           // [T, k]
  float* weights;         // [T, k]
};

// The groups taken, as bits, from the values that lane g has for group g; *sure: no other
// choice is within `off` of it.
template <class T>
MX_DEVINL uint32_t take_groups(T value, int groups, int top, T off, bool* sure) {
  const int lane = threadIdx.x & 31;
  int rank = 0;
  for (int g = 0; g < groups; ++g) {
    const T v = __shfl_sync(FULL, value, g);
    if (v > value || (v == value && g < lane)) ++rank;
  }
  const uint32_t taken = __ballot_sync(FULL, lane < groups && rank < top);
  const uint32_t last = __ballot_sync(FULL, lane < groups && rank == top - 1);
  const uint32_t next = __ballot_sync(FULL, lane < groups && rank == top);
  if (next) {
    const T a = __shfl_sync(FULL, value, __ffs(last) - 1), b = __shfl_sync(FULL, value, __ffs(next) - 1);
    *sure = a - b > off || (a == b && isinf(a));
  }
  return taken;
}

// The two largest of a group's values, added.
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
  return size > 1 ? a + b : a;
}

// A token's experts in double precision, by one warp: lane j returns the j-th.
template <bool WIDE, bool SIGMOID>
__device__ __noinline__ int route_exactly(const RouteParams& p, const void* row, double* c) {
  const int lane = threadIdx.x & 31;
  const int E = p.E, n = (E + 31) / 32;
  __syncwarp();
  double most = -INFINITY, z = 0;
  for (int i = 0; i < n; ++i) {
    const int e = lane + 32 * i;
    if (e < E) most = fmax(most, (double)logit<WIDE>(row, e));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) most = fmax(most, __shfl_xor_sync(FULL, most, o));
  if (most == -INFINITY) most = 0;
  for (int i = 0; i < n; ++i) {
    const int e = lane + 32 * i;
    if (e >= E) continue;
    const double l = logit<WIDE>(row, e);
    const double v = SIGMOID ? 1 / (1 + exp(-l)) : exp(l - most);
    c[e] = v;
    z += v;
  }
  z = warp_sum(z);
  for (int i = 0; i < n; ++i) {
    const int e = lane + 32 * i;
    if (e >= E) continue;
    double v = SIGMOID ? c[e] : z > 0 ? c[e] / z : 0.0;
    if (p.bias) v += (double)p.bias[e];
    if (logit<WIDE>(row, e) == -INFINITY) v = -INFINITY;
    c[e] = v;
  }
  __syncwarp();
  uint32_t taken = 0;  // bit i: expert lane + 32 i is chosen, or of no group that is
  if (p.groups > 1) {
    const int size = E / p.groups;
    bool sure = true;
    const double v = lane < p.groups ? group_value(c + lane * size, size, lane % size) : 0.0;
    const uint32_t in = take_groups(v, p.groups, p.top_groups, 0.0, &sure);
    for (int i = 0; i < n; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !(in >> (e / size) & 1)) taken |= 1u << i;
    }
  }
  if (!p.bias) {  // the logits' own order
    __syncwarp();
    for (int i = 0; i < n; ++i) {
      const int e = lane + 32 * i;
      if (e < E) c[e] = logit<WIDE>(row, e);
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

// A warp has a token; lane i experts i V to i V + V - 1.
template <int V, bool WIDE, bool SIGMOID>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) moe_route_kernel(RouteParams p) {
  extern __shared__ double s_c[];
  pdl_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp;
  if (t >= p.T) return;
  double* const buf = s_c + (size_t)warp * p.E;
  const int E = p.E, k = p.k, first = lane * V;
  const void* row = reinterpret_cast<const uint8_t*>(p.logits) + (size_t)t * E * (WIDE ? 4 : 2);
  float l[V];
  bool bad = false;
  float most = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    l[i] = first + i < E ? logit<WIDE>(row, first + i) : -INFINITY;
    bad |= l[i] != l[i] || (!SIGMOID && l[i] == INFINITY);
    most = fmaxf(most, l[i]);
  }
  float inv = 1.0f;
  const bool need_scores = p.bias || p.groups > 1;
  if (!SIGMOID) {
    most = warp_max(most);
    if (most == -INFINITY) most = 0.0f;
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) z += expf(l[i] - most);
    z = warp_sum(z);
    inv = z > 0.0f ? 1.0f / z : 0.0f;
  }
  auto score = [&](float x) { return SIGMOID ? 1.0f / (1.0f + expf(-x)) : expf(x - most) * inv; };
  uint32_t key[V];
  float c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] = l[i];
    if (need_scores) {
      const float s = score(l[i]);
      float b = 0.0f;
      if (p.bias && first + i < E) b = p.bias[first + i];
      bad |= b != b;
      c[i] = l[i] == -INFINITY ? -INFINITY : s + b;
      bad |= c[i] != c[i];
    }
    key[i] = first + i < E ? key_of(p.bias ? c[i] : l[i]) : 0;
  }
  if (__any_sync(FULL, bad)) {  // no order: the first k, and weights that say so
    if (lane < k) {
      p.ids[t * k + lane] = lane;
      p.weights[t * k + lane] = __uint_as_float(0x7FC00000u);
    }
    return;
  }
  bool sure = true;
  if (p.groups > 1) {
    const int size = E / p.groups;
    float* cf = reinterpret_cast<float*>(buf);
    float largest = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (first + i < E) {
        cf[first + i] = c[i];
        if (c[i] != -INFINITY) largest = fmaxf(largest, fabsf(c[i]));
      }
    __syncwarp();
    const float v = lane < p.groups ? group_value(cf + lane * size, size, lane % size) : 0.0f;
    // a score is off by 2^-18 of the largest at most, a sum of two by twice that; c and the sum are rounded
    const float off = 0x1p-16f * (SIGMOID ? 1.0f : inv) + 0x1p-20f * warp_max(largest);
    const uint32_t in = take_groups(v, p.groups, p.top_groups, off, &sure);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (first + i < E && !(in >> ((first + i) / size) & 1)) key[i] = 0;
  }
  // the k largest, and the one behind them
  uint32_t best = 0;
  int at = 0;
  auto find = [&] {
    best = key[0];
    at = 0;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (key[i] > best) { best = key[i]; at = i; }
  };
  find();
  uint32_t mine = 0, next = 0;  // keys of the lane's expert and of the one behind it
  int id = 0, next_id = 0;
  for (int j = 0; j <= k; ++j) {
    const uint32_t top = __reduce_max_sync(FULL, best);
    const int owner = __ffs(__ballot_sync(FULL, best == top)) - 1;  // of equal ones the lowest lane has the lowest numbers
    const int e = __shfl_sync(FULL, first + at, owner);
    if (lane == j) { mine = top; id = e; }
    if (lane == j - 1) { next = top; next_id = e; }
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == at) key[i] = 0;
      find();
    }
  }
  float x = lane < k ? logit<WIDE>(row, id) : 0.0f;
  float s = lane < k ? score(x) : 0.0f;
  if (p.bias && lane < k && next) {
    const float x2 = logit<WIDE>(row, next_id), s2 = score(x2);
    const float c1 = of_key(mine), c2 = of_key(next);
    const bool equal = (x == x2 && p.bias[id] == p.bias[next_id]) || (c1 == c2 && isinf(c1));
    const float u1 = fmaxf(s, 0x1p-126f), u2 = fmaxf(s2, 0x1p-126f);
    float off = (u1 + u2) * 0x1p-21f + 0x1p-23f * (fabsf(c1) + fabsf(c2));
    if (!SIGMOID) off += 0x1p-18f * fabsf(s - s2) - 0x1p-23f * (u1 * __logf(u1) + u2 * __logf(u2));
    if (!equal && !(c1 - c2 > off)) sure = false;
  }
  if (!__all_sync(FULL, sure)) {
    id = route_exactly<WIDE, SIGMOID>(p, row, buf);
    x = lane < k ? logit<WIDE>(row, id) : 0.0f;
    s = lane < k ? score(x) : 0.0f;
  }
  const float total = p.renorm ? warp_sum(s) + 1e-20f : 1.0f;
  if (lane < k) {
    p.ids[t * k + lane] = id;
    p.weights[t * k + lane] = p.scale * (s / total);
  }
}

struct RouteBwdParams {
  const float* dweights;  // [T, k]
  const void* logits;     // [T, E]
  const int32_t* ids;     // [T, k]
  int64_t T;
  int32_t E, k;
  int renorm;
  float scale;
  void* dlogits;          // [T, E], the logits' type
  int32_t* err;
};

// ds_j = scale (dw_j - (sum dw s) / t) / t with t = sum s + 1e-20 (scale dw_j without renormalisation);
// softmax: dl = s (ds - sum ds s), where sum ds s = scale (sum dw s) 1e-20 / t^2 with renormalisation;
// sigmoid: dl = ds s (1 - s).  An expert that is named twice gets both gradients.
template <int V, bool WIDE, bool SIGMOID>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) moe_route_bwd_kernel(RouteBwdParams p) {
  pdl_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp;
  if (t >= p.T) return;
  const int E = p.E, k = p.k, first = lane * V;
  const void* row = reinterpret_cast<const uint8_t*>(p.logits) + (size_t)t * E * (WIDE ? 4 : 2);
  float l[V];
  float most = -INFINITY, z = 0.0f, inv = 1.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    l[i] = first + i < E ? logit<WIDE>(row, first + i) : -INFINITY;
    most = fmaxf(most, l[i]);
  }
  if (!SIGMOID) {
    most = warp_max(most);
    if (most == -INFINITY) most = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) z += expf(l[i] - most);
    z = warp_sum(z);
    inv = z != 0.0f ? 1.0f / z : 0.0f;
  }
  int id = lane < k ? p.ids[t * k + lane] : -1;
  const float dw = lane < k ? p.dweights[t * k + lane] : 0.0f;
  if (lane < k && (id < 0 || id >= E)) {
    record_error(p.err, MX_ERR_BAD_OFFSETS);
    id = -1;
  }
  const float x = id >= 0 ? logit<WIDE>(row, id) : 0.0f;
  const float s = id < 0 ? 0.0f : SIGMOID ? 1.0f / (1.0f + expf(-x)) : expf(x - most) * inv;
  float ds = p.scale * dw, back = 0.0f;  // back: sum ds s
  const float dot = warp_sum(id >= 0 ? dw * s : 0.0f);
  if (p.renorm) {
    const float total = warp_sum(s) + 1e-20f;
    ds = p.scale * (dw - dot / total) / total;
    back = p.scale * (dot / total) * (1e-20f / total);
  } else {
    back = p.scale * dot;
  }
  float out[V];
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int e = __shfl_sync(FULL, id, j);
    const float v = __shfl_sync(FULL, ds, j);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e == first + i) out[i] += v;
  }
  uint8_t* dst = reinterpret_cast<uint8_t*>(p.dlogits) + (size_t)t * E * (WIDE ? 4 : 2);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (first + i >= E) break;
    float d;
    if (SIGMOID) {
      const float q = expf(-fabsf(l[i]));  // s (1 - s) = q / (1 + q)^2
      d = out[i] == 0.0f ? 0.0f : out[i] * (q / ((1.0f + q) * (1.0f + q)));
    } else {
      d = expf(l[i] - most) * inv * (out[i] - back);
    }
    if (WIDE) reinterpret_cast<float*>(dst)[first + i] = d;
    else reinterpret_cast<uint16_t*>(dst)[first + i] = (uint16_t)f32_to_bf16_bits(d);
  }
}

// ---------------------------------------------------------------- grouping

constexpr int TG_WARPS = 8;

// Rows r0 to r1 of a warp, 32 at a time in order: f(row, expert or -1, lanes of the same expert).
template <class F>
MX_DEVINL void walk(const int32_t* expert_of, int64_t r0, int64_t r1, int32_t E, F&& f) {
  const int lane = threadIdx.x & 31;
  for (int64_t rb = r0; rb < r1; rb += 32) {
    const int64_t r = rb + lane;
    int32_t e = r < r1 ? expert_of[r] : -1;
    if (e < 0 || e >= E) e = -1;
    const unsigned peers = __match_any_sync(FULL, e >= 0 ? e : -1 - lane);
    f(r, e, peers);
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

// Each CTA adds up the chunks before its own and all of them, and places its rows: a row's place is its group's start,
// plus the group's rows in chunks before, in warps before, in earlier steps of the warp and in lower lanes.
__global__ void __launch_bounds__(TG_WARPS * 32)
    token_group_place_kernel(const int32_t* __restrict__ expert_of, int64_t R, int32_t E, int64_t chunk,
                             const int32_t* __restrict__ counts, int32_t* __restrict__ offs,
                             int32_t* __restrict__ row_dst, int32_t* __restrict__ row_src, int32_t* err) {
  extern __shared__ int32_t sm[];
  int32_t* next = sm;              // [TG_WARPS][E]
  int32_t* total = sm + TG_WARPS * E;  // [E], then the groups' ends
  __shared__ int32_t warp_total[TG_WARPS];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_chunks = gridDim.x, mine = blockIdx.x;
  const int64_t c0 = mine * chunk, c1 = min(R, c0 + chunk), share = chunk / TG_WARPS;
  const int64_t w0 = min(c1, c0 + warp * share), w1 = min(c1, w0 + share);
  int32_t* h = next + warp * E;
  for (int e = tid; e < TG_WARPS * E; e += blockDim.x) next[e] = 0;
  __syncthreads();
  walk(expert_of, w0, w1, E, [&](int64_t, int32_t e, unsigned peers) {
    if (e >= 0 && lane == __ffs(peers) - 1) h[e] += __popc(peers);
    __syncwarp();
  });
  __syncthreads();
  for (int e = tid; e < E; e += blockDim.x) {
    int32_t before = 0, all = 0;
    if (n_chunks > 1) {
      for (int c = 0; c < n_chunks; ++c) {
        const int32_t n = counts[(int64_t)c * E + e];
        all += n;
        if (c < mine) before += n;
      }
    } else {
      for (int w = 0; w < TG_WARPS; ++w) all += next[w * E + e];
    }
    total[e] = all;
    for (int w = 0; w < TG_WARPS; ++w) {
      const int32_t n = next[w * E + e];
      next[w * E + e] = before;
      before += n;
    }
  }
  __syncthreads();
  // ends of the groups: each thread adds up neighbours, then the threads before it
  const int per = (E + blockDim.x - 1) / blockDim.x, e0 = tid * per;
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
    for (int w = 0; w < TG_WARPS; ++w) next[w * E + e0 + i] += run;
    run += n;
    total[e0 + i] = run;
    if (mine == 0) offs[e0 + i] = run;
  }
  __syncthreads();
  const int32_t placed = total[E - 1];
  bool bad = false;
  walk(expert_of, w0, w1, E, [&](int64_t r, int32_t e, unsigned peers) {
    const int32_t pos = e >= 0 ? h[e] + __popc(peers & ((1u << lane) - 1u)) : -1;
    __syncwarp();
    if (e >= 0 && lane == __ffs(peers) - 1) h[e] += __popc(peers);
    __syncwarp();
    if (r < w1) {
      row_dst[r] = pos;
      if (e >= 0) row_src[pos] = (int32_t)r;
      else bad = true;
      if (r >= placed) row_src[r] = -1;
    }
  });
  if (__any_sync(FULL, bad) && lane == 0) record_error(err, MX_ERR_BAD_OFFSETS);
}

int64_t group_chunk(int64_t R) {
  const int64_t most = 2 * (int64_t)num_sms();
  const int64_t c = std::max<int64_t>(1024, (R + most - 1) / most);
  return (c + 32 * TG_WARPS - 1) / (32 * TG_WARPS) * (32 * TG_WARPS);
}

template <int V, bool WIDE>
cudaError_t route_v(const RouteLaunch& a, cudaStream_t stream) {
  RouteParams p{};
  p.logits = a.logits; p.bias = a.bias; p.T = a.T; p.E = a.E; p.k = a.k; p.groups = a.groups; p.top_groups = a.top_groups;
  p.renorm = a.renorm; p.scale = a.scale; p.ids = a.ids; p.weights = a.weights;
  const size_t smem = (size_t)ROUTE_WARPS * a.E * 8;
  const unsigned grid = (unsigned)((a.T + ROUTE_WARPS - 1) / ROUTE_WARPS);
  auto kern = a.score == MX_SCORE_SIGMOID ? moe_route_kernel<V, WIDE, true> : moe_route_kernel<V, WIDE, false>;
  return launch_overlapped(kern, grid, ROUTE_WARPS * 32, smem, stream, 1, p);
}

template <int V, bool WIDE>
cudaError_t route_bwd_v(const RouteBwdLaunch& a, cudaStream_t stream) {
  RouteBwdParams p{};
  p.dweights = a.dweights; p.logits = a.logits; p.ids = a.ids; p.T = a.T; p.E = a.E; p.k = a.k; p.renorm = a.renorm;
  p.scale = a.scale; p.dlogits = a.dlogits; p.err = a.err;
  const unsigned grid = (unsigned)((a.T + ROUTE_WARPS - 1) / ROUTE_WARPS);
  auto kern = a.score == MX_SCORE_SIGMOID ? moe_route_bwd_kernel<V, WIDE, true> : moe_route_bwd_kernel<V, WIDE, false>;
  return launch_overlapped(kern, grid, ROUTE_WARPS * 32, 0, stream, 1, p);
}

}  // namespace

int launch_moe_route(const RouteLaunch& a, cudaStream_t stream) {
  count_launch(MX_KERNEL_ROUTE);
  auto go = [&](auto f16, auto f32) { return a.wide ? f32(a, stream) : f16(a, stream); };
  cudaError_t e;
  if (a.E <= 32) e = go(route_v<1, false>, route_v<1, true>);
  else if (a.E <= 64) e = go(route_v<2, false>, route_v<2, true>);
  else if (a.E <= 128) e = go(route_v<4, false>, route_v<4, true>);
  else if (a.E <= 256) e = go(route_v<8, false>, route_v<8, true>);
  else if (a.E <= 512) e = go(route_v<16, false>, route_v<16, true>);
  else e = go(route_v<32, false>, route_v<32, true>);
  return cuda_status(e, "moe_route_kernel launch");
}

int launch_moe_route_bwd(const RouteBwdLaunch& a, cudaStream_t stream) {
  count_launch(MX_KERNEL_ROUTE);
  auto go = [&](auto f16, auto f32) { return a.wide ? f32(a, stream) : f16(a, stream); };
  cudaError_t e;
  if (a.E <= 32) e = go(route_bwd_v<1, false>, route_bwd_v<1, true>);
  else if (a.E <= 64) e = go(route_bwd_v<2, false>, route_bwd_v<2, true>);
  else if (a.E <= 128) e = go(route_bwd_v<4, false>, route_bwd_v<4, true>);
  else if (a.E <= 256) e = go(route_bwd_v<8, false>, route_bwd_v<8, true>);
  else if (a.E <= 512) e = go(route_bwd_v<16, false>, route_bwd_v<16, true>);
  else e = go(route_bwd_v<32, false>, route_bwd_v<32, true>);
  return cuda_status(e, "moe_route_bwd_kernel launch");
}

size_t token_group_workspace(int64_t R, int32_t E) {
  // for any number of SMs: a chunk has 1024 rows at least
  return (size_t)((R + 1023) / 1024) * (size_t)E * 4;
}

int launch_token_group(const int32_t* expert_of, int64_t R, int32_t E, int32_t* offs, int32_t* row_dst, int32_t* row_src,
                       void* workspace, int32_t* err, cudaStream_t stream) {
  const int64_t chunk = group_chunk(R);
  const unsigned grid = (unsigned)((R + chunk - 1) / chunk);
  int32_t* counts = reinterpret_cast<int32_t*>(workspace);
  cudaError_t e;
  if (grid > 1) {
    count_launch(MX_KERNEL_DISPATCH);
    e = launch_overlapped(token_group_count_kernel, grid, TG_WARPS * 32, (size_t)E * 4, stream, 1, expert_of, R, E, chunk, counts);
    if (e != cudaSuccess) return cuda_status(e, "token_group_count_kernel launch");
  }
  count_launch(MX_KERNEL_DISPATCH);
  e = launch_overlapped(token_group_place_kernel, grid, TG_WARPS * 32, (size_t)(TG_WARPS + 1) * E * 4, stream, 1, expert_of, R,
                        E, chunk, (const int32_t*)counts, offs, row_dst, row_src, err);
  return cuda_status(e, "token_group_place_kernel launch");
}

}  // namespace mx
