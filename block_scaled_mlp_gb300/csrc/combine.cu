// combine.cu - expert rows back to tokens: the weighted sum of a token's k rows, and its gradients.
//
//   out[t] = add[t] + sum_j w[t, j] rows[dst[t k + j]]             in fp32, one rounding to bf16
//   drows[dst[t k + j]] = w[t, j] dout[t],   dw[t, j] = dout[t] . rows[dst[t k + j]]
//
// A negative dst is a row that was not placed (it adds nothing, its dw is 0); rows that hold no routed
// row (src < 0: padding) get zeros.
// Both are bound by HBM: the forward pass reads the rows, the backward pass reads and writes them, and goes by
// tokens rather than by rows, so that dout is read once (by rows it would be read k times, from HBM where
// [T, d] does not fit L2).  On a GB300 whose copy runs at 6.78 TB/s: 16384 tokens of 8 rows of 7168 with an addend 378 us
// (6.2 TB/s) and, backward, 600 us (6.6 TB/s); 8 tokens 3.1 and 2.9 us.
#include "common.cuh"
#include "kernels.h"

namespace mx {

namespace {

constexpr int CB_THREADS = 256;

struct CombineParams {
  const uint4* rows;      // [n_rows, d] bf16
  int64_t n_rows;
  uint32_t d8;            // d / 8
  const int32_t* dst;     // [T k]
  int64_t T;
  int32_t k;
  const float* weights;   // [T, k] or NULL
  const uint4* add;       // [T, d] or NULL
  uint4* out;             // [T, d]
  int32_t* err;
};

MX_DEVINL void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
MX_DEVINL uint4 pack_bf16x8(const float (&f)[8]) {
  return make_uint4(f2_to_bf16x2(f2_pack(f[0], f[1])), f2_to_bf16x2(f2_pack(f[2], f[3])), f2_to_bf16x2(f2_pack(f[4], f[5])),
                    f2_to_bf16x2(f2_pack(f[6], f[7])));
}

// A thread has 8 columns of a token.
__global__ void __launch_bounds__(CB_THREADS) moe_combine_kernel(CombineParams p) {
  pdl_begin();
  const int64_t t = blockIdx.x;
  const uint32_t c = blockIdx.y * CB_THREADS + threadIdx.x;
  if (c >= p.d8) return;
  float acc[8] = {};
  if (p.add) unpack8(__ldg(p.add + t * p.d8 + c), acc);
  const int32_t* dst = p.dst + t * p.k;
  const float* w = p.weights ? p.weights + t * p.k : nullptr;
  bool bad = false;
#pragma unroll 4
  for (int j = 0; j < p.k; ++j) {
    const int32_t r = dst[j];
    bad |= r >= p.n_rows;
    if (r < 0 || r >= p.n_rows) continue;
    float f[8];
    unpack8(__ldg(p.rows + r * (int64_t)p.d8 + c), f);
    const float wj = w ? w[j] : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(wj, f[i], acc[i]);
  }
  if (bad && c == 0) record_error(p.err, MX_ERR_BAD_OFFSETS);
  p.out[t * p.d8 + c] = pack_bf16x8(acc);
}

struct CombineBwdParams {
  const uint4* dout;      // [T, d] bf16
  const uint4* rows;      // [n_rows, d]
  int64_t n_rows;
  uint32_t d8;
  const int32_t* dst;     // [T k]
  const int32_t* src;     // [n_rows]
  int64_t T;
  int32_t k;
  const float* weights;   // [T, k]
  uint4* drows;           // [n_rows, d]
  float* dweights;        // [T, k]
  int32_t* err;
};

constexpr int CB_WARPS = CB_THREADS / 32;

// A CTA has a token, and all of its rows or (few tokens) one of them; its share of the rows without a routed row besides.
// One row of a token at a time, in step: with rows on their way ahead of one another, or without the barrier between them,
// more rows are open at once than DRAM's pages bear (16384 tokens of 8 rows of 7168: 604 against 818 and 646 us).
__global__ void __launch_bounds__(CB_THREADS) moe_combine_bwd_kernel(CombineBwdParams p) {
  __shared__ float part[CB_WARPS];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t = blockIdx.x;
  const int j0 = gridDim.y > 1 ? blockIdx.y : 0, j1 = gridDim.y > 1 ? j0 + 1 : p.k;
  for (int j = j0; j < j1; ++j) {
    const int32_t r = p.dst[t * p.k + j];
    float dot = 0.0f;
    bool bad = r >= p.n_rows;
    if (r >= 0 && r < p.n_rows) {
      const float w = p.weights[t * p.k + j];
      bad = p.src[r] != t * p.k + j;  // another's row: not written
      for (uint32_t c = tid; c < p.d8; c += CB_THREADS) {
        float g[8], f[8];
        unpack8(__ldg(p.dout + t * p.d8 + c), g);
        unpack8(__ldg(p.rows + r * (int64_t)p.d8 + c), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot = fmaf(g[i], f[i], dot);
          g[i] *= w;
        }
        if (!bad) p.drows[r * (int64_t)p.d8 + c] = pack_bf16x8(g);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
    __syncthreads();
    if (lane == 0) part[warp] = dot;
    __syncthreads();
    if (tid == 0) {
      float s = 0.0f;
      for (int i = 0; i < CB_WARPS; ++i) s += part[i];
      p.dweights[t * p.k + j] = s;
      if (bad) record_error(p.err, MX_ERR_BAD_OFFSETS);
    }
  }
  // a lane looks at a row, all threads write the zeros
  const int64_t ctas = (int64_t)gridDim.x * gridDim.y, share = (p.n_rows + ctas - 1) / ctas;
  const int64_t i0 = (t * gridDim.y + blockIdx.y) * share, i1 = min(p.n_rows, i0 + share);
  for (int64_t base = i0; base < i1; base += 32) {
    const int64_t i = base + lane;
    const int32_t s = i < i1 ? p.src[i] : -1;
    const bool lost = s >= 0 && (s >= p.T * p.k || p.dst[s] != i);  // no token's
    if (lost && warp == 0) record_error(p.err, MX_ERR_BAD_OFFSETS);
    for (uint32_t spare = __ballot_sync(0xFFFFFFFFu, i < i1 && (s < 0 || lost)); spare; spare &= spare - 1) {
      uint4* row = p.drows + (base + __ffs(spare) - 1) * p.d8;
      for (uint32_t c = tid; c < p.d8; c += CB_THREADS) row[c] = make_uint4(0, 0, 0, 0);
    }
  }
}

}  // namespace

int launch_moe_combine(const CombineLaunch& a, cudaStream_t stream) {
  CombineParams p{};
  p.rows = (const uint4*)a.rows; p.n_rows = a.n_rows; p.d8 = (uint32_t)(a.d / 8); p.dst = a.row_dst; p.T = a.T; p.k = a.k;
  p.weights = a.weights; p.add = (const uint4*)a.add; p.out = (uint4*)a.out; p.err = a.err;
  const dim3 grid((unsigned)a.T, (p.d8 + CB_THREADS - 1) / CB_THREADS);
  count_launch(MX_KERNEL_DISPATCH);
  return cuda_status(launch_overlapped(moe_combine_kernel, grid, CB_THREADS, 0, stream, 1, p), "moe_combine_kernel launch");
}

int launch_moe_combine_bwd(const CombineLaunch& a, cudaStream_t stream) {
  CombineBwdParams p{};
  p.dout = (const uint4*)a.dout; p.rows = (const uint4*)a.rows; p.n_rows = a.n_rows; p.d8 = (uint32_t)(a.d / 8);
  p.dst = a.row_dst; p.src = a.row_src; p.T = a.T; p.k = a.k; p.weights = a.weights; p.drows = (uint4*)a.drows;
  p.dweights = a.dweights; p.err = a.err;
  count_launch(MX_KERNEL_DISPATCH);
  // a CTA for each row while all of them are one wave (8 tokens of 8 rows of 7168: 2.9 against 10.2 us)
  const dim3 grid((unsigned)a.T, a.T * a.k <= 4 * (int64_t)num_sms() ? (unsigned)a.k : 1u);
  return cuda_status(launch_overlapped(moe_combine_bwd_kernel, grid, CB_THREADS, 0, stream, 1, p),
                     "moe_combine_bwd_kernel launch");
}

}  // namespace mx
