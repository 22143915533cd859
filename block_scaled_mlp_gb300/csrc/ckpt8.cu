// ckpt8.cu - 8-bit activation checkpoints (format: ckpt8.cuh) by themselves,
// and SwiGLU with [g | u] kept as one: the forward pass writes y and the
// checkpoint from one read of h13, the backward pass reads the checkpoint.
//
//   y  = g s u,  s = 1 / (1 + e^-g)                 from the unrounded h13
//   dg = dy u s (1 + g (1 - s)),  du = dy g s,  y' = g s u
//                                                   from the checkpoint's g, u
// in fp32, each result rounded once to bf16.
//
// All four kernels are bound by HBM (8.06, 10.06 and 3.03 bytes an element
// against about 30 instructions), so the layout is the plainest that keeps
// every access full: a lane holds eight consecutive elements (16 bytes of
// bf16, 8 bytes of codes), four lanes one block, and no shared memory.  Two
// vectors a thread put enough loads in flight and share one reduction of the
// block maxima.  On a GB300 whose copy runs at 6.78 TB/s: saving and loading
// 16384 x 7168 52 us each (6.8 TB/s; 65 and 62 with one vector a thread); SwiGLU
// of 8192 x 14336 140 us forward (6.8 TB/s; 172) and 184 us backward with y'
// (6.4 TB/s; 191), where five streams share the bus.  2048 elements or less are
// one launch's latency (1.5 to 3 us).
#include "ckpt8.cuh"
#include "kernels.h"

namespace mx {

namespace {

constexpr int C8_THREADS = 256;

// s = 1 / (1 + e^-g) by the approximate exponential and division.  CUDA's bounds for
// them are 2 + 1.173 |g| units in the last place and two units: s is off by some 5
// units of 2^-23 near g = 0, 30 at g = -20 and 110 at -87, 1.3e-5 of itself, where a
// bf16 result is rounded by 2^-9.  For 8192 x 14336, forward and backward, it takes
// 140 and 183 us; with expf, to one unit, 145 and 194, with an IEEE division besides
// 160 and 236.  Below g = -87.3 the denominator passes 2^126 and s is 0 (1e-38).
MX_DEVINL float sigmoid_approx(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// A thread has vectors i and i + C8_THREADS of its CTA's 2 * C8_THREADS.
__global__ void __launch_bounds__(C8_THREADS)
    ckpt8_save_kernel(const uint4* __restrict__ x, int64_t n8, uint2* __restrict__ codes, uint8_t* __restrict__ scales) {
  pdl_begin();
  const int64_t i = (int64_t)blockIdx.x * (2 * C8_THREADS) + threadIdx.x, j = i + C8_THREADS;
  const uint4 z = make_uint4(0, 0, 0, 0);
  const uint4 a = i < n8 ? ld_once(x + i) : z, b = j < n8 ? ld_once(x + j) : z;  // whole blocks: four lanes together
  const uint32_t s2 = ckpt8_block_scales(a, b), inv2 = inv_pow2_bf16x2(s2);
  if (i < n8) {
    codes[i] = ckpt8_encode(a, (uint16_t)inv2);
    if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)s2;
  }
  if (j < n8) {
    codes[j] = ckpt8_encode(b, (uint16_t)(inv2 >> 16));
    if ((threadIdx.x & 3) == 0) scales[j >> 2] = (uint8_t)(s2 >> 16);
  }
}

__global__ void __launch_bounds__(C8_THREADS)
    ckpt8_load_kernel(const uint2* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t n8,
                      uint4* __restrict__ x) {
  pdl_begin();
  const int64_t i = (int64_t)blockIdx.x * (2 * C8_THREADS) + threadIdx.x, j = i + C8_THREADS;
  if (i >= n8) return;
  const bool two = j < n8;
  const uint2 a = ld_once(codes + i), b = two ? ld_once(codes + j) : make_uint2(0, 0);
  const uint32_t sa = scales[i >> 2], sb = two ? scales[j >> 2] : 0;
  float v[8];
  values8(a, pow2_of_byte(sa), v);
  x[i] = pack8(v);
  if (two) {
    values8(b, pow2_of_byte(sb), v);
    x[j] = pack8(v);
  }
}

struct SwigluCkptParams {
  const uint4* h13;       // [M, 2h] bf16 (forward)
  const uint4* dy;        // [M, h] bf16 (backward)
  uint2* codes;           // [M, 2h]
  uint8_t* scales;        // [M, 2h/32]
  uint4* y;               // [M, h] bf16; backward: the recomputed y, or NULL
  uint4* dh13;            // [M, 2h] bf16 (backward)
  int64_t n8;             // M * h / 8
  uint32_t h8;            // h / 8
};

// Row and 8-element column of vector i of an [M, h] matrix (n8 < 2^32, or the
// 64-bit division).
MX_DEVINL void row_col(int64_t i, uint32_t h8, bool narrow, int64_t& row, uint32_t& c) {
  if (narrow) {
    row = (uint32_t)i / h8;
    c = (uint32_t)i - (uint32_t)row * h8;
  } else {
    row = i / h8;
    c = (uint32_t)(i - row * h8);
  }
}

// Both kernels: SW vectors a thread, C8_THREADS apart, all loads before the
// first use.
constexpr int SW = 2;

struct SwigluAt {
  int64_t i;    // vector of the [M, h] matrices; of g and of u in [M, 2h]
  int64_t gi, ui;
  bool in;
};
MX_DEVINL SwigluAt swiglu_at(const SwigluCkptParams& p, int k) {
  SwigluAt a;
  a.i = (int64_t)blockIdx.x * (SW * C8_THREADS) + k * C8_THREADS + threadIdx.x;
  a.in = a.i < p.n8;
  int64_t row;
  uint32_t c;
  row_col(a.in ? a.i : 0, p.h8, p.n8 <= 0xFFFFFFFFll, row, c);
  a.gi = row * 2 * p.h8 + c;
  a.ui = a.gi + p.h8;
  return a;
}

__global__ void __launch_bounds__(C8_THREADS) swiglu_ckpt8_fwd_kernel(SwigluCkptParams p) {
  pdl_begin();
  SwigluAt at[SW];
  uint4 gp[SW], up[SW];
#pragma unroll
  for (int k = 0; k < SW; ++k) {
    at[k] = swiglu_at(p, k);
    const uint4 z = make_uint4(0, 0, 0, 0);
    gp[k] = at[k].in ? ld_once(p.h13 + at[k].gi) : z;
    up[k] = at[k].in ? ld_once(p.h13 + at[k].ui) : z;
  }
#pragma unroll
  for (int k = 0; k < SW; ++k) {
    const uint32_t s2 = ckpt8_block_scales(gp[k], up[k]), inv2 = inv_pow2_bf16x2(s2);
    if (!at[k].in) continue;
    p.codes[at[k].gi] = ckpt8_encode(gp[k], (uint16_t)inv2);
    p.codes[at[k].ui] = ckpt8_encode(up[k], (uint16_t)(inv2 >> 16));
    if ((threadIdx.x & 3) == 0) {
      p.scales[at[k].gi >> 2] = (uint8_t)s2;
      p.scales[at[k].ui >> 2] = (uint8_t)(s2 >> 16);
    }
    float g[8], u[8], y[8];
    unpack8(gp[k], g);
    unpack8(up[k], u);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = g[i] * sigmoid_approx(g[i]) * u[i];
    p.y[at[k].i] = pack8(y);
  }
}

__global__ void __launch_bounds__(C8_THREADS) swiglu_ckpt8_bwd_kernel(SwigluCkptParams p) {
  pdl_begin();
  SwigluAt at[SW];
  uint4 dp[SW];
  uint2 gc[SW], uc[SW];
  uint32_t sg[SW], su[SW];
#pragma unroll
  for (int k = 0; k < SW; ++k) {
    at[k] = swiglu_at(p, k);
    if (!at[k].in) continue;
    dp[k] = ld_once(p.dy + at[k].i);
    gc[k] = ld_once(p.codes + at[k].gi);
    uc[k] = ld_once(p.codes + at[k].ui);
    sg[k] = p.scales[at[k].gi >> 2];
    su[k] = p.scales[at[k].ui >> 2];
  }
#pragma unroll
  for (int k = 0; k < SW; ++k) {
    if (!at[k].in) continue;
    float g[8], u[8], dy[8], y[8];
    unpack8(dp[k], dy);
    values8(gc[k], pow2_of_byte(sg[k]), g);
    values8(uc[k], pow2_of_byte(su[k]), u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid_approx(g[i]);
      const float a = g[i] * s;
      const float dg = dy[i] * u[i] * (s + a * (1.0f - s));
      y[i] = a * u[i];
      u[i] = dy[i] * a;
      g[i] = dg;
    }
    p.dh13[at[k].gi] = pack8(g);
    p.dh13[at[k].ui] = pack8(u);
    if (p.y) p.y[at[k].i] = pack8(y);
  }
}

int grid_of(int64_t n8, int per_thread, unsigned* grid) {
  const int64_t b = (n8 + per_thread * C8_THREADS - 1) / (per_thread * C8_THREADS);
  if (b > INT32_MAX) return fail(MX_ERR_UNSUPPORTED, "8-bit checkpoint: too many elements");
  *grid = (unsigned)b;
  return MX_OK;
}

}  // namespace

int launch_ckpt8_save(const void* x, int64_t rows, int64_t cols, void* codes, void* scales, cudaStream_t stream) {
  const int64_t n8 = rows * (cols / 8);
  unsigned grid;
  if (int rc = grid_of(n8, 2, &grid)) return rc;
  count_launch(MX_KERNEL_CKPT8);
  return cuda_status(launch_overlapped(ckpt8_save_kernel, grid, C8_THREADS, 0, stream, 1, (const uint4*)x, n8, (uint2*)codes,
                                       (uint8_t*)scales),
                     "ckpt8_save_kernel launch");
}

int launch_ckpt8_load(const void* codes, const void* scales, int64_t rows, int64_t cols, void* x, cudaStream_t stream) {
  const int64_t n8 = rows * (cols / 8);
  unsigned grid;
  if (int rc = grid_of(n8, 2, &grid)) return rc;
  count_launch(MX_KERNEL_CKPT8);
  return cuda_status(launch_overlapped(ckpt8_load_kernel, grid, C8_THREADS, 0, stream, 1, (const uint2*)codes,
                                       (const uint8_t*)scales, n8, (uint4*)x),
                     "ckpt8_load_kernel launch");
}

int launch_swiglu_ckpt8_fwd(const void* h13, int64_t M, int64_t h, void* y, void* codes, void* scales,
                            cudaStream_t stream) {
  SwigluCkptParams p{};
  p.h13 = (const uint4*)h13; p.y = (uint4*)y; p.codes = (uint2*)codes; p.scales = (uint8_t*)scales;
  p.n8 = M * (h / 8); p.h8 = (uint32_t)(h / 8);
  unsigned grid;
  if (int rc = grid_of(p.n8, SW, &grid)) return rc;
  count_launch(MX_KERNEL_CKPT8);
  return cuda_status(launch_overlapped(swiglu_ckpt8_fwd_kernel, grid, C8_THREADS, 0, stream, 1, p),
                     "swiglu_ckpt8_fwd_kernel launch");
}

int launch_swiglu_ckpt8_bwd(const void* dy, const void* codes, const void* scales, int64_t M, int64_t h, void* dh13,
                            void* y, cudaStream_t stream) {
  SwigluCkptParams p{};
  p.dy = (const uint4*)dy; p.codes = (uint2*)const_cast<void*>(codes);
  p.scales = (uint8_t*)const_cast<void*>(scales);
  p.dh13 = (uint4*)dh13; p.y = (uint4*)y;
  p.n8 = M * (h / 8); p.h8 = (uint32_t)(h / 8);
  unsigned grid;
  if (int rc = grid_of(p.n8, SW, &grid)) return rc;
  count_launch(MX_KERNEL_CKPT8);
  return cuda_status(launch_overlapped(swiglu_ckpt8_bwd_kernel, grid, C8_THREADS, 0, stream, 1, p),
                     "swiglu_ckpt8_bwd_kernel launch");
}

}  // namespace mx
