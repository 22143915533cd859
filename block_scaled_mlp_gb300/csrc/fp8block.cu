// fp8block.cu - E4M3 codes with one fp32 scale for 128 elements of a row, or for a 128 x 128 block of a weight.
//
//   m = max |x| of the block, 2^-100 at least;  scale = RN_f32(m / 448);  code = RN_e4m3(448 x / m)
//
// The quotient is rounded once, straight to a code.  It lies half way between two codes often (whenever 7 divides
// the fraction of m and the rest fits), so a quotient that fp32 rounds first would go to the wrong side: x and m have
// 8 bits, a tie t has 5, so 448 x / m is either t or at least 2^-13 of it away, and what has to be exact is t itself.
// 448 / m is split in two, r = hi + lo with hi of 16 bits: x hi is exact in fp32, and fma(x, lo, x hi) is within
// 2^-38 of the quotient before its rounding, so a tie comes out as itself.
// A block that holds a NaN or an infinity has a NaN scale and codes 0x7F.
#include "common.cuh"
#include "kernels.h"

namespace mx {

namespace {

constexpr float FB_LEAST = 0x1p-100f;

MX_DEVINL uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  // |max| with NaN passed on; the sign bits of the result mean nothing
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The largest magnitude of a vector of 8 bf16 values, as bf16 bits.
MX_DEVINL uint32_t amax8(uint4 v) {
  const uint32_t m = max_abs_bf16x2(max_abs_bf16x2(v.x, v.y), max_abs_bf16x2(v.z, v.w)) & 0x7FFF7FFFu;
  return max(m & 0xFFFFu, m >> 16);  // magnitudes are ordered as whole numbers are, NaN above all
}

struct BlockScale {
  float hi, lo;   // 448 / m
  float scale;    // m / 448
  bool ok;
};

MX_DEVINL BlockScale block_scale(uint32_t amax_bits) {
  BlockScale b;
  b.ok = amax_bits < 0x7F80u;
  const float m = fmaxf(__uint_as_float(amax_bits << 16), FB_LEAST);
  b.scale = b.ok ? __fdiv_rn(m, 448.0f) : __uint_as_float(0x7FC00000u);
  const float r = __fdiv_rn(448.0f, m);
  b.hi = __uint_as_float(__float_as_uint(r) & 0xFFFFFF00u);
  // the rest of the quotient: 448 - hi m is exact (an fma), m is not subnormal
  b.lo = __fdiv_rn(fmaf(-b.hi, m, 448.0f), m);
  return b;
}

MX_DEVINL uint32_t codes4(uint32_t a, uint32_t b, const BlockScale& s) {
  const f2 hi = f2_splat(s.hi), lo = f2_splat(s.lo);
  const f2 x = f2_from_bf16x2(a), y = f2_from_bf16x2(b);
  const f2 p = f2_fma(x, lo, f2_mul(x, hi)), q = f2_fma(y, lo, f2_mul(y, hi));
  return cvt_e4m3x2(p.x, p.y) | cvt_e4m3x2(q.x, q.y) << 16;
}
MX_DEVINL uint2 codes8(uint4 v, const BlockScale& s) {
  return s.ok ? make_uint2(codes4(v.x, v.y, s), codes4(v.z, v.w, s)) : make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

struct RowsParams {
  const uint4* x;         // [rows_in, cols] bf16
  int64_t rows_in;
  const int32_t* src;     // [rows] or NULL
  int64_t rows;
  int32_t div;
  uint32_t c8;            // cols / 8
  uint2* codes;           // [rows, cols]
  float* scales;          // [ceil(cols / 128), rows]
  int32_t* err;
};

constexpr int FR_THREADS = 256;

// 16 lanes have a block.
__global__ void __launch_bounds__(FR_THREADS) fp8_block_rows_kernel(RowsParams p) {
  pdl_begin();
  const uint32_t blocks = (p.c8 + 15) / 16;
  const int64_t n = p.rows * blocks, g = ((int64_t)blockIdx.x * FR_THREADS + threadIdx.x) >> 4;
  if (((int64_t)blockIdx.x * FR_THREADS + (threadIdx.x & ~31)) >> 4 >= n) return;  // whole warps: the lanes talk
  const int sub = threadIdx.x & 15;
  const int64_t row = g / blocks;
  const uint32_t b = (uint32_t)(g - row * blocks), c = b * 16 + sub;
  const bool in = g < n && c < p.c8;
  int64_t from = row;
  if (p.src && g < n) {
    const int32_t s = p.src[row];
    from = s < 0 ? -1 : s / p.div;
    if (from >= p.rows_in) {
      if (sub == 0) record_error(p.err, MX_ERR_BAD_OFFSETS);
      from = -1;
    }
  }
  const uint4 v = in && from >= 0 ? __ldg(p.x + from * p.c8 + c) : make_uint4(0, 0, 0, 0);
  uint32_t m = amax8(v);
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const BlockScale s = block_scale(m);
  if (in) p.codes[row * p.c8 + c] = codes8(v, s);
  if (sub == 0 && g < n) p.scales[b * p.rows + row] = s.scale;
}

struct WeightParams {
  const uint4* w;         // [E, N, K] bf16
  int64_t N, K;
  uint2* codes;           // [E, N, K]
  uint8_t* codes_t;       // [E, K, N] or NULL
  float* scales;          // [E, ceil(N / 128), ceil(K / 128)]
};

constexpr int FW_THREADS = 256;

// A CTA has a 128 x 128 block: 16 vectors a row, 16 rows a step, 8 steps.
__global__ void __launch_bounds__(FW_THREADS) fp8_block_weight_kernel(WeightParams p) {
  __shared__ uint32_t part[FW_THREADS / 32];
  __shared__ uint8_t tile[128][132];
  pdl_begin();
  const int tid = threadIdx.x, cv = tid & 15, r0 = tid >> 4;
  const int64_t e = blockIdx.z, n0 = (int64_t)blockIdx.y * 128, k0 = (int64_t)blockIdx.x * 128;
  const uint32_t k8 = (uint32_t)(p.K / 8);
  const bool in_k = k0 + cv * 8 < p.K;
  uint4 v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = n0 + r0 + i * 16;
    v[i] = in_k && n < p.N ? __ldg(p.w + (e * p.N + n) * k8 + k0 / 8 + cv) : make_uint4(0, 0, 0, 0);
    m = max(m, amax8(v[i]));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((tid & 31) == 0) part[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FW_THREADS / 32; ++i) m = max(m, part[i]);
  const BlockScale s = block_scale(m);
  if (tid == 0) p.scales[(e * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = s.scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = n0 + r0 + i * 16;
    const uint2 q = codes8(v[i], s);
    if (in_k && n < p.N) p.codes[(e * p.N + n) * k8 + k0 / 8 + cv] = q;
    if (p.codes_t) {
      *reinterpret_cast<uint32_t*>(&tile[r0 + i * 16][cv * 8]) = q.x;
      *reinterpret_cast<uint32_t*>(&tile[r0 + i * 16][cv * 8 + 4]) = q.y;
    }
  }
  if (!p.codes_t) return;
  __syncthreads();
  // 16 codes of a column a thread: 8 threads a column, 32 columns a step (N is a multiple of 16)
  const int nv = tid & 7;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int col = (tid >> 3) + i * 32;
    if (k0 + col >= p.K || n0 + nv * 16 >= p.N) continue;
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      q[j] = tile[nv * 16 + j * 4][col] | tile[nv * 16 + j * 4 + 1][col] << 8 | tile[nv * 16 + j * 4 + 2][col] << 16 |
             (uint32_t)tile[nv * 16 + j * 4 + 3][col] << 24;
    *reinterpret_cast<uint4*>(p.codes_t + (e * p.K + k0 + col) * p.N + n0 + nv * 16) = make_uint4(q[0], q[1], q[2], q[3]);
  }
}

}  // namespace

int launch_fp8_block_rows(const void* x, int64_t rows_in, int64_t cols, const int32_t* src, int64_t rows, int32_t div, void* codes,
                          float* scales, int32_t* err, cudaStream_t stream) {
  RowsParams p{};
  p.x = (const uint4*)x; p.rows_in = rows_in; p.src = src; p.rows = rows; p.div = div; p.c8 = (uint32_t)(cols / 8);
  p.codes = (uint2*)codes; p.scales = scales; p.err = err;
  const int64_t n = rows * ((cols + 127) / 128);
  count_launch(MX_KERNEL_FP8_BLOCK);
  return cuda_status(launch_overlapped(fp8_block_rows_kernel, (unsigned)((n + FR_THREADS / 16 - 1) / (FR_THREADS / 16)), FR_THREADS,
                                       0, stream, 1, p),
                     "fp8_block_rows_kernel launch");
}

int launch_fp8_block_weight(const void* w, int64_t E, int64_t N, int64_t K, void* codes, void* codes_t, float* scales,
                            cudaStream_t stream) {
  WeightParams p{};
  p.w = (const uint4*)w; p.N = N; p.K = K; p.codes = (uint2*)codes; p.codes_t = (uint8_t*)codes_t; p.scales = scales;
  const dim3 grid((unsigned)((K + 127) / 128), (unsigned)((N + 127) / 128), (unsigned)E);
  count_launch(MX_KERNEL_FP8_BLOCK);
  return cuda_status(launch_overlapped(fp8_block_weight_kernel, grid, FW_THREADS, 0, stream, 1, p), "fp8_block_weight_kernel launch");
}

}  // namespace mx
