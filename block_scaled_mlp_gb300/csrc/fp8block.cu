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
//
// Bound by HBM (rows 3.03 bytes an element, weights 3 or 4) but for gathered rows, which read x from L2 as often as it is
// routed and are bound by instructions, some 4 an element.  On a GB300 whose copy runs at 6.78 TB/s: 16384 x 7168 57 us (6.2
// TB/s); 4096 x 7168 each to 8 groups 70 us (235 MB of codes written, 470 MB read through L2; at 6.78 TB/s the least is 45);
// weights of 16 x 5120 x 8192 425 us with transposed codes (6.3 TB/s), 285 without; 64 gathered rows 1.9 us.
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
};

MX_DEVINL BlockScale block_scale(uint32_t amax_bits) {
  BlockScale b;
  const float m = fmaxf(__uint_as_float(amax_bits << 16), FB_LEAST);
  // m / 448 from 1 / 448 and the exact rest of that quotient (Markstein's correction): the nearest for each of a bf16's
  // 128 fractions
  const float q = m * (1.0f / 448.0f);
  b.scale = fmaf(fmaf(-448.0f, q, m), 1.0f / 448.0f, q);
  // 448 / m by its fraction f in [1, 2): an approximate reciprocal c, hi = 448 c cut off at 16 bits, the rest (448 - hi f) c;
  // 448 - hi f is exact in an fma, so hi + lo is within 2^-37 of the quotient.  Then both times 2^-e.
  const uint32_t u = __float_as_uint(m), E = u >> 23;
  const float f = __uint_as_float((u & 0x007FFFFFu) | 0x3F800000u);
  float c;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(c) : "f"(f));
  const float hi = __uint_as_float(__float_as_uint(448.0f * c) & 0xFFFFFF00u), lo = fmaf(-hi, f, 448.0f) * c;
  const float p = __uint_as_float(E < 254 ? (254 - E) << 23 : 0x00400000u);
  b.hi = hi * p;
  b.lo = lo * p;
  if (amax_bits >= 0x7F80u) b.scale = b.hi = __uint_as_float(0x7FC00000u);  // NaN products convert to 0x7F
  return b;
}

MX_DEVINL uint32_t codes4(uint32_t a, uint32_t b, const BlockScale& s) {
  const f2 hi = f2_splat(s.hi), lo = f2_splat(s.lo);
  const f2 x = f2_from_bf16x2(a), y = f2_from_bf16x2(b);
  const f2 p = f2_fma(x, lo, f2_mul(x, hi)), q = f2_fma(y, lo, f2_mul(y, hi));
  return cvt_e4m3x2(p.x, p.y) | cvt_e4m3x2(q.x, q.y) << 16;
}
MX_DEVINL uint2 codes8(uint4 v, const BlockScale& s) {
  return make_uint2(codes4(v.x, v.y, s), codes4(v.z, v.w, s));
}

struct RowsParams {
  const uint8_t* x;       // [rows_in, cols] bf16
  int64_t rows_in;
  const int32_t* src;     // [rows] or NULL
  int64_t rows;
  int32_t div;
  int32_t cols;
  int32_t blocks;         // of a row
  int32_t share;          // blocks of a row that a warp takes
  int32_t splits;         // warps that share eight rows
  uint8_t* codes;         // [rows, cols]
  float* scales;          // [blocks, rows]
  int32_t* err;
};

constexpr int FR_THREADS = 128;

// 32 elements of a row: two loads of 32 bytes, or four of 16 where rows are not on 32 bytes.
struct Quarter {
  uint32_t w[16];
};
template <bool WIDE>
MX_DEVINL Quarter load_quarter(const uint8_t* x, int left) {  // left: elements up to the row's end
  Quarter q;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t* w = q.w + h * 8;
    if (left >= (h + 1) * 16) {   // cols is a multiple of 16
      if (WIDE) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(x + h * 32));
      } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(x + h * 32)), b = __ldg(reinterpret_cast<const uint4*>(x + h * 32 + 16));
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 0;
    }
  }
  return q;
}

// A warp has eight rows, four lanes each, and goes along their blocks: 32 elements a lane, so a block's largest takes two
// exchanges, the scales of eight rows leave as one sector, and a row's src is read once.
template <bool WIDE>
__global__ void __launch_bounds__(FR_THREADS, 8) fp8_block_rows_kernel(RowsParams p) {
  pdl_begin();
  const int lane = threadIdx.x & 31, sub = lane & 3;
  const int64_t w = (int64_t)blockIdx.x * (FR_THREADS / 32) + (threadIdx.x >> 5);
  const int64_t group = w / p.splits;
  const int32_t b0 = (int32_t)(w - group * p.splits) * p.share, b1 = min(p.blocks, b0 + p.share);
  const int64_t row = group * 8 + (lane >> 2);
  if (group * 8 >= p.rows) return;  // whole warps: the lanes talk
  const bool live = row < p.rows;
  int64_t from = row;
  if (p.src && live) {
    const int32_t s = p.src[row];
    from = s < 0 ? -1 : s / p.div;
    if (from >= p.rows_in) {
      if (sub == 0 && b0 == 0) record_error(p.err, MX_ERR_BAD_OFFSETS);
      from = -1;
    }
  }
  const bool read = live && from >= 0;
  const int c0 = b0 * 128 + sub * 32;   // this lane's columns of the first block
  const uint8_t* x = p.x + (read ? from * p.cols + c0 : 0) * 2;
  uint8_t* codes = p.codes + row * p.cols + c0;
  float* scales = p.scales + b0 * p.rows + row;
  // the next block on its way while one is cast: 64 registers and 32 warps an SM, which is worth more than a second block on
  // its way (32768 gathered rows of 7168: 74 against 108 us when it was changed, 70 now)
  Quarter next = load_quarter<WIDE>(x, read ? p.cols - c0 : 0);
  for (int32_t b = b0; b < b1; ++b) {
    const int left = p.cols - b * 128 - sub * 32;
    const Quarter q = next;
    x += 256;
    next = load_quarter<WIDE>(x, read && b + 1 < b1 ? left - 128 : 0);
    uint32_t m = q.w[0];
#pragma unroll
    for (int j = 1; j < 16; ++j) m = max_abs_bf16x2(m, q.w[j]);
    m &= 0x7FFF7FFFu;
    m = max(m & 0xFFFFu, m >> 16);  // magnitudes are ordered as whole numbers are, NaN above all
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const BlockScale s = block_scale(m);
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = codes4(q.w[2 * j], q.w[2 * j + 1], s);
    if (live) {
      if (WIDE && left >= 32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(codes), "r"(c[0]), "r"(c[1]), "r"(c[2]),
                     "r"(c[3]), "r"(c[4]), "r"(c[5]), "r"(c[6]), "r"(c[7])
                     : "memory");
      } else {
        if (left >= 16) reinterpret_cast<uint4*>(codes)[0] = make_uint4(c[0], c[1], c[2], c[3]);
        if (left >= 32) reinterpret_cast<uint4*>(codes)[1] = make_uint4(c[4], c[5], c[6], c[7]);
      }
      if (sub == 0) *scales = s.scale;
    }
    codes += 128;
    scales += p.rows;
  }
}

struct WeightParams {
  const uint4* w;         // [E, N, K] bf16
  int64_t N, K;
  uint2* codes;           // [E, N, K]
  uint8_t* codes_t;       // [E, K, N] or NULL
  float* scales;          // [E, ceil(N / 128), ceil(K / 128)]
};

constexpr int FW_THREADS = 256;

// A CTA has a 128 x 128 block in registers: 16 vectors a row, 16 rows a step, 8 steps.  The transposed codes go through
// shared memory in rows of 132 bytes, so that neither the words of a row nor the bytes of a column meet in one bank often.
__global__ void __launch_bounds__(FW_THREADS) fp8_block_weight_kernel(WeightParams p) {
  __shared__ uint32_t part[FW_THREADS / 32];
  __shared__ uint32_t tile[128][33];   // written as words (which it lies on by its type), read as bytes
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
      tile[r0 + i * 16][cv * 2] = q.x;
      tile[r0 + i * 16][cv * 2 + 1] = q.y;
    }
  }
  if (!p.codes_t) return;
  __syncthreads();
  // 16 codes of a column a thread: 8 threads a column, 32 columns a step (N is a multiple of 16)
  const int nv = tid & 7;
  const uint8_t* bytes = reinterpret_cast<const uint8_t*>(tile[nv * 16]);
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int col = (tid >> 3) + i * 32;
    if (k0 + col >= p.K || n0 + nv * 16 >= p.N) continue;
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      q[j] = bytes[j * 4 * 132 + col] | bytes[(j * 4 + 1) * 132 + col] << 8 | bytes[(j * 4 + 2) * 132 + col] << 16 |
             (uint32_t)bytes[(j * 4 + 3) * 132 + col] << 24;
    *reinterpret_cast<uint4*>(p.codes_t + (e * p.K + k0 + col) * p.N + n0 + nv * 16) = make_uint4(q[0], q[1], q[2], q[3]);
  }
}

}  // namespace

int launch_fp8_block_rows(const void* x, int64_t rows_in, int64_t cols, const int32_t* src, int64_t rows, int32_t div, void* codes,
                          float* scales, int32_t* err, cudaStream_t stream) {
  RowsParams p{};
  p.x = (const uint8_t*)x; p.rows_in = rows_in; p.src = src; p.rows = rows; p.div = div; p.cols = (int32_t)cols;
  p.blocks = (int32_t)((cols + 127) / 128);
  p.codes = (uint8_t*)codes; p.scales = scales; p.err = err;
  // few rows: their blocks shared out until each SM has 32 warps
  const int64_t groups = (rows + 7) / 8, want = 32 * (int64_t)num_sms();
  p.splits = (int32_t)std::min<int64_t>(p.blocks, (want + groups - 1) / groups);
  p.share = (p.blocks + p.splits - 1) / p.splits;
  p.splits = (p.blocks + p.share - 1) / p.share;
  const bool wide = cols % 32 == 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(codes)) & 31) == 0;
  const int64_t n = groups * p.splits;
  count_launch(MX_KERNEL_FP8_BLOCK);
  return cuda_status(launch_overlapped(wide ? fp8_block_rows_kernel<true> : fp8_block_rows_kernel<false>,
                                       (unsigned)((n + FR_THREADS / 32 - 1) / (FR_THREADS / 32)), FR_THREADS, 0, stream, 1, p),
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
