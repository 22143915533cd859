// norm.cu - residual addition and root-mean-square norm with the result in
// MXFP8 (rows, or rows and columns) and / or bf16, and the backward pass.
//
//   r = RN_bf16(x + residual),  n = (sum_j r_j^2 / d + eps)^-1/2,  y = r n w
//   dr = n (dy w - r n c) + dres,  c = n / d sum_j dy_j w_j r_j
//   dw = sum over rows of dy r n
//
// Sums are fp32; n is kept as an unevaluated pair of fp32 values and r w is
// exact in fp32 (two bf16 factors), and y keeps enough of r w n that the codes
// and the bf16 values are r w n rounded once (see norm2).  The sum r is what
// the model carries on in bf16, so the norm is taken of the rounded value, the
// one that the backward pass has.  Each input is read once and each output
// written once, a row staying in registers or shared memory between its two
// uses.  Times below are device times on a GB300 whose copy runs at 6.78 TB/s.
#include "ckpt8.cuh"
#include "kernels.h"
#include "tile_quant.cuh"

#include <string.h>

#include <atomic>
#include <type_traits>

namespace mx {

namespace {

constexpr int NB_MAX_STAGES = 6;          // backward: rows in a CTA's ring, at most
constexpr int NB_MAX_SMEM = 220 * 1024;   // of all rings of an SM; every call's limit (see NC_MAX_SMEM)

struct NormFwdParams {
  const uint4* x;        // [M, d] bf16
  const uint4* res;      // [M, d] bf16 or NULL
  const uint4* w;        // [d] bf16
  uint4* r;              // [M, d] bf16: x + res, or NULL
  float* rstd;           // [M]
  uint4* y;              // [M, d] bf16 or NULL
  uint8_t* q_row;        // [M, d] E4M3 or NULL
  ScaleDst s_row;
  uint8_t* q_col;        // [d, M] E4M3 or NULL
  ScaleDst s_col;
  uint8_t* ck;           // [M, d] checkpoint codes of r, or NULL
  uint8_t* ck_s;         // [M, d/32]
  int64_t M;
  int32_t d8;            // d / 8
  float d, eps;
  uint32_t rceil;
};

// r of eight elements: the bf16 sums (rounded once), packed.
MX_DEVINL uint4 add8(const uint4& a, const uint4& b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(x[i]), "r"(y[i]));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

MX_DEVINL float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Unevaluated sums hi + lo; one that is infinite or NaN stays so.
MX_DEVINL f2 pair_add(f2 a, f2 b) {
  const float s = __fadd_rn(a.x, b.x), t = __fsub_rn(s, a.x);
  const float e = __fadd_rn(__fsub_rn(a.x, __fsub_rn(s, t)), __fsub_rn(b.x, t));  // s + e = a.x + b.x
  const float l = __fadd_rn(e, __fadd_rn(a.y, b.y)), h = __fadd_rn(s, l);
  return fabsf(s) < __uint_as_float(0x7F800000u) ? f2_pack(h, __fsub_rn(l, __fsub_rn(h, s))) : f2_pack(s, 0.0f);
}
MX_DEVINL void squares8(const uint4& a, f2& s) {
  sumsq_bf16x2(a.x, s);
  sumsq_bf16x2(a.y, s);
  sumsq_bf16x2(a.z, s);
  sumsq_bf16x2(a.w, s);
}

// Sums of squares as hi + lo: the squares are exact, four of them (in the two-axis
// kernel eight) are added in fp32, and from there on each addition's rounding error
// goes to lo.  So a row's sum is off by three (four) roundings of 2^-24 at most,
// whatever its length: by 3e-9 (6e-9) on average for normal values, by 1e-8 and
// at worst 1.4e-7 of 2000 rows where one channel in 256 is twenty times larger.
// hi alone says whether a sum is finite (lo is then NaN); settle() before use.
// Two sums at once, and one of hi + lo with another.
MX_DEVINL f2 f2_sub(f2 a, f2 b) { return f2_fma(b, f2_splat(-1.0f), a); }
MX_DEVINL void sum_add2(f2& hi, f2& lo, f2 v) {
  const f2 s = f2_add(hi, v), t = f2_sub(s, hi);
  lo = f2_add(lo, f2_add(f2_sub(hi, f2_sub(s, t)), f2_sub(v, t)));
  hi = s;
}
MX_DEVINL void sum_add(f2& a, f2 b) {
  const float s = __fadd_rn(a.x, b.x), t = __fsub_rn(s, a.x);
  const float e = __fadd_rn(__fsub_rn(a.x, __fsub_rn(s, t)), __fsub_rn(b.x, t));
  a = f2_pack(s, __fadd_rn(__fadd_rn(a.y, b.y), e));
}
MX_DEVINL f2 settle(f2 a) { return pair_add(f2_pack(a.x, 0.0f), f2_pack(0.0f, a.y)); }
template <int FROM>
MX_DEVINL f2 warp_sum_add(f2 v) {
#pragma unroll
  for (int o = FROM; o > 0; o >>= 1)
    sum_add(v, f2_pack(__shfl_xor_sync(0xFFFFFFFFu, v.x, o), __shfl_xor_sync(0xFFFFFFFFu, v.y, o)));
  return v;
}
// The warp's sums of four rows (two a pair), row lane / 8 in each lane: a lane
// hands on the rows of the other half, so 12 exchanges and not 40.
MX_DEVINL f2 warp_sum_rows(const f2 (&hi)[2], const f2 (&lo)[2]) {
  const int lane = threadIdx.x & 31;
  const bool up = lane & 16;
  f2 h = up ? hi[1] : hi[0], l = up ? lo[1] : lo[0];
  const f2 sh = up ? hi[0] : hi[1], sl = up ? lo[0] : lo[1];
  auto other = [](f2 v, int o) {
    return f2_pack(__shfl_xor_sync(0xFFFFFFFFu, v.x, o), __shfl_xor_sync(0xFFFFFFFFu, v.y, o));
  };
  sum_add2(h, l, other(sh, 16));
  l = f2_add(l, other(sl, 16));
  const bool second = lane & 8;
  f2 v = second ? f2_pack(h.y, l.y) : f2_pack(h.x, l.x);
  sum_add(v, other(second ? f2_pack(h.x, l.x) : f2_pack(h.y, l.y), 8));
  return warp_sum_add<4>(v);
}

// n = (ss / d + eps)^-1/2 as a pair for norm2: the rounded root and one Newton
// step's correction.  A root that is not finite (or zero) stays as it is.  rstd: n in
// fp32.
//   EXACT: where m = ss / d + eps is the square of a number a of 12 bits or less (rows
// of one magnitude, say), y = r w / a may be an exact number.  The last bit of n's
// correction (2^-47 of n) says so to norm2: clear where it may, set elsewhere.  In such
// a row n is raised by 2^-38 of itself, past the pair's own error (some 2^-46): an
// exact y comes out of norm2's truncation whole, and any other stays on its side of
// every tie (a tie T of nine bits differs from r w / a by 1 / (T a), 2^-21, or more).
template <bool EXACT>
MX_DEVINL f2 rstd_pair(f2 ss, float d, float eps, float& rstd) {
  const float q = __fdiv_rn(ss.x, d);
  const float ql = __fdividef(__fadd_rn(__fmaf_rn(-q, d, ss.x), ss.y), d);
  const f2 m = pair_add(f2_pack(q, ql), f2_pack(eps, 0.0f));
  const float n = __frsqrt_rn(m.x), t = __fmul_rn(n, n);
  float e = __fmaf_rn(-m.x, t, 1.0f);
  e = __fmaf_rn(-m.x, __fmaf_rn(n, n, -t), e);
  e = __fmaf_rn(-m.y, t, e);
  float lo = __fmul_rn(__fmul_rn(0.5f, n), e);
  const bool valid = fabsf(lo) < n;
  if (!valid) lo = 0.0f;
  rstd = n + lo;
  if (EXACT && valid) {
    const float a = __uint_as_float((__float_as_uint(__fmul_rn(m.x, n)) + 0x800u) & ~0xFFFu);  // 12 bits of the root
    const bool square = m.y == 0.0f && __fmaf_rn(a, a, -m.x) == 0.0f;
    lo = __uint_as_float(square ? __float_as_uint(__fmaf_rn(n, 0x1p-38f, lo)) & ~1u : __float_as_uint(lo) | 1u);
  }
  return f2_pack(n, lo);
}

// y of two and of eight elements, fp32, rounded to odd: truncated, and the last
// bit set (EXACT: unless y may be an exact number, see above).  Such a value lies on
// the same side of every E4M3 and bf16 tie as r w n itself, so the rounding that
// follows is that of r w n, where an fp32 value to nearest lands on the tie itself
// once in a million times and goes to the even side: of 117 million codes 64 to 75
// then differed from the 64-bit result, and 2 to 5 do with this and the sums above.
//   EXACT goes by eps alone (short_number): with an eps of many bits no row's m is a
// short square, unless the row makes up for eps bit by bit.  Asking every element's
// row costs up to 5% of the two-axis kernel (registers) and 1 to 3% of the others.
// Zero becomes 2^-149, which rounds to a zero code and a zero bf16.  Where |r w|
// passes fp32 y is NaN; multiplying r n by w for such weights cost 2.5% of every
// call.  (Where a row's sum of squares passes it, n is zero, and y with it.)
template <bool EXACT>
MX_DEVINL float to_odd(float y, f2 n) {
  uint32_t v = __float_as_uint(y) | 1u;
  if (EXACT)  // y | (n.y & 1) in one instruction
    asm("lop3.b32 %0, %1, %2, 1, 0xF8;" : "=r"(v) : "r"(__float_as_uint(y)), "r"(__float_as_uint(n.y)));
  return __uint_as_float(v);
}
template <bool EXACT>
MX_DEVINL f2 norm2(uint32_t r, f2 n, uint32_t w) {
  const f2 rw = mul_bf16x2(r, w);
  const f2 y = __ffma2_rz(rw, f2_splat(n.x), f2_mul(rw, f2_splat(n.y)));
  return f2_pack(to_odd<EXACT>(y.x, n), to_odd<EXACT>(y.y, n));
}
template <bool EXACT>
MX_DEVINL void norm8(const uint4& r, f2 n, const uint4& w, f2 (&y)[4]) {
  y[0] = norm2<EXACT>(r.x, n, w.x);
  y[1] = norm2<EXACT>(r.y, n, w.y);
  y[2] = norm2<EXACT>(r.z, n, w.z);
  y[3] = norm2<EXACT>(r.w, n, w.w);
}
// Whether eps has 12 significant bits or less (0, a power of two).
bool short_number(float eps) {
  uint32_t bits;
  memcpy(&bits, &eps, 4);
  return (bits & 0xFFFu) == 0;
}

// ---- rows: one CTA per row, or (WARP) one warp, ROW_WARPS of them a CTA; the
// row in registers, V vectors of eight a thread.  Rows past M only clear the
// scale layout's padding rows.  Bound by HBM from some hundred rows on: 16384 x
// 7168 with a residual into row codes and bf16 158 us (6.7 TB/s), 8192 x 4096 into
// bf16 22.5 us (6.0 TB/s); below that by the latency of one row (1 x 7168: 3.0 us).
constexpr int ROW_WARPS = 4;
template <int V, bool WARP, bool EXACT>
__global__ void __launch_bounds__(512) add_rmsnorm_row_kernel(NormFwdParams p) {
  pdl_begin();
  const int lane = threadIdx.x & 31;
  const int T = WARP ? 32 : blockDim.x, t = WARP ? lane : threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  if (p.q_row && p.s_row.mma) {
    // zeros where the layout is padded (to 128 rows): whole rows past M, columns past d / 32
    const int S = p.d8 / 4, S4 = (S + 3) & ~3;
    for (int c = (row < p.M ? S : 0) + t; c < S4; c += T) p.s_row.put(row, c, 0);
  }
  if (row >= p.M) return;
  const int64_t base = row * p.d8;
  uint4 v[V];
  f2 ss = f2_splat(0.0f), ss_lo = ss;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = t + k * T;
    v[k] = c < p.d8 ? ld_once(p.x + base + c) : make_uint4(0, 0, 0, 0);
  }
  if (p.res) {
    uint4 a[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = t + k * T;
      a[k] = c < p.d8 ? ld_once(p.res + base + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = t + k * T;
      v[k] = add8(v[k], a[k]);
      if (c < p.d8) p.r[base + c] = v[k];
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    f2 sq = f2_splat(0.0f);
    squares8(v[k], sq);
    sum_add2(ss, ss_lo, sq);
  }
  f2 sum = f2_pack(ss.x, ss_lo.x);
  sum_add(sum, f2_pack(ss.y, ss_lo.y));
  sum = warp_sum_add<16>(sum);
  if (!WARP) {
    __shared__ f2 part[16];
    if (lane == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = warp_sum_add<8>((lane & 15) < (T >> 5) ? part[lane & 15] : f2_splat(0.0f));
  }
  sum = settle(sum);
  float rstd;
  const f2 n = rstd_pair<EXACT>(sum, p.d, p.eps, rstd);
  if (t == 0) p.rstd[row] = rstd;
  const uint32_t up = p.rceil ? 0x1FFFFFu : 0u;
  // two vectors of the row at a time (V = 1: one, and zeros), so that two
  // blocks share the scales' exchange
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    const int c0 = t + k * T, c1 = c0 + T;
    const bool in0 = c0 < p.d8, in1 = V > 1 && c1 < p.d8;
    const uint4 z = make_uint4(0, 0, 0, 0), v0 = v[k], v1 = V > 1 ? v[k + (V > 1)] : z;
    if (p.ck) {
      const uint32_t s2 = ckpt8_block_scales(v0, v1), inv2 = inv_pow2_bf16x2(s2);
      if (in0) {
        reinterpret_cast<uint2*>(p.ck)[base + c0] = ckpt8_encode(v0, (uint16_t)inv2);
        if ((c0 & 3) == 0) p.ck_s[(base + c0) >> 2] = (uint8_t)s2;
      }
      if (in1) {
        reinterpret_cast<uint2*>(p.ck)[base + c1] = ckpt8_encode(v1, (uint16_t)(inv2 >> 16));
        if ((c1 & 3) == 0) p.ck_s[(base + c1) >> 2] = (uint8_t)(s2 >> 16);
      }
    }
    f2 y0[4], y1[4];
    norm8<EXACT>(v0, n, in0 ? __ldg(p.w + c0) : z, y0);
    norm8<EXACT>(v1, n, in1 ? __ldg(p.w + c1) : z, y1);
    if (p.y) {
      if (in0) p.y[base + c0] = pack8(y0);
      if (in1) p.y[base + c1] = pack8(y1);
    }
    if (p.q_row) {
      const uint32_t s2 = mx_block_scales(y0, y1, up);
      if (in0) {
        reinterpret_cast<uint2*>(p.q_row)[base + c0] = mx_encode(y0, s2 & 0xFF);
        if ((c0 & 3) == 0) p.s_row.put(row, c0 >> 2, s2 & 0xFF);
      }
      if (in1) {
        reinterpret_cast<uint2*>(p.q_row)[base + c1] = mx_encode(y1, s2 >> 16);
        if ((c1 & 3) == 0) p.s_row.put(row, c1 >> 2, s2 >> 16);
      }
    }
  }
}

// ---- rows and columns: a cluster of CTAs per 32 rows, each with a slice of
// the columns.  r of the slice stays in shared memory in bf16; the rows' sums of
// squares are exchanged through distributed shared memory, so one pass over HBM
// gives both quantizations (a second kernel for the columns would read r again:
// 10 bytes an element instead of 8).  16384 x 7168 with a residual into both
// codes and a checkpoint takes 197 us (5.4 TB/s), without either 126 us (3.8 TB/s), of
// which the loads and sums take 44 by themselves, either quantization some 40: 32
// warps an SM do not cover the loads, the exchange and the quantizations of one
// another.
//
// Row passes: a warp has four rows, a lane eight elements of each, four lanes
// one block.  Column pass: lanes l and l ^ 16 have rows 0-15 and 16-31 of one
// column pair (16 rows keep the registers low enough for four CTAs an SM, where
// the tiles leave room: 8192 x 4096, 60 us against 68 with three).  The tile's
// 16-byte vectors of rows 16-31 sit at vector index ^ 4, so that the two
// half-warps of the column pass read different banks.
constexpr int NC_ROWS = 32;
constexpr int NC_THREADS = 256;
constexpr int NC_MAX_CTAS = 16;
constexpr int NC_CTAS_SM = 4;
constexpr int NC_PORTABLE_CTAS = 8;  // a cluster that every device holds
// Shared memory of the widest slice.  The kernels' limit is this for every call: it is
// the function's, not the launch's, and another thread may launch with another width.
constexpr int NC_MAX_SMEM = NC_ROWS * (int)(kNormMaxD / NC_PORTABLE_CTAS) * 2;

MX_DEVINL void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
MX_DEVINL void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
MX_DEVINL void copy_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Scale bytes of row r at columns c, c + step, ...: the first one's address
// and the distance for eight further columns.
struct ScaleRow {
  uint8_t* at;
  int32_t step8;
};
MX_DEVINL ScaleRow scale_row(const ScaleDst& d, int64_t r, int32_t c) {
  return d.mma ? ScaleRow{d.base + mma_scale_offset(r, c, d.tiles_per_row), 1024} : ScaleRow{d.base + r * d.ld + c, 8};
}

template <bool RES, bool CK, bool Y, bool ROW, bool EXACT>
__global__ void __launch_bounds__(NC_THREADS, NC_CTAS_SM) add_rmsnorm_col_kernel(NormFwdParams p, int32_t slice8) {
  extern __shared__ __align__(16) uint4 tile[];   // [32][slice8]
  __shared__ __align__(16) f2 part[NC_MAX_CTAS][NC_ROWS];    // sums of squares by CTA and row
  __shared__ __align__(16) f2 s_n[NC_ROWS];
  pdl_begin();
  const int rank = (int)cluster_ctarank();
  const int ctas = (int)(gridDim.y);
  const int64_t r0 = (int64_t)blockIdx.x * NC_ROWS;
  const int c0 = rank * slice8;                                  // first vector of the slice
  const int n8 = min(slice8, p.d8 - c0);                         // its vectors
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool live = r0 < p.M;  // else: a row block of the scale layout's padding

  if (p.s_col.mma && rank == ctas - 1) {
    // zeros where the layouts are padded: rows past M, columns past d
    const int S = p.d8 / 4, first = live ? S : 0, cols = ((S + 3) & ~3) - first;
    if (ROW)
      for (int i = threadIdx.x; i < cols * NC_ROWS; i += NC_THREADS) p.s_row.put(r0 + i % NC_ROWS, first + i / NC_ROWS, 0);
    for (int64_t c = (live ? p.d8 * 8 : 0) + threadIdx.x; c < ((p.d8 * 8 + 127) & ~127); c += NC_THREADS)
      p.s_col.put(c, r0 >> 5, 0);
  }
  if (!live) return;  // the whole cluster
  __syncwarp();
  cluster_arrive();   // waited for before the first store into another CTA, behind the loads

  const int rw = warp * 4;                                       // the warp's first row
  const int64_t at0 = (r0 + rw) * p.d8 + c0 + lane;              // its first vector
  uint4* trow = tile + rw * slice8 + (lane ^ (rw >= 16 ? 4 : 0));
  f2 ss[2] = {}, ss_lo[2] = {};
  // x goes to the tile by asynchronous copies, all of them in flight at once;
  // the residual's vectors are loaded one step ahead, from L2 after the first
  // step (16384 x 7168 with a checkpoint: 199 us, 211 without the prefetch, 207 with
  // it before the copies of x)
  const int steps = (n8 + 31) / 32;
  for (int i = 0; i < steps; ++i)
    if (i * 32 + lane < n8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) copy_async16(trow + k * slice8 + i * 32, p.x + at0 + i * 32 + k * p.d8);
    }
  uint4 a[4];
  auto load_res = [&](int cb) {
    if (RES && cb + lane < n8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) a[k] = ld_once(p.res + at0 + cb + k * p.d8);
    }
  };
  load_res(0);
  if (RES && (lane & 7) == 0)  // a lane a 128-byte line
    for (int cb = 32; cb + lane < n8; cb += 32) {
#pragma unroll
      for (int k = 0; k < 4; ++k) prefetch_l2(p.res + at0 + cb + k * p.d8);
    }
  copy_async_wait_all();  // a lane reads only what it copied itself
  for (int cb = 0; cb < n8; cb += 32) {
    const bool in = cb + lane < n8;
    const int64_t at = at0 + cb;
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = in ? trow[k * slice8 + cb] : make_uint4(0, 0, 0, 0);
    if (RES) {
      if (in) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = add8(v[k], a[k]);
          trow[k * slice8 + cb] = v[k];
          p.r[at + k * p.d8] = v[k];
        }
      }
      load_res(cb + 32);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      f2 a2 = f2_splat(0.0f), b2 = a2;
      squares8(v[2 * k], a2);
      squares8(v[2 * k + 1], b2);
      sum_add2(ss[k], ss_lo[k], f2_pack(a2.x + a2.y, b2.x + b2.y));
    }
    if (CK) {
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const uint32_t s2 = ckpt8_block_scales(v[k], v[k + 1]), inv2 = inv_pow2_bf16x2(s2);
        if (in) {
          const int64_t e0 = at + k * p.d8, e1 = e0 + p.d8;
          reinterpret_cast<uint2*>(p.ck)[e0] = ckpt8_encode(v[k], (uint16_t)inv2);
          reinterpret_cast<uint2*>(p.ck)[e1] = ckpt8_encode(v[k + 1], (uint16_t)(inv2 >> 16));
          if ((lane & 3) == 0) {
            p.ck_s[e0 >> 2] = (uint8_t)s2;
            p.ck_s[e1 >> 2] = (uint8_t)(s2 >> 16);
          }
        }
      }
    }
  }
  const int n8_all = n8 & ~31;
  const f2 sum = warp_sum_rows(ss, ss_lo);
  __syncwarp();
  cluster_wait();  // the other CTAs have started
  // lane: this CTA's sum of row lane / 8 of the warp to CTAs lane % 8 and + 8 of the cluster
  for (int j = lane & 7; j < ctas; j += 8)
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(cluster_map(smem_u32(&part[rank][rw + (lane >> 3)]), j)),
                 "f"(sum.x), "f"(sum.y)
                 : "memory");
  __syncwarp();
  cluster_sync();  // every CTA's sums are here; the tile is complete too
  if (threadIdx.x < NC_ROWS) {
    f2 t = part[0][threadIdx.x];
    for (int j = 1; j < ctas; ++j) sum_add(t, part[j][threadIdx.x]);  // the same order in every CTA
    float rstd;
    s_n[threadIdx.x] = rstd_pair<EXACT>(settle(t), p.d, p.eps, rstd);
    if (rank == 0) p.rstd[r0 + threadIdx.x] = rstd;
  }
  __syncthreads();

  // rows
  if (Y || ROW) {
    const uint32_t up = p.rceil ? 0x1FFFFFu : 0u;
    f2 n[4];
    ScaleRow sr[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      n[k] = s_n[rw + k];
      if (ROW) sr[k] = scale_row(p.s_row, r0 + rw + k, (c0 + lane) >> 2);
    }
    auto quant_rows = [&](int cb, auto all) {
      const bool in = decltype(all)::value || cb + lane < n8;
      const uint4 z = make_uint4(0, 0, 0, 0), w = in ? __ldg(p.w + c0 + cb + lane) : z;
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        f2 y0[4], y1[4];
        norm8<EXACT>(in ? trow[k * slice8 + cb] : z, n[k], w, y0);
        norm8<EXACT>(in ? trow[(k + 1) * slice8 + cb] : z, n[k + 1], w, y1);
        const int64_t e0 = at0 + cb + k * p.d8, e1 = e0 + p.d8;
        if (Y && in) {
          p.y[e0] = pack8(y0);
          p.y[e1] = pack8(y1);
        }
        if (ROW) {
          const uint32_t s2 = mx_block_scales(y0, y1, up);
          if (in) {
            reinterpret_cast<uint2*>(p.q_row)[e0] = mx_encode(y0, s2 & 0xFF);
            reinterpret_cast<uint2*>(p.q_row)[e1] = mx_encode(y1, s2 >> 16);
            if ((lane & 3) == 0) {
              *sr[k].at = (uint8_t)s2;
              *sr[k + 1].at = (uint8_t)(s2 >> 16);
            }
          }
          sr[k].at += sr[k].step8;
          sr[k + 1].at += sr[k + 1].step8;
        }
      }
    };
    for (int cb = 0; cb < n8_all; cb += 32) quant_rows(cb, std::true_type{});
    if (n8_all < n8) quant_rows(n8_all, std::false_type{});
  }

  // columns: 16 pairs a warp at a time
  const int rh = lane >> 4;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(tile) + rh * 16 * slice8 * 4;
  const uint32_t* ww = reinterpret_cast<const uint32_t*>(p.w + c0);
  const f2* nr = s_n + rh * 16;
  uint8_t* sc = p.s_col.base + (p.s_col.mma ? ((r0 >> 7) << 9) + ((r0 >> 5) & 3) : r0 >> 5);
  const bool v8 = ((uintptr_t)p.q_col & 31) == 0;  // rows r0 .. of a column: M and r0 are multiples of 32
  for (int pb = warp * 16; pb < n8 * 4; pb += NC_THREADS / 2) {
    const int pc = pb + (lane & 15);                // n8 is a multiple of 4: all 16 pairs exist
    const uint32_t w = __ldg(ww + pc);
    const uint32_t* src = words + (pc ^ (rh << 4));
    f2 y[16];
    float ma = 0, mb = 0;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float4 nn = *reinterpret_cast<const float4*>(nr + i);
      y[i] = norm2<EXACT>(src[i * slice8 * 4], f2_pack(nn.x, nn.y), w);
      y[i + 1] = norm2<EXACT>(src[(i + 1) * slice8 * 4], f2_pack(nn.z, nn.w), w);
      ma = max3_abs(ma, y[i].x, y[i + 1].x);
      mb = max3_abs(mb, y[i].y, y[i + 1].y);
    }
    ma = max_abs(ma, __shfl_xor_sync(0xFFFFFFFFu, ma, 16));
    mb = max_abs(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, 16));
    const uint32_t sa = e8m0_from_amax_f32(ma, p.rceil), sb = e8m0_from_amax_f32(mb, p.rceil);
    const f2 inv = f2_pack(inv_pow2(sa == 0xFF ? 127u : sa), inv_pow2(sb == 0xFF ? 127u : sb));
    uint32_t ca[4], cb[4], out[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f2 t[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) t[k] = f2_mul(y[4 * i + k], inv);
      ca[i] = sa == 0xFF ? 0x7F7F7F7Fu : cvt_e4m3x2(t[0].x, t[1].x) | (cvt_e4m3x2(t[2].x, t[3].x) << 16);
      cb[i] = sb == 0xFF ? 0x7F7F7F7Fu : cvt_e4m3x2(t[0].y, t[1].y) | (cvt_e4m3x2(t[2].y, t[3].y) << 16);
    }
    col16x2_gather(ca, cb, rh, out);                // lane: all 32 rows of one column
    const int64_t col = (int64_t)c0 * 8 + 2 * pc + rh;
    store32_codes(p.q_col + col * p.M + r0, out, v8);
    sc[p.s_col.mma ? (col >> 7) * p.s_col.tiles_per_row * 512 + (col & 31) * 16 + ((col >> 5) & 3) * 4 : col * p.s_col.ld] =
        (uint8_t)(rh ? sb : sa);
  }
}

// ---- backward: each CTA takes every G-th row.  Bulk copies bring the rows of
// dy, r (or its codes) and dres into a ring in shared memory, NB_STAGES - 1
// rows ahead, so that registers hold only the thread's columns of w and of the
// weight gradient (fp32, over all of the CTA's rows).  A row is read twice from
// shared memory: for the sum, which takes the row's one barrier, and for dx.
// Bound by HBM: 16384 x 7168 takes 126 us from a checkpoint (6.6 TB/s) and 137 us
// from bf16 (6.9 TB/s).  Rows held in registers, with the next row's loads in
// flight, took 128 of them, one CTA an SM, and 167 us from a checkpoint.  The
// CTAs' partial weight gradients go to the workspace [G][d] and a second kernel
// adds them in a fixed order: results do not change from run to run.  A CTA's
// sum is an fp32 chain of M / G rows, off by M / G times 2^-24 of its magnitudes at
// most (108 times for 16384 rows on one CTA an SM), below the 2^-9 of dw in bf16.
struct NormBwdParams {
  const uint8_t* dy;     // [M, d] bf16
  const uint8_t* r;      // [M, d] bf16, or (CK) its checkpoint codes
  const uint8_t* ck_s;   // [M, d/32]
  const float* rstd;     // [M]
  const uint4* w;        // [d]
  const uint8_t* dres;   // [M, d] bf16 or NULL
  uint4* dx;             // [M, d] bf16
  float* part;           // [G][d]
  int64_t M;
  int32_t d8;
  int32_t stages, stage_bytes;
  float inv_d;
};

// Eight saved values of r: bf16, or codes of a block with its power of two.
template <bool CK> struct Saved;
template <> struct Saved<false> {
  static constexpr int BYTES = 16;
  f2 v[4];
  MX_DEVINL void read(const uint8_t* at, float) {
    const uint4 x = *reinterpret_cast<const uint4*>(at);
    v[0] = f2_from_bf16x2(x.x); v[1] = f2_from_bf16x2(x.y); v[2] = f2_from_bf16x2(x.z); v[3] = f2_from_bf16x2(x.w);
  }
};
template <> struct Saved<true> {
  static constexpr int BYTES = 8;
  f2 v[4];
  MX_DEVINL void read(const uint8_t* at, float scale) {
    float f[8];
    values8(*reinterpret_cast<const uint2*>(at), scale, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_pack(f[2 * i], f[2 * i + 1]);
  }
};

template <int V, int T_MAX, int CTAS, bool CK>
__global__ void __launch_bounds__(T_MAX, CTAS) add_rmsnorm_bwd_kernel(NormBwdParams p) {
  extern __shared__ __align__(128) uint8_t ring[];   // [stages][dy | r | dres]
  __shared__ float sums[2][T_MAX / 32];
  __shared__ __align__(8) uint64_t full[NB_MAX_STAGES];
  const int T = blockDim.x, warps = T >> 5;
  const int64_t row_b = (int64_t)p.d8 * 16, saved_b = (int64_t)p.d8 * Saved<CK>::BYTES;
  auto load = [&](int64_t row, int s) {
    uint8_t* dst = ring + s * p.stage_bytes;
    mbar_arrive_expect_tx(&full[s], (uint32_t)(row_b + saved_b + (p.dres ? row_b : 0)));
    bulk_load(dst, p.dy + row * row_b, (uint32_t)row_b, &full[s]);
    bulk_load(dst + row_b, p.r + row * saved_b, (uint32_t)saved_b, &full[s]);
    if (p.dres) bulk_load(dst + row_b + saved_b, p.dres + row * row_b, (uint32_t)row_b, &full[s]);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  pdl_wait();
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages - 1; ++s)
      if (blockIdx.x + (int64_t)s * gridDim.x < p.M) load(blockIdx.x + (int64_t)s * gridDim.x, s);
  }
  uint4 w[V];
  f2 acc[V][4];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = threadIdx.x + k * T;
    w[k] = c < p.d8 ? __ldg(p.w + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[k][i] = f2_splat(0.0f);
  }
  __syncthreads();
  int stage = 0, par = 0;
  uint32_t phase = 0;
  // the statistic and the scale bytes of a row, fetched a row ahead
  float n_next = 0;
  uint32_t s_next[V] = {};
  auto fetch = [&](int64_t row) {
    n_next = p.rstd[row];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = threadIdx.x + k * T;
      if (CK && c < p.d8) s_next[k] = p.ck_s[row * (p.d8 >> 2) + (c >> 2)];
    }
  };
  bool lost = false;
  if (blockIdx.x < p.M) fetch(blockIdx.x);
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, par ^= 1) {
    const uint8_t* in = ring + stage * p.stage_bytes;
    const float n = n_next;
    float scale[V];
#pragma unroll
    for (int k = 0; k < V; ++k) scale[k] = CK ? pow2_of_byte(s_next[k]) : 0.0f;
    if (row + gridDim.x < p.M) fetch(row + gridDim.x);
    const bool here = mbar_wait(&full[stage], phase, nullptr);
    f2 dot2 = f2_splat(0.0f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = threadIdx.x + k * T;
      if (c < p.d8) {
        const uint4 dy = *reinterpret_cast<const uint4*>(in + c * 16);
        Saved<CK> r;
        r.read(in + row_b + c * Saved<CK>::BYTES, scale[k]);
        dot2 = f2_fma(mul_bf16x2(dy.x, w[k].x), r.v[0], dot2);
        dot2 = f2_fma(mul_bf16x2(dy.y, w[k].y), r.v[1], dot2);
        dot2 = f2_fma(mul_bf16x2(dy.z, w[k].z), r.v[2], dot2);
        dot2 = f2_fma(mul_bf16x2(dy.w, w[k].w), r.v[3], dot2);
      }
    }
    float dot = warp_sum(dot2.x + dot2.y);
    if ((threadIdx.x & 31) == 0) sums[par][threadIdx.x >> 5] = dot;
    // the row's barrier (the next row writes the other buffer); a wait that
    // ran out of its bound ends the kernel for the whole CTA, once the rows
    // still on their way have come (or run out of the bound as well), and makes
    // dw NaN
    if (!__syncthreads_and(here)) {
      for (int k = 1; k < p.stages - 1 && row + (int64_t)k * gridDim.x < p.M; ++k)
        mbar_wait(&full[(stage + k) % p.stages], stage + k < p.stages ? phase : phase ^ 1, nullptr);
      lost = true;
      break;
    }
    if (threadIdx.x == 0) {
      // every thread is past the previous row: its stage takes the next one
      const int64_t next = row + (int64_t)(p.stages - 1) * gridDim.x;
      if (next < p.M) load(next, stage == 0 ? p.stages - 1 : stage - 1);
    }
    dot = 0;
    for (int i = 0; i < warps; ++i) dot += sums[par][i];
    // n dot first, which has the size of dy w: n^2 passes fp32 where |r| < 2^-64
    const f2 n2 = f2_splat(n), c2 = f2_splat(-(n * dot * p.inv_d * n));
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = threadIdx.x + k * T;
      if (c >= p.d8) continue;
      const uint4 dy = *reinterpret_cast<const uint4*>(in + c * 16);
      const uint4 dr = p.dres ? *reinterpret_cast<const uint4*>(in + row_b + saved_b + c * 16) : make_uint4(0, 0, 0, 0);
      Saved<CK> r;
      r.read(in + row_b + c * Saved<CK>::BYTES, scale[k]);
      const uint32_t g[4] = {dy.x, dy.y, dy.z, dy.w}, ww[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
      const uint32_t dd[4] = {dr.x, dr.y, dr.z, dr.w};
      f2 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[k][i] = f2_fma(f2_from_bf16x2(g[i]), f2_mul(r.v[i], n2), acc[k][i]);
        o[i] = f2_fma(n2, f2_fma(c2, r.v[i], mul_bf16x2(g[i], ww[i])), f2_from_bf16x2(dd[i]));
      }
      p.dx[row * p.d8 + c] = pack8(o);
    }
    if (++stage == p.stages) { stage = 0; phase ^= 1; }
  }
  // Not before: waiting CTAs of the sums' kernel beside this one's (8192 x 4096,
  // call after call) took 47 us instead of 36.
  pdl_allow_next();
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = threadIdx.x + k * T;
    if (c >= p.d8) continue;
    float4* dst = reinterpret_cast<float4*>(p.part + ((int64_t)blockIdx.x * p.d8 + c) * 8);
    if (lost) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = f2_splat(__int_as_float(0x7FC00000));
    dst[0] = make_float4(acc[k][0].x, acc[k][0].y, acc[k][1].x, acc[k][1].y);
    dst[1] = make_float4(acc[k][2].x, acc[k][2].y, acc[k][3].x, acc[k][3].y);
  }
}

// dw[c] = sum over g of part[g][c]: C columns a block, R threads a column with every
// R-th row of the partials each, then their sums in order.  Bound by latency (2 of the
// 35 us of 8192 x 4096): few columns a block where a row has too few for all SMs
// (65536 x 512: 36 us in all with 8, 42 with 32), many for few partials (600 x 1536:
// 5.8 us with 32, 6.9 with 8; 300 x 7168 6.5 and 9.0).
constexpr int NB_SUM_THREADS = 1024;
template <int C>
__global__ void __launch_bounds__(NB_SUM_THREADS) norm_dw_kernel(const float* __restrict__ part, int32_t G, int32_t d,
                                                                 __nv_bfloat16* __restrict__ dw) {
  constexpr int R = NB_SUM_THREADS / C;
  static_assert(C <= NB_SUM_THREADS / 32, "a warp a column");
  __shared__ float s[C][R + 1];
  pdl_begin();  // the partials of the kernel before
  const int x = threadIdx.x % C, g0 = threadIdx.x / C, c = blockIdx.x * C + x;
  float t = 0;
  if (c < d) {
#pragma unroll 4
    for (int g = g0; g < G; g += R) t += part[(int64_t)g * d + c];
  }
  s[x][g0] = t;
  __syncthreads();
  const int col = threadIdx.x >> 5, lane = threadIdx.x & 31;  // warp: a column
  if (col >= C) return;
  t = 0;
#pragma unroll
  for (int i = lane; i < R; i += 32) t += s[col][i];
  t = warp_sum(t);
  if (lane == 0 && blockIdx.x * C + col < d) dw[blockIdx.x * C + col] = __float2bfloat16_rn(t);
}

// How a row is held: vectors of eight a thread, and by a warp or a CTA.
//   Few rows (two an SM or fewer): many threads a row (1 x 7168: 3.2 against 3.4
// us with two vectors against four; 152 x 1024: 1.8 against 2.1 with one and two).
//   Else as many loads in flight as the registers allow, which is four vectors,
// or two of x and two of the residual: without one, 8192 x 4096 takes 22.5 us with
// four and 27.0 with two, 16384 x 7168 75.9 and 92.3; with one 48.0 and 49.1, 158
// and 162; 16384 x 2048 47 with two, 58 with one.  Past 8192 columns a CTA's 512
// threads need four (without a residual 128 us; 131 with eight), or take eight
// (with one: 184 us for 8192 x 16384; 198 with four).
//   Up to 512 columns, and to 1024 without a residual, a warp has a row: CTAs of
// one row cannot start faster (65536 x 512: 23 us, 66 with them; 32768 x 1024
// without a residual 22 against 33, with one 48 against 47).
struct RowShape {
  int V;
  bool warp;
};
RowShape row_shape(int64_t M, int d8, bool res) {
  if (M <= 2 * (int64_t)num_sms()) return {d8 <= 256 ? 1 : d8 <= 1024 ? 2 : 4, false};
  if (d8 <= 64) return {2, true};
  if (d8 <= 128 && !res) return {4, true};
  return {d8 > 1024 ? (res ? 8 : 4) : res ? 2 : 4, false};
}
int threads_of(int d8, int V) { return ((d8 + V - 1) / V + 31) / 32 * 32; }

// Backward: vectors and threads, CTAs an SM, ring stages.  Four vectors a thread:
// few warps meet at a row's barrier, and several rows are under way.  512 threads
// an SM from a checkpoint (with a residual gradient, against 896 threads with two
// vectors: 8192 x 8192 77 us and 104, 16384 x 5120 94 and 103), 384 from bf16, whose
// rows need fewer instructions and fill the ring sooner (16384 x 8192 153 us, 158
// with 512; 16384 x 5120 without a residual gradient 77 and 87).  Up to 512 columns
// a warp has a row, 24 of them an SM (65536 x 512: 42 us; 51 and 56 with 24 and 16
// before the sum of its partials was spread over more blocks).
struct NormBwdShape {
  int V, T, ctas, stages, stage_bytes;
};
NormBwdShape bwd_shape(int64_t d, bool ck, bool dres) {
  NormBwdShape s;
  const int d8 = (int)(d / 8);
  s.V = d8 <= 32 ? 1 : d8 <= 64 ? 2 : 4;
  s.T = threads_of(d8, s.V);
  s.stage_bytes = (int)((d * (2 + (ck ? 1 : 2) + (dres ? 2 : 0)) + 127) / 128 * 128);
  const int smem = NB_MAX_SMEM;
  s.ctas = std::max(1, s.V < 4 ? 24 : (ck ? 512 : 384) / s.T);
  while (s.ctas > 1 && (smem / s.ctas - 1024) / s.stage_bytes < 2) --s.ctas;
  s.stages = std::min(NB_MAX_STAGES, (smem / s.ctas - 1024) / s.stage_bytes);
  return s;
}

// Two-axis kernels by [exact][residual][checkpoint][bf16 y][row codes].
using ColKernel = void (*)(NormFwdParams, int32_t);
#define MX_NC(R, C, X) {{add_rmsnorm_col_kernel<R, C, false, false, X>, add_rmsnorm_col_kernel<R, C, false, true, X>}, \
                        {add_rmsnorm_col_kernel<R, C, true, false, X>, add_rmsnorm_col_kernel<R, C, true, true, X>}}
const ColKernel col_kernels[2][2][2][2][2] = {
    {{MX_NC(false, false, false), MX_NC(false, true, false)}, {MX_NC(true, false, false), MX_NC(true, true, false)}},
    {{MX_NC(false, false, true), MX_NC(false, true, true)}, {MX_NC(true, false, true), MX_NC(true, true, true)}}};
#undef MX_NC

int col_attributes(ColKernel k) {
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, NC_MAX_SMEM);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return cuda_status(e, "cudaFuncSetAttribute");
}

// CTAs of a cluster, at most: sixteen, or eight where no part of the device (a slice of
// one, say) holds sixteen.  The kernels differ in nothing that counts for it, so one
// is asked about, once a device.
std::atomic<int> g_col_limit;  // mx_selftest_norm_clusters
int col_cluster_limit(int* most) {
  static std::atomic<int> held[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e, "cudaGetDevice");
  int n = held[dev & 63].load(std::memory_order_relaxed);
  if (n == 0) {
    const ColKernel k = col_kernels[0][1][1][1][1];
    if (int rc = col_attributes(k)) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, NC_MAX_CTAS);
    cfg.blockDim = dim3(NC_THREADS);
    cfg.dynamicSmemBytes = NC_ROWS * (kNormMaxD / NC_MAX_CTAS) * 2;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = NC_MAX_CTAS;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int m = 0;
    e = cudaOccupancyMaxActiveClusters(&m, k, &cfg);
    if (e != cudaSuccess) return cuda_status(e, "cudaOccupancyMaxActiveClusters");
    n = m > 0 ? NC_MAX_CTAS : NC_PORTABLE_CTAS;
    held[dev & 63].store(n, std::memory_order_relaxed);
  }
  const int limit = g_col_limit.load(std::memory_order_relaxed);
  *most = limit ? std::min(limit, n) : n;
  return MX_OK;
}

}  // namespace

void set_norm_cluster_limit(int most) { g_col_limit.store(most, std::memory_order_relaxed); }

// CTAs of the backward pass: each with two rows at least, beyond two an SM (1200 x
// 1024: 7.2 us, 8.0 with a row each, whose partial gradients outweigh it).
int bwd_grid(int64_t M, int ctas_sm) {
  const int64_t sms = num_sms();
  return (int)std::min(std::min(M, ctas_sm * sms), std::max(2 * sms, M / 2));
}
// Rows of partial weight gradients, whatever is kept of r and with or without
// a residual gradient.
int norm_bwd_ctas(int64_t M, int64_t d) { return bwd_grid(M, bwd_shape(d, true, false).ctas); }

int launch_add_rmsnorm_fwd(const NormFwdLaunch& a, cudaStream_t stream) {
  NormFwdParams p{};
  p.x = (const uint4*)a.x; p.res = (const uint4*)a.residual; p.w = (const uint4*)a.w;
  p.r = (uint4*)a.r; p.rstd = a.rstd; p.y = (uint4*)a.y;
  p.M = a.M; p.d8 = (int32_t)(a.d / 8); p.d = (float)a.d; p.eps = a.eps;
  p.rceil = a.floor_scale ? 0u : 1u;
  const bool mma = a.layout == MX_SCALE_MMA;
  const int64_t Sr = a.d / 32, Sc = a.M / 32;
  p.q_row = (uint8_t*)a.q_row; p.s_row = ScaleDst{(uint8_t*)a.s_row, (Sr + 3) / 4, Sr, mma};
  p.q_col = (uint8_t*)a.q_col; p.s_col = ScaleDst{(uint8_t*)a.s_col, (Sc + 3) / 4, Sc, mma};
  p.ck = (uint8_t*)a.ck; p.ck_s = (uint8_t*)a.ck_scales;
  const int64_t padded = mma && (a.q_row || a.q_col) ? (a.M + 127) / 128 * 128 : a.M;  // rows of the scale layout
  if (padded > INT32_MAX) return fail(MX_ERR_UNSUPPORTED, "norm: too many rows");
  if (a.q_col) {
    // Slices of a multiple of 256 columns (whole warps).  Enough rows: at least
    // 512 columns, so that clusters stay small (16384 x 2048: 63 us on four CTAs,
    // 72 on eight), on up to eleven CTAs, whose tiles of 768 columns leave an SM four
    // of them (before the residual's prefetch, 16384 x 7168: 212 us on ten, 219 on
    // seven; 16384 x 8192: 240 on eleven, 248 on eight), sixteen where slices would pass that (8192 x 16384).  Few rows
    // (under two 512-column slices an SM): as many CTAs as there can be (32 x 7168:
    // 6.7 us on fourteen, 9.4 on seven; 1024 x 2048: 7.3 us on eight, 8.5 on four).
    const bool few = padded / NC_ROWS * ((p.d8 + 63) / 64) <= 2 * (int64_t)num_sms();
    int limit;
    if (int rc = col_cluster_limit(&limit)) return rc;
    const int most = std::min(limit, few || p.d8 > 11 * 96 ? NC_MAX_CTAS : 11);
    const int slice8 = std::max(few ? 32 : 64, ((p.d8 + 31) / 32 + most - 1) / most * 32);
    const int ctas = (p.d8 + slice8 - 1) / slice8;
    const size_t smem = (size_t)NC_ROWS * slice8 * 16;
    const ColKernel k =
        col_kernels[short_number(p.eps)][p.res != nullptr][p.ck != nullptr][p.y != nullptr][p.q_row != nullptr];
    if (int rc = col_attributes(k)) return rc;
    count_launch(MX_KERNEL_NORM);
    return cuda_status(launch_overlapped(k, dim3((unsigned)(padded / NC_ROWS), (unsigned)ctas), NC_THREADS, smem, stream,
                                         dim3(1, (unsigned)ctas), p, (int32_t)slice8),
                       "add_rmsnorm_col_kernel launch");
  }
  const RowShape sh = row_shape(a.M, p.d8, p.res != nullptr);
  count_launch(MX_KERNEL_NORM);
  using Kernel = void (*)(NormFwdParams);
  // [exact]: a row a warp, V = 2 and 4; a row a CTA, V = 1, 2, 4 and 8
#define MX_NR(X) {add_rmsnorm_row_kernel<2, true, X>, add_rmsnorm_row_kernel<4, true, X>, add_rmsnorm_row_kernel<1, false, X>, \
                  add_rmsnorm_row_kernel<2, false, X>, add_rmsnorm_row_kernel<4, false, X>, add_rmsnorm_row_kernel<8, false, X>}
  static const Kernel kernels[2][6] = {MX_NR(false), MX_NR(true)};
#undef MX_NR
  const Kernel k = kernels[short_number(p.eps)][sh.warp ? sh.V / 4 : sh.V == 1 ? 2 : sh.V == 2 ? 3 : sh.V == 4 ? 4 : 5];
  const int64_t grid = sh.warp ? (padded + ROW_WARPS - 1) / ROW_WARPS : padded;
  const int threads = sh.warp ? ROW_WARPS * 32 : threads_of(p.d8, sh.V);
  return cuda_status(launch_overlapped(k, (unsigned)grid, threads, 0, stream, 1, p), "add_rmsnorm_row_kernel launch");
}

int launch_add_rmsnorm_bwd(const NormBwdLaunch& a, cudaStream_t stream) {
  const NormBwdShape s = bwd_shape(a.d, a.ck != nullptr, a.dres != nullptr);
  NormBwdParams p{};
  p.dy = (const uint8_t*)a.dy; p.r = (const uint8_t*)(a.ck ? a.ck : a.r); p.ck_s = (const uint8_t*)a.ck_scales;
  p.rstd = a.rstd; p.w = (const uint4*)a.w; p.dres = (const uint8_t*)a.dres; p.dx = (uint4*)a.dx;
  p.part = (float*)a.workspace;
  p.M = a.M; p.d8 = (int32_t)(a.d / 8); p.inv_d = 1.0f / (float)a.d;
  p.stages = s.stages; p.stage_bytes = s.stage_bytes;
  const int G = bwd_grid(a.M, s.ctas);
  const size_t smem = (size_t)s.stages * s.stage_bytes;
  using Kernel = void (*)(NormBwdParams);
#define MX_NB(V, T, C) {add_rmsnorm_bwd_kernel<V, T, C, false>, add_rmsnorm_bwd_kernel<V, T, C, true>}
  static const Kernel kernels[3][2] = {MX_NB(1, 32, 24), MX_NB(2, 32, 24), MX_NB(4, 512, 1)};
#undef MX_NB
  const Kernel k = kernels[s.V == 1 ? 0 : s.V == 2 ? 1 : 2][a.ck != nullptr];
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, NB_MAX_SMEM);
  if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute");
  count_launch(MX_KERNEL_NORM);
  e = launch_overlapped(k, G, s.T, smem, stream, 1, p);
  if (e != cudaSuccess) return cuda_status(e, "add_rmsnorm_bwd_kernel launch");
  count_launch(MX_KERNEL_NORM);
  // columns a block of the sum: 32 for few partials or where that gives every SM a block
  const int C = G <= 2 * num_sms() || a.d >= 32 * num_sms() ? 32 : a.d >= 16 * num_sms() ? 16 : 8;
  auto sum = C == 32 ? norm_dw_kernel<32> : C == 16 ? norm_dw_kernel<16> : norm_dw_kernel<8>;
  return cuda_status(launch_overlapped(sum, (unsigned)((a.d + C - 1) / C), NB_SUM_THREADS, 0, stream, 1, (const float*)p.part,
                                       (int32_t)G, (int32_t)a.d, (__nv_bfloat16*)a.dw),
                     "norm_dw_kernel launch");
}

}  // namespace mx
