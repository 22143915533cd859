// fp8mm.cu - matrix products of E4M3 operands with one fp32 scale for 128 contraction elements of a token row and for
// 128 x 128 of a weight, dense or grouped by expert.
//
//   FWD    out[t, n] = sum_b sx[b, t] sw[e, n / 128, b] sum_{k in block b} x[t, k] w[e, n, k]
//   DGRAD  dx[t, k]  = sum_b sd[b, t] sw[e, b, k / 128] sum_{n in block b} dout[t, n] w[e, n, k]
//
// (DGRAD reads the transposed codes, so both are one product: features F, contraction C.)  The inner sums are tensor core
// products (tcgen05, kind::f8f6f4) of 128 elements, each into an accumulator of its own in TMEM; the epilogue warps
// bring it out, multiply it by its scales in fp32 and add it to sums in registers.  One rounding to bf16 at the end.
//
// What that bounds: an accumulator of 128 x 256 is 128 KB to be read and 32768 FMAs to be done in the 512 cycles that its
// MMAs take, and its columns are free for the next but one only when both CTAs of a pair have read them.  So there are
// two kernels.
//   Many rows a group: tokens on the M side, so that a lane of the epilogue has one token and a K block's scale is
// one number for it (with tokens on the N side a scale a column comes from shared memory, which the MMAs' operands
// fill already: 715 against 413 us for 8192 x 4096 x 14336 at the first build of both).  CTA pairs, 256 x 256.
//   Few rows: tokens on the N side (any multiple of 32 at run time), features on the M side, so that a group's last tile
// costs what its rows cost; one CTA a tile, or several that share its contraction.
//
// On a GB300 (twice the bf16 library rate: 3.9 PFLOP/s; copies 6.78 TB/s): 8192 x 4096 x 14336 309 us (3.1 PFLOP/s; 2.7 in
// long runs, by the power limit), 131072 rows over 64 experts of 4096 x 7168 both ways 5.95 ms (2.6 PFLOP/s); 64 rows over 64
// of them, 31 hit, 144 us (6.3 TB/s of weights); 8 rows of 4096 x 7168 8.3 us (9.4 from HBM); 800 rows over 8 of 2048 x 2048 12.5 us.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace mx {

namespace {

constexpr int FM_EPI = 8;                 // epilogue warps
constexpr int FM_MAX_E = 1024;
constexpr int FM_THREADS = 128 + FM_EPI * 32;
constexpr int FM_REGS = 168;              // a thread at launch; after the split 88 + 2 * 208 or 56 + 2 * 224 = 3 * 168

// A CTA has 128 features; BT: columns of a token tile; S: CTAs that share a tile's contraction.
template <int BT, int S>
struct FCfg {
  static constexpr int A_BYTES = 128 * 128;              // 128 features x 128 contraction elements
  static constexpr int B_BYTES = BT * 128;
  static constexpr int TX = A_BYTES + B_BYTES;
  static constexpr int EPI_BYTES = FM_EPI * 2048;        // a warp's 32 x 32 bf16 block
  static constexpr int TABLE = FM_MAX_E * 8;             // group ends and running unit numbers
  static constexpr int PART = BT * 128 * 4;              // one CTA's sums
  static constexpr int PARTS = (S - 1) * PART;           // in a tile's first CTA: the others'
  static constexpr int BUFS = 4;                         // accumulators, and the scales of their K blocks
  static constexpr int SC_BYTES = BUFS * BT * 4;
  static constexpr int TMEM = BUFS * BT;
  static constexpr uint32_t IDESC = (1u << 4) | ((128u >> 4) << 24);
  static constexpr int STAGES = (226 * 1024 - EPI_BYTES - SC_BYTES - PARTS - TABLE - 1536) / TX;
  static constexpr size_t SMEM = (size_t)STAGES * TX + EPI_BYTES + SC_BYTES + PARTS + TABLE + 512 /*barriers*/ + 1024 /*align*/;
  static_assert(BT == 64 || BT == 32, "tile widths");
  static_assert(S == 1 || S == 2 || S == 4, "CTAs of a cluster");
  static_assert(STAGES >= 3, "shared memory");
  static_assert((2 * STAGES + 2 * BUFS + 2 + FM_EPI) * 8 <= 512, "barriers");
  static_assert(SMEM + 1024 /*static*/ <= 227 * 1024, "shared memory");
};

struct MmParams {
  int64_t M;                // token rows
  int32_t F, C;             // features, contraction length
  int32_t E;
  const int32_t* offs;      // NULL: one group of all rows
  const float* st;          // [ceil(C / 128), M]
  const float* sw;          // of expert e, feature block f, contraction block c: sw[e * sw_e + f * sw_f + c * sw_c]
  int64_t sw_e, sw_f, sw_c;
  uint8_t* out;             // [M, F] bf16
  int32_t* err;
};

MX_DEVINL void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Four values into another CTA of the cluster, counted by a barrier there: the sender waits for nothing (stores and an arrival
// that releases them take it 2000 cycles).
MX_DEVINL void st_async_4(uint32_t dst, f2 a, f2 b, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst), "f"(a.x),
               "f"(a.y), "f"(b.x), "f"(b.y), "r"(bar)
               : "memory");
}

// warp_wait by the barrier's shared memory address.
MX_DEVINL bool mbar_try_wait_at(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// `done`: an earlier try's outcome.
MX_DEVINL bool warp_wait_at(uint32_t bar, uint32_t parity, int32_t* err, bool done = false) {
  if (__all_sync(0xFFFFFFFFu, done)) return true;
  done = mbar_try_wait_at(bar, parity);
  if (!done) {
    const uint64_t t0 = globaltimer_ns();
    while (!(done = mbar_try_wait_at(bar, parity)))
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        record_error(err, MX_ERR_TIMEOUT);
        break;
      }
  }
  return __all_sync(0xFFFFFFFFu, done);
}

// acc += (a s, b t), where it stands: as a volatile statement it stays behind the TMEM load that was issued before it (left
// to the compiler's order, 356 against 342 us for 8192 x 4096 x 14336).
MX_DEVINL void fma_here(f2& acc, uint32_t a, uint32_t b, float s, float t) {
  asm volatile(
      "{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%0, %1};\n"
      " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;\n}"
      : "+f"(acc.x), "+f"(acc.y)
      : "r"(a), "r"(b), "f"(s), "f"(t));
}

// Bounded wait for arrivals from other CTAs of the cluster, whose writes it makes visible.
MX_DEVINL bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, int32_t* err) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      record_error(err, MX_ERR_TIMEOUT);
      return false;
    }
  }
}

template <int R>
MX_DEVINL void regs_give() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
MX_DEVINL void regs_take() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }

// tcgen05.wait::ld that the loaded registers pass through: no use of them moves ahead of it.
MX_DEVINL void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

struct Unit {
  int32_t e;
  int32_t f0;       // first feature
  int64_t t0;       // first token row
  int32_t tn;       // live rows of the tile
  int32_t n_eff;    // tn rounded up to the MMA's multiple of 32
};

// Tiles of BT token rows and FT features.
template <int BT, int FT>
MX_DEVINL Unit unit_of(const MmParams& p, const int32_t* ends, const int32_t* unit_end, int32_t u) {
  // u's group: as many as end before u, by blocks of 32 and within one (a warp calls this together)
  const int lane = threadIdx.x & 31;
  const int32_t b = 32 * __popc(__ballot_sync(0xFFFFFFFFu, 32 * lane + 31 < p.E && unit_end[min(32 * lane + 31, p.E - 1)] <= u));
  const int lo = b + __popc(__ballot_sync(0xFFFFFFFFu, b + lane < p.E && unit_end[min(b + lane, p.E - 1)] <= u));
  Unit r;
  r.e = lo;
  const uint32_t f_tiles = (uint32_t)(p.F + FT - 1) / FT;
  const uint32_t v = u - (lo ? unit_end[lo - 1] : 0);
  const int32_t start = lo ? ends[lo - 1] : 0, rows = ends[lo] - start;
  const uint32_t t_tiles = (uint32_t)(rows + BT - 1) / BT;
  int32_t t = 0, f = v;
  if (t_tiles > 1) {
    if (rows <= p.F) {  // the rows are the smaller operand: re-read them, stream the weights once
      f = v / t_tiles;
      t = v - f * t_tiles;
    } else {
      t = v / f_tiles;
      f = v - t * f_tiles;
    }
  }
  r.f0 = f * FT;
  r.t0 = (int64_t)start + (int64_t)t * BT;
  r.tn = min(BT, rows - t * BT);
  r.n_eff = (r.tn + 31) & ~31;
  return r;
}

// By all threads: group ends as they lie.
MX_DEVINL void load_ends(const MmParams& p, int32_t* ends) {
  for (int e = threadIdx.x; e < p.E; e += FM_THREADS) ends[e] = __ldg(p.offs + e);
}

// By one thread, without group ends: one group of all rows.
template <int BT, int FT>
MX_DEVINL void one_group(const MmParams& p, int32_t* ends, int32_t* unit_end, int* s_ok, int* s_units) {
  ends[0] = (int32_t)p.M;
  *s_units = unit_end[0] = (int32_t)((p.M + BT - 1) / BT) * ((p.F + FT - 1) / FT);
  *s_ok = 1;
}

// By one warp: group ends checked, and the running number of work units.
template <int BT, int FT>
MX_DEVINL void read_ends(const MmParams& p, const int32_t* ends, int32_t* unit_end, int* s_ok, int* s_units) {
  const int lane = threadIdx.x & 31;
  const int32_t f_tiles = (p.F + FT - 1) / FT;
  int32_t prev = 0, units = 0;
  bool ok = true;
  for (int base = 0; base < p.E; base += 32) {
    const int e = base + lane;
    const int32_t v = e >= p.E ? 0x7FFFFFFF : ends[e];
    int32_t before = __shfl_up_sync(0xFFFFFFFFu, v, 1);
    if (lane == 0) before = prev;
    const bool in = e < p.E;
    if (in && (v < before || v < 0 || (int64_t)v > p.M)) ok = false;
    int32_t n = in && ok ? (v - before + BT - 1) / BT * f_tiles : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t m = __shfl_up_sync(0xFFFFFFFFu, n, o);
      if (lane >= o) n += m;
    }
    if (in) unit_end[e] = units + n;
    units += __shfl_sync(0xFFFFFFFFu, n, 31);
    prev = __shfl_sync(0xFFFFFFFFu, v, min(31, p.E - 1 - base));
  }
  ok = __all_sync(0xFFFFFFFFu, ok);
  if (lane == 0) {
    *s_ok = ok;
    *s_units = ok ? units : 0;
    if (!ok && blockIdx.x == 0) record_error(p.err, MX_ERR_BAD_OFFSETS);
  }
}

// By the epilogue's threads: rows past the last group (all rows, if the ends were refused) are zeros.
MX_DEVINL void zero_spare_rows(const MmParams& p, int64_t first, int thread) {
  uint4* dst = reinterpret_cast<uint4*>(p.out + first * p.F * 2);
  const int64_t n = (p.M - first) * p.F / 8;
  for (int64_t i = (int64_t)blockIdx.x * (FM_EPI * 32) + thread; i < n; i += (int64_t)gridDim.x * (FM_EPI * 32))
    dst[i] = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------- tokens on the N side

template <int BT, int S>
__global__ void __launch_bounds__(FM_THREADS, 1)
    fp8_mm_narrow_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, MmParams p) {
  using C = FCfg<BT, S>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + C::STAGES * C::A_BYTES;
  uint8_t* sEpi = sB + C::STAGES * C::B_BYTES;
  float* sScale = reinterpret_cast<float*>(sEpi + C::EPI_BYTES);
  uint8_t* sParts = sEpi + C::EPI_BYTES + C::SC_BYTES;
  int32_t* ends = reinterpret_cast<int32_t*>(sParts + C::PARTS);
  int32_t* unit_end = ends + FM_MAX_E;
  uint64_t* full = reinterpret_cast<uint64_t*>(sParts + C::PARTS + C::TABLE);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + C::BUFS;
  uint64_t* parts_bar = acc_empty + C::BUFS;   // S > 1, by epilogue warp: the other pairs' sums are here
  uint64_t* done_bar = parts_bar + FM_EPI;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done_bar + 1);
  __shared__ int s_ok, s_units;

  // by way of a shuffle the compiler knows it to be one number for the warp: without, the roles spill (24 bytes, read back
  // in their loops)
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int part = S > 1 ? (int)cluster_ctarank() : 0;   // this CTA's share of the contraction
  const int32_t unit0 = blockIdx.x / S, ustep = gridDim.x / S;
  const int32_t kb0 = (p.C + 127) / 128 * part / S, num_kb = (p.C + 127) / 128 * (part + 1) / S - kb0;   // this CTA's K blocks

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int a = 0; a < C::BUFS; ++a) { mbar_init(&acc_full[a], 2); mbar_init(&acc_empty[a], FM_EPI); }
    for (int e = 0; e < FM_EPI; ++e) mbar_init(&parts_bar[e], 1);
    mbar_init(done_bar, 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 96 && !p.offs) one_group<BT, 128>(p, ends, unit_end, &s_ok, &s_units);
  if (warp == 1) { tmem_alloc(tmem_holder, C::TMEM); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (S > 1) cluster_sync();  // the others' barriers exist before any remote arrive
  const uint32_t tmem = *tmem_holder;
  if (p.offs) {
    pdl_begin();     // all of the above overlaps the kernel before
    load_ends(p, ends);
    __syncthreads();
    if (warp == 2) read_ends<BT, 128>(p, ends, unit_end, &s_ok, &s_units);
    __syncthreads();
  } else {
    // The warps that load and store wait, when they have worked out where: at every tile, as a role's first is not always the
    // CTA's (the second scale warp has none in a tile of one K block); behind the first a wait returns at once.
    pdl_allow_next();
  }
  const int32_t n_units = s_units;

  if (warp < 4) {
    regs_give<88>();
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      const bool leader = elect_one();
      if (leader) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
      }
      int stage = 0; uint32_t phase = 0;
      bool ok = true;
      for (int32_t u = unit0; u < n_units && ok; u += ustep) {
        const Unit t = unit_of<BT, 128>(p, ends, unit_end, u);
        if (!p.offs) pdl_wait();
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!warp_wait(&empty[stage], phase ^ 1, p.err)) { ok = false; break; }
          if (leader) {
            mbar_arrive_expect_tx(&full[stage], C::TX);
            tma_load_3d(sA + stage * C::A_BYTES, &tmA, (kb0 + kb) * 128, t.f0, t.e, &full[stage]);
            tma_load_2d(sB + stage * C::B_BYTES, &tmB, (kb0 + kb) * 128, (int32_t)t.t0, &full[stage]);
          }
          __syncwarp();
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMAs
      const bool leader = elect_one();
      // K-major: 8-row atoms 1024 bytes apart, 32 elements = 32 bytes along the row
      const uint64_t a0 = smem_desc(smem_u32(sA), 16, 1024, 2);
      const uint64_t b0 = smem_desc(smem_u32(sB), 16, 1024, 2);
      int stage = 0; uint32_t phase = 0;
      int buf = 0; uint32_t buf_phase = 0;
      bool ok = true;
      for (int32_t u = unit0; u < n_units && ok; u += ustep) {
        const Unit t = unit_of<BT, 128>(p, ends, unit_end, u);
        const uint32_t idesc = C::IDESC | ((uint32_t)(t.n_eff >> 3) << 17);
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!warp_wait(&acc_empty[buf], buf_phase ^ 1, p.err)) { ok = false; break; }
          if (!warp_wait(&full[stage], phase, p.err)) { ok = false; break; }
          tc_fence_after();
          if (leader) {
            const uint32_t d = tmem + (uint32_t)(buf * BT);
            const uint64_t ad = a0 + (uint64_t)((stage * C::A_BYTES) >> 4);
            const uint64_t bd = b0 + (uint64_t)((stage * C::B_BYTES) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f8(d, ad + k * 2, bd + k * 2, idesc, k > 0);
            tc_commit(&empty[stage]);
            tc_commit(&acc_full[buf]);
          }
          __syncwarp();
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
          if (++buf == C::BUFS) { buf = 0; buf_phase ^= 1; }
        }
      }
      if (leader) tc_commit(done_bar);
      __syncwarp();
      mbar_wait(done_bar, 0, p.err);
      __syncwarp();
    } else {
      // ------------------------------------------------------------ scales
      // Every other K block of a warp's: those of the tile's tokens times the one of the CTA's features, loaded four turns
      // ahead.  They are part of what an accumulator's acc_full stands for, and their place is free when it is.
      constexpr int PER = BT / 32;
      int32_t next_u = unit0, next_kb = warp - 2;  // K blocks are numbered through all units
      bool fresh = true;
      const float *st = nullptr, *w = nullptr;
      int live = 0;
      float s[4][PER], f[4];
      bool have[4];
      auto load = [&](int i) {
        while (next_kb >= num_kb && next_u < n_units) { next_kb -= num_kb; next_u += ustep; fresh = true; }
        have[i] = next_u < n_units;
        if (!have[i]) return;
        if (fresh) {
          const Unit t = unit_of<BT, 128>(p, ends, unit_end, next_u);
          st = p.st + (kb0 + next_kb) * p.M + t.t0 + lane;
          w = p.sw + t.e * p.sw_e + (t.f0 >> 7) * p.sw_f + (kb0 + next_kb) * p.sw_c;
          live = t.tn - lane;
          fresh = false;
          if (!p.offs) pdl_wait();
        }
#pragma unroll
        for (int c = 0; c < PER; ++c) s[i][c] = 32 * c < live ? __ldg(st + 32 * c) : 0.0f;
        f[i] = __ldg(w);
        st += 2 * p.M, w += 2 * p.sw_c;
        next_kb += 2;
      };
      int buf = warp - 2; uint32_t phase = 0;
      bool ok = num_kb > 0;
      if (ok) {
#pragma unroll
        for (int i = 0; i < 4; ++i) load(i);
      }
      while (ok) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!ok || !have[i]) { ok = false; break; }
          if (!warp_wait(&acc_empty[buf], phase ^ 1, p.err)) { ok = false; break; }
          float* dst = sScale + buf * BT + lane;
#pragma unroll
          for (int c = 0; c < PER; ++c) dst[32 * c] = s[i][c] * f[i];
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_full[buf]);
          buf += 2;
          if (buf >= C::BUFS) { buf -= C::BUFS; phase ^= 1; }
          load(i);
        }
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    regs_take<208>();
    const int ew = warp - 4, q = warp & 3, half = ew >> 2;
    if (!p.offs) pdl_wait();
    uint8_t* stg = sEpi + ew * 2048;
    const int c = half * 32;                     // this warp's columns (BT = 32: half of the warps have none)
    const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16);
    const int qr = lane >> 2, qc = (lane & 3) * 8;
    const uint32_t full_at = smem_u32(acc_full), scales = smem_u32(sScale);
    int buf = 0; uint32_t buf_phase = 0;
    bool ok = true;
    for (int32_t u = unit0; u < n_units && ok; u += ustep) {
      const Unit t = unit_of<BT, 128>(p, ends, unit_end, u);
      const int32_t f = t.f0 + q * 32;   // this warp's features
      const bool here = c < t.tn;
      f2 acc[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = f2_splat(0.0f);
      for (int kb = 0; kb < num_kb; ++kb) {
        ok = warp_wait_at(full_at + buf * 8, buf_phase, p.err);
        if (!ok) break;
        tc_fence_after();
        if (here) {
          const uint32_t sc = scales + (buf * BT + c) * 4;
          uint32_t v[32];
          tmem_ld_32cols(tb + (uint32_t)(buf * BT + c), v);
          tmem_ld_wait(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float4 m;
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(m.x), "=f"(m.y), "=f"(m.z), "=f"(m.w) : "r"(sc + i * 16));
            fma_here(acc[2 * i], v[4 * i], v[4 * i + 1], m.x, m.y);
            fma_here(acc[2 * i + 1], v[4 * i + 2], v[4 * i + 3], m.z, m.w);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
        if (++buf == C::BUFS) { buf = 0; buf_phase ^= 1; }
      }
      if (!ok || f >= p.F || !here) continue;
      if constexpr (S > 1) {
        // the other CTAs' sums to the first, which adds them in order: 8 vectors of 4 tokens a lane
        const uint32_t at = (uint32_t)((BT == 32 ? q : ew) * 32 + lane) * 16;
        constexpr int V_STEP = (BT == 32 ? 4 : 8) * 512;
        if (part) {
          const uint32_t dst = cluster_map(smem_u32(sParts), 0) + (part - 1) * C::PART + at;
          const uint32_t bar = cluster_map(smem_u32(&parts_bar[ew]), 0);
#pragma unroll
          for (int i = 0; i < 8; ++i) st_async_4(dst + i * V_STEP, acc[2 * i], acc[2 * i + 1], bar);
          continue;
        }
        if (lane == 0) mbar_arrive_expect_tx(&parts_bar[ew], (S - 1) * 32 * 128);
        __syncwarp();
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&parts_bar[ew], 0, p.err));
        if (!ok) {
          mbar_wait_cluster(&parts_bar[ew], 0, p.err);   // once more for what may still come, before this CTA leaves
          break;
        }
#pragma unroll 1
        for (int o = 0; o < S - 1; ++o)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(sParts + o * C::PART + at + i * V_STEP);
            acc[2 * i] = f2_add(acc[2 * i], f2_pack(v.x, v.y));
            acc[2 * i + 1] = f2_add(acc[2 * i + 1], f2_pack(v.z, v.w));
          }
      }
      // a lane has one feature of all 32 tokens: turned through shared memory
      uint8_t* dst = p.out + ((t.t0 + c + qr) * p.F + f + qc) * 2;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t v = f2_to_bf16x2(acc[i]);
        *reinterpret_cast<uint16_t*>(stg + (2 * i) * 64 + lane * 2) = (uint16_t)v;
        *reinterpret_cast<uint16_t*>(stg + (2 * i + 1) * 64 + lane * 2) = (uint16_t)(v >> 16);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i * 8 + qr < t.tn && f + qc < p.F)
          *reinterpret_cast<uint4*>(dst + (int64_t)(i * 8) * p.F * 2) =
              *reinterpret_cast<const uint4*>(stg + (i * 8 + qr) * 64 + (lane & 3) * 16);
    }
    zero_spare_rows(p, s_ok ? ends[p.E - 1] : 0, ew * 32 + lane);
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (S > 1) cluster_sync();  // no store or arrive from another CTA targets an exited one
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::TMEM);
}

// ---------------------------------------------------------------- tokens on the M side

// 128 tokens and 256 features a CTA, 256 tokens a pair.
struct WCfg {
  static constexpr int A_BYTES = 128 * 128;              // 128 tokens x 128 contraction elements
  static constexpr int B_BYTES = 128 * 128;              // this CTA's half of the tile's features
  static constexpr int TX = A_BYTES + B_BYTES;
  static constexpr int TABLE = FM_MAX_E * 8;
  static constexpr int SLOTS = 4;                        // K blocks whose scales are at hand
  static constexpr int SC_BYTES = SLOTS * 256 * 4;       // 128 tokens x 2 feature blocks each
  static constexpr int OUTS = 3;                         // 32 x 32 bf16 blocks of a warp on their way out
  static constexpr int EPI_BYTES = FM_EPI * OUTS * 2048;
  static constexpr int TILES = 16;                       // tiles that the epilogue is told of by the scales' warps
  static constexpr int TILE_BYTES = TILES * 2 * 16;
  static constexpr int BUFS = 4;                         // accumulators of 128 columns, two for either feature block
  static constexpr int TMEM = BUFS * 128;
  static constexpr uint32_t IDESC = (1u << 4) | ((128u >> 3) << 17) | ((256u >> 4) << 24);
  static constexpr int STAGES = (226 * 1024 - EPI_BYTES - SC_BYTES - TILE_BYTES - TABLE - 1536) / TX;
  static constexpr size_t SMEM = (size_t)STAGES * TX + EPI_BYTES + SC_BYTES + TILE_BYTES + TABLE + 512 /*barriers*/ + 1024 /*align*/;
  static_assert((2 * STAGES + 2 * BUFS + 2) * 8 <= 512, "barriers");
  static_assert(SMEM + 1024 /*static*/ <= 227 * 1024, "shared memory");
};

__global__ void __launch_bounds__(FM_THREADS, 1)
    fp8_mm_wide_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmC, MmParams p) {
  using C = WCfg;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + C::STAGES * C::A_BYTES;
  uint8_t* sEpi = sB + C::STAGES * C::B_BYTES;
  float* sScale = reinterpret_cast<float*>(sEpi + C::EPI_BYTES);
  int4* sTile = reinterpret_cast<int4*>(sScale + C::SLOTS * 256);
  int32_t* ends = reinterpret_cast<int32_t*>(sTile + C::TILES * 2);
  int32_t* unit_end = ends + FM_MAX_E;
  uint64_t* full = reinterpret_cast<uint64_t*>(unit_end + FM_MAX_E);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + C::BUFS;
  uint64_t* done_bar = acc_empty + C::BUFS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done_bar + 1);
  __shared__ int s_ok, s_units;

  // by way of a shuffle the compiler knows it to be one number for the warp: without, the roles spill (24 bytes, read back
  // in their loops)
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const int32_t unit0 = blockIdx.x / 2, ustep = gridDim.x / 2;
  const int32_t num_kb = (p.C + 127) / 128;

  if (threadIdx.x == 0) {
    // the even CTA's full and acc_empty barriers serve the pair
    for (int s = 0; s < C::STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int a = 0; a < C::BUFS; ++a) { mbar_init(&acc_full[a], 2); mbar_init(&acc_empty[a], FM_EPI); }
    mbar_init(done_bar, 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 96 && !p.offs) one_group<256, 256>(p, ends, unit_end, &s_ok, &s_units);
  if (warp == 1) { tmem_alloc_pair(tmem_holder, C::TMEM); tmem_relinquish_pair(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // the peer's barriers exist before any remote arrive or pair copy
  const uint32_t tmem = *tmem_holder;
  if (p.offs) {
    pdl_begin();     // all of the above overlaps the kernel before
    load_ends(p, ends);
    __syncthreads();
    if (warp == 2) read_ends<256, 256>(p, ends, unit_end, &s_ok, &s_units);
    __syncthreads();
  } else {
    pdl_allow_next();   // as above: the warps that load and store wait
  }
  const int32_t n_units = s_units;

  if (warp < 4) {
    regs_give<56>();
    if (warp == 0) {
      // ---------------------------------------------------------- loads
      const bool leader = elect_one();
      if (leader) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
      }
      int stage = 0; uint32_t phase = 0;
      bool ok = true;
      for (int32_t u = unit0; u < n_units && ok; u += ustep) {
        const Unit t = unit_of<256, 256>(p, ends, unit_end, u);
        const int32_t row = (int32_t)t.t0 + rank * 128, f = t.f0 + rank * 64;
        if (!p.offs) pdl_wait();
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!warp_wait(&empty[stage], phase ^ 1, p.err)) { ok = false; break; }
          if (leader) {
            const uint32_t bar = cluster_map(smem_u32(&full[stage]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * C::TX);
            tma_load_2d_pair(sA + stage * C::A_BYTES, &tmA, kb * 128, row, bar);
            // 64 of either block's 128 features: the MMA's N side is both CTAs' rows
            tma_load_3d_pair(sB + stage * C::B_BYTES, &tmB, kb * 128, f, t.e, bar);
            tma_load_3d_pair(sB + stage * C::B_BYTES + 8192, &tmB, kb * 128, f + 128, t.e, bar);
          }
          __syncwarp();
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMAs
      if (rank == 0) {
        const bool leader = elect_one();
        const uint64_t a0 = smem_desc(smem_u32(sA), 16, 1024, 2);
        const uint64_t b0 = smem_desc(smem_u32(sB), 16, 1024, 2);
        int stage = 0; uint32_t phase = 0;
        uint32_t phases = 0;  // bit b: of accumulator b of either feature block
        bool ok = true;
        for (int32_t u = unit0; u < n_units && ok; u += ustep) {
          for (int kb = 0; kb < num_kb; ++kb) {
            const int buf = kb & 1;  // each tile begins with accumulator 0
            if (!warp_wait(&full[stage], phase, p.err)) { ok = false; break; }
            const uint64_t ad = a0 + (uint64_t)((stage * C::A_BYTES) >> 4);
            const uint64_t bd = b0 + (uint64_t)((stage * C::B_BYTES) >> 4);
#pragma unroll
            for (int half = 0; half < 2; ++half) {   // feature blocks
              if (ok) ok = warp_wait(&acc_empty[half * 2 + buf], ~(phases >> buf) & 1, p.err);
              if (!ok) break;
              tc_fence_after();
              if (leader) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_f8_pair(tmem + (uint32_t)((half * 2 + buf) * 128), ad + k * 2, bd + half * 512 + k * 2, C::IDESC, k > 0);
                if (half == 1) tc_commit_pair_mc(&empty[stage], 0x3);
                tc_commit_pair_mc(&acc_full[half * 2 + buf], 0x3);
              }
              __syncwarp();
            }
            phases ^= 1u << buf;
            if (!ok) break;
            if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
          }
        }
        if (leader) tc_commit_pair_mc(done_bar, 0x1);
        __syncwarp();
        mbar_wait(done_bar, 0, p.err);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- scales
      // A warp for either feature block: the scales of the CTA's 128 tokens times the block's, loaded four K blocks ahead.
      // They are part of what an accumulator's acc_full stands for, so the epilogue waits once for both (a barrier of their
      // own cost it 30 us of 340).  A slot is free when the accumulator's last product is done: its MMA waited for the
      // epilogue to be through with the one before, four K blocks ago at most.
      const int half = warp - 2;
      int32_t next_u = unit0, next_kb = 0;
      const float *st = nullptr, *sw = nullptr;
      int live = 0, tile = 0;
      float s[4][4], f[4];
      auto load = [&](int i) {
        if (next_u >= n_units) return;
        if (next_kb == 0) {
          const Unit t = unit_of<256, 256>(p, ends, unit_end, next_u);
          st = p.st + t.t0 + rank * 128 + lane;
          sw = p.sw + t.e * p.sw_e + min((t.f0 >> 7) + half, (p.F - 1) >> 7) * p.sw_f;
          live = t.tn - rank * 128;
          if (lane == 0) sTile[half * C::TILES + tile] = make_int4((int32_t)t.t0 + rank * 128, live, t.f0, 0);
          tile = (tile + 1) & (C::TILES - 1);
          if (!p.offs) pdl_wait();
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) s[i][c] = lane + 32 * c < live ? __ldg(st + 32 * c) : 0.0f;
        f[i] = __ldg(sw);
        st += p.M, sw += p.sw_c;
        if (++next_kb == num_kb) { next_kb = 0; next_u += ustep; }
      };
      float* dst = sScale + half * 128 + lane;
      int32_t u = unit0, kb = 0;
      uint32_t phases = 0;  // bit b: of the block's accumulator b
      bool ok = true;
#pragma unroll
      for (int i = 0; i < 4; ++i) load(i);
      while (u < n_units && ok) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (u >= n_units || !ok) break;
          const int buf = kb & 1;
          ok = warp_wait(&acc_full[half * 2 + buf], ~(phases >> buf) & 1, p.err);
#pragma unroll
          for (int c = 0; c < 4; ++c) dst[i * 256 + 32 * c] = s[i][c] * f[i];
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_full[half * 2 + buf]);
          phases ^= 1u << buf;
          load(i);
          if (++kb == num_kb) { kb = 0; u += ustep; }
        }
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    regs_take<224>();
    // A warp has 32 tokens and one feature block, the other warp of its scheduler the other: their MMAs come one after the
    // other, so one adds while the other waits or loads (both warps on half of either block: 377 us against 364 for 8192 x
    // 4096 x 14336).  Registers are what is short (128 sums, 64 values on their way): barriers by their addresses, and the
    // unit is worked out again for the stores.
    const uint32_t half = (uint32_t)(warp - 4) >> 2;
    if (!p.offs) pdl_wait();
    const uint32_t tb = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 256;
    const uint32_t bars = smem_u32(acc_full) + half * 16;                      // acc_full, acc_empty
    const uint32_t give = cluster_map(bars + C::BUFS * 8, 0);                  // the even CTA's acc_empty
    uint32_t ph0 = 0, ph1 = 0;   // phases of the accumulators
    bool ok = true;
    const uint32_t scales = smem_u32(sScale) + (half * 128 + (warp & 3) * 32 + lane) * 4;
    uint32_t slot = 0;
    uint8_t* const stg0 = sEpi + (warp - 4) * (C::OUTS * 2048);
    uint8_t* stg = stg0;
    int tile = 0;
    for (int32_t u = unit0; u < n_units && ok; u += ustep) {
      f2 acc[4][16];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[j][i] = f2_splat(0.0f);
      // one load from TMEM is always on its way: a block of 32 columns is loaded while the one before it is added, the
      // first of the next K block while the last of this one is
      uint32_t v[2][32];
      ok = warp_wait_at(bars, ph0, p.err);
      tc_fence_after();
      tmem_ld_32cols(tb, v[0]);
      // K block kb, in accumulator BUF
      auto step = [&](auto buf_c, int kb) {
        constexpr int BUF = decltype(buf_c)::value;
        float s;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"(scales + slot * 1024));
        slot = (slot + 1) & (C::SLOTS - 1);
        const bool more = kb + 1 < num_kb;
        bool ready = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j == 3 && more) ready = mbar_try_wait_at(bars + (BUF ^ 1) * 8, BUF ? ph0 : ph1);
          tmem_ld_wait(v[j & 1]);
          if (j < 3) {
            tmem_ld_32cols(tb + BUF * 128 + (j + 1) * 32, v[(j + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(give + BUF * 8);
            if (BUF) ph1 ^= 1; else ph0 ^= 1;
            if (more) {
              if (ok) ok = warp_wait_at(bars + (BUF ^ 1) * 8, BUF ? ph0 : ph1, p.err, ready);
              tc_fence_after();
              tmem_ld_32cols(tb + (BUF ^ 1) * 128, v[0]);
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) fma_here(acc[j][i], v[j & 1][2 * i], v[j & 1][2 * i + 1], s, s);
        }
      };
      for (int kb = 0; kb < num_kb && ok; kb += 2) {
        step(std::integral_constant<int, 0>{}, kb);
        if (kb + 1 < num_kb && ok) step(std::integral_constant<int, 1>{}, kb + 1);
      }
      if (!ok) break;
      // 32 columns at a time through shared memory (chunks of 16 bytes, in the order of TMA's 64-byte swizzle, which meets no
      // bank twice), from where TMA takes blocks of 32 live rows.  An SM writes some 20 bytes a cycle, so a tile takes it
      // 3300 cycles, which the warps need not wait for (32768 rows over 16 of 5120 x 2048: 264 against 274 us with a block a
      // warp on its way and a stage more for the loads).  The tile is known from the scales' warp, which worked it out ahead
      // (here some 1000 cycles that no MMA runs beside).
      const int4 t = sTile[half * C::TILES + tile];   // first row, live rows, first feature
      tile = (tile + 1) & (C::TILES - 1);
      const int32_t r0 = (warp & 3) * 32, f = t.z + (int32_t)half * 128;
      const bool whole = r0 + 32 <= t.y;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (lane == 0) bulk_wait_read<C::OUTS - 1>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) w[m] = f2_to_bf16x2(acc[j][4 * i + m]);
          *reinterpret_cast<uint4*>(stg + lane * 64 + (i ^ ((lane >> 1) & 3)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (whole) fence_async_smem();
        __syncwarp();
        if (whole) {
          if (lane == 0 && f + j * 32 < p.F) tma_store_2d(&tmC, stg, f + j * 32, t.x + r0);
        } else {
          const int32_t c = f + j * 32 + (lane & 3) * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2);
            if (r0 + r < t.y && c < p.F)
              *reinterpret_cast<uint4*>(p.out + ((int64_t)(t.x + r0 + r) * p.F + c) * 2) =
                  *reinterpret_cast<const uint4*>(stg + r * 64 + ((lane & 3) ^ ((r >> 1) & 3)) * 16);
          }
        }
        if (lane == 0) bulk_commit();
        stg = stg == stg0 + (C::OUTS - 1) * 2048 ? stg0 : stg + 2048;
      }
    }
    if (lane == 0) bulk_wait<0>();
    zero_spare_rows(p, s_ok ? ends[p.E - 1] : 0, (warp - 4) * 32 + lane);
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no pair MMA, copy or remote arrive targets an exited CTA
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, C::TMEM);
}


// Clusters of a kernel that can be resident at once (none, if no part of the device holds one), by device; KIND tells the
// kernels apart.  A kernel's register split needs the registers that it was written for.
template <int KIND, class Kernel>
int resident_clusters(Kernel k, size_t smem, int ctas, int* n) {
  static std::atomic<int> resident[64];  // the number + 1, once known; any thread may be the one that asks
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e, "cudaGetDevice");
  int r = resident[dev & 63].load(std::memory_order_relaxed);
  if (r == 0) {
    cudaFuncAttributes a{};
    if ((e = cudaFuncGetAttributes(&a, k)) != cudaSuccess) return cuda_status(e, "cudaFuncGetAttributes");
    if (a.numRegs != FM_REGS)
      return fail(MX_ERR_UNSUPPORTED, "the FP8 product was built with %d registers a thread, not %d", a.numRegs, FM_REGS);
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
      return cuda_status(e, "cudaFuncSetAttribute");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas * (num_sms() / ctas));
    cfg.blockDim = dim3(FM_THREADS);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int m = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&m, k, &cfg)) != cudaSuccess) return cuda_status(e, "cudaOccupancyMaxActiveClusters");
    r = m + 1;
    resident[dev & 63].store(r, std::memory_order_relaxed);
  }
  *n = r - 1;
  return MX_OK;
}

// Tiles of bt token rows, at most: any group that has rows may end in a part of one.
int64_t tile_bound(const MmParams& p, int bt) {
  const int64_t groups = std::min<int64_t>(p.E, p.M), ft = bt == 256 ? 256 : 128;
  return (p.M + groups * (bt - 1)) / bt * ((p.F + ft - 1) / ft);
}

// KIND tells the kernels apart; ctas: of a cluster.  whole: a cluster has one tile at most (S > 1: its buffer for the
// other pairs' sums is written once).  args: the kernel's.
template <int KIND, class... A>
int launch_cfg(void (*k)(A...), size_t smem, int bt, int ctas, bool whole, const MmParams& p, cudaStream_t stream, const A&... args) {
  const int64_t units = tile_bound(p, bt);
  if (units > INT32_MAX / 8) return fail(MX_ERR_UNSUPPORTED, "FP8 product: too many tiles");
  int nres = 0;
  if (int rc = resident_clusters<KIND>(k, smem, ctas, &nres)) return rc;
  if (nres <= 0) return cuda_status(cudaErrorInvalidConfiguration, "cudaOccupancyMaxActiveClusters");
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute");
  const int64_t clusters = std::max<int64_t>(1, whole ? units : std::min<int64_t>(units, nres));
  count_launch(MX_KERNEL_FP8_BLOCK);
  return cuda_status(launch_overlapped(k, (unsigned)(ctas * clusters), FM_THREADS, smem, stream, ctas, args...), "FP8 product launch");
}

// Token rows to a tile (256: tokens on the M side, CTA pairs) and CTAs to a tile's contraction.
//   Few tiles: an SM takes in some 50 bytes a cycle, so a long contraction is shared by the CTAs of a cluster, in one wave (8
// rows of one group, us with one, two and four CTAs: 4096 x 7168 14.5, 9.7, 8.3; 512 x 7168 14.0, 9.0, 6.6; 7168 x 2048 5.9,
// 5.7; 1024 x 1024 4.1, 4.0, 4.2; 128 rows of 4096 x 7168 by 64 16.0, 11.7).
//   Small tiles while they are one wave or the weights' bytes count, large ones where the tensor cores or the rows' bytes do.
// us with 32 / 64 / 256 (128 of the first kind was ahead for groups of 96 rows only, by 3 to 6%): 512 rows of one 1024 x 1024
// 4.7 / 4.7 / 6.4; 1000 of one 1024 x 4096 - / 10.5 / 13.6; 2048 of one 2048 x 2048 - / - / 10.3; 64 over 64 of 4096 x 7168
// 146 / 144 / 166; 1024 over 64 of 2048 x 2048 45.3 / 43.7 / 54.8; 256 over 8 of it 12.2 / 10.7 / 11.5; 800 over 8 19.7 / 13.5 /
// 12.4; 2041 over 16 of 1424 x 1008 18.2 / 13.8 / 13.9, of 1008 x 1424 16.7 / 13.8 / 10.9; 1000 over 16 of 5120 x 8192 162 / 123 /
// 129; 4096 over 16 500 / 288 / 187; 3000 over 64 of 4096 x 2048 111 / 92 / 108; 6000 over 64 183 / 122 / 115.
//   Groups' sizes are on the device only, so the rule takes their mean, over groups without rows too.  The other way round,
// 64 / 256: 4096 rows of which one of 64 experts has 4033, of 4096 x 7168 439 / 378, of 2048 x 2048 74 / 67; shared out evenly
// 305 / 311 of 4096 x 7168.
struct TokenShape {
  int bt, share;
};
int token_shape(const MmParams& p, TokenShape* s) {
  int n2 = 0, n4 = 0, rc;
  if ((rc = resident_clusters<642>(fp8_mm_narrow_kernel<64, 2>, FCfg<64, 2>::SMEM, 2, &n2)) ||
      (rc = resident_clusters<324>(fp8_mm_narrow_kernel<32, 4>, FCfg<32, 4>::SMEM, 4, &n4)))
    return rc;
  const int64_t t32 = tile_bound(p, 32), t64 = tile_bound(p, 64), n1 = num_sms();
  if (p.C >= 2048 && t32 <= n4) *s = TokenShape{32, 4};
  else if (p.C >= 2048 && t32 <= n2) *s = TokenShape{32, 2};
  else if (p.C >= 2048 && t64 <= n2) *s = TokenShape{64, 2};
  else if (t32 <= n1) *s = TokenShape{32, 1};
  else if (t64 <= n1 || p.M <= 64 * (int64_t)p.E) *s = TokenShape{64, 1};
  else *s = TokenShape{256, 1};
  return MX_OK;
}

}  // namespace

int launch_fp8_block_mm(const Fp8MmLaunch& g, cudaStream_t stream) {
  const bool fwd = g.mode == MX_RAGGED_FWD;
  MmParams p{};
  p.M = g.M; p.E = g.offs ? g.E : 1; p.offs = g.offs; p.out = (uint8_t*)g.c; p.err = g.err;
  p.F = (int32_t)(fwd ? g.N : g.K);
  p.C = (int32_t)(fwd ? g.K : g.N);
  const int64_t nb = (g.N + 127) / 128, kb = (g.K + 127) / 128;
  p.st = g.sa; p.sw = g.sw; p.sw_e = nb * kb; p.sw_f = fwd ? kb : 1; p.sw_c = fwd ? 1 : kb;
  TokenShape s{};
  int rc = token_shape(p, &s);
  if (rc) return rc;
  const bool wide = s.bt == 256;
  CUtensorMap w, a;
  uint64_t dw[3] = {(uint64_t)p.C, (uint64_t)p.F, (uint64_t)p.E}, sw[2] = {(uint64_t)p.C, (uint64_t)p.C * p.F};
  uint32_t bw[3] = {128, wide ? 64u : 128u, 1};
  uint64_t da[2] = {(uint64_t)p.C, (uint64_t)p.M}, sa[1] = {(uint64_t)p.C};
  uint32_t ba[2] = {128, wide ? 128u : (uint32_t)s.bt};
  rc = make_tmap(&w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(g.w), dw, sw, bw, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!rc) rc = make_tmap(&a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(g.a), da, sa, ba, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc) return rc;
  if (wide) {
    CUtensorMap c;
    uint64_t dc[2] = {(uint64_t)p.F, (uint64_t)p.M}, sc[1] = {(uint64_t)p.F * 2};
    uint32_t bc[2] = {32, 32};
    rc = make_tmap(&c, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.c, dc, sc, bc, CU_TENSOR_MAP_SWIZZLE_64B);
    if (rc) return rc;
    return launch_cfg<2561>(fp8_mm_wide_kernel, WCfg::SMEM, 256, 2, false, p, stream, a, w, c, p);
  }
#define MX_NARROW(BT, S)                                                                                            \
  if (s.bt == BT && s.share == S)                                                                                   \
    return launch_cfg<BT * 10 + S>(fp8_mm_narrow_kernel<BT, S>, FCfg<BT, S>::SMEM, BT, S, S > 1, p, stream, w, a, p);
  MX_NARROW(32, 1) MX_NARROW(32, 2) MX_NARROW(32, 4) MX_NARROW(64, 1) MX_NARROW(64, 2)
#undef MX_NARROW
  return fail(MX_ERR_UNSUPPORTED, "FP8 product: no kernel for the shape");
}

}  // namespace mx
