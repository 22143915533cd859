// ragged.cu - bf16 matrix products grouped by expert with ragged group sizes.
//
//   FWD    out[t, n] = sum_k x[t, k] w[e, n, k]       t in group e
//   DGRAD  dx[t, k]  = sum_n dout[t, n] w[e, n, k]
//   WGRAD  dw[e, n, k] = sum_{t in e} dout[t, n] x[t, k]
//
// on the tcgen05 tensor cores: bf16 operands, fp32 accumulation in TMEM over
// the whole contraction, one rounding to bf16.  Group ends may be any
// non-decreasing numbers; nothing is padded in memory.
//
// Token groups are ragged, so tokens are the N side of the MMA (any multiple
// of 32 at run time) and weight features the M side (256 per CTA pair): the
// last tile of a group costs what its rows cost, and rows of the next group
// that a tile's load brings along are columns of the accumulator that nobody
// reads.  The accumulator comes out with features along its lanes; the
// epilogue turns 32 x 32 blocks in shared memory and writes token rows.
// In WGRAD both operands contract over tokens and are read where they lie
// (token-major, the "MN-major" operand form), with no transposed copies; the
// last partial step of 16 tokens is overwritten with zeros behind the group's
// end in shared memory first, in both operands, so that nothing the next group
// holds (NaN included) enters the sum.
//
// Where tiles are fewer than pairs, the pairs of a cluster share a tile's
// contraction (S of them); the first pair adds the others' fp32 sums, sent
// through distributed shared memory, in order.
//
// One persistent CTA pair per two SMs, roles as in gemm.cu: warp 0 loads
// (TMA), warp 1 issues MMAs (even CTA), warps 2-9 drain accumulators (two of
// them, so a tile's stores overlap the next tile's MMAs), warp 10 clears
// WGRAD tails.
//
// On a GB300 (bf16 library products at 1.94 PFLOP/s, copies at 6.78 TB/s): 32768
// rows over 16 experts, 5120 x 8192, 1.41 to 1.6 ms each way (up to the full
// rate; longer runs are bound by the power limit, 1.55 to 1.85 PFLOP/s).  64 rows
// over 64 experts, 4096 x 7168, 220 us (6.8 TB/s of weights).  Between the two,
// partial tiles bring 32 KB a step and CTA from L2 for little work, and the last
// wave is not full: 4096 rows over 16 experts, 5120 x 8192, 281 / 272 / 317 us,
// 1.1 to 1.3 PFLOP/s and 4.2 to 4.9 TB/s of weights.
#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace mx {

namespace {

constexpr int RG_FWD = 0, RG_DGRAD = 1, RG_WGRAD = 2;
constexpr int RG_EPI = 8;                 // epilogue warps
constexpr int RG_MAX_E = 1024;
constexpr int RG_F = 256;                 // features per pair tile

// BT: columns of a token tile; S: CTA pairs that share a tile's contraction.
template <int MODE, int BT, int S>
struct RCfg {
  static constexpr bool A_MN = MODE != RG_FWD, B_MN = MODE == RG_WGRAD;
  static constexpr int A_BYTES = 128 * 128;              // 128 features x 64 contraction elements
  static constexpr int B_BYTES = (BT / 2) * 128;         // this CTA's half of the tile
  static constexpr int TX = A_BYTES + B_BYTES;
  static constexpr int EPI_WARP = MODE == RG_WGRAD ? 4096 : 2048;  // a warp's 32 x 64 or 32 x 32 bf16 block
  static constexpr int EPI_BYTES = RG_EPI * EPI_WARP;
  // Group ends and running unit numbers.  WGRAD needs the ends only, and its
  // 64-column blocks leave room for 128: with more experts every role reads them
  // from global memory (620 against 575 us for 64 experts of 8 rows, 4096 x 7168).
  static constexpr int ENDS = MODE == RG_WGRAD ? 128 : RG_MAX_E;
  static constexpr int TABLE = ENDS * (MODE == RG_WGRAD ? 4 : 8);
  static constexpr int PART = BT * 128 * 4;              // one CTA's accumulator
  static constexpr int PARTS = (S - 1) * PART;           // in a tile's first pair: the other pairs'
  static constexpr int TMEM = 2 * BT;                    // two accumulators
  static constexpr int THREADS = 64 + RG_EPI * 32 + (MODE == RG_WGRAD ? 32 : 0);
  static constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | (A_MN ? 1u << 15 : 0u) |
                                    (B_MN ? 1u << 16 : 0u) | ((uint32_t)(RG_F >> 4) << 24);
  static constexpr int STAGES = (226 * 1024 - EPI_BYTES - PARTS - TABLE - 1536) / TX;
  static constexpr size_t SMEM = (size_t)STAGES * TX + EPI_BYTES + PARTS + TABLE + 512 /*barriers*/ + 1024 /*align*/;
  static_assert(BT == 256 ? S == 1 : MODE != RG_WGRAD && (BT == 128 ? S == 1 : BT == 64 || BT == 32), "tile widths");
  static_assert(S == 1 || S == 2 || S == 4, "at most eight CTAs a cluster");
  static_assert(STAGES >= 4, "shared memory");
  static_assert(SMEM + 1024 /*static*/ <= 227 * 1024, "shared memory");
};

struct RaggedParams {
  int64_t M;                // token rows
  int32_t F;                // features on the M side (FWD, WGRAD: N; DGRAD: K)
  int32_t C;                // contraction length (FWD: K; DGRAD: N)
  int32_t T;                // WGRAD: columns of the N side (K)
  int32_t E;
  const int32_t* offs;
  uint8_t* out;             // [M, F] (FWD, DGRAD) or [E, F, T] (WGRAD), bf16
  int32_t* err;
};

// Arrival in the even CTA for an accumulator that is drained: its values are in
// registers (tcgen05.wait::ld), nothing else is handed over, so the arrival
// need not release anything.  With release at cluster scope it waits for the
// acknowledgement of the tile's global stores (1391 against 1169 us, at that
// stage, for the weight gradients of 512 rows over 64 experts, 4096 x 7168).
MX_DEVINL void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// WGRAD: boxes of 1, 2, 4 and 8 rows of 64 elements.
struct ZeroMaps {
  CUtensorMap rows[4];
};

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

struct Unit {
  int32_t e;
  int32_t f0;       // first feature
  int64_t t0;       // first token row (FWD, DGRAD) or N-side column (WGRAD)
  int32_t tn;       // live rows / columns of the tile
  int32_t n_eff;    // tn rounded up to the MMA's multiple of 32
  int32_t num_kb;   // contraction steps of 64
  int64_t k0;       // WGRAD: first token
  int32_t tail;     // WGRAD: tokens of the last step (1 to 64)
};

template <int MODE, int BT>
MX_DEVINL Unit unit_of(const RaggedParams& p, const int32_t* ends, const int32_t* unit_end, int32_t u) {
  Unit r{};
  const int32_t f_tiles = (p.F + RG_F - 1) / RG_F;
  if (MODE == RG_WGRAD) {
    const int32_t t_tiles = (p.T + BT - 1) / BT, per = f_tiles * t_tiles;
    r.e = u / per;
    const int32_t v = u - r.e * per;
    r.f0 = (v % f_tiles) * RG_F;
    r.t0 = (int64_t)(v / f_tiles) * BT;
    r.tn = (int32_t)min((int64_t)BT, p.T - r.t0);
    r.k0 = r.e && ends ? ends[r.e - 1] : 0;
    const int32_t rows = ends ? ends[r.e] - (int32_t)r.k0 : 0;
    r.num_kb = (rows + 63) / 64;
    r.tail = rows - (r.num_kb - 1) * 64;
  } else {
    int lo = 0, hi = p.E - 1;  // first group whose unit_end is > u
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (unit_end[mid] > u) hi = mid; else lo = mid + 1;
    }
    r.e = lo;
    const int32_t v = u - (lo ? unit_end[lo - 1] : 0);
    const int64_t start = lo ? ends[lo - 1] : 0;
    const int32_t rows = ends[lo] - (int32_t)start;
    const int32_t t_tiles = (rows + BT - 1) / BT;
    int32_t t, f;
    if (rows <= p.F) {  // the rows are the smaller operand: re-read them, stream the weights once
      f = v / t_tiles;
      t = v - f * t_tiles;
    } else {
      t = v / f_tiles;
      f = v - t * f_tiles;
    }
    // the group's rows shared out evenly over its tiles, in multiples of 32 (a
    // last tile of a few rows would load as much of the weights as a full one)
    const int32_t share = ((rows + t_tiles - 1) / t_tiles + 31) & ~31;
    r.f0 = f * RG_F;
    r.t0 = start + (int64_t)t * share;
    r.tn = min(share, rows - t * share);
    r.num_kb = (p.C + 63) / 64;
  }
  r.n_eff = (r.tn + 31) & ~31;
  return r;
}

template <int MODE, int BT, int S>
__global__ void __launch_bounds__(RCfg<MODE, BT, S>::THREADS, 1)
    ragged_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ ZeroMaps tmZ, RaggedParams p) {
  using C = RCfg<MODE, BT, S>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + C::STAGES * C::A_BYTES;
  uint8_t* sEpi = sB + C::STAGES * C::B_BYTES;
  uint8_t* sParts = sEpi + C::EPI_BYTES;
  int32_t* s_ends = reinterpret_cast<int32_t*>(sParts + C::PARTS);
  int32_t* unit_end = s_ends + C::ENDS;  // not WGRAD
  const int32_t* ends = s_ends;
  uint64_t* full = reinterpret_cast<uint64_t*>(sParts + C::PARTS + C::TABLE);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* done_bar = acc_empty + 2;
  uint64_t* tail_bar = done_bar + 1;   // WGRAD, by stage: a tail's bytes are here
  uint64_t* parts_bar = tail_bar + C::STAGES;  // S > 1, by epilogue warp: the other pairs' sums are here
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(parts_bar + RG_EPI);
  __shared__ int s_ok, s_units;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int crank = (int)cluster_ctarank();
  const int rank = crank & 1, lead = crank & ~1;   // of the pair; its even CTA
  const int part = crank >> 1;                     // the pair's share of the contraction
  const int32_t unit0 = blockIdx.x / (2 * S), ustep = gridDim.x / (2 * S);
  const int32_t f_tiles = (p.F + RG_F - 1) / RG_F;

  if (threadIdx.x == 0) {
    // the even CTA's full and acc_empty barriers serve the pair
    for (int s = 0; s < C::STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(&acc_full[a], 1); mbar_init(&acc_empty[a], 2 * RG_EPI); }
    for (int s = 0; s < C::STAGES; ++s) mbar_init(&tail_bar[s], 1);
    mbar_init(done_bar, 1);
    for (int w = 0; w < RG_EPI; ++w) mbar_init(&parts_bar[w], S > 1 ? 32 * (S - 1) : 1);
    fence_mbar_init();
  }
  if (warp == 1) { tmem_alloc_pair(tmem_holder, C::TMEM); tmem_relinquish_pair(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // the peer's barriers exist before any remote arrive or pair copy
  const uint32_t tmem = *tmem_holder;
  pdl_begin();     // all of the above overlaps the kernel before
  if (warp == 2) {
    // group ends, checked, and the running number of work units
    int32_t prev = 0, units = 0;
    bool ok = true;
    for (int base = 0; base < p.E; base += 32) {
      const int e = base + lane;
      const int32_t v = e < p.E ? p.offs[e] : 0x7FFFFFFF;
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
      if (in && e < C::ENDS) {
        s_ends[e] = v;
        if (MODE != RG_WGRAD) unit_end[e] = units + n;
      }
      units += __shfl_sync(0xFFFFFFFFu, n, 31);
      prev = __shfl_sync(0xFFFFFFFFu, v, min(31, p.E - 1 - base));
    }
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (lane == 0) {
      s_ok = ok;
      s_units = MODE == RG_WGRAD ? p.E * f_tiles * ((p.T + BT - 1) / BT) : ok ? units : 0;
      if (!ok && blockIdx.x == 0) record_error(p.err, MX_ERR_BAD_OFFSETS);
    }
  }
  __syncthreads();
  const int32_t n_units = s_units;
  if (MODE == RG_WGRAD) ends = !s_ok ? nullptr /* refused: every group empty, zeros */ : p.E <= C::ENDS ? s_ends : p.offs;

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
      const Unit t = unit_of<MODE, BT>(p, ends, unit_end, u);
      const int32_t f = t.f0 + rank * 128;
      const int32_t b0 = (int32_t)(t.t0 + rank * (t.n_eff / 2));
      const int kb0 = t.num_kb * part / S, kb1 = t.num_kb * (part + 1) / S;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait(&empty[stage], phase ^ 1, p.err)) { ok = false; break; }
        if (leader) {
          uint8_t* dA = sA + stage * C::A_BYTES;
          uint8_t* dB = sB + stage * C::B_BYTES;
          const int32_t k = (int32_t)(t.k0 + kb * 64);
          const bool clear = MODE == RG_WGRAD && kb == t.num_kb - 1 && (t.tail & 15);
          uint32_t bar;
          if (clear) {
            // the step's bytes complete on this CTA's own barrier, and the
            // zeros that follow them on the pair's full barrier
            mbar_arrive_expect_tx(&tail_bar[stage], C::TX);
            bar = cluster_map(smem_u32(&tail_bar[stage]), crank);
          } else {
            bar = cluster_map(smem_u32(&full[stage]), lead);
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * C::TX);
          }
          if (MODE == RG_FWD) {
            tma_load_3d_pair(dA, &tmA, k, f, t.e, bar);
            tma_load_2d_pair(dB, &tmB, k, b0, bar);
          } else if (MODE == RG_DGRAD) {
            tma_load_3d_pair(dA, &tmA, f, k, t.e, bar);
            tma_load_3d_pair(dA + 8192, &tmA, f + 64, k, t.e, bar);
            tma_load_2d_pair(dB, &tmB, k, b0, bar);
          } else {
            tma_load_2d_pair(dA, &tmA, f, k, bar);
            tma_load_2d_pair(dA + 8192, &tmA, f + 64, k, bar);
            tma_load_2d_pair(dB, &tmB, b0, k, bar);
            tma_load_2d_pair(dB + 8192, &tmB, b0 + 64, k, bar);
          }
        }
        __syncwarp();
        if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    if (rank == 0) {
      const bool leader = elect_one();
      // K-major: 8-row atoms 1024 bytes apart, 16 elements = 32 bytes along the row.
      // MN-major: 64-element columns 8192 bytes apart, 8-row atoms 1024 apart, 16
      // contraction rows = 2048 bytes.
      const uint64_t a0 = smem_desc(smem_u32(sA), C::A_MN ? 8192 : 16, 1024, 2);
      const uint64_t b0 = smem_desc(smem_u32(sB), C::B_MN ? 8192 : 16, 1024, 2);
      constexpr uint64_t a_step = C::A_MN ? 128 : 2, b_step = C::B_MN ? 128 : 2;
      int stage = 0; uint32_t phase = 0;
      int acc = 0; uint32_t acc_phase = 0;
      bool ok = true;
      for (int32_t u = unit0; u < n_units && ok; u += ustep) {
        const Unit t = unit_of<MODE, BT>(p, ends, unit_end, u);
        if (t.num_kb == 0) continue;
        if (!warp_wait(&acc_empty[acc], acc_phase ^ 1, p.err)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * BT);
        const uint32_t idesc = C::IDESC | ((uint32_t)(t.n_eff >> 3) << 17);
        const int kb0 = t.num_kb * part / S, kb1 = t.num_kb * (part + 1) / S;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!warp_wait(&full[stage], phase, p.err)) { ok = false; break; }
          tc_fence_after();
          const uint64_t ad = a0 + (uint64_t)((stage * C::A_BYTES) >> 4);
          const uint64_t bd = b0 + (uint64_t)((stage * C::B_BYTES) >> 4);
          const int nk = MODE == RG_WGRAD && kb == t.num_kb - 1 ? (t.tail + 15) / 16 : 4;
          if (leader) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < nk) mma_bf16_pair(d, ad + k * a_step, bd + k * b_step, idesc, kb > kb0 || k > 0);
            tc_commit_pair_mc(&empty[stage], (uint16_t)(0x3 << lead));
          }
          __syncwarp();
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        if (leader) tc_commit_pair_mc(&acc_full[acc], (uint16_t)(0x3 << lead));
        __syncwarp();
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if (leader) tc_commit_pair_mc(done_bar, (uint16_t)(0x1 << lead));
      __syncwarp();
      mbar_wait(done_bar, 0, p.err);
    }
    __syncwarp();
  } else if (MODE == RG_WGRAD && warp == 2 + RG_EPI) {
    // ------------------------------------------------------------ tails
    // Zeros over rows tail .. the next multiple of 16 of both operands' 64-column
    // blocks, once the step's own bytes are here: TMA loads of rows past the
    // end of the tensor (8, 4, 2 and 1 of them), which read as zeros and complete on
    // the pair's full barrier.  Stores from a warp took a fence and, in the odd CTA,
    // an arrival with release at cluster scope, which waits for the epilogue's global
    // stores too: 948 against 833 us for 64 experts of 250 rows (4096 x 7168).
    const bool leader = elect_one();
    int stage = 0; uint32_t phases = 0;  // bit s: the parity that tail_bar[s] completes next
    for (int32_t u = unit0; u < n_units; u += ustep) {
      const Unit t = unit_of<MODE, BT>(p, ends, unit_end, u);
      if (t.num_kb == 0) continue;
      stage = (stage + t.num_kb - 1) % C::STAGES;  // the last step's stage
      const int rows = -t.tail & 15;
      if (rows) {
        if (!warp_wait(&tail_bar[stage], (phases >> stage) & 1, p.err)) break;
        phases ^= 1u << stage;
        if (leader) {
          const uint32_t bar = cluster_map(smem_u32(&full[stage]), lead);
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * 4 * rows * 128);
          for (int b = 0; b < 4; ++b) {
            uint8_t* at = (b < 2 ? sA + stage * C::A_BYTES + b * 8192 : sB + stage * C::B_BYTES + (b - 2) * 8192) + t.tail * 128;
            for (int i = 0; i < 4; ++i)
              if (rows >> i & 1) {
                tma_load_2d_pair(at, &tmZ.rows[i], 0, (int32_t)p.M, bar);
                at += 128 << i;
              }
          }
        }
        __syncwarp();
      }
      if (++stage == C::STAGES) stage = 0;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int ew = warp - 2, q = warp & 3, half = ew >> 2;
    uint8_t* stg = sEpi + ew * C::EPI_WARP;
    int acc = 0; uint32_t acc_phase = 0;
    // WGRAD: row n, column col of the tile, of dw[e]
    auto dw_at = [&](const Unit& t, int32_t n, int32_t col) {
      return p.out + (((int64_t)t.e * p.F + n) * p.T + t.t0 + col) * 2;
    };
    constexpr int NC = BT <= 64 ? 1 : BT / 64, STEP = NC == 1 ? 1 : 2;
    // columns of the warp's block j: pairs of neighbours in WGRAD (whole
    // 128-byte lines of a row), every other one else, so that a short tile keeps both
    // warps of a lane quarter busy
    auto col_of = [half](int j) { return MODE == RG_WGRAD ? (j >> 1) * 128 + half * 64 + (j & 1) * 32 : (2 * j + half) * 32; };
    const int qr = MODE == RG_WGRAD ? lane >> 3 : lane >> 2;            // this lane's row and columns in a block's stores
    const int qc = MODE == RG_WGRAD ? (lane & 7) * 8 : (lane & 3) * 8;
    // FWD, DGRAD: a block of 32 tokens from column c of the tile on; a lane has
    // one feature of all of them: turned through shared memory
    auto store_tokens = [&](const Unit& t, int32_t f, int c, const uint32_t (&r)[32]) {
      uint8_t* dst = p.out + ((t.t0 + c + qr) * p.F + f + qc) * 2;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t v = f2_to_bf16x2(f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])));
        *reinterpret_cast<uint16_t*>(stg + (2 * i) * 64 + lane * 2) = (uint16_t)v;
        *reinterpret_cast<uint16_t*>(stg + (2 * i + 1) * 64 + lane * 2) = (uint16_t)(v >> 16);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i * 8 + qr < t.tn && f + qc < p.F)
          *reinterpret_cast<uint4*>(dst + (int64_t)(i * 8) * p.F * 2) =
              *reinterpret_cast<const uint4*>(stg + (i * 8 + qr) * 64 + (lane & 3) * 16);
    };
    for (int32_t u = unit0; u < n_units; u += ustep) {
      const Unit t = unit_of<MODE, BT>(p, ends, unit_end, u);
      const int32_t f = t.f0 + rank * 128 + q * 32;   // this warp's features
      if (t.num_kb == 0) {                            // WGRAD: an empty group's zeros
        for (int c = half; c * 32 < t.tn; c += 2)
          for (int j = 0; j < 4; ++j)
            if (f + j * 8 < p.F && c * 32 + (lane & 3) * 8 < t.tn)
              *reinterpret_cast<uint4*>(dw_at(t, f + j * 8 + (lane >> 2), c * 32 + (lane & 3) * 8)) = make_uint4(0, 0, 0, 0);
        continue;
      }
      if (!warp_wait(&acc_full[acc], acc_phase, p.err)) break;
      tc_fence_after();
      const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BT);
      // two blocks at a time: both loads in flight and one wait, and few enough
      // registers that nothing spills (four at a time spilled 12 to 88 bytes, which
      // L1, nearly all shared memory here, does not hold: 1169 against 683 us for
      // a store-bound weight gradient)
#pragma unroll 1
      for (int j0 = 0; j0 < NC; j0 += STEP) {
        uint32_t r[STEP][32];
#pragma unroll
        for (int j = 0; j < STEP; ++j)
          if (col_of(j0 + j) < t.tn) tmem_ld_32cols(tb + col_of(j0 + j), r[j]);
        tmem_ld_wait();
        if (j0 + STEP == NC) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (rank != 0) mbar_arrive_cluster_relaxed(cluster_map(smem_u32(&acc_empty[acc]), lead));
            else mbar_arrive(&acc_empty[acc]);
          }
        }
        if (f >= p.F) continue;
        if (S > 1 && col_of(0) < t.tn) {
          // the other pairs' sums of this block to the first pair, which adds them in order:
          // 8 vectors of 4 tokens a lane
          const uint32_t at = (uint32_t)(ew * 32 + lane) * 16;
          constexpr int V_STEP = RG_EPI * 512 / (BT == 32 ? 2 : 1);
          if (part) {
            const uint32_t dst = cluster_map(smem_u32(sParts), rank) + (part - 1) * C::PART + at;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + i * V_STEP), "r"(r[0][4 * i]),
                           "r"(r[0][4 * i + 1]), "r"(r[0][4 * i + 2]), "r"(r[0][4 * i + 3])
                           : "memory");
            mbar_arrive_cluster(cluster_map(smem_u32(&parts_bar[ew]), rank));
            continue;
          }
          if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&parts_bar[ew], 0, p.err))) break;
#pragma unroll
          for (int o = 0; o < S - 1; ++o)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 v = *reinterpret_cast<const float4*>(sParts + o * C::PART + at + i * V_STEP);
              r[0][4 * i] = __float_as_uint(__uint_as_float(r[0][4 * i]) + v.x);
              r[0][4 * i + 1] = __float_as_uint(__uint_as_float(r[0][4 * i + 1]) + v.y);
              r[0][4 * i + 2] = __float_as_uint(__uint_as_float(r[0][4 * i + 2]) + v.z);
              r[0][4 * i + 3] = __float_as_uint(__uint_as_float(r[0][4 * i + 3]) + v.w);
            }
        }
        if (MODE == RG_WGRAD) {
          // lane: a row of dw, 64 columns of it; through shared memory (16-byte
          // chunk k of row r at k ^ (r & 7)) so that eight lanes write a row's line
          const int c = col_of(j0);
          if (c >= t.tn) continue;
          uint8_t* dst = dw_at(t, f + qr, c + qc);
          __syncwarp();
#pragma unroll
          for (int j = 0; j < STEP; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t v[4];
#pragma unroll
              for (int l = 0; l < 4; ++l)
                v[l] = f2_to_bf16x2(f2_pack(__uint_as_float(r[j][8 * k + 2 * l]), __uint_as_float(r[j][8 * k + 2 * l + 1])));
              *reinterpret_cast<uint4*>(stg + lane * 128 + (((j * 4 + k) ^ (lane & 7)) * 16)) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int rr = k * 4 + qr;
            if (f + k * 4 < p.F && c + qc < t.tn)  // F is a multiple of 8
              *reinterpret_cast<uint4*>(dst + (int64_t)k * 4 * p.T * 2) =
                  *reinterpret_cast<const uint4*>(stg + rr * 128 + (((lane & 7) ^ (rr & 7)) * 16));
          }
        } else {
#pragma unroll
          for (int j = 0; j < STEP; ++j) {
            const int c = col_of(j0 + j);
            if (c >= t.tn) break;
            store_tokens(t, f, c, r[j]);
          }
        }
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
    if (MODE != RG_WGRAD) {
      // rows past the last group (all rows, if the ends were refused) are zeros
      const int64_t first = s_ok ? ends[p.E - 1] : 0;
      uint4* dst = reinterpret_cast<uint4*>(p.out + first * p.F * 2);
      const int64_t n = (p.M - first) * p.F / 8;
      for (int64_t i = (int64_t)blockIdx.x * (RG_EPI * 32) + ew * 32 + lane; i < n; i += (int64_t)gridDim.x * (RG_EPI * 32))
        dst[i] = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no pair MMA, copy or remote arrive targets an exited CTA
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, C::TMEM);
}

// Clusters that can be resident at once (none, if no part of the device holds one), by device.
template <int MODE, int BT, int S>
int resident_clusters(int* n) {
  using C = RCfg<MODE, BT, S>;
  static std::atomic<int> resident[64];  // the number + 1, once known; any thread may be the one that asks
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e, "cudaGetDevice");
  int r = resident[dev & 63].load(std::memory_order_relaxed);
  if (r == 0) {
    auto k = ragged_kernel<MODE, BT, S>;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * S * (num_sms() / (2 * S)));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int m = 0;
    e = cudaOccupancyMaxActiveClusters(&m, k, &cfg);
    if (e != cudaSuccess) return cuda_status(e, "cudaOccupancyMaxActiveClusters");
    r = m + 1;
    resident[dev & 63].store(r, std::memory_order_relaxed);
  }
  *n = r - 1;
  return MX_OK;
}

template <int MODE, int BT, int S>
int launch_cfg(const CUtensorMap& tA, const CUtensorMap& tB, const ZeroMaps& tZ, const RaggedParams& p, int64_t units,
               cudaStream_t stream) {
  using C = RCfg<MODE, BT, S>;
  auto k = ragged_kernel<MODE, BT, S>;
  int nres = 0;
  if (int rc = resident_clusters<MODE, BT, S>(&nres)) return rc;
  if (nres <= 0) return cuda_status(cudaErrorInvalidConfiguration, "cudaOccupancyMaxActiveClusters");
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute");
  // S > 1: a cluster has one tile at most (its buffer for the other pairs' sums is written once)
  const int64_t clusters = std::max<int64_t>(1, S > 1 ? units : std::min<int64_t>(units, nres));
  count_launch(MX_KERNEL_RAGGED);
  return cuda_status(launch_overlapped(k, (unsigned)(2 * S * clusters), C::THREADS, C::SMEM, stream, 2 * S, tA, tB, tZ, p),
                     "ragged_kernel launch");
}


// Tiles of bt token rows, at most: any group that has rows may end in a part of one.
int64_t tile_bound(const RaggedLaunch& g, const RaggedParams& p, int bt) {
  const int64_t groups = std::min<int64_t>(g.E, g.M);
  return (g.M + groups * (bt - 1)) / bt * ((p.F + RG_F - 1) / RG_F);
}

// Token rows to a tile and pairs to a tile's contraction (FWD, DGRAD).
//   Few tiles: an SM takes in some 110 GB/s, so a long contraction is shared by
// the pairs of a cluster, in one wave of clusters (8 rows of one group, us without,
// with two and with four pairs: 512 x 7168 21.3, 13.3, 9.4; 2048 x 4096 13.9, 9.9,
// 7.9; 1024 x 1024 6.0, 5.8, 5.7; 200 rows of 1024 x 1024 6.2, 6.5 with two; 100 rows
// of 4096 x 4096 15.3, 12.6 with two and tiles of 64 rows).
//   At most 16 rows a group, or in one wave: 32 rows a tile.  The weights' bytes
// count, and a narrow tile leaves shared memory to 11 stages of them.  At most 64 a
// group, or in one wave: 128; else 256.  Forward, us, with 32 / 128 / 256: 30 rows over
// 16 of 1024 x 2048 11 / - / 19; 400 over 43 of 1176 x 1176 23.1 / 24.3 / 28.8; 256 over 8
// of 2048 x 2048 19.4 / 15.4 / 16.0; 343 over 8 of 4744 x 2248 40.8 / 32.7 / 37.4; 4096
// over 64 of 2048 x 2048 108 / 87.5 / 90.8; 800 over 8 of them 27 / 20.7 / 17.6; 500 of one
// 1024 x 1024 6.8 / - / 9.9; 1000 of one 1024 x 4096 25 / 15.4 / 23.1.
struct TokenShape {
  int bt, pairs;
};
template <int MODE>
int token_shape(const RaggedLaunch& g, const RaggedParams& p, TokenShape* s) {
  int n1 = 0, n2 = 0, n4 = 0, rc;
  if ((rc = resident_clusters<MODE, 32, 1>(&n1)) || (rc = resident_clusters<MODE, 64, 2>(&n2)) ||
      (rc = resident_clusters<MODE, 64, 4>(&n4)))
    return rc;
  const int64_t t32 = tile_bound(g, p, 32), t64 = tile_bound(g, p, 64), t128 = tile_bound(g, p, 128);
  if (p.C >= 1024 && t32 <= n4) *s = TokenShape{32, 4};
  else if (p.C >= 1024 && t64 <= n4) *s = TokenShape{64, 4};
  else if (p.C >= 1536 && t32 <= n2) *s = TokenShape{32, 2};
  else if (p.C >= 1536 && t64 <= n2) *s = TokenShape{64, 2};
  else if (g.M <= 16 * (int64_t)g.E || t32 <= n1) *s = TokenShape{32, 1};
  else if (g.M <= 64 * (int64_t)g.E || t128 <= n1) *s = TokenShape{128, 1};
  else *s = TokenShape{256, 1};
  return MX_OK;
}

template <int MODE>
int launch_tokens(const CUtensorMap& tA, const CUtensorMap& tB, const RaggedParams& p, TokenShape s, int64_t units,
                  cudaStream_t stream) {
  const ZeroMaps none{};
  if (s.bt == 32)
    return s.pairs == 1   ? launch_cfg<MODE, 32, 1>(tA, tB, none, p, units, stream)
           : s.pairs == 2 ? launch_cfg<MODE, 32, 2>(tA, tB, none, p, units, stream)
                          : launch_cfg<MODE, 32, 4>(tA, tB, none, p, units, stream);
  if (s.bt == 64)
    return s.pairs == 2 ? launch_cfg<MODE, 64, 2>(tA, tB, none, p, units, stream)
                        : launch_cfg<MODE, 64, 4>(tA, tB, none, p, units, stream);
  if (s.bt == 128)
    return launch_cfg<MODE, 128, 1>(tA, tB, none, p, units, stream);
  return launch_cfg<MODE, 256, 1>(tA, tB, none, p, units, stream);
}

}  // namespace

int launch_ragged(const RaggedLaunch& g, cudaStream_t stream) {
  const int mode = g.mode;
  CUtensorMap tA, tB;
  ZeroMaps tZ{};
  int rc;
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  auto map2 = [&](CUtensorMap* m, const void* base, int64_t cols, uint32_t rows,
                  CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B) {
    uint64_t dims[2] = {(uint64_t)cols, (uint64_t)g.M};
    uint64_t strides[1] = {(uint64_t)cols * 2};
    uint32_t box[2] = {64, rows};
    return make_tmap(m, bf, 2, const_cast<void*>(base), dims, strides, box, swz);
  };
  auto map_w = [&](CUtensorMap* m, uint32_t rows) {
    uint64_t dims[3] = {(uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.E};
    uint64_t strides[2] = {(uint64_t)g.K * 2, (uint64_t)g.K * g.N * 2};
    uint32_t box[3] = {64, rows, 1};
    return make_tmap(m, bf, 3, const_cast<void*>(g.b), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  RaggedParams p{};
  p.M = g.M; p.E = g.E; p.offs = g.offs; p.out = (uint8_t*)g.c; p.err = g.err;
  if (mode != MX_RAGGED_WGRAD) {
    const bool fwd = mode == MX_RAGGED_FWD;
    p.F = (int32_t)(fwd ? g.N : g.K);
    p.C = (int32_t)(fwd ? g.K : g.N);
    TokenShape s;
    if ((rc = fwd ? token_shape<RG_FWD>(g, p, &s) : token_shape<RG_DGRAD>(g, p, &s))) return rc;
    const int64_t units = tile_bound(g, p, s.bt);
    if (units > INT32_MAX - 1024) return fail(MX_ERR_UNSUPPORTED, "ragged product: too many tiles");
    if ((rc = map_w(&tA, fwd ? 128 : 64)) || (rc = map2(&tB, g.a, p.C, s.bt / 2))) return rc;
    return fwd ? launch_tokens<RG_FWD>(tA, tB, p, s, units, stream) : launch_tokens<RG_DGRAD>(tA, tB, p, s, units, stream);
  }
  p.F = (int32_t)g.N; p.T = (int32_t)g.K;
  if ((rc = map2(&tA, g.a, g.N, 64)) || (rc = map2(&tB, g.b, g.K, 64))) return rc;
  for (int i = 0; i < 4; ++i)
    if ((rc = map2(&tZ.rows[i], g.b, g.K, 1u << i, CU_TENSOR_MAP_SWIZZLE_NONE))) return rc;
  const int64_t units = (int64_t)g.E * ((g.N + RG_F - 1) / RG_F) * ((g.K + 255) / 256);
  if (units > INT32_MAX - 1024) return fail(MX_ERR_UNSUPPORTED, "ragged product: too many tiles");
  return launch_cfg<RG_WGRAD, 256, 1>(tA, tB, tZ, p, units, stream);
}

}  // namespace mx
