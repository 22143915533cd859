// warp_on_cpu.h - runs a warp of a CUDA kernel's source on the host: 32 fibres, each of which runs until the next exchange
// of the warp.  Indexes that the kernel works out from its data are checked and counted, not followed.
// For kernels whose warps keep to themselves and whose exchanges are of all 32 lanes.
#pragma once
#include <ucontext.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <type_traits>
#include <vector>

#define MX_DEVINL inline
#define __device__
#define __noinline__
#define __global__
#define __constant__ static const
#define __grid_constant__
#define __launch_bounds__(...)

struct float2 { float x, y; };
struct float4 { float x, y, z, w; };
struct uint4 { uint32_t x, y, z, w; };
struct Index { unsigned x, y, z; };
inline Index threadIdx, blockIdx, blockDim;

inline float2 make_float2(float a, float b) { return {a, b}; }
template <class T>
T __ldg(const T* p) { return *p; }
inline uint32_t __float_as_uint(float f) { uint32_t u; std::memcpy(&u, &f, 4); return u; }
inline float __uint_as_float(uint32_t u) { float f; std::memcpy(&f, &u, 4); return f; }
inline float __fadd_rn(float a, float b) { return a + b; }
inline float __fsub_rn(float a, float b) { return a - b; }
inline float __fmul_rn(float a, float b) { return a * b; }
inline float __fmaf_rn(float a, float b, float c) { return fmaf(a, b, c); }
inline float __frcp_rn(float a) { return 1.0f / a; }
inline float __fdiv_rn(float a, float b) { return a / b; }
inline float log_on_cpu(float a) { return logf(a); }
#define __logf log_on_cpu
inline int __popc(uint32_t v) { return __builtin_popcount(v); }
inline int __ffs(uint32_t v) { return __builtin_ffs((int)v); }
inline void pdl_begin() {}

namespace warp {
constexpr int LANES = 32;
inline int lane;                     // the one that runs
inline uint64_t box[2][LANES];       // values given in an exchange; the next one uses the other
inline int kind[2][LANES], next_box[LANES];
inline bool done[LANES];
inline ucontext_t main_context, context[LANES];
inline std::vector<char> stack[LANES];
inline void (*entry)();
inline long faults;
inline char first_fault[128];

inline void fault(const char* what, long at, long n) {
  if (!faults++) std::snprintf(first_fault, sizeof(first_fault), "%s[%ld] of %ld", what, at, n);
}
// The values of all lanes, once each has given one.
inline const uint64_t* exchange(uint64_t v, int k) {
  const int me = lane, b = next_box[me];
  box[b][me] = v;
  kind[b][me] = k;
  next_box[me] ^= 1;
  swapcontext(&context[me], &main_context);
  for (int i = 0; i < LANES; ++i)
    if (kind[b][i] != k) { fault("another exchange", kind[b][i], k); break; }
  return box[b];
}
template <class T>
uint64_t pack(T v) { uint64_t u = 0; std::memcpy(&u, &v, sizeof(T)); return u; }
template <class T>
T unpack(uint64_t u) { T v; std::memcpy(&v, &u, sizeof(T)); return v; }

inline void run_lane() {
  entry();
  done[lane] = true;
  swapcontext(&context[lane], &main_context);
}
inline void run(void (*f)()) {
  entry = f;
  for (int i = 0; i < LANES; ++i) {
    stack[i].resize(1 << 16);
    getcontext(&context[i]);
    context[i].uc_stack.ss_sp = stack[i].data();
    context[i].uc_stack.ss_size = stack[i].size();
    context[i].uc_link = &main_context;
    makecontext(&context[i], run_lane, 0);
    done[i] = false;
    next_box[i] = 0;
  }
  for (int left = LANES, steps = 0; left && steps < 1000000; ++steps) {
    left = 0;
    for (int i = 0; i < LANES; ++i) {
      if (done[i]) continue;
      lane = i;
      threadIdx.x = i;
      swapcontext(&main_context, &context[i]);
      left += !done[i];
    }
  }
  for (int i = 0; i < LANES; ++i)
    if (!done[i]) { fault("lanes without an end", i, 0); break; }
}

// An array of n whose indexes are checked.
template <class T>
struct Checked {
  T* p;
  long n;
  const char* name;
  T& operator[](long i) const {
    static thread_local T nothing;
    if (i >= 0 && i < n) return p[i];
    fault(name, i, n);
    return nothing = T{};
  }
  operator T*() const { return p; }
};
}  // namespace warp

inline void __syncwarp() { warp::exchange(0, 1); }
template <class T>
T __shfl_sync(uint32_t, T v, int l) { return warp::unpack<T>(warp::exchange(warp::pack(v), 2)[l & 31]); }
template <class T>
T __shfl_xor_sync(uint32_t, T v, int o) { const int me = warp::lane; return warp::unpack<T>(warp::exchange(warp::pack(v), 3)[me ^ o]); }
template <class T>
T __shfl_down_sync(uint32_t, T v, int o) {
  const int me = warp::lane;
  const uint64_t* b = warp::exchange(warp::pack(v), 4);
  return me + o > 31 ? v : warp::unpack<T>(b[me + o]);
}
inline uint32_t __ballot_sync(uint32_t, bool p) {
  const uint64_t* b = warp::exchange(p, 5);
  uint32_t r = 0;
  for (int i = 0; i < 32; ++i) r |= (uint32_t)(b[i] != 0) << i;
  return r;
}
inline bool __any_sync(uint32_t m, bool p) { return __ballot_sync(m, p) != 0; }
inline bool __all_sync(uint32_t m, bool p) { return __ballot_sync(m, p) == ~0u; }
inline uint32_t __reduce_max_sync(uint32_t, uint32_t v) {
  const uint64_t* b = warp::exchange(v, 6);
  uint32_t r = 0;
  for (int i = 0; i < 32; ++i) r = std::max(r, (uint32_t)b[i]);
  return r;
}
inline uint32_t __reduce_or_sync(uint32_t, uint32_t v) {
  const uint64_t* b = warp::exchange(v, 7);
  uint32_t r = 0;
  for (int i = 0; i < 32; ++i) r |= (uint32_t)b[i];
  return r;
}
