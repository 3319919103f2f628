// recur.cuh -- the gated linear recurrence: shared device code.
//
// Per channel, with the gate g and the value v of a step,
//   b = (1 - floor) sigmoid(-g),   a = 1 - b,   h <- a h + b v.
// b has its digits however small it is.  So has a: from b = 1/2 on it is formed from the
// sigmoid's other side, floor + (1 - floor) sigmoid(g), so that a state that a gate throws
// away (a reset) leaves nothing but a times itself.  (h + b (v - h) rounds v - h, at the size
// of the state that goes: 1e8 before a value of 1 left 0.)
// A stretch of steps maps the state that enters it to the one that leaves,
//   h -> P h + e,   P = prod a,   e the state it leaves from h = 0.
// Beside P, Q = 1 - P is formed as Q <- a Q + b, so that each has its digits where it is
// small, and Q is kept where it is at most 1/2, as -Q in P's place: the state then moves
// by e - Q h.  With a rounded P near 1 a long memory would be off by P's rounding times
// all of the state, stretch after stretch and the same way (a state of 1 under steady
// values of 1 was off by 4e-4 to 2e-3 after 65536 steps); as e and Q are formed alike,
// what is steady stays.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "layers.h"

namespace ssm {
namespace recur {

// One access of a lane: VEC channels of a step, at most 4 bytes, so that a warp
// reads 128 bytes of a row.
template <typename T, int VEC> struct Cell;
template <> struct Cell<float, 1> {
  using Word = float;
  static __device__ __forceinline__ void get(Word w, float (&f)[1]) { f[0] = w; }
  static __device__ __forceinline__ Word put(const float (&f)[1]) { return f[0]; }
};
template <> struct Cell<__nv_bfloat16, 1> {
  using Word = unsigned short;
  static __device__ __forceinline__ void get(Word w, float (&f)[1]) {
    f[0] = __uint_as_float(static_cast<unsigned>(w) << 16);
  }
  static __device__ __forceinline__ Word put(const float (&f)[1]) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
  }
};
template <> struct Cell<__nv_bfloat16, 2> {
  using Word = unsigned;
  static __device__ __forceinline__ void get(Word w, float (&f)[2]) {
    f[0] = __uint_as_float(w << 16);
    f[1] = __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ Word put(const float (&f)[2]) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[0], f[1]);
    return *reinterpret_cast<const Word*>(&v);
  }
};

// 1 / x for x >= 1/2 (0 past 2^126), within 1 ulp.
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// g <- e^g / 2, within 7 2^-24 of itself whatever g: 2^t with t = g log2(e) rounded, times
// half of what the rounding, and log2(e)'s own, took.  That is near 1/2 where e^g is neither
// infinite nor flushed to 0 (below 2^-126), and kept within [0, 1] elsewhere.
template <int V>
__device__ __forceinline__ void half_exps(float (&g)[V], float) {
  float down[V], r[V], k[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    // e^89 is infinite, 1 / (1 + e^g) 0; no infinity less infinity below
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(g[v]) : "f"(g[v]), "f"(89.f));
    k[v] = kLog2e;
  }
  vscale<V>(down, g, -kLog2e);  // -t
  vfma<V>(r, g, k, down);
#pragma unroll
  for (int v = 0; v < V; ++v) k[v] = 1.92596299e-8f;  // log2(e) - kLog2e
  vfma<V>(r, g, k, r);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    r[v] = __saturatef(fmaf(r[v], 0.346573590f, 0.5f));  // ln(2) / 2; NaN becomes 0
    g[v] = ex2(-down[v]);
  }
  vmul<V>(g, g, r);
}
// The same for gates of 8 significant bits, whose product with 16 of log2(e) is exact.
template <int V>
__device__ __forceinline__ void half_exps(float (&g)[V], __nv_bfloat16) {
  float t[V];
  vscale<V>(t, g, 1.44268798828125f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    g[v] = __saturatef(fmaf(g[v], 2.44427e-6f, 0.5f));  // (log2(e) - the above) ln(2) / 2
    t[v] = ex2(t[v]);
  }
  vmul<V>(g, g, t);
}

// A channel's floor: 1 - floor, and half of it.
template <int V> struct Floor {
  float at[V], keep[V], half[V];
  __device__ __forceinline__ void set(int v, float f) {
    at[v] = f;
    keep[v] = 1.f - f;
    half[v] = 0.5f * keep[v];
  }
};

// The gates of a step: open = 2 sigmoid(-g) (0 for a gate of +infinity, 2 for -infinity, NaN
// for NaN), b = (1 - floor) sigmoid(-g) and a = 1 - b.  T: the gate's type; g becomes e^g / 2.
template <typename T, int V>
__device__ __forceinline__ void gates(float (&g)[V], const Floor<V>& floor, float (&open)[V],
                                      float (&b)[V], float (&a)[V]) {
  float t[V], far[V];
  half_exps<V>(g, T());
#pragma unroll
  for (int v = 0; v < V; ++v) t[v] = 0.5f;
  vadd<V>(t, g, t);
#pragma unroll
  for (int v = 0; v < V; ++v) open[v] = rcp(t[v]);
  vmul<V>(b, floor.half, open);
  vmul<V>(far, g, open);
  vfma<V>(far, floor.keep, far, floor.at);
#pragma unroll
  for (int v = 0; v < V; ++v) a[v] = b[v] > 0.5f ? far[v] : 1.f - b[v];  // e^g < 1 in the first
}
// sigmoid(g) from e^g / 2 and 2 sigmoid(-g), within 18 2^-24 of itself; where the latter is 0
// it is 0 too.
__device__ __forceinline__ float holding(float e, float open) { return fminf(e, 4e37f) * open; }

// How P is kept (Q of 0: P is 1), and h through what is kept of a stretch.
__device__ __forceinline__ float kept(float P, float Q) { return Q > 0.f && Q <= 0.5f ? -Q : P; }
// 1 where Q is kept, 0 where P is.
__device__ __forceinline__ float is_rest(float c) {
  float k;
  asm("set.lt.f32.f32 %0, %1, 0f00000000;" : "=f"(k) : "f"(c));
  return k;
}
__device__ __forceinline__ float through(float c, float h, float e) {
  return fmaf(is_rest(c), h, fmaf(c, h, e));
}
// P and Q from what is kept.
__device__ __forceinline__ float product(float c) { return c + is_rest(c); }
__device__ __forceinline__ float remainder(float c) { return (1.f - is_rest(c)) - c; }

__device__ __forceinline__ int64_t valid_of(const int32_t* valid_len, int64_t b, int64_t seqlen) {
  if (!valid_len) return seqlen;
  const int64_t v = valid_len[b];
  return v < 0 ? 0 : v > seqlen ? seqlen : v;
}

// Rows of a batch with valid lengths go to the CTAs longest first (CTAs start in
// index order, so that the short ones fill the end): the row of rank r among up to
// 32, a lane per row, ties by index; larger batches stay in index order.  All lanes of the warp call it.
__device__ __forceinline__ int64_t by_length(const int32_t* valid_len, int64_t batch,
                                             int64_t seqlen, int64_t r) {
  const int lane = threadIdx.x & 31, n = static_cast<int>(batch);
  const int64_t len = lane < n ? valid_of(valid_len, lane, seqlen) : -1;
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const int64_t other = __shfl_sync(0xffffffffu, len, j);
    rank += other > len || (other == len && j < lane);
  }
  return __ffs(__ballot_sync(0xffffffffu, lane < n && rank == r)) - 1;
}

}  // namespace recur
}  // namespace ssm
