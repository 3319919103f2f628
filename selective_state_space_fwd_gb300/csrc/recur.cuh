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
#pragma once
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

// 1 / x for x >= 1 (0 past 2^126), within 1 ulp.
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// g <- e^g, within 7 2^-24 of itself whatever g: 2^t with t = g log2(e) rounded, times
// what the rounding, and log2(e)'s own, took.  That is below 2^-16 where e^g is neither
// infinite nor flushed to 0 (below 2^-126); beyond, where it may be infinite or none, it is
// kept small.
template <int V>
__device__ __forceinline__ void exps(float (&g)[V]) {
  constexpr float kFar = 0x1p-13f;
  float down[V], r[V], k[V];
  vscale<V>(down, g, -kLog2e);  // -t
#pragma unroll
  for (int v = 0; v < V; ++v) k[v] = kLog2e;
  vfma<V>(r, g, k, down);
#pragma unroll
  for (int v = 0; v < V; ++v) k[v] = 1.92596299e-8f;  // log2(e) - kLog2e
  vfma<V>(r, g, k, r);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    r[v] = fmaxf(fminf(r[v], kFar), -kFar);
    g[v] = ex2(-down[v]);
  }
  float ln2[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    ln2[v] = 0.693147181f;
    k[v] = 1.f;
  }
  vfma<V>(r, r, ln2, k);
  vmul<V>(g, g, r);
}
__device__ __forceinline__ float expg(float g) {
  float e[1] = {g};
  exps<1>(e);
  return e[0];
}
// The gates of a step: open = sigmoid(-g) (0 for a gate of +infinity, 1 for -infinity, NaN
// for NaN), b = keep open and a = 1 - b, with keep = 1 - floor.  g becomes e^g.
template <int V>
__device__ __forceinline__ void gates(float (&g)[V], const float (&keep)[V], const float (&floor)[V],
                                      float (&open)[V], float (&b)[V], float (&a)[V]) {
  float t[V], far[V];
  exps<V>(g);
#pragma unroll
  for (int v = 0; v < V; ++v) t[v] = 1.f;
  vadd<V>(t, g, t);
#pragma unroll
  for (int v = 0; v < V; ++v) open[v] = rcp(t[v]);
  vmul<V>(b, keep, open);
  vmul<V>(far, g, open);
  vfma<V>(far, keep, far, floor);
#pragma unroll
  for (int v = 0; v < V; ++v) a[v] = b[v] > 0.5f ? far[v] : 1.f - b[v];  // e^g < 1 in the first
}
// sigmoid(g) from e^g and sigmoid(-g), within 18 2^-24 of itself; e^g where it still has a
// reciprocal (its product with a reciprocal of 0 would be NaN at infinity).  NaN is left to
// the reciprocal.
__device__ __forceinline__ float holding(float e, float open) { return fminf(e, 8.5e37f) * open; }

__device__ __forceinline__ int64_t valid_of(const int32_t* valid_len, int64_t b, int64_t seqlen) {
  if (!valid_len) return seqlen;
  const int64_t v = valid_len[b];
  return v < 0 ? 0 : v > seqlen ? seqlen : v;
}

// Rows of a batch with valid lengths go to the CTAs longest first (CTAs start in
// index order, so that the short ones fill the end): the row of rank r among up to
// 32, a lane per row, ties by index.  All lanes of the warp call it.
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
