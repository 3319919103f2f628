// recur.cuh -- the gated linear recurrence: shared device code.
//
// Per channel, with the gate g and the value v of a step,
//   b = (1 - floor) sigmoid(-g),   a = 1 - b,   h <- a h + b v = h + b (v - h).
// A stretch of steps maps the state that enters it to the one that leaves:
//   h -> h + (e - C h),   C = 1 - prod a,   e the state it leaves from h = 0.
// C, not the product, is what is kept: where a channel remembers for thousands of
// steps every b is far below 1, and a rounded a, or a product of them, would lose
// most of b's digits, in the same direction at every step.
#pragma once
#include "common.cuh"
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
// sigmoid(-g): 0 for a gate of +infinity, 1 for -infinity, NaN for NaN.
__device__ __forceinline__ float opening(float g) { return rcp(1.f + ex2(g * kLog2e)); }
// The same, and hold = sigmoid(g), both with full relative precision: where e^g
// has left fp32's range (its product with 0 would be NaN) it is 1.
__device__ __forceinline__ float opening(float g, float& hold) {
  const float e = ex2(g * kLog2e), r = rcp(1.f + e);
  hold = e > 1e30f ? 1.f : e * r;
  return r;
}

// The state that leaves a stretch (c, e) which x enters.
__device__ __forceinline__ float through(float x, float c, float e) { return e + fmaf(-c, x, x); }

__device__ __forceinline__ int64_t valid_of(const int32_t* valid_len, int64_t b, int64_t seqlen) {
  if (!valid_len) return seqlen;
  const int64_t v = valid_len[b];
  return v < 0 ? 0 : v > seqlen ? seqlen : v;
}

}  // namespace recur
}  // namespace ssm
