// conv.cuh -- device code shared by the forms of the short causal convolution
// (kernel_conv.cu, kernel_conv_tma.cu): a thread holds VEC consecutive channels,
// their taps and the last width - 1 rows in registers.
#pragma once
#include "common.cuh"
#include "f32x2.cuh"
#include "layers.h"
#include "vec.cuh"

namespace ssm {

__device__ __forceinline__ int64_t conv_valid(const ConvParams& p, int64_t b) {
  if (p.valid_len == nullptr) return p.seqlen;
  const int64_t v = p.valid_len[b];
  return v < 0 ? 0 : (v > p.seqlen ? p.seqlen : v);
}

// Row `row` of the carried state: the step width - 1 - row before step 0.
template <typename T, int K, int VEC>
__device__ __forceinline__ Raw<T, VEC> state_row(const void* state0, int64_t b, int64_t dim,
                                                 int64_t d0, int row) {
  Raw<T, VEC> r;
  if (state0 == nullptr) {
    raw_zero<T, VEC>(r);
    return r;
  }
  return raw_load<T, VEC>(static_cast<const T*>(state0) + (b * (K - 1) + row) * dim + d0);
}

template <int K, int VEC>
__device__ __forceinline__ void load_taps(const float* weight, const float* bias, int64_t d0,
                                          float (&w)[K][VEC], float (&bv)[VEC]) {
  if constexpr (VEC > 1) {  // VEC * K consecutive floats, 16-byte aligned (the caller's check)
    float t[VEC * K];
    if constexpr (VEC * K % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VEC * K / 4; ++i) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(weight + d0 * K) + i);
        t[4 * i] = v.x; t[4 * i + 1] = v.y; t[4 * i + 2] = v.z; t[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC * K; ++i) t[i] = __ldg(weight + d0 * K + i);
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v)
#pragma unroll
      for (int k = 0; k < K; ++k) w[k][v] = t[v * K + k];
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][0] = __ldg(weight + d0 * K + k);
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) bv[v] = bias ? __ldg(bias + d0 + v) : 0.f;
}

// pre of the row `cur` after the window `win` (oldest row first).
template <int K, int VEC>
__device__ __forceinline__ void taps(const float (&w)[K][VEC], const float (&bv)[VEC],
                                     const float (&win)[K - 1][VEC], const float (&cur)[VEC],
                                     float (&pre)[VEC]) {
  vfma<VEC>(pre, w[0], win[0], bv);
#pragma unroll
  for (int k = 1; k < K - 1; ++k) vfma<VEC>(pre, w[k], win[k], pre);
  vfma<VEC>(pre, w[K - 1], cur, pre);
}

// 1 / v with the MUFU unit (PTX rcp.approx.ftz.f32: within 1 ulp; 0 for
// infinities, which a sigmoid's denominator may be).
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// s = sigmoid(v) = 1 / (1 + e^-v).
template <int VEC>
__device__ __forceinline__ void sigmoid(const float (&v)[VEC], float (&s)[VEC]) {
  float one[VEC];
  vscale<VEC>(s, v, -kLog2e);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    s[i] = ex2(s[i]);
    one[i] = 1.f;
  }
  vadd<VEC>(s, s, one);
#pragma unroll
  for (int i = 0; i < VEC; ++i) s[i] = rcp(s[i]);
}

template <int K, int VEC>
__device__ __forceinline__ void push(float (&win)[K - 1][VEC], const float (&cur)[VEC]) {
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
#pragma unroll
    for (int k = 0; k + 1 < K - 1; ++k) win[k][v] = win[k + 1][v];
    win[K - 2][v] = cur[v];
  }
}

// silu of pre, elementwise.
template <int VEC>
__device__ __forceinline__ void apply_silu(float (&pre)[VEC]) {
  float s[VEC];
  sigmoid<VEC>(pre, s);
  vmul<VEC>(pre, pre, s);
}

// dpre = dy silu'(pre), in place of dy: silu'(v) = s (1 + v (1 - s)), s = sigmoid(v).
template <int VEC>
__device__ __forceinline__ void apply_dsilu(const float (&pre)[VEC], float (&g)[VEC]) {
  float s[VEC], t[VEC], one[VEC];
  sigmoid<VEC>(pre, s);
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    t[v] = 1.f - s[v];
    one[v] = 1.f;
  }
  vfma<VEC>(t, pre, t, one);
  vmul<VEC>(t, t, s);
  vmul<VEC>(g, g, t);
}

// dx of a step: the taps against the window of later dpre (`dp`, oldest first)
// and the newest, g.
template <int K, int VEC>
__device__ __forceinline__ void dx_taps(const float (&w)[K][VEC], const float (&dp)[K - 1][VEC],
                                        const float (&g)[VEC], float (&a)[VEC]) {
  vmul<VEC>(a, w[0], g);
#pragma unroll
  for (int k = 1; k < K; ++k) vfma<VEC>(a, w[k], dp[K - 1 - k], a);
}

// dw += dpre x over the window and the current row.
template <int K, int VEC>
__device__ __forceinline__ void add_dw(float (&dw)[K][VEC], float (&db)[VEC], const float (&g)[VEC],
                                       const float (&win)[K - 1][VEC], const float (&cur)[VEC]) {
  vadd<VEC>(db, db, g);
#pragma unroll
  for (int k = 0; k < K - 1; ++k) vfma<VEC>(dw[k], g, win[k], dw[k]);
  vfma<VEC>(dw[K - 1], g, cur, dw[K - 1]);
}

}  // namespace ssm
