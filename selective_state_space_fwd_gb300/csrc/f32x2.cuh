// f32x2.cuh -- elementwise fp32 arithmetic on VEC values, two per instruction
// (the f32x2 forms do the work of two scalar ones in one issue slot, with the
// same rounding).  An odd VEC falls back to scalar instructions.
#pragma once

namespace ssm {

__device__ __forceinline__ void fma_pair(float& d0, float& d1, float a0, float a1, float b0,
                                         float b1, float c0, float c1) {
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul_pair(float& d0, float& d1, float a0, float a1, float b0,
                                         float b1) {
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void add_pair(float& d0, float& d1, float a0, float a1, float b0,
                                         float b1) {
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// d = a b + c, elementwise.
template <int VEC>
__device__ __forceinline__ void vfma(float (&d)[VEC], const float (&a)[VEC], const float (&b)[VEC],
                                     const float (&c)[VEC]) {
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int v = 0; v < VEC; v += 2)
      fma_pair(d[v], d[v + 1], a[v], a[v + 1], b[v], b[v + 1], c[v], c[v + 1]);
  } else {
#pragma unroll
    for (int v = 0; v < VEC; ++v) d[v] = fmaf(a[v], b[v], c[v]);
  }
}
// d = a b.
template <int VEC>
__device__ __forceinline__ void vmul(float (&d)[VEC], const float (&a)[VEC],
                                     const float (&b)[VEC]) {
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int v = 0; v < VEC; v += 2) mul_pair(d[v], d[v + 1], a[v], a[v + 1], b[v], b[v + 1]);
  } else {
#pragma unroll
    for (int v = 0; v < VEC; ++v) d[v] = a[v] * b[v];
  }
}
// d = a + b.
template <int VEC>
__device__ __forceinline__ void vadd(float (&d)[VEC], const float (&a)[VEC],
                                     const float (&b)[VEC]) {
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int v = 0; v < VEC; v += 2) add_pair(d[v], d[v + 1], a[v], a[v + 1], b[v], b[v + 1]);
  } else {
#pragma unroll
    for (int v = 0; v < VEC; ++v) d[v] = a[v] + b[v];
  }
}
// The same with one value for b or c.
template <int VEC>
__device__ __forceinline__ void vscale(float (&d)[VEC], const float (&a)[VEC], float b) {
  float t[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) t[v] = b;
  vmul<VEC>(d, a, t);
}

}  // namespace ssm
