// vec.cuh -- VEC consecutive elements of a row, moved in accesses of up to 16
// bytes and widened to fp32 (bf16 widens exactly; stores round to nearest
// even).  The raw form keeps loaded rows in their storage type, so that many
// loads can be in flight per thread for few registers.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace ssm {

template <typename T, int VEC> struct Raw {
  static constexpr int kWords = VEC * static_cast<int>(sizeof(T)) / 4;
  static_assert(kWords * 4 == VEC * static_cast<int>(sizeof(T)), "whole 32-bit words");
  static_assert(kWords <= 2 || kWords % 4 == 0, "accesses of up to 16 bytes");
  uint32_t w[kWords];
};
template <> struct Raw<float, 1> { float w; };
template <> struct Raw<__nv_bfloat16, 1> { __nv_bfloat16 w; };

template <typename T, int VEC>
__device__ __forceinline__ void raw_zero(Raw<T, VEC>& r) {
  if constexpr (VEC == 1) {
    r.w = T(0.f);
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T, VEC>::kWords; ++i) r.w[i] = 0u;
  }
}

// p is aligned to the access: 8 or 16 bytes when VEC > 1.
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> raw_load(const T* p) {
  Raw<T, VEC> r;
  if constexpr (VEC == 1) {
    r.w = __ldg(p);
  } else if constexpr (Raw<T, VEC>::kWords == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T, VEC>::kWords / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
      r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
  }
  return r;
}

// The same for memory that this kernel also writes (a state or a stream
// updated in place), so not through the read-only path.
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> raw_load_rw(const T* p) {
  Raw<T, VEC> r;
  if constexpr (VEC == 1) {
    r.w = *p;
  } else if constexpr (Raw<T, VEC>::kWords == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T, VEC>::kWords / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
  }
  return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void raw_store(T* p, const Raw<T, VEC>& r) {
  if constexpr (VEC == 1) {
    *p = r.w;
  } else if constexpr (Raw<T, VEC>::kWords == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T, VEC>::kWords / 4; ++i)
      reinterpret_cast<uint4*>(p)[i] =
          make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
  }
}

template <int VEC>
__device__ __forceinline__ void widen(const Raw<float, VEC>& r, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = r.w;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = __uint_as_float(r.w[i]);
  }
}
template <int VEC>
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16, VEC>& r, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = __bfloat162float(r.w);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      f[2 * i] = __uint_as_float(r.w[i] << 16);
      f[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
  }
}

template <int VEC>
__device__ __forceinline__ void narrow(const float (&f)[VEC], Raw<float, VEC>& r) {
  if constexpr (VEC == 1) {
    r.w = f[0];
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.w[i] = __float_as_uint(f[i]);
  }
}
template <int VEC>
__device__ __forceinline__ void narrow(const float (&f)[VEC], Raw<__nv_bfloat16, VEC>& r) {
  if constexpr (VEC == 1) {
    r.w = __float2bfloat16_rn(f[0]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      r.w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void load_f(const T* p, float (&f)[VEC]) {
  widen<VEC>(raw_load<T, VEC>(p), f);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_f(T* p, const float (&f)[VEC]) {
  Raw<T, VEC> r;
  narrow<VEC>(f, r);
  raw_store<T, VEC>(p, r);
}

}  // namespace ssm
