// vec8.cuh -- groups of 8 consecutive fp32 or bf16 elements in registers, for
// the streaming kernels: one access of 16 bytes (bf16) or 32 (fp32).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sm100.cuh"

namespace muon {

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(v);
  else return v;
}
// Rounds to nearest even, once, where T is bf16.
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
  else return v;
}

// 8 elements as loaded: kept raw until they are used, so that several loads
// can be in flight in few registers.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};

// p 16-byte aligned for bf16, 32-byte for fp32: 8 fp32 are one whole sector per
// lane (two 16-byte accesses would each touch half of every sector).
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* p) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 4) sm100::ld_global_v8(p, r.w[0], r.w[1]);
  else r.w[0] = *reinterpret_cast<const uint4*>(p);
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  } else {
    const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
  }
}
// The same 8 as four pairs, for packed fp32 arithmetic (one instruction per
// pair; per lane the rounding of the single form).
template <typename T>
__device__ __forceinline__ void unpack4x2(const Raw8<T>& r, float2 (&v)[4]) {
  float s[8];
  unpack8(r, s);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = make_float2(s[2 * k], s[2 * k + 1]);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  const Raw8<T> r = load_raw8(p);
  unpack8(r, v);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    const uint4 lo = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    const uint4 hi = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    sm100::st_global_v8(p, lo, hi);
  }
}

}  // namespace muon
