// e4m3.cuh -- checkpoint codes (8-bit floats, 4 exponent and 3 mantissa bits)
// to bf16, in packed integer and bf16 arithmetic.
//
// The code's exponent and mantissa bits, moved to the low end of bf16's
// exponent and the high end of its mantissa, read as the value times 2^-120
// (bf16 subnormals and the code's line up), so one exact multiply by a power of
// two gives the restored value.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace muon {

// Codes in bytes 1 and 3 (bytes 0 and 2) of w as two bf16 times 2^-120.
__device__ __forceinline__ uint32_t codes13(uint32_t w) { return ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u); }
__device__ __forceinline__ uint32_t codes02(uint32_t w) { return ((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u); }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t f) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 16 codes of one exponent -> 16 bf16 in two 16-byte units, features 1 and 2
// of every four exchanged.
__device__ __forceinline__ void restore16(const uint4& q, int e, uint4& lo, uint4& hi) {
  // 2^(120 + e - 127) fits bf16 up to e = 134; beyond, a second factor follows
  const int p = e == 255 ? 0 : min(e - 7, 127);
  uint32_t f = e == 255 ? 0x7fffu : static_cast<uint32_t>(p + 127) << 7;
  f |= f << 16;
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = mul_bf16x2(codes02(w[i]), f);
    r[2 * i + 1] = mul_bf16x2(codes13(w[i]), f);
  }
  if (e > 134 && e != 255) {
    uint32_t g = static_cast<uint32_t>(e - 134 + 127) << 7;
    g |= g << 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = mul_bf16x2(r[i], g);
  }
  lo = make_uint4(r[0], r[1], r[2], r[3]);
  hi = make_uint4(r[4], r[5], r[6], r[7]);
}

}  // namespace muon
