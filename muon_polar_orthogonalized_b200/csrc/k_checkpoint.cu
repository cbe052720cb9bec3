// k_checkpoint.cu -- activation checkpoints in 8 bits.
//
// A checkpoint of x [rows, cols] holds, per row and block of 128 features, one
// exponent byte e and 128 codes in the 8-bit float format with 4 exponent and
// 3 mantissa bits (e4m3, largest value 448): value = code * 2^(e - 127).  e is
// the smallest power of two that brings the block's largest magnitude to at
// most 448, but not below 2^-124.  A power of two costs a floating-point code
// no precision, and makes every value exact in bf16 (4 significant bits; the
// smallest multiple, 2^-9 * 2^-124, is bf16's own smallest), so the tensor
// cores take restored values without a further rounding.  A block that holds
// an infinity or NaN gets e = 255, which stands for NaN throughout.
//
//   pack         x -> codes, exponents     reads x once, writes cols + cols/128 bytes per row
//   unpack       the reverse
// The weight gradient from a checkpoint is in k_weight_grad.cu.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "grad_params.cuh"
#include "pdl.cuh"
#include "vec8.cuh"

namespace muon {

constexpr int kCkThreads = 256;
constexpr int kCkWarps = kCkThreads / 32;
constexpr int kNanExp = 255;

__device__ __forceinline__ float exp2i(int p) {   // 2^p, -126 <= p <= 127
  return __uint_as_float(static_cast<uint32_t>(p + 127) << 23);
}

// Exponent byte of a block whose largest magnitude has these bits:
// 448 = 1.75 * 2^8, so magnitude m * 2^E (1 <= m < 2) needs E - 8 where
// m <= 1.75 and E - 7 beyond.  Subnormal magnitudes need the least exponent.
__device__ __forceinline__ int block_exponent(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return kNanExp;
  if (amax_bits == 0) return 127;
  const int E = static_cast<int>(amax_bits >> 23) - 127;
  const int p = E - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (p < -124 ? -124 : p) + 127;
}

// A warp packs 256 columns of a row: lane l the 8 columns from 8 l, so that
// 16 lanes share a block.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kCkThreads) checkpoint_pack_kernel(const CkptParams p, int nseg) {
  pdl_launch_dependents();
  pdl_wait();
  const long long task = static_cast<long long>(blockIdx.x) * kCkWarps + (threadIdx.x >> 5);
  const long long row = task / nseg;
  if (row >= p.rows) return;
  const int lane = threadIdx.x & 31;
  const int c = static_cast<int>(task - row * nseg) * 256 + lane * 8;
  const T* x = static_cast<const T*>(p.x) + row * p.x_ld;
  float v[8] = {};
  if constexpr (VEC) {
    if (c < p.cols) load8(x + c, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + k < p.cols) v[k] = to_f32(x[c + k]);
  }
  uint32_t amax = 0;   // magnitudes order like their bits; NaN is the largest
#pragma unroll
  for (int k = 0; k < 8; ++k) amax = max(amax, __float_as_uint(v[k]) & 0x7fffffffu);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int e = block_exponent(amax);
  if (c >= p.q_ld) return;
  const float f = e == kNanExp ? 0.f : exp2i(127 - e);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h] * f, v[4 * h + 1] * f), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b =
        __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h + 2] * f, v[4 * h + 3] * f), __NV_SATFINITE, __NV_E4M3);
    w[h] = a | (b << 16);
  }
  *reinterpret_cast<uint2*>(p.q + row * p.q_ld + c) = make_uint2(w[0], w[1]);
  if ((lane & 15) == 0 && c < p.cols) p.exps[row * p.nblk + c / kCkptBlock] = static_cast<uint8_t>(e);
}

// 2 codes -> 2 floats, exact.
__device__ __forceinline__ float2 codes2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// The factor of an exponent byte; 255 gives NaN.
__device__ __forceinline__ float block_factor(int e) {
  return e == kNanExp ? __uint_as_float(0x7fffffffu) : exp2i(e - 127);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kCkThreads) checkpoint_unpack_kernel(const CkptParams p, int nseg) {
  pdl_launch_dependents();
  pdl_wait();
  const long long task = static_cast<long long>(blockIdx.x) * kCkWarps + (threadIdx.x >> 5);
  const long long row = task / nseg;
  if (row >= p.rows) return;
  const int lane = threadIdx.x & 31;
  const int c = static_cast<int>(task - row * nseg) * 256 + lane * 8;
  if (c >= p.cols) return;
  const uint2 q = *reinterpret_cast<const uint2*>(p.q + row * p.q_ld + c);
  const float f = block_factor(p.exps[row * p.nblk + c / kCkptBlock]);
  float v[8];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const float2 u = codes2(((h < 2 ? q.x : q.y) >> ((h & 1) * 16)) & 0xffffu);
    v[2 * h] = u.x * f;
    v[2 * h + 1] = u.y * f;
  }
  T* out = static_cast<T*>(p.out) + row * p.out_ld;
  if constexpr (VEC) {
    store8(out + c, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + k < p.cols) out[c + k] = from_f32<T>(v[k]);
  }
}

// ---------------------------------------------------------------- launchers
static int ck_segments(long long cols) { return static_cast<int>((cols + 255) / 256); }
static dim3 ck_grid(long long tasks) { return dim3(static_cast<unsigned>((tasks + kCkWarps - 1) / kCkWarps)); }

template <typename T, bool VEC>
static cudaError_t pack_typed(const CkptParams& p, cudaStream_t s) {
  const int nseg = ck_segments(p.q_ld);
  return launch_pdl(checkpoint_pack_kernel<T, VEC>, ck_grid(p.rows * nseg), dim3(kCkThreads), 0, s, p, nseg);
}
cudaError_t launch_checkpoint_pack(const CkptParams& p, cudaStream_t s) {
  if (p.bf16) return p.vec ? pack_typed<__nv_bfloat16, true>(p, s) : pack_typed<__nv_bfloat16, false>(p, s);
  return p.vec ? pack_typed<float, true>(p, s) : pack_typed<float, false>(p, s);
}
template <typename T, bool VEC>
static cudaError_t unpack_typed(const CkptParams& p, cudaStream_t s) {
  const int nseg = ck_segments(p.cols);
  return launch_pdl(checkpoint_unpack_kernel<T, VEC>, ck_grid(p.rows * nseg), dim3(kCkThreads), 0, s, p, nseg);
}
cudaError_t launch_checkpoint_unpack(const CkptParams& p, cudaStream_t s) {
  if (p.bf16) return p.vec ? unpack_typed<__nv_bfloat16, true>(p, s) : unpack_typed<__nv_bfloat16, false>(p, s);
  return p.vec ? unpack_typed<float, true>(p, s) : unpack_typed<float, false>(p, s);
}

}  // namespace muon
