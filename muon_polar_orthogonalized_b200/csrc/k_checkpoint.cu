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
// Both are bound by HBM: 16384 x 14336 bf16 there and back in 223 us, 0.97 of the
// copy rate.  The weight gradient from a checkpoint is in k_weight_grad.cu.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "grad_params.cuh"
#include "pdl.cuh"
#include "vec8.cuh"

namespace muon {

// Launch shape: blocks of eight warps, `wx` side by side along a row and 8 / wx
// rows apart.  A lane takes 16 adjacent features at a time (8 lanes share an
// exponent), kCkUnits times, 512 apart; no index is divided.
constexpr int kCkWarps = 8;
constexpr int kCkUnits = 2;
constexpr int kCkCols = 512 * kCkUnits;   // of a warp
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

// 16 features from column c on; zeros past the row.
template <typename T>
struct Feat16 {
  Raw8<T> r[2];
  __device__ __forceinline__ void load(const T* row, int c, int cols) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      r[h] = Raw8<T>{};
      if (c + 8 * h < cols) r[h] = load_raw8(row + c + 8 * h);
    }
  }
  // bits of the largest magnitude as fp32 (magnitudes order like their bits; NaN is the largest)
  __device__ __forceinline__ uint32_t amax() const {
    if constexpr (sizeof(T) == 2) {
      __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w[4] = {r[h].w[0].x, r[h].w[0].y, r[h].w[0].z, r[h].w[0].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a = w[k] & 0x7fff7fffu;
          m = __hmax2_nan(m, *reinterpret_cast<const __nv_bfloat162*>(&a));
        }
      }
      const uint32_t b = *reinterpret_cast<const uint32_t*>(&m);
      return max(b << 16, b & 0xffff0000u);
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[8];
        unpack8(r[h], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
      }
      return m;
    }
  }
  // codes of the values times f, a power of two.  In bf16 the product is exact
  // but where it falls below 2^-126, far under half the smallest code.
  __device__ __forceinline__ uint4 codes(float f) const {
    uint32_t out[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
      if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 ff = __float2bfloat162_rn(f);
        uint4 w = r[h].w[0];
        uint32_t* q = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&q[k]), ff);
          q[k] = *reinterpret_cast<const uint32_t*>(&p);
        }
        Raw8<T> s;
        s.w[0] = w;
        unpack8(s, v);
      } else {
        unpack8(r[h], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= f;
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t a =
            __nv_cvt_float2_to_fp8x2(make_float2(v[4 * q], v[4 * q + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t b =
            __nv_cvt_float2_to_fp8x2(make_float2(v[4 * q + 2], v[4 * q + 3]), __NV_SATFINITE, __NV_E4M3);
        out[2 * h + q] = a | (b << 16);
      }
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
  }
};

// Rows that 16-byte accesses do not fit: a lane takes every 32nd feature of a
// block of 128, so that neighbouring lanes' accesses adjoin.
template <typename T>
__global__ void __launch_bounds__(32 * kCkWarps) checkpoint_pack_odd_kernel(const CkptParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.z + threadIdx.z;
  if (row >= p.rows) return;
  const T* x = static_cast<const T*>(p.x) + row * p.x_ld;
  uint8_t* q = p.q + row * p.q_ld;
  const int c0 = (blockIdx.y * blockDim.y + threadIdx.y) * kCkCols;
  for (int b = c0; b < min(static_cast<int>(p.q_ld), c0 + kCkCols); b += kCkptBlock) {
    float v[4];
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = b + k * 32 + threadIdx.x;
      v[k] = c < p.cols ? to_f32(x[c]) : 0.f;
      amax = max(amax, __float_as_uint(v[k]) & 0x7fffffffu);
    }
    const int e = block_exponent(__reduce_max_sync(0xffffffffu, amax));
    const float f = e == kNanExp ? 0.f : exp2i(127 - e);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = b + k * 32 + threadIdx.x;
      if (c < p.q_ld) q[c] = __nv_cvt_float_to_fp8(v[k] * f, __NV_SATFINITE, __NV_E4M3);
    }
    if (threadIdx.x == 0 && b < p.cols) p.exps[row * p.nblk + b / kCkptBlock] = static_cast<uint8_t>(e);
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kCkWarps) checkpoint_unpack_odd_kernel(const CkptParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.z + threadIdx.z;
  if (row >= p.rows) return;
  T* out = static_cast<T*>(p.out) + row * p.out_ld;
  const uint8_t* q = p.q + row * p.q_ld;
  const int c0 = (blockIdx.y * blockDim.y + threadIdx.y) * kCkCols;
  for (int b = c0; b < min(p.cols, c0 + kCkCols); b += kCkptBlock) {
    const int e = p.exps[row * p.nblk + b / kCkptBlock];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = b + k * 32 + threadIdx.x;
      if (c < p.cols) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(q[c], __NV_E4M3);
        const float f = e == kNanExp ? __uint_as_float(0x7fffffffu) : exp2i(e - 127);
        out[c] = from_f32<T>(__half2float(*reinterpret_cast<const __half*>(&h)) * f);
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kCkWarps) checkpoint_pack_kernel(const CkptParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.z + threadIdx.z;
  if (row >= p.rows) return;
  const int c0 = (blockIdx.y * blockDim.y + threadIdx.y) * kCkCols + threadIdx.x * 16;
  const T* x = static_cast<const T*>(p.x) + row * p.x_ld;
  Feat16<T> v[kCkUnits];
#pragma unroll
  for (int u = 0; u < kCkUnits; ++u) v[u].load(x, c0 + 512 * u, p.cols);
#pragma unroll
  for (int u = 0; u < kCkUnits; ++u) {
    const int c = c0 + 512 * u;
    uint32_t amax = v[u].amax();
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int e = block_exponent(amax);
    if (c < p.q_ld)
      *reinterpret_cast<uint4*>(p.q + row * p.q_ld + c) = v[u].codes(e == kNanExp ? 0.f : exp2i(127 - e));
    if ((threadIdx.x & 7) == 0 && c < p.cols) p.exps[row * p.nblk + c / kCkptBlock] = static_cast<uint8_t>(e);
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kCkWarps) checkpoint_unpack_kernel(const CkptParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.z + threadIdx.z;
  if (row >= p.rows) return;
  const int c0 = (blockIdx.y * blockDim.y + threadIdx.y) * kCkCols + threadIdx.x * 16;
  T* out = static_cast<T*>(p.out) + row * p.out_ld;
  uint4 q[kCkUnits];
  int e[kCkUnits];
#pragma unroll
  for (int u = 0; u < kCkUnits; ++u) {
    const int c = c0 + 512 * u;
    if (c >= p.cols) break;
    q[u] = *reinterpret_cast<const uint4*>(p.q + row * p.q_ld + c);
    e[u] = p.exps[row * p.nblk + c / kCkptBlock];
  }
#pragma unroll
  for (int u = 0; u < kCkUnits; ++u) {
    const int c = c0 + 512 * u;
    if (c >= p.cols) break;
    uint4 r[2];
    restore16(q[u], e[u], r[0], r[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // features 1 and 2 of every four back in place
      Raw8<__nv_bfloat16> b;
      b.w[0] = make_uint4(__byte_perm(r[h].x, r[h].y, 0x5410), __byte_perm(r[h].x, r[h].y, 0x7632),
                          __byte_perm(r[h].z, r[h].w, 0x5410), __byte_perm(r[h].z, r[h].w, 0x7632));
      const int cc = c + 8 * h;
      if (cc >= p.cols) break;
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(out + cc) = b.w[0];
      } else {
        float v[8];
        unpack8(b, v);
        store8(out + cc, v);
      }
    }
  }
}

// ---------------------------------------------------------------- launchers
static void ck_shape(long long rows, long long cols, dim3& grid, dim3& block) {
  const unsigned segs = static_cast<unsigned>((cols + kCkCols - 1) / kCkCols);
  unsigned wx = 1;
  while (wx < kCkWarps && wx < segs) wx *= 2;
  block = dim3(32, wx, kCkWarps / wx);
  while (block.z > 1 && rows * segs < 8 * 148 * block.z) block.z /= 2;   // few rows: spread over the SMs
  grid = dim3(static_cast<unsigned>((rows + block.z - 1) / block.z), (segs + wx - 1) / wx);
}

template <typename T>
static cudaError_t pack_typed(const CkptParams& p, cudaStream_t s) {
  dim3 grid, block;
  ck_shape(p.rows, p.q_ld, grid, block);
  return launch_pdl(p.vec ? checkpoint_pack_kernel<T> : checkpoint_pack_odd_kernel<T>, grid, block, 0, s, p);
}
cudaError_t launch_checkpoint_pack(const CkptParams& p, cudaStream_t s) {
  return p.bf16 ? pack_typed<__nv_bfloat16>(p, s) : pack_typed<float>(p, s);
}
template <typename T>
static cudaError_t unpack_typed(const CkptParams& p, cudaStream_t s) {
  dim3 grid, block;
  ck_shape(p.rows, p.cols, grid, block);
  return launch_pdl(p.vec ? checkpoint_unpack_kernel<T> : checkpoint_unpack_odd_kernel<T>, grid, block, 0, s, p);
}
cudaError_t launch_checkpoint_unpack(const CkptParams& p, cudaStream_t s) {
  return p.bf16 ? unpack_typed<__nv_bfloat16>(p, s) : unpack_typed<float>(p, s);
}

}  // namespace muon
