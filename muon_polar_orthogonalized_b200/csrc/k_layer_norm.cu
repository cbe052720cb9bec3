// k_layer_norm.cu -- layer norm, its backward pass and its weights' gradient.
//
//   forward   mean = sum x / D;  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps)
//             y = (x - mean) * rstd * gain + bias
//   backward  xh = (x - mean) * rstd;  gy = dy * gain
//             dx = rstd * (gy - mean(gy) - xh * mean(gy * xh))
//             dgain (+)= sum over rows of dy * xh;  dbias (+)= sum over rows of dy
//
// All sums are in fp32 and in an order that depends on the shape alone.  The
// floor is HBM: x and y (forward), x, dy and dx (backward), once each.
//
// A row lives in the registers of one warp (up to 1024 columns) or of one
// block, so x is read once and the variance is taken about the mean in a
// second pass over registers (a one-pass sum of squares would cancel for rows
// far from zero).  The backward kernel is persistent: a block walks rows
// b, b + blocks, ... and keeps its columns' dgain and dbias sums on chip, then
// writes one partial row per block; a second kernel adds the partial rows in
// order.  The number of blocks depends on the shape and the SM count only.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "grad_params.cuh"
#include "pdl.cuh"
#include "vec8.cuh"

namespace muon {

// Sum over the threads of a row group (a warp, or the whole block), the same
// bits in every thread.  `red` holds 2 x 32 floats, used alternately so that
// one barrier per sum suffices.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float* red, int& flip) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s[n] += __shfl_xor_sync(0xffffffffu, s[n], o);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* r = red + flip * N * 32;
    flip ^= 1;
    if (lane == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) r[n * 32 + warp] = s[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float t = lane < W ? r[n * 32 + lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      s[n] = t;
    }
  }
}

// A thread's share of a row: ITEMS units of 8 adjacent columns (VEC), or
// ITEMS * 8 single columns; neighbouring threads hold neighbouring units.
template <int TPR, bool VEC>
struct Share {
  // column of element e (0..7) of unit i for thread `t` of the row group
  static __device__ __forceinline__ int col(int t, int i, int e) {
    return VEC ? (i * TPR + t) * 8 + e : (i * 8 + e) * TPR + t;
  }
  template <typename T>
  static __device__ __forceinline__ void load(const T* row, int t, int i, int cols, float (&v)[8]) {
    if constexpr (VEC) {
      if (col(t, i, 0) < cols) {
        load8(row + col(t, i, 0), v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = col(t, i, e) < cols ? to_f32(row[col(t, i, e)]) : 0.f;
    }
  }
  template <typename T>
  static __device__ __forceinline__ void store(T* row, int t, int i, int cols, const float (&v)[8]) {
    if constexpr (VEC) {
      if (col(t, i, 0) < cols) store8(row + col(t, i, 0), v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col(t, i, e) < cols) row[col(t, i, e)] = from_f32<T>(v[e]);
    }
  }
};

// ---------------------------------------------------------------- forward
constexpr int kFwdItems = 4;   // 32 columns per thread
template <typename X, typename Y, int TPR, bool VEC>
__global__ void __launch_bounds__(TPR < 256 ? (TPR == 32 ? 256 : TPR) : TPR)
layer_norm_kernel(const NormParams p) {
  constexpr int ROWS = TPR == 32 ? 8 : 1;   // rows per block
  using S = Share<TPR, VEC>;
  __shared__ float red[64];
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x % TPR;
  const long long row = static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / TPR;
  if (row >= p.rows) return;   // ROWS > 1: whole warps
  int flip = 0;
  const X* x = static_cast<const X*>(p.x) + row * p.x_ld;
  float v[kFwdItems][8];
#pragma unroll
  for (int i = 0; i < kFwdItems; ++i) S::load(x, t, i, p.cols, v[i]);
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < kFwdItems; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] += v[i][e];
  row_sum<TPR>(s, red, flip);
  const float n = static_cast<float>(p.cols);
  const float mean = s[0] / n;   // divided, not scaled: the mean of equal values is that value
  float q[1] = {0.f};
#pragma unroll
  for (int i = 0; i < kFwdItems; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[i][e] = S::col(t, i, e) < p.cols ? v[i][e] - mean : 0.f;
      q[0] = fmaf(v[i][e], v[i][e], q[0]);
    }
  row_sum<TPR>(q, red, flip);
  const float rstd = 1.f / sqrtf(q[0] / n + p.eps);
  if (t == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
  Y* y = static_cast<Y*>(p.y) + row * p.y_ld;
#pragma unroll
  for (int i = 0; i < kFwdItems; ++i) {
    float g[8], b[8] = {};
    S::load(p.gain, t, i, p.cols, g);
    if (p.bias) S::load(p.bias, t, i, p.cols, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = fmaf(v[i][e] * rstd, g[e], b[e]);
    S::store(y, t, i, p.cols, v[i]);
  }
}

// --------------------------------------------------------------- backward
// dgain and dbias sums per thread in shared memory, at slots that only this
// thread touches: [unit element][thread].
constexpr int kBwdItems = 2;   // 16 columns per thread
template <typename X, int TPR, bool VEC>
__global__ void __launch_bounds__(TPR) layer_norm_grad_kernel(const NormParams p) {
  using S = Share<TPR, VEC>;
  __shared__ float red[128];
  extern __shared__ float acc[];
  const int t = threadIdx.x;
  constexpr int E = kBwdItems * 8;
  float* dg = acc;
  float* db = acc + E * TPR;
#pragma unroll
  for (int e = 0; e < E; ++e) dg[e * TPR + t] = db[e * TPR + t] = 0.f;
  int flip = 0;
  pdl_launch_dependents();
  pdl_wait();
  const float inv = 1.f / static_cast<float>(p.cols);
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const X* x = static_cast<const X*>(p.x) + row * p.x_ld;
    const X* dy = static_cast<const X*>(p.dy) + row * p.dy_ld;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float xh[kBwdItems][8], gy[kBwdItems][8];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kBwdItems; ++i) {
      S::load(x, t, i, p.cols, xh[i]);
      S::load(dy, t, i, p.cols, gy[i]);
    }
#pragma unroll
    for (int i = 0; i < kBwdItems; ++i) {
      float g[8];
      S::load(p.gain, t, i, p.cols, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[i][e] = S::col(t, i, e) < p.cols ? (xh[i][e] - mean) * rstd : 0.f;
        float* a = dg + (i * 8 + e) * TPR + t;
        float* b = db + (i * 8 + e) * TPR + t;
        *a = fmaf(gy[i][e], xh[i][e], *a);
        *b += gy[i][e];
        gy[i][e] *= g[e];
        s[0] += gy[i][e];
        s[1] = fmaf(gy[i][e], xh[i][e], s[1]);
      }
    }
    row_sum<TPR>(s, red, flip);
    const float c1 = s[0] * inv, c2 = s[1] * inv;
    X* dx = static_cast<X*>(p.y) + row * p.y_ld;
#pragma unroll
    for (int i = 0; i < kBwdItems; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) gy[i][e] = rstd * (gy[i][e] - c1 - xh[i][e] * c2);
      S::store(dx, t, i, p.cols, gy[i]);
    }
  }
  float* out = p.partial + static_cast<long long>(blockIdx.x) * 2 * p.cols;
#pragma unroll
  for (int i = 0; i < kBwdItems; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = S::col(t, i, e);
      if (c < p.cols) {
        out[c] = dg[(i * 8 + e) * TPR + t];
        out[p.cols + c] = db[(i * 8 + e) * TPR + t];
      }
    }
}

// dgain / dbias (+)= the blocks' partial rows, added in a fixed tree: 16
// threads per column take every 16th row each, then their sums are added.
constexpr int kColThreads = 16;
template <typename G>
__global__ void __launch_bounds__(32 * kColThreads) layer_norm_column_kernel(const NormParams p) {
  __shared__ float part[kColThreads][33];
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = 0;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int which = blockIdx.y;   // 0: dgain, 1: dbias
  G* out = static_cast<G*>(which ? p.dbias : p.dgain);
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < p.cols)
#pragma unroll 4
    for (int b = w; b < p.blocks; b += kColThreads)
      s += p.partial[(static_cast<long long>(b) * 2 + which) * p.cols + c];
  part[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < p.cols) {
    float v = part[0][lane];
#pragma unroll
    for (int k = 1; k < kColThreads; ++k) v += part[k][lane];
    if (p.accumulate) v += to_f32(out[c]);
    out[c] = from_f32<G>(v);
  }
}

// ---------------------------------------------------------------- launchers
template <typename X, typename Y, int TPR, bool VEC>
static cudaError_t forward_launch(const NormParams& p, cudaStream_t s) {
  constexpr int ROWS = TPR == 32 ? 8 : 1;
  return launch_pdl(layer_norm_kernel<X, Y, TPR, VEC>, dim3(static_cast<unsigned>((p.rows + ROWS - 1) / ROWS)),
                    dim3(TPR * ROWS), 0, s, p);
}
template <typename X, typename Y, bool VEC>
static cudaError_t forward_width(const NormParams& p, cudaStream_t s) {
  constexpr int E = kFwdItems * 8;
  if (p.cols <= 32 * E) return forward_launch<X, Y, 32, VEC>(p, s);
  if (p.cols <= 64 * E) return forward_launch<X, Y, 64, VEC>(p, s);
  if (p.cols <= 128 * E) return forward_launch<X, Y, 128, VEC>(p, s);
  if (p.cols <= 256 * E) return forward_launch<X, Y, 256, VEC>(p, s);
  return forward_launch<X, Y, 512, VEC>(p, s);
}
template <typename X, typename Y>
static cudaError_t forward_typed(const NormParams& p, cudaStream_t s) {
  return p.vec ? forward_width<X, Y, true>(p, s) : forward_width<X, Y, false>(p, s);
}
static_assert(512 * kFwdItems * 8 >= kNormMaxCols && 1024 * kBwdItems * 8 >= kNormMaxCols, "row capacity");
cudaError_t launch_layer_norm(const NormParams& p, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (p.x_bf16) return p.y_bf16 ? forward_typed<B, B>(p, s) : forward_typed<B, float>(p, s);
  return p.y_bf16 ? forward_typed<float, B>(p, s) : forward_typed<float, float>(p, s);
}

static int grad_threads(int cols) {
  for (int t = 32; t < 1024; t *= 2)
    if (cols <= t * kBwdItems * 8) return t;
  return 1024;
}
int layer_norm_grad_blocks(long long rows, int cols, int sms) {
  const int per_sm = 1024 / grad_threads(cols);   // blocks an SM holds: 1024 threads
  const long long cap = static_cast<long long>(sms) * (per_sm > 8 ? 8 : per_sm);
  return static_cast<int>(rows < cap ? rows : cap);
}
template <typename X, int TPR, bool VEC>
static cudaError_t backward_launch(const NormParams& p, cudaStream_t s) {
  constexpr int kSmem = 2 * kBwdItems * 8 * TPR * 4;
  const cudaError_t e = cudaFuncSetAttribute(layer_norm_grad_kernel<X, TPR, VEC>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(layer_norm_grad_kernel<X, TPR, VEC>, dim3(p.blocks), dim3(TPR), kSmem, s, p);
}
template <typename X, bool VEC>
static cudaError_t backward_width(const NormParams& p, cudaStream_t s) {
  switch (grad_threads(p.cols)) {
    case 32: return backward_launch<X, 32, VEC>(p, s);
    case 64: return backward_launch<X, 64, VEC>(p, s);
    case 128: return backward_launch<X, 128, VEC>(p, s);
    case 256: return backward_launch<X, 256, VEC>(p, s);
    case 512: return backward_launch<X, 512, VEC>(p, s);
    default: return backward_launch<X, 1024, VEC>(p, s);
  }
}
cudaError_t launch_layer_norm_grad(const NormParams& p, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (p.x_bf16) return p.vec ? backward_width<B, true>(p, s) : backward_width<B, false>(p, s);
  return p.vec ? backward_width<float, true>(p, s) : backward_width<float, false>(p, s);
}
cudaError_t launch_layer_norm_columns(const NormParams& p, cudaStream_t s) {
  const dim3 grid((p.cols + 31) / 32, p.dbias ? 2 : 1);
  if (p.grad_bf16)
    return launch_pdl(layer_norm_column_kernel<__nv_bfloat16>, grid, dim3(32 * kColThreads), 0, s, p);
  return launch_pdl(layer_norm_column_kernel<float>, grid, dim3(32 * kColThreads), 0, s, p);
}

}  // namespace muon
