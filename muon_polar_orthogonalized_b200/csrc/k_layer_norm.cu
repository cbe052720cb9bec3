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
// A group of threads shares a row, 8 or 16 columns per thread, and the variance
// is taken about the mean in a second pass over the row (a one-pass sum of
// squares would cancel for rows far from zero).  Blocks are persistent, and
// every thread copies its columns of the rows ahead into a ring of its own in
// shared memory (cp.async): the next rows are in flight at no cost in registers
// and with no barrier, since no thread reads another's copy, and each pass over
// a row reads it from there again.  What bounds it then is the chain of a row's
// two sums (exchange, barrier, exchange: about 1.2 us a row for the few groups
// an SM holds), so a group takes R rows at a time and sums all of them in one
// exchange.  Measured: 32768 x 4096 bf16 forward in 104 us (0.79 of the copy
// rate) and backward in 153 us (0.81), where 70% and 62% of the cycles issue an
// instruction; 8192 x 4096 fp32 in 48 us (0.85) and 68 us (0.91).  Gain and bias stay in registers (read from L1 for every row, they
// kept it 82% busy).  Backward, a thread keeps its columns' dgain and dbias sums
// in registers; the block's groups are added in order into one partial row per
// block, and a second kernel adds the partial rows in order.  Rows that 16-byte
// accesses do not fit (odd widths) are loaded element by element, without the
// ring.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "grad_params.cuh"
#include "pdl.cuh"
#include "vec8.cuh"

namespace muon {

constexpr int kNormThreads = 256;   // of a block that holds several groups

// Where a row's columns live: blockDim.x threads (a multiple of 32) per group,
// blockDim.y groups.  Unit i of thread t is 8 columns: adjacent ones (bf16 rows),
// two runs of 4 (fp32 rows, so that neighbouring threads' 16-byte accesses adjoin
// there too: with 8 adjacent ones every sector is fetched twice), or, without
// VEC, 8 that lie blockDim.x apart.
template <bool VEC, bool SPLIT>
struct Cols {
  static __device__ __forceinline__ int at(int i, int e) {
    const int t = threadIdx.x, n = blockDim.x;
    if (!VEC) return (i * 8 + e) * n + t;
    return SPLIT ? ((2 * i + e / 4) * n + t) * 4 + e % 4 : (i * n + t) * 8 + e;
  }
  // whether a unit holds any of the row's columns
  static __device__ __forceinline__ bool inside(int i, int cols) { return at(i, 0) < cols; }
  // units that are inside only; columns past the row load as zeros
  template <typename T>
  static __device__ __forceinline__ void load(const T* row, int i, int cols, float2 (&v)[4]) {
    if constexpr (VEC && !SPLIT) {
      unpack4x2(load_raw8(row + at(i, 0)), v);
    } else if constexpr (VEC) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const T* q = row + at(i, 4 * h);
        const bool in = at(i, 4 * h) < cols;
        if constexpr (sizeof(T) == 4) {
          const float4 f = in ? *reinterpret_cast<const float4*>(q) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[2 * h] = make_float2(f.x, f.y);
          v[2 * h + 1] = make_float2(f.z, f.w);
        } else {
          const uint2 w = in ? *reinterpret_cast<const uint2*>(q) : make_uint2(0, 0);
          v[2 * h] = make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
          v[2 * h + 1] = make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
        }
      }
    } else {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = at(i, e) < cols ? to_f32(row[at(i, e)]) : 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = make_float2(f[2 * k], f[2 * k + 1]);
    }
  }
  template <typename T>
  static __device__ __forceinline__ void store(T* row, int i, int cols, const float2 (&v)[4]) {
    const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
    if constexpr (VEC && !SPLIT) {
      store8(row + at(i, 0), f);
    } else if constexpr (VEC) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        T* q = row + at(i, 4 * h);
        if (at(i, 4 * h) >= cols) continue;
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<float4*>(q) = make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
        } else {
          const __nv_bfloat162 a = __floats2bfloat162_rn(f[4 * h], f[4 * h + 1]);
          const __nv_bfloat162 b = __floats2bfloat162_rn(f[4 * h + 2], f[4 * h + 3]);
          *reinterpret_cast<uint2*>(q) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at(i, e) < cols) row[at(i, e)] = from_f32<T>(f[e]);
    }
  }
  // zeros in an inside unit's columns past the row
  static __device__ __forceinline__ void trim(int i, int cols, float2 (&v)[4]) {
    if constexpr (VEC && SPLIT) {
      if (at(i, 4) >= cols) v[2] = v[3] = make_float2(0.f, 0.f);
    } else if constexpr (!VEC) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (at(i, 2 * k) >= cols) v[k].x = 0.f;
        if (at(i, 2 * k + 1) >= cols) v[k].y = 0.f;
      }
    }
  }
};

// A thread's ring of K stages in shared memory: PER 16-byte pieces per stage, each
// at its own slot of the block's threads (neighbouring threads, neighbouring
// slots).
template <int K, int PER>
struct Ring {
  uint4* slots;
  int threads, tid;
  __device__ __forceinline__ explicit Ring(void* smem)
      : slots(static_cast<uint4*>(smem)), threads(blockDim.x * blockDim.y), tid(threadIdx.y * blockDim.x + threadIdx.x) {}
  __device__ __forceinline__ uint4* slot(int stage, int piece) const {
    return slots + (stage * PER + piece) * threads + tid;
  }
  // zeros in the slots past the row, which `copy` never fills (and only those:
  // nothing orders a plain store before a later asynchronous copy's).  Split
  // units alone are read where a half of them is past the row.  OPS operands of
  // UNITS units, sizeof(T) / 2 pieces each.
  template <typename C, typename T, int UNITS, int OPS>
  __device__ __forceinline__ void clear(int cols) const {
    constexpr int H = static_cast<int>(sizeof(T) / 2);
#pragma unroll
    for (int k = 0; k < K * PER; ++k)
      if (C::at(k / (OPS * H) % UNITS, k % H * 8 / H) >= cols) slots[k * threads + tid] = make_uint4(0, 0, 0, 0);
  }
  // unit i of a row, in sizeof(T) / 2 pieces from `piece` on
  template <typename C, typename T>
  __device__ __forceinline__ void copy(int stage, int piece, const T* row, int i, int cols) const {
    constexpr int H = static_cast<int>(sizeof(T) / 2);
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int c = C::at(i, h * 8 / H);
      const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(slot(stage, piece + h)));
      if (c < cols) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(row + c) : "memory");
    }
  }
  template <typename T>
  __device__ __forceinline__ void get(int stage, int piece, float2 (&v)[4]) const {
    Raw8<T> r;
#pragma unroll
    for (int h = 0; h < static_cast<int>(sizeof(T) / 2); ++h) r.w[h] = *slot(stage, piece + h);
    unpack4x2(r, v);
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // the oldest of the K stages in flight has arrived
  static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(K - 1) : "memory"); }
};

__device__ __forceinline__ void group_barrier() {
  asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(blockDim.x) : "memory");
}

// Sums of N values (a power of two) over a group's threads, the same bits in
// every thread.  Within a warp the values are halved among the lanes first
// (lane bit 4 keeps the upper half, and so on), so that N values cost N - 1 +
// 5 - log2 N exchanges, not 5 N.  `red` holds 2 x N x 32 floats, used
// alternately, so that one barrier per sum suffices.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red, int& flip) {
  const int lane = threadIdx.x & 31;
  int live = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (live > 1) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i >= live / 2) break;
        const float keep = up ? v[i + live / 2] : v[i];
        const float send = up ? v[i] : v[i + live / 2];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
      live /= 2;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
  // lane l now has the warp's sum of value l / SPAN
  constexpr int SPAN = 32 / N;
  float s = v[0];
  const int warps = blockDim.x >> 5;
  if (warps > 1) {
    const int first = threadIdx.y * warps;
    float* r = red + flip * N * 32;
    flip ^= 1;
    if (lane % SPAN == 0) r[(lane / SPAN) * 32 + first + (threadIdx.x >> 5)] = s;
    group_barrier();
    s = 0.f;
    for (int w = lane % SPAN; w < warps; w += SPAN) s += r[(lane / SPAN) * 32 + first + w];
#pragma unroll
    for (int o = SPAN / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, s, i * SPAN);
}

// ---------------------------------------------------------------- forward
// R: rows a group takes at a time; K: stages of R rows in the ring; HOLD: gain
// and bias stay in registers.
template <typename X, typename Y, bool VEC, int UNITS, int MAXT, int MINB, int R, int K, bool HOLD>
__global__ void __launch_bounds__(MAXT, MINB) layer_norm_kernel(const NormParams p) {
  using C = Cols<VEC, sizeof(X) == 4>;
  constexpr int UP = static_cast<int>(sizeof(X)) / 2;   // 16-byte pieces per unit
  extern __shared__ uint4 ring_smem[];
  __shared__ float red[2 * R * 32];
  const Ring<K, R * UNITS * UP> ring(ring_smem);
  int flip = 0;
  pdl_launch_dependents();
  if constexpr (VEC && sizeof(X) == 4) ring.template clear<C, X, UNITS, 1>(p.cols);
  pdl_wait();
  const float n = static_cast<float>(p.cols);
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y * R;
  long long row0 = (static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y) * R;
  auto fetch = [&](long long first, int stage) {
    if constexpr (VEC) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (first + r >= p.rows) break;
        const X* x = static_cast<const X*>(p.x) + (first + r) * p.x_ld;
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
          ring.template copy<C>(stage, (r * UNITS + i) * UP, x, i, p.cols);
      }
    }
    ring.commit();
  };
#pragma unroll
  for (int k = 0; k < K - 1; ++k) fetch(row0 + k * step, k);
  float2 g[UNITS][4], b[UNITS][4] = {};
  auto weights = [&](int i) {
    if (!C::inside(i, p.cols)) return;
    C::load(p.gain, i, p.cols, g[i]);
    if (p.bias) C::load(p.bias, i, p.cols, b[i]);
  };
  if (HOLD) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) weights(i);
  }
  int stage = 0;
  for (; row0 < p.rows; row0 += step) {
    fetch(row0 + (K - 1) * step, stage == 0 ? K - 1 : stage - 1);
    ring.wait();
    const int live = static_cast<int>(min(static_cast<long long>(R), p.rows - row0));
    // without the ring, a short row stays in registers (R is 1)
    constexpr bool KEEP = !VEC && R == 1;
    float2 held[KEEP ? UNITS : 1][4];
    if constexpr (KEEP)
#pragma unroll
      for (int i = 0; i < UNITS; ++i) C::load(static_cast<const X*>(p.x) + row0 * p.x_ld, i, p.cols, held[i]);
    auto unit = [&](int r, int i, float2 (&v)[4]) {
      if constexpr (VEC) {
        ring.template get<X>(stage, (r * UNITS + i) * UP, v);
      } else if constexpr (!KEEP) {
        C::load(static_cast<const X*>(p.x) + (row0 + r) * p.x_ld, i, p.cols, v);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = held[i][k];
      }
    };
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 s = both(0.f);
      if (r < live)
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
          if (C::inside(i, p.cols)) {
            float2 v[4];
            unit(r, i, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) s = __fadd2_rn(s, v[k]);
          }
      mean[r] = s.x + s.y;
    }
    group_sum<R>(mean, red, flip);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] /= n;   // divided, not scaled: the mean of equal values is that value
      float2 s = both(0.f);
      if (r < live)
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
          if (C::inside(i, p.cols)) {
            float2 v[4];
            unit(r, i, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __fadd2_rn(v[k], both(-mean[r]));
            C::trim(i, p.cols, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) s = __ffma2_rn(v[k], v[k], s);
          }
      rstd[r] = s.x + s.y;
    }
    group_sum<R>(rstd, red, flip);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= live) break;
      rstd[r] = 1.f / sqrtf(rstd[r] / n + p.eps);
      if (threadIdx.x == 0) {
        p.mean[row0 + r] = mean[r];
        p.rstd[row0 + r] = rstd[r];
      }
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      if (!C::inside(i, p.cols)) continue;
      if (!HOLD) weights(i);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= live) break;
        float2 v[4];
        unit(r, i, v);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[k] = __ffma2_rn(__fmul2_rn(__fadd2_rn(v[k], both(-mean[r])), both(rstd[r])), g[i][k], b[i][k]);
        C::store(static_cast<Y*>(p.y) + (row0 + r) * p.y_ld, i, p.cols, v);
      }
    }
    if (++stage == K) stage = 0;
  }
}

// --------------------------------------------------------------- backward
template <typename X, bool VEC, int UNITS, int MAXT, int MINB, int R, int K, bool HOLD>
__global__ void __launch_bounds__(MAXT, MINB) layer_norm_grad_kernel(const NormParams p) {
  using C = Cols<VEC, sizeof(X) == 4>;
  constexpr int UP = static_cast<int>(sizeof(X)) / 2;
  extern __shared__ uint4 ring_smem[];
  __shared__ float red[2 * 2 * R * 32];
  const Ring<K, 2 * R * UNITS * UP> ring(ring_smem);   // per row and unit: x, then dy
  int flip = 0;
  float2 dg[UNITS][4] = {}, db[UNITS][4] = {}, g[UNITS][4] = {};
  pdl_launch_dependents();
  if constexpr (VEC && sizeof(X) == 4) ring.template clear<C, X, UNITS, 2>(p.cols);
  pdl_wait();
  const float n = static_cast<float>(p.cols);
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y * R;
  long long row0 = (static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y) * R;
  auto fetch = [&](long long first, int stage) {
    if constexpr (VEC) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (first + r >= p.rows) break;
        const X* x = static_cast<const X*>(p.x) + (first + r) * p.x_ld;
        const X* dy = static_cast<const X*>(p.dy) + (first + r) * p.dy_ld;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
          ring.template copy<C>(stage, (r * UNITS + i) * 2 * UP, x, i, p.cols);
          ring.template copy<C>(stage, (r * UNITS + i) * 2 * UP + UP, dy, i, p.cols);
        }
      }
    }
    ring.commit();
  };
  float mean_next[R], rstd_next[R];
  auto stats = [&](long long first) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean_next[r] = first + r < p.rows ? p.mean[first + r] : 0.f;
      rstd_next[r] = first + r < p.rows ? p.rstd[first + r] : 0.f;
    }
  };
#pragma unroll
  for (int k = 0; k < K - 1; ++k) fetch(row0 + k * step, k);
  stats(row0);
  if (HOLD) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
      if (C::inside(i, p.cols)) C::load(p.gain, i, p.cols, g[i]);
  }
  int stage = 0;
  for (; row0 < p.rows; row0 += step) {
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = mean_next[r];
      rstd[r] = rstd_next[r];
    }
    fetch(row0 + (K - 1) * step, stage == 0 ? K - 1 : stage - 1);
    stats(row0 + step);
    ring.wait();
    const int live = static_cast<int>(min(static_cast<long long>(R), p.rows - row0));
    // without the ring, a short row stays in registers (R is 1)
    constexpr bool KEEP = !VEC && UNITS == 1;
    float2 held[KEEP ? UNITS : 1][2][4];
    if constexpr (KEEP)
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        C::load(static_cast<const X*>(p.x) + row0 * p.x_ld, i, p.cols, held[i][0]);
        C::load(static_cast<const X*>(p.dy) + row0 * p.dy_ld, i, p.cols, held[i][1]);
      }
    // xh and dy of a unit that is inside, zeros past the row
    auto unit = [&](int r, int i, float2 (&xh)[4], float2 (&dy)[4]) {
      if constexpr (VEC) {
        ring.template get<X>(stage, (r * UNITS + i) * 2 * UP, xh);
        ring.template get<X>(stage, (r * UNITS + i) * 2 * UP + UP, dy);
      } else if constexpr (KEEP) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          xh[k] = held[i][0][k];
          dy[k] = held[i][1][k];
        }
      } else {
        C::load(static_cast<const X*>(p.x) + (row0 + r) * p.x_ld, i, p.cols, xh);
        C::load(static_cast<const X*>(p.dy) + (row0 + r) * p.dy_ld, i, p.cols, dy);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) xh[k] = __fmul2_rn(__fadd2_rn(xh[k], both(-mean[r])), both(rstd[r]));
      C::trim(i, p.cols, xh);
    };
    float s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 s1 = both(0.f), s2 = both(0.f);
      if (r < live)
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
          if (C::inside(i, p.cols)) {
            float2 xh[4], dy[4];
            unit(r, i, xh, dy);
            if (!HOLD) C::load(p.gain, i, p.cols, g[i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              dg[i][k] = __ffma2_rn(dy[k], xh[k], dg[i][k]);
              db[i][k] = __fadd2_rn(db[i][k], dy[k]);
              const float2 gy = __fmul2_rn(dy[k], g[i][k]);
              s1 = __fadd2_rn(s1, gy);
              s2 = __ffma2_rn(gy, xh[k], s2);
            }
          }
      s[2 * r] = s1.x + s1.y;
      s[2 * r + 1] = s2.x + s2.y;
    }
    group_sum<2 * R>(s, red, flip);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= live) break;
      const float2 c1 = both(-s[2 * r] / n), c2 = both(-s[2 * r + 1] / n);
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        if (!C::inside(i, p.cols)) continue;
        float2 xh[4], dy[4];
        unit(r, i, xh, dy);
        if (!HOLD) C::load(p.gain, i, p.cols, g[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          dy[k] = __fmul2_rn(__ffma2_rn(xh[k], c2, __ffma2_rn(dy[k], g[i][k], c1)), both(rstd[r]));
        C::store(static_cast<X*>(p.y) + (row0 + r) * p.y_ld, i, p.cols, dy);
      }
    }
    if (++stage == K) stage = 0;
  }
  if (blockDim.y > 1) __syncthreads();   // the ring is done with
  float* fold = reinterpret_cast<float*>(ring_smem);
  // the groups' sums, in order
  for (int k = 0; k < static_cast<int>(blockDim.y); ++k) {
    if (static_cast<int>(threadIdx.y) == k) {
      float* out = p.partial + static_cast<long long>(blockIdx.x) * 2 * p.cols;
      const bool last = k == static_cast<int>(blockDim.y) - 1;
#pragma unroll
      for (int i = 0; i < UNITS; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = C::at(i, e);
          if (c >= p.cols) continue;
          float vg = e & 1 ? dg[i][e >> 1].y : dg[i][e >> 1].x, vb = e & 1 ? db[i][e >> 1].y : db[i][e >> 1].x;
          if (k > 0) {
            vg += fold[c];
            vb += fold[p.cols + c];
          }
          (last ? out : fold)[c] = vg;
          (last ? out : fold)[p.cols + c] = vb;
        }
    }
    if (blockDim.y > 1) __syncthreads();
  }
}

// dgain / dbias (+)= the blocks' partial rows, added in a fixed tree: 32
// threads per column take every 32nd row each, then their sums are added.
constexpr int kColThreads = 32;
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
#pragma unroll 8
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
namespace {
int round32(int x) { return (x + 31) / 32 * 32; }
// Threads and groups (eight at most) of a block for rows of `cols` columns.
dim3 norm_block(int units_per_thread, int cols) {
  const int units = (cols + 7) / 8;
  const int t = round32((units + units_per_thread - 1) / units_per_thread);
  return dim3(t, t >= kNormThreads ? 1 : kNormThreads / t);
}
}  // namespace

template <typename X, typename Y, bool VEC, int UNITS, int MAXT, int MINB, int R, int K, bool HOLD>
static cudaError_t forward_launch(const NormParams& p, cudaStream_t s) {
  dim3 block = norm_block(UNITS, p.cols);
  // a block of several groups only where there are rows for every SM
  while (block.y > 1 && static_cast<long long>(block.y) * R * p.sms > p.rows) block.y = (block.y + 1) / 2;
  const auto kern = layer_norm_kernel<X, Y, VEC, UNITS, MAXT, MINB, R, K, HOLD>;
  const size_t smem = VEC ? static_cast<size_t>(K) * R * UNITS * 8 * sizeof(X) * block.x * block.y : 0;
  if (smem > 32 * 1024) {   // beyond the default limit of 48 KB with the static part
    const cudaError_t e = allow_smem(kern, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const long long per = static_cast<long long>(block.y) * R;
  const long long want = (p.rows + per - 1) / per, cap = static_cast<long long>(p.sms) * MINB * (MAXT / (block.x * block.y));
  return launch_pdl(kern, dim3(static_cast<unsigned>(want < cap ? want : cap)), block, smem, s, p);
}
template <typename X, typename Y, bool VEC>
static cudaError_t forward_shape(const NormParams& p, cudaStream_t s) {
  if constexpr (!VEC) {
    // 8192 rows of 2563 and 4095 bf16: 82 and 93 us with two blocks per SM, 101
    // and 103 with three, whose registers spill.  Above 4096, one row kept in
    // registers or four read again, 8191 wide: fp32 195 and 212 us, bf16 253 and
    // 199.
    if (p.cols <= 2048) return forward_launch<X, Y, false, 1, kNormThreads, 4, 1, 1, true>(p, s);
    if (p.cols <= 4096) return forward_launch<X, Y, false, 2, kNormThreads, 2, 4, 1, true>(p, s);
    if (p.cols <= 8192) return forward_launch<X, Y, false, 2, 512, 1, sizeof(X) == 2 ? 4 : 1, 1, true>(p, s);
    return forward_launch<X, Y, false, 2, 1024, 1, 2, 1, false>(p, s);
  } else {
    // One row at a time up to 8 rows per SM, several per exchange beyond (bf16,
    // one and several: 333 x 4096 3.6 and 5.1 us, 1000 x 4096 6.8 and 7.2; 2048 x
    // 4096 11.4 and 10.1, 4096 x 1664 12.5 and 9.5).  Backward, one row at a time
    // gained nothing over 333 to 1184 rows as a whole.
    const bool few = p.rows <= 8ll * p.sms;
    constexpr bool B16 = sizeof(X) == 2;
    if (p.cols <= 2048)
      return few ? forward_launch<X, Y, VEC, 1, kNormThreads, 4, 1, 2, true>(p, s)
                 : forward_launch<X, Y, VEC, 1, kNormThreads, B16 ? 4 : 3, 4, 2, true>(p, s);
    if (p.cols <= 4096)
      return few ? forward_launch<X, Y, VEC, 2, kNormThreads, 3, 1, 2, true>(p, s)
                 : forward_launch<X, Y, VEC, 2, kNormThreads, 3, B16 ? 4 : 2, 2, true>(p, s);
    if (p.cols <= 8192) return forward_launch<X, Y, VEC, 2, 512, 1, B16 ? 4 : 2, 2, true>(p, s);
    return forward_launch<X, Y, VEC, 2, 1024, 1, B16 ? 2 : 1, 2, false>(p, s);
  }
}
template <typename X, typename Y>
static cudaError_t forward_typed(const NormParams& p, cudaStream_t s) {
  return p.vec ? forward_shape<X, Y, true>(p, s) : forward_shape<X, Y, false>(p, s);
}
static_assert(1024 * 2 * 8 >= kNormMaxCols, "row capacity");
cudaError_t launch_layer_norm(const NormParams& p, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (p.x_bf16) return p.y_bf16 ? forward_typed<B, B>(p, s) : forward_typed<B, float>(p, s);
  return p.y_bf16 ? forward_typed<float, B>(p, s) : forward_typed<float, float>(p, s);
}

// The backward kernel's classes of widths: units per thread, largest block, blocks per SM.
struct GradClass {
  int units, max_threads, per_sm;
};
static GradClass grad_class(int cols) {
  if (cols <= 2048) return {1, kNormThreads, 2};
  if (cols <= 4096) return {2, kNormThreads, 2};
  if (cols <= 8192) return {2, 512, 1};
  return {2, 1024, 1};
}
int layer_norm_grad_blocks(long long rows, int cols, int sms) {
  const GradClass c = grad_class(cols);
  const dim3 block = norm_block(c.units, cols);
  const long long per_sm = static_cast<long long>(c.per_sm) * (c.max_threads / (block.x * block.y));
  const long long want = (rows + block.y - 1) / block.y, cap = sms * per_sm;
  return static_cast<int>(want < cap ? want : cap);
}
template <typename X, bool VEC, int UNITS, int MAXT, int MINB, int R, int K, bool HOLD>
static cudaError_t backward_launch(const NormParams& p, cudaStream_t s) {
  const dim3 block = norm_block(UNITS, p.cols);
  const auto kern = layer_norm_grad_kernel<X, VEC, UNITS, MAXT, MINB, R, K, HOLD>;
  size_t smem = VEC ? static_cast<size_t>(K) * R * 2 * UNITS * 8 * sizeof(X) * block.x * block.y : 0;
  if (block.y > 1) smem = smem > static_cast<size_t>(8) * p.cols ? smem : static_cast<size_t>(8) * p.cols;
  if (smem > 32 * 1024) {
    const cudaError_t e = allow_smem(kern, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(p.blocks), block, smem, s, p);
}
template <typename X, bool VEC>
static cudaError_t backward_shape(const NormParams& p, cudaStream_t s) {
  if constexpr (!VEC) {
    if (p.cols <= 2048) return backward_launch<X, false, 1, kNormThreads, 2, 1, 1, true>(p, s);
    if (p.cols <= 4096) return backward_launch<X, false, 2, kNormThreads, 2, 2, 1, true>(p, s);
    if (p.cols <= 8192) return backward_launch<X, false, 2, 512, 1, 2, 1, true>(p, s);
    return backward_launch<X, false, 2, 1024, 1, 1, 1, false>(p, s);
  } else {
    constexpr bool B16 = sizeof(X) == 2;
    if (p.cols <= 2048) return backward_launch<X, VEC, 1, kNormThreads, 2, B16 ? 4 : 2, B16 ? 2 : 3, true>(p, s);
    if (p.cols <= 4096) return backward_launch<X, VEC, 2, kNormThreads, 2, B16 ? 2 : 1, 2, true>(p, s);
    if (p.cols <= 8192) return backward_launch<X, VEC, 2, 512, 1, B16 ? 2 : 1, 2, true>(p, s);
    return backward_launch<X, VEC, 2, 1024, 1, 1, B16 ? 3 : 1, false>(p, s);
  }
}
template <typename X>
static cudaError_t backward_typed(const NormParams& p, cudaStream_t s) {
  return p.vec ? backward_shape<X, true>(p, s) : backward_shape<X, false>(p, s);
}
cudaError_t launch_layer_norm_grad(const NormParams& p, cudaStream_t s) {
  return p.x_bf16 ? backward_typed<__nv_bfloat16>(p, s) : backward_typed<float>(p, s);
}
cudaError_t launch_layer_norm_columns(const NormParams& p, cudaStream_t s) {
  const dim3 grid((p.cols + 31) / 32, p.dbias ? 2 : 1);
  if (p.grad_bf16)
    return launch_pdl(layer_norm_column_kernel<__nv_bfloat16>, grid, dim3(32 * kColThreads), 0, s, p);
  return launch_pdl(layer_norm_column_kernel<float>, grid, dim3(32 * kColThreads), 0, s, p);
}

}  // namespace muon
