// k_embedding.cu -- embedding lookup and the table's gradient.
//
//   embedding       out[t] = scale * E[id_t]  (zeros where id_t is no row of E)
//   embedding_sort  the token positions in order of (id, position)
//   embedding_grad  dE[v] (+)= scale * sum over t with id_t = v of dout[t],
//                   in fp32, in an order that depends on the ids alone
//
// Lookup and gradient stream: their floor is the rows read and written.  The
// gradient never adds into memory from several threads: the ids are sorted,
// so each row of E has one run of sorted positions [lo, hi), and one warp per
// row and column segment sums the run in order and writes the row once (an
// empty run writes zeros, or nothing when accumulating).  Frequent tokens
// have runs of thousands of positions; runs longer than kEmbedLongRun are cut
// at multiples of kEmbedChunk sorted positions, every whole chunk is summed
// by its own warp into the workspace, and the row's warp adds the ragged
// head, the chunk sums and the ragged tail, again in order.
//
// The sort is a least-significant-digit radix sort (stable, so positions stay
// ascending within an id) by ONE thread-block cluster: the blocks exchange
// digit counts through distributed shared memory and wait for one another at
// the hardware's cluster barrier, so a whole sort is one launch with no
// grid-wide spinning.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "grad_params.cuh"
#include "pdl.cuh"
#include "vec8.cuh"

namespace muon {
namespace cg = cooperative_groups;

constexpr int kEmbThreads = 256;
constexpr int kEmbWarps = kEmbThreads / 32;

// The row of the table a token asks for, or -1.
__device__ __forceinline__ long long token_row(const void* ids, int ids64, long long t, long long vocab) {
  const long long id = ids64 ? static_cast<const long long*>(ids)[t] : static_cast<const int*>(ids)[t];
  return (id >= 0 && id < vocab) ? id : -1;
}

// Columns per warp task: 8 per lane and unit with 16-byte accesses, or single
// columns, lanes adjacent.
template <bool VEC>
constexpr int kSegCols = VEC ? 256 : 128;

// One warp per (token, column segment).
template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(kEmbThreads) embedding_kernel(const EmbedParams p, int nseg) {
  pdl_launch_dependents();
  pdl_wait();
  const long long task = static_cast<long long>(blockIdx.x) * kEmbWarps + (threadIdx.x >> 5);
  const long long t = task / nseg;
  if (t >= p.n) return;
  const int lane = threadIdx.x & 31;
  const int c0 = static_cast<int>(task - t * nseg) * kSegCols<VEC>;
  const long long row = token_row(p.ids, p.ids64, t, p.vocab);
  const T* src = static_cast<const T*>(p.table) + (row < 0 ? 0 : row) * p.dim;
  O* dst = static_cast<O*>(p.out) + t * p.out_ld;
  if constexpr (VEC) {
    const int c = c0 + lane * 8;
    if (c >= p.dim) return;
    float v[8] = {};
    if (row >= 0) {
      load8(src + c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= p.scale;
    }
    store8(dst + c, v);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + k * 32 + lane;
      if (c < p.dim) dst[c] = from_f32<O>(row < 0 ? 0.f : to_f32(src[c]) * p.scale);
    }
  }
}

// ------------------------------------------------------------------- sort
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxBits = 9;
constexpr int kSortBins = 1 << kSortMaxBits;
constexpr int kSortCluster = 8;
constexpr int kSortSmem = (kSortWarps * kSortBins + 2 * kSortBins) * 4;

// Lanes of the warp that hold the same digit as this one.
__device__ __forceinline__ uint32_t same_digit(uint32_t active, uint32_t d) { return __match_any_sync(active, d); }

__global__ void __launch_bounds__(kSortThreads, 1) embedding_sort_kernel(const EmbedGradParams p) {
  extern __shared__ uint32_t sm[];
  uint32_t* hist = sm;                                  // [warp][bin]
  uint32_t* total = sm + kSortWarps * kSortBins;        // [bin] of this block, read by the cluster
  uint32_t* scan = total + kSortBins;                   // [bin]
  __shared__ uint32_t warp_sum[kSortWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int nb = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bins = 1 << p.bits;
  pdl_launch_dependents();
  pdl_wait();

  if (rank == 0 && tid == 0) *p.status = 0;
  // no id has been seen yet
  for (long long v = static_cast<long long>(rank) * kSortThreads + tid; v < p.vocab;
       v += static_cast<long long>(nb) * kSortThreads) {
    p.lo[v] = 0;
    p.hi[v] = 0;
  }
  // each warp owns one contiguous range of positions, a multiple of 32 long
  const long long warps = static_cast<long long>(nb) * kSortWarps;
  const long long per = ((p.n + warps - 1) / warps + 31) / 32 * 32;
  const long long begin = (static_cast<long long>(rank) * kSortWarps + warp) * per;
  const long long end = begin + per < p.n ? begin + per : p.n;

  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const uint32_t* kin = p.keys[(pass + 1) & 1];
    const uint32_t* pin = p.pos[(pass + 1) & 1];
    uint32_t* kout = p.keys[pass & 1];
    uint32_t* pout = p.pos[pass & 1];
    auto key_at = [&](long long i) -> uint32_t {
      if (pass) return kin[i];
      const long long row = token_row(p.ids, p.ids64, i, p.vocab);
      return static_cast<uint32_t>(row < 0 ? p.vocab : row);
    };
    for (int b = tid; b < kSortWarps * bins; b += kSortThreads) hist[(b / bins) * kSortBins + (b % bins)] = 0;
    __syncthreads();
    uint32_t* mine = hist + warp * kSortBins;
    for (long long i0 = begin; i0 < end; i0 += 32) {
      const long long i = i0 + lane;
      const uint32_t act = __ballot_sync(0xffffffffu, i < end);
      if (i < end) {
        const uint32_t d = (key_at(i) >> shift) & (bins - 1);
        const uint32_t peers = same_digit(act, d);
        if (lane == __ffs(peers) - 1) mine[d] += __popc(peers);
      }
      __syncwarp();
    }
    __syncthreads();
    // per bin: exclusive scan over this block's warps
    if (tid < bins) {
      uint32_t run = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = hist[w * kSortBins + tid];
        hist[w * kSortBins + tid] = run;
        run += c;
      }
      total[tid] = run;
    }
    cluster.sync();
    // per bin: counts of the blocks before this one, and of all blocks
    uint32_t before = 0, all = 0;
    if (tid < bins) {
      for (int r = 0; r < nb; ++r) {
        const uint32_t c = cluster.map_shared_rank(total, r)[tid];
        if (r < rank) before += c;
        all += c;
      }
    }
    // exclusive scan of `all` over the bins
    uint32_t inc = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    if (warp == 0) {
      uint32_t s = warp_sum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
      }
      warp_sum[lane] = s;
    }
    __syncthreads();
    if (tid < bins) scan[tid] = inc - all + (warp ? warp_sum[warp - 1] : 0) + before;
    __syncthreads();
    for (long long i0 = begin; i0 < end; i0 += 32) {
      const long long i = i0 + lane;
      const uint32_t act = __ballot_sync(0xffffffffu, i < end);
      if (i < end) {
        const uint32_t key = key_at(i);
        const uint32_t from = pass ? pin[i] : static_cast<uint32_t>(i);
        const uint32_t d = (key >> shift) & (bins - 1);
        const uint32_t peers = same_digit(act, d);
        const uint32_t rk = __popc(peers & ((1u << lane) - 1));
        const uint32_t dst = scan[d] + mine[d] + rk;
        __syncwarp(act);
        if (rk == 0) mine[d] += __popc(peers);
        kout[dst] = key;
        pout[dst] = from;
      }
      __syncwarp();
    }
    // the next pass (or the run boundaries) reads what every block wrote
    __threadfence();
    cluster.sync();
  }

  const uint32_t* keys = p.keys[(p.passes + 1) & 1];
  for (long long i = static_cast<long long>(rank) * kSortThreads + tid; i < p.n;
       i += static_cast<long long>(nb) * kSortThreads) {
    const uint32_t k = keys[i];
    if (k >= p.vocab) continue;
    if (i == 0 || keys[i - 1] != k) p.lo[k] = static_cast<uint32_t>(i);
    if (i == p.n - 1 || keys[i + 1] != k) p.hi[k] = static_cast<uint32_t>(i + 1);
  }
}

// ---------------------------------------------------------------- gradient
// The columns a lane sums: 8 adjacent ones, or 4 that lie 32 apart.
template <bool VEC>
struct Acc {
  static constexpr int N = VEC ? 8 : 4;
  float v[N];
};

template <typename D, bool VEC>
__device__ __forceinline__ void add_row(const D* row, int c0, int lane, int dim, Acc<VEC>& a) {
  if constexpr (VEC) {
    const int c = c0 + lane * 8;
    if (c < dim) {
      float v[8];
      load8(row + c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) a.v[k] += v[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + k * 32 + lane;
      if (c < dim) a.v[k] += to_f32(row[c]);
    }
  }
}

// a += the rows at sorted positions [lo, hi), in order.
template <typename D, bool VEC>
__device__ __forceinline__ void add_run(const EmbedGradParams& p, const uint32_t* pos, uint32_t lo, uint32_t hi,
                                        int c0, int lane, Acc<VEC>& a) {
  const D* dout = static_cast<const D*>(p.dout);
  for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t mine = i0 + lane < hi ? pos[i0 + lane] : 0;
    const int cnt = min(32u, hi - i0);
#pragma unroll 4
    for (int j = 0; j < cnt; ++j) {
      const uint32_t t = __shfl_sync(0xffffffffu, mine, j);
      add_row<D, VEC>(dout + static_cast<long long>(t) * p.dout_ld, c0, lane, p.dim, a);
    }
  }
}

// One warp per (whole chunk of a long run, column segment).
template <typename D, bool VEC>
__global__ void __launch_bounds__(kEmbThreads) embedding_chunk_kernel(const EmbedGradParams p, int nseg) {
  pdl_launch_dependents();
  pdl_wait();
  const long long task = static_cast<long long>(blockIdx.x) * kEmbWarps + (threadIdx.x >> 5);
  const long long chunk = task / nseg;
  if ((chunk + 1) * kEmbedChunk > p.n) return;
  const int lane = threadIdx.x & 31;
  const int c0 = static_cast<int>(task - chunk * nseg) * kSegCols<VEC>;
  const uint32_t* keys = p.keys[(p.passes + 1) & 1];
  const uint32_t* pos = p.pos[(p.passes + 1) & 1];
  const uint32_t lo = static_cast<uint32_t>(chunk * kEmbedChunk), hi = lo + kEmbedChunk;
  const uint32_t k = keys[lo];
  if (k >= p.vocab || keys[hi - 1] != k || p.hi[k] - p.lo[k] <= kEmbedLongRun) return;
  Acc<VEC> a = {};
  add_run<D, VEC>(p, pos, lo, hi, c0, lane, a);
  float* out = p.partial + chunk * p.dim;
  if constexpr (VEC) {
    const int c = c0 + lane * 8;
    if (c < p.dim) store8(out + c, a.v);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + j * 32 + lane;
      if (c < p.dim) out[c] = a.v[j];
    }
  }
}

// One warp per (row of the table, column segment).
template <typename D, typename G, bool VEC>
__global__ void __launch_bounds__(kEmbThreads) embedding_row_kernel(const EmbedGradParams p, int nseg) {
  pdl_launch_dependents();
  pdl_wait();
  const long long task = static_cast<long long>(blockIdx.x) * kEmbWarps + (threadIdx.x >> 5);
  const long long v = task / nseg;
  if (v >= p.vocab) return;
  const int lane = threadIdx.x & 31;
  const int c0 = static_cast<int>(task - v * nseg) * kSegCols<VEC>;
  const uint32_t lo = p.lo[v], hi = p.hi[v];
  if (lo == hi && p.accumulate) return;
  const uint32_t* pos = p.pos[(p.passes + 1) & 1];
  Acc<VEC> a = {};
  if (hi - lo <= kEmbedLongRun) {
    add_run<D, VEC>(p, pos, lo, hi, c0, lane, a);
  } else {
    const uint32_t first = (lo + kEmbedChunk - 1) / kEmbedChunk, last = hi / kEmbedChunk;   // whole chunks
    add_run<D, VEC>(p, pos, lo, first * kEmbedChunk, c0, lane, a);
#pragma unroll 8
    for (uint32_t c = first; c < last; ++c)
      add_row<float, VEC>(p.partial + static_cast<long long>(c) * p.dim, c0, lane, p.dim, a);
    add_run<D, VEC>(p, pos, last * kEmbedChunk, hi, c0, lane, a);
  }
  G* out = static_cast<G*>(p.grad) + v * p.dim;
  if constexpr (VEC) {
    const int c = c0 + lane * 8;
    if (c < p.dim) {
      float o[8] = {};
      if (p.accumulate) load8(out + c, o);
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = fmaf(p.scale, a.v[k], o[k]);
      store8(out + c, o);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + k * 32 + lane;
      if (c < p.dim) out[c] = from_f32<G>(fmaf(p.scale, a.v[k], p.accumulate ? to_f32(out[c]) : 0.f));
    }
  }
}

// ---------------------------------------------------------------- launchers
template <bool VEC>
static int segments(int dim) { return (dim + kSegCols<VEC> - 1) / kSegCols<VEC>; }
static dim3 warp_grid(long long tasks) { return dim3(static_cast<unsigned>((tasks + kEmbWarps - 1) / kEmbWarps)); }

template <typename T, typename O, bool VEC>
static cudaError_t embedding_typed(const EmbedParams& p, cudaStream_t s) {
  const int nseg = segments<VEC>(p.dim);
  return launch_pdl(embedding_kernel<T, O, VEC>, warp_grid(p.n * nseg), dim3(kEmbThreads), 0, s, p, nseg);
}
cudaError_t launch_embedding(const EmbedParams& p, cudaStream_t s) {
  using F = cudaError_t (*)(const EmbedParams&, cudaStream_t);
  using B = __nv_bfloat16;
  static const F table[2][2][2] = {
      {{embedding_typed<float, float, false>, embedding_typed<float, float, true>},
       {embedding_typed<float, B, false>, embedding_typed<float, B, true>}},
      {{embedding_typed<B, float, false>, embedding_typed<B, float, true>},
       {embedding_typed<B, B, false>, embedding_typed<B, B, true>}}};
  return table[p.table_bf16][p.out_bf16][p.vec](p, s);
}

cudaError_t launch_embedding_sort(const EmbedGradParams& p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(embedding_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSortCluster);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = kSortSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSortCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, embedding_sort_kernel, p);
}

template <typename D, bool VEC>
static cudaError_t chunks_typed(const EmbedGradParams& p, cudaStream_t s) {
  const int nseg = segments<VEC>(p.dim);
  return launch_pdl(embedding_chunk_kernel<D, VEC>, warp_grid(p.n / kEmbedChunk * nseg), dim3(kEmbThreads), 0, s, p,
                    nseg);
}
cudaError_t launch_embedding_chunks(const EmbedGradParams& p, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (p.dout_bf16) return p.vec ? chunks_typed<B, true>(p, s) : chunks_typed<B, false>(p, s);
  return p.vec ? chunks_typed<float, true>(p, s) : chunks_typed<float, false>(p, s);
}

template <typename D, typename G, bool VEC>
static cudaError_t rows_typed(const EmbedGradParams& p, cudaStream_t s) {
  const int nseg = segments<VEC>(p.dim);
  return launch_pdl(embedding_row_kernel<D, G, VEC>, warp_grid(p.vocab * nseg), dim3(kEmbThreads), 0, s, p, nseg);
}
cudaError_t launch_embedding_rows(const EmbedGradParams& p, cudaStream_t s) {
  using F = cudaError_t (*)(const EmbedGradParams&, cudaStream_t);
  using B = __nv_bfloat16;
  static const F table[2][2][2] = {
      {{rows_typed<float, float, false>, rows_typed<float, float, true>},
       {rows_typed<float, B, false>, rows_typed<float, B, true>}},
      {{rows_typed<B, float, false>, rows_typed<B, float, true>}, {rows_typed<B, B, false>, rows_typed<B, B, true>}}};
  return table[p.dout_bf16][p.grad_bf16][p.vec](p, s);
}

}  // namespace muon
