// k_embedding.cu -- embedding lookup and the table's gradient.
//
//   embedding       out[t] = scale * E[id_t]  (zeros where id_t is no row of E)
//   embedding_sort  the token positions in order of (id, position)
//   embedding_grad  dE[v] (+)= scale * sum over t with id_t = v of dout[t],
//                   in fp32, in an order that depends on the ids alone
//
// Lookup and gradient stream: their floor is the rows read and written.  The
// gradient never adds into memory from several threads: the ids are sorted, so
// that each row of E has one run of sorted positions, and a warp per run and
// row piece adds the run in order and writes the row once.  Frequent tokens
// have runs of thousands of positions; runs longer than kEmbedLongRun are cut
// into pieces of kEmbedPiece positions, a block sums each piece (eight warps, an
// eighth each), and the pieces of a run are added in order by another block.
// Rows without a token are written as zeros by one warp of each block, beside
// the warps that add.  (Writing zeros everywhere beside the sort instead made
// the sort, which waits for L2, four times as long.)  Measured: the lookup of
// 32768 x 4096 in 80 us (0.89 of the copy rate); the gradient of 65536 tokens x
// 1664 in 158 us (0.62), of which the rows take 121, short of loads in flight,
// and the sort 28 (both under a profiler).
//
// The sort is a least-significant-digit radix sort (stable, so positions stay
// ascending within an id) by ONE thread-block cluster: the blocks exchange
// digit counts through distributed shared memory and wait for one another at
// the hardware's cluster barrier, so a whole sort is one launch with no
// grid-wide spinning.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "grad_params.cuh"
#include "pdl.cuh"
#include "sm100.cuh"
#include "vec8.cuh"

namespace muon {
namespace cg = cooperative_groups;

// Launch shape of the streaming kernels: blocks of eight warps, `wx` side by
// side along a row and 8 / wx rows apart, over a grid of (rows, row pieces);
// a warp takes a piece of a row, and where rows are short, its lanes share
// them out in groups of `lpr` lanes, a row each.  No index is divided.
constexpr int kEmbWarps = 8;
constexpr int kSegUnits = 4;    // 8-column units per lane: lookup
constexpr int kSumUnits = 1;    // gradient, which holds sums and several rows' units in registers
struct EmbedShape {
  int lpr;        // lanes per row: 32, or fewer for rows of at most lpr * 8 * units columns
  int wx;
  int cols;       // of a warp: 32 * 8 * units
};
// Lane `l` of `lpr` holds, in unit u, 8 adjacent columns (VEC) or 8 that lie lpr apart.
template <bool VEC>
__device__ __forceinline__ int seg_col(int c0, int lpr, int l, int u, int e) {
  return VEC ? c0 + (u * lpr + l) * 8 + e : c0 + (u * 8 + e) * lpr + l;
}

// The row of the table a token asks for, or -1.
__device__ __forceinline__ long long token_row(const void* ids, int ids64, long long t, long long vocab) {
  const long long id = ids64 ? static_cast<const long long*>(ids)[t] : static_cast<const int*>(ids)[t];
  return (id >= 0 && id < vocab) ? id : -1;
}

// This lane's row (of the grid's rows) and its first column.
struct LaneRow {
  long long row;
  int l, c0;
};
__device__ __forceinline__ LaneRow lane_row(const EmbedShape& sh) {
  const int lane = threadIdx.x, per_warp = 32 / sh.lpr;
  const long long slot = static_cast<long long>(blockIdx.x) * blockDim.z + threadIdx.z;
  return {slot * per_warp + lane / sh.lpr, lane % sh.lpr, static_cast<int>(blockIdx.y * sh.wx + threadIdx.y) * sh.cols};
}

template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(32 * kEmbWarps) embedding_kernel(const EmbedParams p, const EmbedShape sh) {
  pdl_launch_dependents();
  pdl_wait();
  const LaneRow w = lane_row(sh);
  if (w.row >= p.n || w.c0 >= p.dim) return;
  const long long row = token_row(p.ids, p.ids64, w.row, p.vocab);
  const T* src = static_cast<const T*>(p.table) + (row < 0 ? 0 : row) * p.dim;
  O* dst = static_cast<O*>(p.out) + w.row * p.out_ld;
  if constexpr (VEC) {
    Raw8<T> r[kSegUnits];
#pragma unroll
    for (int u = 0; u < kSegUnits; ++u) {
      const int c = seg_col<true>(w.c0, sh.lpr, w.l, u, 0);
      r[u] = Raw8<T>{};
      if (row >= 0 && c < p.dim) r[u] = load_raw8(src + c);
    }
#pragma unroll
    for (int u = 0; u < kSegUnits; ++u) {
      const int c = seg_col<true>(w.c0, sh.lpr, w.l, u, 0);
      if (c >= p.dim) break;
      float v[8];
      unpack8(r[u], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = row < 0 ? 0.f : v[e] * p.scale;
      store8(dst + c, v);
    }
  } else {
#pragma unroll
    for (int u = 0; u < kSegUnits; ++u) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = seg_col<false>(w.c0, sh.lpr, w.l, u, e);
        v[e] = row >= 0 && c < p.dim ? to_f32(src[c]) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = seg_col<false>(w.c0, sh.lpr, w.l, u, e);
        if (c < p.dim) dst[c] = from_f32<O>(row < 0 ? 0.f : v[e] * p.scale);
      }
    }
  }
}

// ------------------------------------------------------------------- sort
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBits = 9;
constexpr int kSortBins = 1 << kSortBits;
constexpr int kSortKeys = 8;         // keys a lane has in flight
constexpr int kSortSmem = (kSortWarps + 2) * kSortBins * 4;

// Lanes of `act` with the same digit: one ballot per bit.  (With the
// match instruction the gradient of 65536 tokens x 1664 took 161 us instead of
// 157.)
__device__ __forceinline__ uint32_t same_digit(uint32_t act, uint32_t d) {
  uint32_t peers = act;
#pragma unroll
  for (int b = 0; b < kSortBits; ++b) {
    const bool set = d & (1u << b);
    const uint32_t m = __ballot_sync(act, set);
    peers &= set ? m : ~m;
  }
  return peers;
}

// Enter the run [lo, hi) of sorted positions of an id.  The order of the entries
// is no one's concern: a run's sum goes to its row, or, for long runs in pieces
// of at most kEmbedPiece positions, to slots from which it is added in order.
// last: the token position of the run's last entry.
__device__ __forceinline__ void list_run(const EmbedGradParams& p, EmbedCounts& counts, uint32_t id, uint32_t lo,
                                         uint32_t hi, uint32_t last) {
  if (hi - lo <= kEmbedLongRun) {
    p.shorts[atomicAdd(&counts.shorts, 1u)] = make_uint4(id, lo, hi, last);
    return;
  }
  const uint32_t pieces = (hi - lo + kEmbedPiece - 1) / kEmbedPiece;
  uint32_t slot = 0;
  if (pieces > 1) {
    slot = atomicAdd(&counts.slots, pieces);
    p.joins[atomicAdd(&counts.joins, 1u)] = make_uint4(id, slot, slot + pieces, 0);
  }
  const uint32_t item = atomicAdd(&counts.items, pieces);
  for (uint32_t q = 0; q < pieces; ++q)
    p.items[item + q] = make_uint4(id, lo + q * kEmbedPiece, min(hi, lo + (q + 1) * kEmbedPiece),
                                   pieces > 1 ? slot + q : kEmbedNoSlot);
}

// Each warp owns one contiguous range of positions.  Counting, it takes its
// keys 32 at a time, in order: lanes with the same digit find one another, a
// key's offset is the warp's count of the digit so far plus the earlier lanes
// of the 32, and the first of them adds their number to the count in shared
// memory.  Placing, a key goes to the start of its digit, plus what earlier
// blocks and warps hold of it, plus its offset.
// ONE: a lane's keys are at most kSortKeys, and stay in its registers between
// counting and placing; else they and their offsets are read again.
template <bool ONE>
__global__ void __launch_bounds__(kSortThreads, 1) embedding_sort_kernel(const EmbedGradParams p) {
  extern __shared__ __align__(128) uint32_t sm[];
  uint32_t* hist = sm;                                  // [warp][bin]
  uint32_t* total = sm + kSortWarps * kSortBins;        // [bin] of this block, read by the cluster
  uint32_t* start = total + kSortBins;                  // [bin] of this block's first key
  __shared__ uint32_t warp_sum[kSortWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t nb = cluster.num_blocks(), rank = cluster.block_rank();
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t n = static_cast<uint32_t>(p.n), vocab = static_cast<uint32_t>(p.vocab);
  pdl_launch_dependents();
  pdl_wait();

  if (rank == 0 && tid == 0) {
    *p.status = 0;
    p.counts->shorts = p.counts->items = p.counts->slots = p.counts->joins = 0;
  }
  // no id has been seen yet (the array is padded to whole 16-byte units)
  for (uint32_t v = rank * kSortThreads + tid; v < (vocab + 3) / 4; v += nb * kSortThreads)
    reinterpret_cast<uint4*>(p.first)[v] = make_uint4(0, 0, 0, 0);
  const uint32_t warps = nb * kSortWarps;
  const uint32_t per = ((n + warps - 1) / warps + 31) / 32 * 32;
  const uint32_t begin = min(n, (rank * kSortWarps + warp) * per), end = min(n, begin + per);

  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * kSortBits;
    const uint2* in = p.sorted[(pass + 1) & 1];
    uint2* out = p.sorted[pass & 1];
    // kSortKeys (key, position)s of this lane from position i0 on, 32 apart
    auto load_keys = [&](uint32_t i0, uint2 (&key)[kSortKeys]) {
#pragma unroll
      for (int k = 0; k < kSortKeys; ++k) {
        const uint32_t i = i0 + k * 32 + lane;
        key[k] = make_uint2(0, i);
        if (i < end) {
          if (pass) {
            key[k] = in[i];
          } else {
            const long long row = token_row(p.ids, p.ids64, i, p.vocab);
            key[k].x = row < 0 ? vocab : static_cast<uint32_t>(row);
          }
        }
      }
    };
    uint32_t* mine = hist + warp * kSortBins;
#pragma unroll
    for (int b = 0; b < kSortBins; b += 128) *reinterpret_cast<uint4*>(mine + b + lane * 4) = make_uint4(0, 0, 0, 0);
    __syncwarp();
    uint2 key[kSortKeys];
    uint32_t off[kSortKeys];
    for (uint32_t i0 = begin; i0 < end; i0 += 32 * kSortKeys) {
      load_keys(i0, key);
#pragma unroll
      for (int k = 0; k < kSortKeys; ++k) {
        if (i0 + k * 32 >= end) break;
        const uint32_t i = i0 + k * 32 + lane;
        const uint32_t act = __ballot_sync(0xffffffffu, i < end);
        if (i < end) {
          const uint32_t d = (key[k].x >> shift) & (kSortBins - 1);
          const uint32_t peers = same_digit(act, d);
          const uint32_t rk = __popc(peers & ((1u << lane) - 1)), so_far = mine[d];
          off[k] = so_far + rk;
          if (!ONE) p.offset[i] = off[k];
          __syncwarp(act);
          if (rk == 0) mine[d] = so_far + __popc(peers);
        }
        __syncwarp();
      }
    }
    __syncthreads();
    // per bin: exclusive scan over this block's warps
    uint32_t own = 0;
    if (tid < kSortBins) {
      uint32_t c[kSortWarps];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[w] = hist[w * kSortBins + tid];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        hist[w * kSortBins + tid] = own;
        own += c[w];
      }
      total[tid] = own;
    }
    // per bin: counts of the blocks before this one, and of all blocks
    uint32_t before = 0, all = own;
    if (nb > 1) {
      cluster.sync();
      if (tid < kSortBins) {
        all = 0;
#pragma unroll
        for (uint32_t r = 0; r < 16; ++r) {
          const uint32_t c = r < nb ? cluster.map_shared_rank(total, r)[tid] : 0;
          if (r < rank) before += c;
          all += c;
        }
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
    if (tid < kSortBins) {
      uint32_t left = 0;
      for (uint32_t w = 0; w < warp; ++w) left += warp_sum[w];
      start[tid] = inc - all + left + before;
    }
    __syncthreads();
    for (uint32_t i0 = begin; i0 < end; i0 += 32 * kSortKeys) {
      if (!ONE) {
        load_keys(i0, key);
#pragma unroll
        for (int k = 0; k < kSortKeys; ++k) {
          const uint32_t i = i0 + k * 32 + lane;
          off[k] = i < end ? p.offset[i] : 0;
        }
      }
#pragma unroll
      for (int k = 0; k < kSortKeys; ++k) {
        if (i0 + k * 32 + lane >= end) break;
        const uint32_t d = (key[k].x >> shift) & (kSortBins - 1);
        out[start[d] + mine[d] + off[k]] = key[k];
      }
    }
    // the next pass (or the run boundaries) reads what every block wrote (the
    // cluster's barrier releases and acquires global memory too)
    cluster.sync();
  }

  // Where runs start (kept per id), then, at their ends, the lists of runs.
  const uint2* sorted = p.sorted[(p.passes + 1) & 1];
  const uint32_t stride = nb * kSortThreads;
  for (uint32_t i0 = rank * kSortThreads + tid; i0 < n; i0 += 4 * stride) {
    uint32_t k[4], left[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t i = i0 + j * stride;
      k[j] = i < n ? sorted[i].x : vocab;
      left[j] = i < n && i > 0 ? sorted[i - 1].x : vocab;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k[j] < vocab && k[j] != left[j]) p.first[k[j]] = i0 + j * stride + 1;
  }
  cluster.sync();
  for (uint32_t i0 = rank * kSortThreads + tid; i0 < n; i0 += 4 * stride) {
    uint32_t k[4], right[4], lo[4], at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t i = i0 + j * stride;
      const uint2 e = i < n ? sorted[i] : make_uint2(vocab, 0);
      k[j] = e.x;
      at[j] = e.y;
      right[j] = i < n - 1 ? sorted[i + 1].x : vocab;
      if (k[j] == right[j]) k[j] = vocab;   // not a run's end
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) lo[j] = k[j] < vocab ? p.first[k[j]] - 1 : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (k[j] < vocab) list_run(p, *p.counts, k[j], lo[j], i0 + j * stride + 1, at[j]);
    }
  }
}

// Few tokens (at most kSmallSort): one block sorts in shared memory, so that it
// needs no more of L2 than its ids, and the launch's other blocks write zeros to
// the whole table meanwhile: the rows that have a token, few here, are written
// again.  (1024 tokens on 50304 x 768 fp32: 44 us with the zeros beside the sums
// as for more tokens, 37 so.  From 8192 tokens on the larger sort, which works
// through L2, takes four times as long beside such a stream of writes.)
constexpr int kSmallSort = 2048;
constexpr int kFillBytes = 32 * 1024;
constexpr int kSmallSmem = kSortSmem + kSmallSort * 8;
static_assert(kFillBytes <= kSmallSmem, "zeros share the sort's shared memory");

__device__ __forceinline__ void fill_table(const EmbedGradParams& p, uint4* zeros) {
  for (int i = threadIdx.x; i < kFillBytes / 16; i += kSortThreads) zeros[i] = make_uint4(0, 0, 0, 0);
  sm100::fence_proxy_async_smem();
  __syncthreads();
  pdl_wait();
  if (threadIdx.x != 0) return;
  const long long bytes = p.vocab * p.dim * (p.grad_bf16 ? 2 : 4), whole = bytes / 16 * 16;
  char* out = static_cast<char*>(p.grad);
  for (long long at = (blockIdx.x - 1ll) * kFillBytes; at < whole; at += (gridDim.x - 1ll) * kFillBytes) {
    sm100::bulk_store(out + at, zeros, static_cast<uint32_t>(min(static_cast<long long>(kFillBytes), whole - at)));
    sm100::bulk_commit_group();
  }
  if (blockIdx.x == 1)
    for (long long at = whole; at < bytes; at += 2) *reinterpret_cast<uint16_t*>(out + at) = 0;
  sm100::bulk_wait_group<0>();   // shared memory stays until it is read, and the zeros are written
}

__global__ void __launch_bounds__(kSortThreads, 1) embedding_sort_small_kernel(const EmbedGradParams p) {
  extern __shared__ __align__(128) uint32_t sm[];
  __shared__ uint32_t warp_sum[kSortWarps];
  __shared__ EmbedCounts counts;
  pdl_launch_dependents();
  if (blockIdx.x > 0) {
    fill_table(p, reinterpret_cast<uint4*>(sm));
    return;
  }
  uint32_t* hist = sm;                                  // [warp][bin]
  uint32_t* start = sm + kSortWarps * kSortBins;        // [bin]
  uint2* buf = reinterpret_cast<uint2*>(start + 2 * kSortBins);   // (id, position), in the order so far
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t n = static_cast<uint32_t>(p.n), vocab = static_cast<uint32_t>(p.vocab);
  constexpr int KEYS = kSmallSort / kSortThreads;
  if (tid == 0) counts = EmbedCounts{};
  pdl_wait();
  uint2 key[KEYS];
  uint32_t off[KEYS];
#pragma unroll
  for (int k = 0; k < KEYS; ++k) {
    const uint32_t i = warp * 32 * KEYS + k * 32 + lane;
    key[k] = make_uint2(vocab, i);
    if (i < n) {
      const long long row = token_row(p.ids, p.ids64, i, p.vocab);
      if (row >= 0) key[k].x = static_cast<uint32_t>(row);
    }
  }
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * kSortBits;
    uint32_t* mine = hist + warp * kSortBins;
#pragma unroll
    for (int b = 0; b < kSortBins; b += 128) *reinterpret_cast<uint4*>(mine + b + lane * 4) = make_uint4(0, 0, 0, 0);
    __syncwarp();
    // positions past n take part with the id `vocab`: they sort last
#pragma unroll
    for (int k = 0; k < KEYS; ++k) {
      const uint32_t d = (key[k].x >> shift) & (kSortBins - 1);
      const uint32_t peers = same_digit(0xffffffffu, d);
      const uint32_t rk = __popc(peers & ((1u << lane) - 1)), so_far = mine[d];
      off[k] = so_far + rk;
      __syncwarp();
      if (rk == 0) mine[d] = so_far + __popc(peers);
      __syncwarp();
    }
    __syncthreads();
    uint32_t own = 0;
    if (tid < kSortBins) {
      uint32_t c[kSortWarps];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[w] = hist[w * kSortBins + tid];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        hist[w * kSortBins + tid] = own;
        own += c[w];
      }
    }
    uint32_t inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    if (tid < kSortBins) {
      uint32_t left = 0;
      for (uint32_t w = 0; w < warp; ++w) left += warp_sum[w];
      start[tid] = inc - own + left;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KEYS; ++k) {
      const uint32_t d = (key[k].x >> shift) & (kSortBins - 1);
      buf[start[d] + mine[d] + off[k]] = key[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KEYS; ++k) key[k] = buf[warp * 32 * KEYS + k * 32 + lane];
  }
  // the lists of runs, at their ends
#pragma unroll
  for (int k = 0; k < KEYS; ++k) {
    const uint32_t i = warp * 32 * KEYS + k * 32 + lane, id = key[k].x;
    if (i < n) p.sorted[(p.passes + 1) & 1][i] = key[k];
    if (id >= vocab || (i + 1 < n && buf[i + 1].x == id)) continue;
    uint32_t lo = 0, step_hi = i;   // first position with this id
    while (lo < step_hi) {
      const uint32_t mid = (lo + step_hi) / 2;
      if (buf[mid].x < id) lo = mid + 1;
      else step_hi = mid;
    }
    list_run(p, counts, id, lo, i + 1, key[k].y);
  }
  __syncthreads();
  if (tid == 0) {
    *p.status = 0;
    *p.counts = counts;
  }
}

// ---------------------------------------------------------------- gradient
// The columns of one row that a lane sums.
template <int UNITS>
struct Sums {
  float v[UNITS][8];
};

template <typename D, bool VEC, int UNITS>
struct RowPiece {
  Raw8<D> raw[UNITS];
  float f[VEC ? 1 : UNITS][8];
  __device__ __forceinline__ void load(const D* row, int dim, int c0, int lpr, int l) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      if constexpr (VEC) {
        const int c = seg_col<true>(c0, lpr, l, u, 0);
        if (c < dim) raw[u] = load_raw8(row + c);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = seg_col<false>(c0, lpr, l, u, e);
          f[u][e] = c < dim ? to_f32(row[c]) : 0.f;
        }
      }
    }
  }
  __device__ __forceinline__ void add_to(Sums<UNITS>& a, int dim, int c0, int lpr, int l) const {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      if constexpr (VEC) {
        if (seg_col<true>(c0, lpr, l, u, 0) >= dim) break;
        float v[8];
        unpack8(raw[u], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) a.v[u][e] += v[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) a.v[u][e] += f[u][e];
      }
    }
  }
};

// a += rows at(lo), ..., at(hi - 1), in that order; AHEAD of them are loaded
// before the first is added.
template <typename D, bool VEC, int AHEAD, int UNITS, typename At>
__device__ __forceinline__ void add_rows(uint32_t lo, uint32_t hi, int dim, int c0, int lpr, int l, Sums<UNITS>& a, At at) {
  uint32_t i = lo;
  for (; i + AHEAD <= hi; i += AHEAD) {
    const D* row[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) row[k] = at(i + k);
    RowPiece<D, VEC, UNITS> r[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) r[k].load(row[k], dim, c0, lpr, l);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) r[k].add_to(a, dim, c0, lpr, l);
  }
  for (; i < hi; ++i) {
    RowPiece<D, VEC, UNITS> r;
    r.load(at(i), dim, c0, lpr, l);
    r.add_to(a, dim, c0, lpr, l);
  }
}

// grad row's columns <- (old +) scale * sums
template <typename G, bool VEC, int UNITS>
__device__ __forceinline__ void write_row(const EmbedGradParams& p, G* out, int c0, int lpr, int l, const Sums<UNITS>& a) {
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    if constexpr (VEC) {
      const int c = seg_col<true>(c0, lpr, l, u, 0);
      if (c >= p.dim) break;
      float o[8] = {};
      if (p.accumulate) load8(out + c, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(p.scale, a.v[u][e], o[e]);
      store8(out + c, o);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = seg_col<false>(c0, lpr, l, u, e);
        if (c < p.dim) out[c] = from_f32<G>(fmaf(p.scale, a.v[u][e], p.accumulate ? to_f32(out[c]) : 0.f));
      }
    }
  }
}

// Sum of the block's adding warps, in order, in warp 0; every one calls it.
__device__ __forceinline__ void adders_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kEmbWarps) : "memory"); }
__device__ __forceinline__ void block_sum(Sums<kSumUnits>& a, float (&part)[kEmbWarps][kSumUnits * 8][32]) {
  const int lane = threadIdx.x, warp = threadIdx.y;
#pragma unroll
  for (int i = 0; i < kSumUnits * 8; ++i) part[warp][i][lane] = a.v[i / 8][i % 8];
  adders_barrier();
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < kSumUnits * 8; ++i) {
      float v = part[0][i][lane];
#pragma unroll
      for (int w = 1; w < kEmbWarps; ++w) v += part[w][i][lane];
      a.v[i / 8][i % 8] = v;
    }
  }
  adders_barrier();
}

// A block's share of a list of pieces (JOIN: of runs' slots), row piece by row
// piece.  Each warp adds a contiguous eighth of the terms.
template <typename D, typename G, bool VEC, bool JOIN>
__device__ __forceinline__ void add_long(const EmbedGradParams& p, uint32_t segs,
                                         float (&part)[kEmbWarps][kSumUnits * 8][32]) {
  const uint2* sorted = p.sorted[(p.passes + 1) & 1];
  const int lane = threadIdx.x, warp = threadIdx.y;
  const uint32_t count = JOIN ? p.counts->joins : p.counts->items;
  for (unsigned long long it = blockIdx.x; it < static_cast<unsigned long long>(count) * segs; it += gridDim.x) {
    const uint32_t i = it <= 0xffffffffull ? static_cast<uint32_t>(it) / segs : static_cast<uint32_t>(it / segs);
    const int c0 = static_cast<int>(it - static_cast<unsigned long long>(i) * segs) * (32 * 8 * kSumUnits);
    const uint4 w = JOIN ? p.joins[i] : p.items[i];
    const uint32_t len = w.z - w.y, b = w.y + len * warp / kEmbWarps, e = w.y + len * (warp + 1) / kEmbWarps;
    Sums<kSumUnits> a = {};
    if constexpr (JOIN)
      add_rows<float, VEC, VEC ? 4 : 2>(b, e, p.dim, c0, 32, lane, a,
                                        [&](uint32_t k) { return p.partial + static_cast<long long>(k) * p.dim; });
    else
      add_rows<D, VEC, VEC ? 4 : 2>(b, e, p.dim, c0, 32, lane, a,
                                    [&](uint32_t k) { return static_cast<const D*>(p.dout) + sorted[k].y * p.dout_ld; });
    block_sum(a, part);
    if (warp != 0) continue;
    if (!JOIN && w.w != kEmbedNoSlot) {
      float* out = p.partial + static_cast<long long>(w.w) * p.dim;
#pragma unroll
      for (int u = 0; u < kSumUnits; ++u) {
        if constexpr (VEC) {
          const int c = seg_col<true>(c0, 32, lane, u, 0);
          if (c < p.dim) store8(out + c, a.v[u]);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int c = seg_col<false>(c0, 32, lane, u, q);
            if (c < p.dim) out[c] = a.v[u][q];
          }
        }
      }
    } else {
      write_row<G, VEC>(p, static_cast<G*>(p.grad) + static_cast<long long>(w.x) * p.dim, c0, 32, lane, a);
    }
  }
}

// Zeros in the rows that have no token, by the block's last warp: a lane per
// row, bulk copies of a zeroed piece of shared memory (436 MB in 69 us; stores
// from registers took 118), or the warp's stores where rows are not whole
// 16-byte units.
constexpr int kZeroBytes = 8192;
constexpr int kRowBlocks = 3;   // of the rows kernel per SM
template <typename G>
__device__ __forceinline__ void fill_rows(const EmbedGradParams& p, const uint4* zeros) {
  const int lane = threadIdx.x;
  const long long bytes = static_cast<long long>(p.dim) * sizeof(G);
  for (long long v0 = static_cast<long long>(blockIdx.x) * 32; v0 < p.vocab; v0 += static_cast<long long>(gridDim.x) * 32) {
    const bool none = v0 + lane < p.vocab && p.first[v0 + lane] == 0;
    if (bytes % 16 == 0) {
      if (none) {
        char* out = static_cast<char*>(p.grad) + (v0 + lane) * bytes;
        for (long long at = 0; at < bytes; at += kZeroBytes)
          sm100::bulk_store(out + at, zeros, static_cast<uint32_t>(min(static_cast<long long>(kZeroBytes), bytes - at)));
        sm100::bulk_commit_group();
      }
    } else {
      for (uint32_t rows = __ballot_sync(0xffffffffu, none); rows; rows &= rows - 1) {
        G* out = static_cast<G*>(p.grad) + (v0 + __ffs(rows) - 1) * p.dim;
        for (int c = lane; c < p.dim; c += 32) out[c] = from_f32<G>(0.f);
      }
    }
  }
  sm100::bulk_wait_group<0>();   // shared memory stays until it is read, and the zeros are written
}

// Every row that is the sum of one run or piece, and the rows without a token.
// Eight warps of a block add: first the pieces of long runs, a block each, then
// the short runs, a warp (or a group of its lanes) per run and row piece, while
// the ninth writes zeros: the reads of some rows and the writes of others share
// the memory's time.
template <typename D, typename G, bool VEC>
__global__ void __launch_bounds__(32 * (kEmbWarps + 1), kRowBlocks) embedding_rows_kernel(const EmbedGradParams p, uint32_t segs,
                                                                                 int lpr) {
  __shared__ float part[kEmbWarps][kSumUnits * 8][32];
  __shared__ __align__(128) uint4 zeros[kZeroBytes / 16];
  pdl_launch_dependents();
  const bool fill = !p.accumulate && p.n > kSmallSort;   // few tokens: the sort's launch has done it
  if (threadIdx.y == kEmbWarps && fill) {
    for (int i = threadIdx.x; i < kZeroBytes / 16; i += 32) zeros[i] = make_uint4(0, 0, 0, 0);
    sm100::fence_proxy_async_smem();
    __syncwarp();
  }
  pdl_wait();
  if (threadIdx.y == kEmbWarps) {
    if (fill) fill_rows<G>(p, zeros);
    return;
  }
  add_long<D, G, VEC, false>(p, segs, part);
  const uint2* sorted = p.sorted[(p.passes + 1) & 1];
  const int l = threadIdx.x % lpr;
  const uint32_t per_warp = 32 / lpr, count = p.counts->shorts;
  // Tasks: row pieces of groups of per_warp runs, BATCH at a time: the runs of
  // the next batch are read while this one's are added, and a run of one token
  // (most are) names it itself, so that only the rows are waited for, together.
  constexpr int BATCH = VEC ? 2 : 1;
  const unsigned long long tasks = static_cast<unsigned long long>((count + per_warp - 1) / per_warp) * segs;
  const unsigned long long step = static_cast<unsigned long long>(gridDim.x) * kEmbWarps;
  const D* dout = static_cast<const D*>(p.dout);
  unsigned long long it = blockIdx.x * kEmbWarps + threadIdx.y;
  uint4 w[BATCH];
  int c0[BATCH];
  auto runs = [&](uint4 (&w)[BATCH], int (&c0)[BATCH], unsigned long long it) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const unsigned long long t = it + k * step;
      const uint32_t q = t <= 0xffffffffull ? static_cast<uint32_t>(t) / segs : static_cast<uint32_t>(t / segs);
      c0[k] = static_cast<int>(t - static_cast<unsigned long long>(q) * segs) * (32 * 8 * kSumUnits);
      const uint32_t i = q * per_warp + threadIdx.x / lpr;
      w[k] = t < tasks && i < count ? p.shorts[i] : make_uint4(0, 0, 0, 0);   // no run: nothing to do
    }
  };
  runs(w, c0, it);
  while (it < tasks) {
    RowPiece<D, VEC, kSumUnits> last[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
      if (w[k].z > w[k].y) last[k].load(dout + w[k].w * p.dout_ld, p.dim, c0[k], lpr, l);
    uint4 w_next[BATCH];
    int c0_next[BATCH];
    it += BATCH * step;
    runs(w_next, c0_next, it);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (w[k].z > w[k].y) {
        Sums<kSumUnits> a = {};
        add_rows<D, VEC, VEC ? 4 : 2>(w[k].y, w[k].z - 1, p.dim, c0[k], lpr, l, a,
                                      [&](uint32_t i) { return dout + sorted[i].y * p.dout_ld; });
        last[k].add_to(a, p.dim, c0[k], lpr, l);
        write_row<G, VEC>(p, static_cast<G*>(p.grad) + static_cast<long long>(w[k].x) * p.dim, c0[k], lpr, l, a);
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      w[k] = w_next[k];
      c0[k] = c0_next[k];
    }
  }
}

// Runs of several pieces.
template <typename G, bool VEC>
__global__ void __launch_bounds__(32 * kEmbWarps) embedding_join_kernel(const EmbedGradParams p, uint32_t segs) {
  __shared__ float part[kEmbWarps][kSumUnits * 8][32];
  pdl_launch_dependents();
  pdl_wait();
  add_long<float, G, VEC, true>(p, segs, part);
}

// ---------------------------------------------------------------- launchers
namespace {
struct EmbedLaunch {
  EmbedShape shape;
  dim3 grid, block;
};
EmbedLaunch embed_launch(long long rows, int dim, int units) {
  EmbedLaunch l;
  l.shape.lpr = 32;
  while (l.shape.lpr > 1 && dim <= l.shape.lpr / 2 * 8 * units) l.shape.lpr /= 2;
  l.shape.cols = 32 * 8 * units;
  const int segs = (dim + l.shape.cols - 1) / l.shape.cols;
  l.shape.wx = 1;
  while (l.shape.wx < kEmbWarps && l.shape.wx < segs) l.shape.wx *= 2;
  l.block = dim3(32, l.shape.wx, kEmbWarps / l.shape.wx);
  const long long per = static_cast<long long>(l.block.z) * (32 / l.shape.lpr);
  l.grid = dim3(static_cast<unsigned>((rows + per - 1) / per), (segs + l.shape.wx - 1) / l.shape.wx);
  return l;
}
}  // namespace

template <typename T, typename O, bool VEC>
static cudaError_t embedding_typed(const EmbedParams& p, cudaStream_t s) {
  const EmbedLaunch l = embed_launch(p.n, p.dim, kSegUnits);
  return launch_pdl(embedding_kernel<T, O, VEC>, l.grid, l.block, 0, s, p, l.shape);
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

// Blocks of the sort's cluster: enough that a lane has few keys.  16 where the
// GPU can place such a cluster (beyond the portable 8).  Only what the GPU can
// place is kept; the attribute that allows such clusters is set before each
// launch, as in allow_smem.
template <bool ONE>
static cudaError_t sort_limit(int* limit) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(embedding_sort_kernel<ONE>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*limit = known[dev].load(std::memory_order_relaxed)) != 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = kSortSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 16;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  *limit = 8;
  if (cudaOccupancyMaxActiveClusters(&clusters, embedding_sort_kernel<ONE>, &cfg) == cudaSuccess && clusters > 0) *limit = 16;
  else cudaGetLastError();
  if (dev < 64) known[dev].store(*limit, std::memory_order_relaxed);
  return cudaSuccess;
}
template <bool ONE>
static cudaError_t sort_launch(const EmbedGradParams& p, unsigned nb, cudaStream_t s) {
  const auto kern = embedding_sort_kernel<ONE>;
  int limit = 8;
  cudaError_t e = allow_smem(kern, kSortSmem);
  if (e == cudaSuccess && nb > 8) e = sort_limit<ONE>(&limit);
  if (e != cudaSuccess) return e;
  if (nb > static_cast<unsigned>(limit)) {
    nb = limit;
    if (ONE && p.n > static_cast<long long>(nb) * kSortThreads * kSortKeys) return sort_launch<false>(p, nb, s);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nb);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = kSortSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nb;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}
cudaError_t launch_embedding_sort(const EmbedGradParams& p, cudaStream_t s) {
  if (p.n <= kSmallSort) {
    const cudaError_t e = allow_smem(embedding_sort_small_kernel, kSmallSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(embedding_sort_small_kernel, dim3(p.accumulate ? 1 : p.sms), dim3(kSortThreads), kSmallSmem, s, p);
  }
  unsigned nb = 1;
  while (nb < 16 && nb < std::max((p.n + 2047) / 2048, p.vocab / 65536)) nb *= 2;
  // per warp, positions are rounded up to 32
  const bool one = p.n <= static_cast<long long>(nb) * kSortThreads * kSortKeys;
  return one ? sort_launch<true>(p, nb, s) : sort_launch<false>(p, nb, s);
}

static uint32_t sum_segments(int dim) { return (dim + 32 * 8 * kSumUnits - 1) / (32 * 8 * kSumUnits); }

template <typename D, typename G, bool VEC>
static cudaError_t rows_typed(const EmbedGradParams& p, cudaStream_t s) {
  int lpr = 32;
  while (lpr > 1 && p.dim <= lpr / 2 * 8 * kSumUnits) lpr /= 2;
  return launch_pdl(embedding_rows_kernel<D, G, VEC>, dim3(kRowBlocks * p.sms), dim3(32, kEmbWarps + 1), 0, s, p,
                    sum_segments(p.dim), lpr);
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

template <typename G, bool VEC>
static cudaError_t join_typed(const EmbedGradParams& p, cudaStream_t s) {
  const uint32_t segs = sum_segments(p.dim);
  const long long most = p.n / (kEmbedPiece + 1) * segs;   // runs of several pieces
  return launch_pdl(embedding_join_kernel<G, VEC>, dim3(static_cast<unsigned>(std::min<long long>(most, 3 * p.sms))),
                    dim3(32, kEmbWarps), 0, s, p, segs);
}
cudaError_t launch_embedding_join(const EmbedGradParams& p, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (p.grad_bf16) return p.vec ? join_typed<B, true>(p, s) : join_typed<B, false>(p, s);
  return p.vec ? join_typed<float, true>(p, s) : join_typed<float, false>(p, s);
}

}  // namespace muon
