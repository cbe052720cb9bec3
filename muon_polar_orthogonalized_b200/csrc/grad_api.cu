// grad_api.cu -- entry points of the operators that make the optimizer's
// gradients: embedding, layer norm and 8-bit activation checkpoints.
// Arguments are checked on the host before any launch; every launch goes to
// the caller's stream, and nothing is allocated.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "grad_params.cuh"
#include "host_api.cuh"

using namespace muon;

namespace {
constexpr int64_t kMaxRows = 1ll << 30;      // tokens, activation rows
constexpr int64_t kMaxVocab = 1ll << 30;
constexpr int64_t kMaxDim = 65536;           // embedding and matrix widths
// Measured costs of a weight gradient's parts, in microseconds: a stage (64
// rows of a tile), a tile's drain, the launch, the launch that joins shared
// tiles, and each worker's sums written and read.
struct WgCost {
  double stage, tile, start, join, part;
};
constexpr WgCost kWgCost[2] = {{0.40, 3.8, 3.0, 3.0, 0.03}, {0.70, 8.0, 4.0, 4.0, 0.17}};   // narrow, wide
constexpr int64_t kMaxTasks = 1ll << 33;     // 128-column pieces of an embedding's rows

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
bool is_dtype(int32_t t) { return t == MUON_F32 || t == MUON_BF16; }
size_t elem(int32_t t) { return t == MUON_BF16 ? 2 : 4; }

// A dense or row-strided activation matrix: pointer aligned to its element,
// pitch at least the width.
muon_status check_rows(const char* what, const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
  if (!is_dtype(dtype)) return api_fail(MUON_ERR_INVALID_ARG, "%s: dtype %d unknown", what, dtype);
  if (ld < cols) return api_fail(MUON_ERR_INVALID_ARG, "%s: row pitch %lld below %lld columns", what,
                                 static_cast<long long>(ld), static_cast<long long>(cols));
  if (ld > (1ll << 40) / std::max<int64_t>(rows, 1))
    return api_fail(MUON_ERR_INVALID_ARG, "%s: %lld rows of pitch %lld out of range", what,
                    static_cast<long long>(rows), static_cast<long long>(ld));
  if (rows > 0 && (!p || !aligned_to(p, elem(dtype))))
    return api_fail(MUON_ERR_INVALID_ARG, "%s: NULL or misaligned", what);
  return MUON_OK;
}
// Rows that can be accessed 8 elements at a time: 16 bytes of bf16, 32 of fp32.
bool rows_vec(const void* p, int32_t dtype, int64_t cols, int64_t ld) {
  return cols % 8 == 0 && aligned_to(p, 8 * elem(dtype)) && ld % 8 == 0;
}
muon_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MUON_OK;
  if (!ws || !aligned_to(ws, 256)) return api_fail(MUON_ERR_WORKSPACE, "workspace NULL or not 256-byte aligned");
  if (have < need) return api_fail(MUON_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", have, need);
  return MUON_OK;
}
muon_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? MUON_OK : api_cuda_fail(e, what);
}

// No C++ exception leaves an entry point.
template <typename F>
muon_status guarded(F&& f) {
  api_clear_error();
  try {
    return f();
  } catch (...) {
    return api_fail(MUON_ERR_CUDA, "out of host memory");
  }
}

muon_status check_embedding(int64_t vocab, int64_t dim, int64_t n, int32_t ids_bits, const void* ids, float scale) {
  if (vocab < 1 || vocab > kMaxVocab) return api_fail(MUON_ERR_INVALID_ARG, "vocab %lld out of range", static_cast<long long>(vocab));
  if (dim < 1 || dim > kMaxDim) return api_fail(MUON_ERR_INVALID_ARG, "dim %lld out of range", static_cast<long long>(dim));
  if (n < 0 || n > kMaxRows) return api_fail(MUON_ERR_INVALID_ARG, "n %lld out of range", static_cast<long long>(n));
  if ((dim + 127) / 128 * std::max(vocab, n) > kMaxTasks)
    return api_fail(MUON_ERR_INVALID_ARG, "vocab or n times dim out of range");
  if (ids_bits != 32 && ids_bits != 64) return api_fail(MUON_ERR_INVALID_ARG, "ids_bits %d is neither 32 nor 64", ids_bits);
  if (n > 0 && (!ids || !aligned_to(ids, ids_bits / 8))) return api_fail(MUON_ERR_INVALID_ARG, "ids: NULL or misaligned");
  if (!std::isfinite(scale)) return api_fail(MUON_ERR_INVALID_ARG, "scale is not finite");
  return MUON_OK;
}

struct EmbedWs {
  size_t keys, runs, shorts, items, joins, partial, total;
};
EmbedWs embed_ws(int64_t vocab, int64_t dim, int64_t n) {
  EmbedWs w;
  w.keys = up256(static_cast<size_t>(n) * 4);
  w.runs = up256(static_cast<size_t>(vocab) * 4);
  w.shorts = up256(static_cast<size_t>(std::min(n, vocab)) * 16);
  w.items = up256(static_cast<size_t>(embed_max_items(n)) * 16);
  w.joins = up256(static_cast<size_t>(n / (kEmbedPiece + 1)) * 16);
  // a run of several pieces has less than two slots per kEmbedPiece positions
  w.partial = up256(static_cast<size_t>(n / kEmbedPiece + n / (kEmbedPiece + 1)) * dim * 4);
  w.total = 256 + 5 * w.keys + w.runs + w.shorts + w.items + w.joins + w.partial;
  return w;
}

muon_status check_norm(int64_t rows, int64_t cols, const float* gain, const float* mean, const float* rstd) {
  if (rows < 0 || rows > kMaxRows) return api_fail(MUON_ERR_INVALID_ARG, "rows %lld out of range", static_cast<long long>(rows));
  if (cols < 1) return api_fail(MUON_ERR_INVALID_ARG, "cols %lld out of range", static_cast<long long>(cols));
  if (cols > kNormMaxCols)
    return api_fail(MUON_ERR_UNSUPPORTED, "layer norm over %lld columns (at most %d)", static_cast<long long>(cols), kNormMaxCols);
  if (!gain || !aligned_to(gain, 16)) return api_fail(MUON_ERR_INVALID_ARG, "gain: NULL or not 16-byte aligned");
  if (rows > 0 && (!mean || !rstd || !aligned_to(mean, 4) || !aligned_to(rstd, 4)))
    return api_fail(MUON_ERR_INVALID_ARG, "mean or rstd: NULL or misaligned");
  return MUON_OK;
}

muon_status check_checkpoint(const void* q, int64_t q_ld, const void* exps, int64_t rows, int64_t cols) {
  if (rows < 0 || rows > kMaxRows) return api_fail(MUON_ERR_INVALID_ARG, "rows %lld out of range", static_cast<long long>(rows));
  if (cols < 1 || cols > kMaxDim) return api_fail(MUON_ERR_INVALID_ARG, "cols %lld out of range", static_cast<long long>(cols));
  if (q_ld < cols || q_ld % 16 != 0 || q_ld > 2 * kMaxDim)
    return api_fail(MUON_ERR_INVALID_ARG, "code pitch %lld: at least cols, a multiple of 16, at most %lld",
                    static_cast<long long>(q_ld), static_cast<long long>(2 * kMaxDim));
  if (rows > 0 && (!q || !exps || !aligned_to(q, 16)))
    return api_fail(MUON_ERR_INVALID_ARG, "codes or exponents: NULL, or codes not 16-byte aligned");
  return MUON_OK;
}

// Plan of a weight gradient: staging of dy, the tile, and who sums what.
struct WeightWs {
  int planes;      // bf16 planes dy is staged in (0: read as it is)
  int64_t pitch;   // of a staged row
  int wide;
  int64_t tiles_n, tiles_k, tiles;
  int kblocks, workers, whole_tiles;
  bool shared;     // some tile is summed by several workers
  size_t staged, total;
  double cost;     // estimated microseconds
};
// The plan for one tile geometry.
WeightWs weight_plan(WeightWs w, int wide, int64_t n, int64_t k) {
  // CTA pairs of a B200 (148 SMs).  A workspace is sized without a device, so the
  // count is fixed; with fewer SMs pairs only queue, since none waits for another.
  constexpr int kPairs = 74;
  const WgCost& c = kWgCost[wide];
  w.wide = wide;
  w.tiles_n = (n + kWgTile[wide].n - 1) / kWgTile[wide].n;
  w.tiles_k = (k + kWgTile[wide].k - 1) / kWgTile[wide].k;
  w.tiles = w.tiles_n * w.tiles_k;
  w.cost = 1e300;
  const double tile_time = w.kblocks * c.stage + c.tile;
  if (w.tiles >= kPairs) {
    // whole tiles only, or whole rounds of them but for the last one and what is
    // left after it, which are dealt out by row blocks
    w.workers = kPairs;
    w.whole_tiles = static_cast<int>(w.tiles);
    w.cost = static_cast<double>((w.tiles + kPairs - 1) / kPairs) * tile_time + c.start;
    const int64_t rounds = w.tiles / kPairs, left = w.tiles % kPairs;
    // what is left joins the last round where it is little (else each of its
    // tiles would be cut into many runs); where it is much, the rounds before
    // it keep their rows in step and share them in L2 (16384 x 4096 x 4096, 128
    // tiles: 434 us with both rounds in runs)
    const int64_t whole_rounds = 2 * left >= kPairs ? rounds : rounds - 1;
    const double shared = static_cast<double>(w.tiles) / kPairs * w.kblocks * c.stage + (rounds + 1) * c.tile + c.start +
                          c.join + 2 * kPairs * c.part;
    if (left != 0 && shared < w.cost) {
      w.whole_tiles = static_cast<int>(whole_rounds * kPairs);
      w.cost = shared;
    }
  } else {
    // several workers per tile where that is faster
    w.whole_tiles = 0;
    for (int64_t per = 1; per <= std::max<int64_t>(w.kblocks, 1) && w.tiles * per <= kPairs; ++per) {
      const double cost = static_cast<double>((w.kblocks + per - 1) / per) * c.stage + c.tile + c.start +
                          (per == 1 ? 0.0 : c.join + static_cast<double>(w.tiles * per) * c.part);
      if (cost < w.cost) {
        w.cost = cost;
        w.workers = static_cast<int>(w.tiles * per);
      }
    }
  }
  const int64_t blocks = (w.tiles - w.whole_tiles) * w.kblocks;
  w.shared = w.kblocks > 1 && (blocks % w.workers != 0 || blocks / w.workers % w.kblocks != 0);
  return w;
}
WeightWs weight_ws(int64_t rows, int64_t n, int64_t k, int32_t dy_dtype, bool dy_aligned) {
  WeightWs w = {};
  w.planes = dy_dtype == MUON_F32 ? 3 : dy_aligned ? 0 : 1;
  w.pitch = (n + 63) / 64 * 64;
  w.staged = up256(static_cast<size_t>(w.planes) * rows * w.pitch * 2);
  w.kblocks = static_cast<int>((rows + 63) / 64 * std::max(w.planes, 1));
  const WeightWs narrow = weight_plan(w, 0, n, k), wide = weight_plan(w, 1, n, k);
  w = wide.cost <= narrow.cost ? wide : narrow;
  w.total = 256 + w.staged +
            (w.shared ? static_cast<size_t>(2 * w.workers) * kWgTile[w.wide].n * kWgTile[w.wide].k * 4 : 0);
  return w;
}
}  // namespace

extern "C" {

// -------------------------------------------------------------- embedding
muon_status muon_embedding_forward(const void* table, int32_t table_dtype, int64_t vocab, int64_t dim,
                                   const void* ids, int32_t ids_bits, int64_t n, float scale, void* out,
                                   int32_t out_dtype, int64_t out_pitch, muon_stream_t stream) {
  return guarded([&]() -> muon_status {
    muon_status st = check_embedding(vocab, dim, n, ids_bits, ids, scale);
    if (st != MUON_OK) return st;
    if (!is_dtype(table_dtype)) return api_fail(MUON_ERR_INVALID_ARG, "table: dtype %d unknown", table_dtype);
    if (!table || !aligned_to(table, 16)) return api_fail(MUON_ERR_INVALID_ARG, "table: NULL or not 16-byte aligned");
    if ((st = check_rows("out", out, out_dtype, n, dim, out_pitch)) != MUON_OK) return st;
    int sms;
    if ((st = api_device(&sms)) != MUON_OK) return st;
    if (n == 0) return MUON_OK;
    EmbedParams p = {};
    p.table = table;
    p.ids = ids;
    p.out = out;
    p.vocab = vocab;
    p.n = n;
    p.out_ld = out_pitch;
    p.dim = static_cast<int>(dim);
    p.ids64 = ids_bits == 64;
    p.table_bf16 = table_dtype == MUON_BF16;
    p.out_bf16 = out_dtype == MUON_BF16;
    p.vec = rows_vec(table, table_dtype, dim, dim) && rows_vec(out, out_dtype, dim, out_pitch);
    p.scale = scale;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launched(api_timed_launch(K_EMBED, s, [&] { return launch_embedding(p, s); }), "embedding launch");
  });
}

size_t muon_embedding_grad_workspace_size(int64_t vocab, int64_t dim, int64_t n) {
  if (vocab < 1 || vocab > kMaxVocab || dim < 1 || dim > kMaxDim || n < 0 || n > kMaxRows) return 0;
  return embed_ws(vocab, dim, n).total;
}

muon_status muon_embedding_grad(const void* dout, int32_t dout_dtype, int64_t dout_pitch, const void* ids,
                                int32_t ids_bits, int64_t n, int64_t vocab, int64_t dim, float scale, void* grad,
                                int32_t grad_dtype, int accumulate, void* workspace, size_t workspace_bytes,
                                muon_stream_t stream) {
  return guarded([&]() -> muon_status {
    muon_status st = check_embedding(vocab, dim, n, ids_bits, ids, scale);
    if (st != MUON_OK) return st;
    if ((st = check_rows("dout", dout, dout_dtype, n, dim, dout_pitch)) != MUON_OK) return st;
    if (!is_dtype(grad_dtype)) return api_fail(MUON_ERR_INVALID_ARG, "grad: dtype %d unknown", grad_dtype);
    if (!grad || !aligned_to(grad, 16)) return api_fail(MUON_ERR_INVALID_ARG, "grad: NULL or not 16-byte aligned");
    const EmbedWs w = embed_ws(vocab, dim, n);
    if ((st = check_workspace(workspace, workspace_bytes, w.total)) != MUON_OK) return st;
    int sms;
    if ((st = api_device(&sms)) != MUON_OK) return st;
    if (n == 0 && accumulate)
      return launched(cudaMemsetAsync(workspace, 0, 4, reinterpret_cast<cudaStream_t>(stream)), "clear status");
    EmbedGradParams p = {};
    p.dout = dout;
    p.ids = ids;
    p.grad = grad;
    p.vocab = vocab;
    p.n = n;
    p.dout_ld = dout_pitch;
    p.dim = static_cast<int>(dim);
    p.ids64 = ids_bits == 64;
    p.dout_bf16 = dout_dtype == MUON_BF16;
    p.grad_bf16 = grad_dtype == MUON_BF16;
    p.accumulate = accumulate != 0;
    p.vec = rows_vec(dout, dout_dtype, dim, dout_pitch) && rows_vec(grad, grad_dtype, dim, dim);
    p.scale = scale;
    p.status = static_cast<unsigned int*>(workspace);
    char* b = static_cast<char*>(workspace) + 256;
    auto take = [&](size_t bytes) {
      char* r = b;
      b += bytes;
      return r;
    };
    for (int i = 0; i < 2; ++i) p.sorted[i] = reinterpret_cast<uint2*>(take(2 * w.keys));
    p.offset = reinterpret_cast<uint32_t*>(take(w.keys));
    p.first = reinterpret_cast<uint32_t*>(take(w.runs));
    p.shorts = reinterpret_cast<uint4*>(take(w.shorts));
    p.counts = reinterpret_cast<EmbedCounts*>(p.status + 4);
    p.items = reinterpret_cast<uint4*>(take(w.items));
    p.joins = reinterpret_cast<uint4*>(take(w.joins));
    p.partial = reinterpret_cast<float*>(take(w.partial));
    p.sms = sms;
    // keys 0 .. vocab (vocab: no token), in passes of 9 bits
    int width = 1;
    while ((vocab >> width) != 0) ++width;
    p.passes = (width + 8) / 9;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    st = launched(api_timed_launch(K_EMBED_SORT, s, [&] { return launch_embedding_sort(p, s); }),
                  "embedding sort launch");
    if (st != MUON_OK) return st;
    st = launched(api_timed_launch(K_EMBED_GRAD, s, [&] { return launch_embedding_rows(p, s); }),
                  "embedding row launch");
    if (st != MUON_OK || n <= kEmbedPiece) return st;   // no run has several pieces
    return launched(api_timed_launch(K_EMBED_GRAD, s, [&] { return launch_embedding_join(p, s); }),
                    "embedding join launch");
  });
}

// ------------------------------------------------------------- layer norm
muon_status muon_layer_norm_forward(const void* x, int32_t x_dtype, int64_t x_pitch, int64_t rows, int64_t cols,
                                    const float* gain, const float* bias, float eps, void* y, int32_t y_dtype,
                                    int64_t y_pitch, float* mean, float* rstd, muon_stream_t stream) {
  return guarded([&]() -> muon_status {
    muon_status st = check_norm(rows, cols, gain, mean, rstd);
    if (st != MUON_OK) return st;
    if (bias && !aligned_to(bias, 16)) return api_fail(MUON_ERR_INVALID_ARG, "bias not 16-byte aligned");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return api_fail(MUON_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if ((st = check_rows("x", x, x_dtype, rows, cols, x_pitch)) != MUON_OK) return st;
    if ((st = check_rows("y", y, y_dtype, rows, cols, y_pitch)) != MUON_OK) return st;
    int sms;
    if ((st = api_device(&sms)) != MUON_OK) return st;
    if (rows == 0) return MUON_OK;
    NormParams p = {};
    p.x = x;
    p.gain = gain;
    p.bias = bias;
    p.y = y;
    p.mean = mean;
    p.rstd = rstd;
    p.rows = rows;
    p.x_ld = x_pitch;
    p.y_ld = y_pitch;
    p.cols = static_cast<int>(cols);
    p.x_bf16 = x_dtype == MUON_BF16;
    p.y_bf16 = y_dtype == MUON_BF16;
    p.vec = rows_vec(x, x_dtype, cols, x_pitch) && rows_vec(y, y_dtype, cols, y_pitch) && aligned_to(gain, 32) &&
            aligned_to(bias, 32);
    p.eps = eps;
    p.sms = sms;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launched(api_timed_launch(K_LAYER_NORM, s, [&] { return launch_layer_norm(p, s); }), "layer norm launch");
  });
}

size_t muon_layer_norm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > kMaxRows || cols < 1 || cols > kNormMaxCols) return 0;
  // one partial row pair per block of the largest launch
  return 256 + up256(static_cast<size_t>(layer_norm_grad_blocks(rows, static_cast<int>(cols), 160)) * 2 * cols * 4);
}

muon_status muon_layer_norm_backward(const void* dy, int64_t dy_pitch, const void* x, int32_t dtype, int64_t x_pitch,
                                     int64_t rows, int64_t cols, const float* gain, const float* mean,
                                     const float* rstd, void* dx, int64_t dx_pitch, void* dgain, void* dbias,
                                     int32_t grad_dtype, int accumulate, void* workspace, size_t workspace_bytes,
                                     muon_stream_t stream) {
  return guarded([&]() -> muon_status {
    muon_status st = check_norm(rows, cols, gain, mean, rstd);
    if (st != MUON_OK) return st;
    if ((st = check_rows("dy", dy, dtype, rows, cols, dy_pitch)) != MUON_OK) return st;
    if ((st = check_rows("x", x, dtype, rows, cols, x_pitch)) != MUON_OK) return st;
    if ((st = check_rows("dx", dx, dtype, rows, cols, dx_pitch)) != MUON_OK) return st;
    if (!is_dtype(grad_dtype)) return api_fail(MUON_ERR_INVALID_ARG, "grad_dtype %d unknown", grad_dtype);
    if (!dgain || !aligned_to(dgain, elem(grad_dtype)) || !aligned_to(dbias, elem(grad_dtype)))
      return api_fail(MUON_ERR_INVALID_ARG, "dgain NULL, or dgain or dbias misaligned");
    if ((st = check_workspace(workspace, workspace_bytes, muon_layer_norm_backward_workspace_size(rows, cols))) != MUON_OK)
      return st;
    int sms;
    if ((st = api_device(&sms)) != MUON_OK) return st;
    NormParams p = {};
    p.x = x;
    p.dy = dy;
    p.gain = gain;
    p.mean = const_cast<float*>(mean);
    p.rstd = const_cast<float*>(rstd);
    p.y = dx;
    p.dgain = dgain;
    p.dbias = dbias;
    p.status = static_cast<unsigned int*>(workspace);
    p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
    p.rows = rows;
    p.x_ld = x_pitch;
    p.dy_ld = dy_pitch;
    p.y_ld = dx_pitch;
    p.cols = static_cast<int>(cols);
    p.x_bf16 = dtype == MUON_BF16;
    p.grad_bf16 = grad_dtype == MUON_BF16;
    p.accumulate = accumulate != 0;
    p.vec = rows_vec(x, dtype, cols, x_pitch) && rows_vec(dy, dtype, cols, dy_pitch) &&
            rows_vec(dx, dtype, cols, dx_pitch) && aligned_to(gain, 32);
    p.sms = std::min(sms, 160);
    p.blocks = layer_norm_grad_blocks(rows, p.cols, p.sms);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows > 0) {
      st = launched(api_timed_launch(K_LAYER_NORM_GRAD, s, [&] { return launch_layer_norm_grad(p, s); }),
                    "layer norm gradient launch");
      if (st != MUON_OK) return st;
    }
    return launched(api_timed_launch(K_LAYER_NORM_GRAD, s, [&] { return launch_layer_norm_columns(p, s); }),
                    "layer norm column launch");
  });
}

// ------------------------------------------------------------ checkpoints
muon_status muon_checkpoint_pack(const void* x, int32_t x_dtype, int64_t x_pitch, int64_t rows, int64_t cols,
                                 uint8_t* codes, int64_t code_pitch, uint8_t* exponents, muon_stream_t stream) {
  return guarded([&]() -> muon_status {
    muon_status st = check_checkpoint(codes, code_pitch, exponents, rows, cols);
    if (st != MUON_OK) return st;
    if ((st = check_rows("x", x, x_dtype, rows, cols, x_pitch)) != MUON_OK) return st;
    int sms;
    if ((st = api_device(&sms)) != MUON_OK) return st;
    if (rows == 0) return MUON_OK;
    CkptParams p = {};
    p.x = x;
    p.q = codes;
    p.exps = exponents;
    p.rows = rows;
    p.x_ld = x_pitch;
    p.q_ld = code_pitch;
    p.cols = static_cast<int>(cols);
    p.nblk = (p.cols + kCkptBlock - 1) / kCkptBlock;
    p.bf16 = x_dtype == MUON_BF16;
    p.vec = rows_vec(x, x_dtype, cols, x_pitch);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launched(api_timed_launch(K_CKPT_PACK, s, [&] { return launch_checkpoint_pack(p, s); }),
                    "checkpoint pack launch");
  });
}

muon_status muon_checkpoint_unpack(const uint8_t* codes, int64_t code_pitch, const uint8_t* exponents, int64_t rows,
                                   int64_t cols, void* out, int32_t out_dtype, int64_t out_pitch,
                                   muon_stream_t stream) {
  return guarded([&]() -> muon_status {
    muon_status st = check_checkpoint(codes, code_pitch, exponents, rows, cols);
    if (st != MUON_OK) return st;
    if ((st = check_rows("out", out, out_dtype, rows, cols, out_pitch)) != MUON_OK) return st;
    int sms;
    if ((st = api_device(&sms)) != MUON_OK) return st;
    if (rows == 0) return MUON_OK;
    CkptParams p = {};
    p.out = out;
    p.q = const_cast<uint8_t*>(codes);
    p.exps = const_cast<uint8_t*>(exponents);
    p.rows = rows;
    p.out_ld = out_pitch;
    p.q_ld = code_pitch;
    p.cols = static_cast<int>(cols);
    p.nblk = (p.cols + kCkptBlock - 1) / kCkptBlock;
    p.bf16 = out_dtype == MUON_BF16;
    p.vec = rows_vec(out, out_dtype, cols, out_pitch);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launched(api_timed_launch(K_CKPT_UNPACK, s, [&] { return launch_checkpoint_unpack(p, s); }),
                    "checkpoint unpack launch");
  });
}

size_t muon_checkpoint_weight_grad_workspace_size(int64_t rows, int64_t n, int64_t k, int32_t dy_dtype,
                                                  int dy_aligned) {
  if (rows < 0 || rows > kMaxRows || n < 1 || n > kMaxDim || k < 1 || k > kMaxDim || !is_dtype(dy_dtype)) return 0;
  return weight_ws(rows, n, k, dy_dtype, dy_aligned && n % 8 == 0).total;
}

muon_status muon_checkpoint_weight_grad(const void* dy, int32_t dy_dtype, int64_t dy_pitch, int64_t rows, int64_t n,
                                        const uint8_t* codes, int64_t code_pitch, const uint8_t* exponents, int64_t k,
                                        void* grad, int32_t grad_dtype, int accumulate, void* workspace,
                                        size_t workspace_bytes, muon_stream_t stream) {
  return guarded([&]() -> muon_status {
    muon_status st = check_checkpoint(codes, code_pitch, exponents, rows, k);
    if (st != MUON_OK) return st;
    if (n < 1 || n > kMaxDim) return api_fail(MUON_ERR_INVALID_ARG, "n %lld out of range", static_cast<long long>(n));
    if ((st = check_rows("dy", dy, dy_dtype, rows, n, dy_pitch)) != MUON_OK) return st;
    if (!is_dtype(grad_dtype)) return api_fail(MUON_ERR_INVALID_ARG, "grad: dtype %d unknown", grad_dtype);
    if (!grad || !aligned_to(grad, 16)) return api_fail(MUON_ERR_INVALID_ARG, "grad: NULL or not 16-byte aligned");
    const WeightWs w = weight_ws(rows, n, k, dy_dtype, rows_vec(dy, dy_dtype, n, dy_pitch));
    if ((st = check_workspace(workspace, workspace_bytes, w.total)) != MUON_OK) return st;
    int sms;
    if ((st = api_device(&sms)) != MUON_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
      if (!accumulate)
        st = launched(cudaMemsetAsync(grad, 0, static_cast<size_t>(n) * k * elem(grad_dtype), s), "zero gradient");
      if (st == MUON_OK) st = launched(cudaMemsetAsync(workspace, 0, 4, s), "clear status");
      return st;
    }
    WeightGradTc p = {};
    char* base = static_cast<char*>(workspace);
    const void* src = dy;
    int64_t ld = dy_pitch;
    if (w.planes > 0) {   // staged as bf16
      src = base + 256;
      ld = w.pitch;
      st = launched(api_timed_launch(K_WEIGHT_GRAD, s, [&] {
                      return launch_weight_grad_stage(dy, dy_dtype == MUON_BF16, rows_vec(dy, dy_dtype, n, dy_pitch),
                                                      dy_pitch, base + 256, rows, static_cast<int>(n),
                                                      static_cast<int>(w.pitch), s);
                    }), "weight gradient staging launch");
      if (st != MUON_OK) return st;
    }
    const int planes = std::max(w.planes, 1);
    const cuuint64_t R = static_cast<cuuint64_t>(rows), row_bytes = static_cast<cuuint64_t>(ld) * 2;
    const cuuint64_t plane_bytes = planes > 1 ? row_bytes * R : row_bytes;   // one plane: never stepped
    // 64-column chunks as a dimension of their own where rows are whole chunks
    const int64_t width = w.planes > 0 ? w.pitch : n;
    p.chunked = width % 64 == 0;
    if (p.chunked) {
      const cuuint64_t dims[4] = {64, R, static_cast<cuuint64_t>(width / 64), static_cast<cuuint64_t>(planes)};
      const cuuint64_t strides[3] = {row_bytes, 128, plane_bytes};
      const cuuint32_t box[4] = {64, 64, 2, 1};
      st = api_tensor_map(&p.tm_dy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(src), dims, strides, box,
                          CU_TENSOR_MAP_SWIZZLE_128B);
    } else {
      const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), R, static_cast<cuuint64_t>(planes)};
      const cuuint64_t strides[2] = {row_bytes, plane_bytes};
      const cuuint32_t box[3] = {64, 64, 1};
      st = api_tensor_map(&p.tm_dy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(src), dims, strides, box,
                          CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (st != MUON_OK) return st;
    {
      const cuuint64_t dims[3] = {static_cast<cuuint64_t>(k), R, 1};
      const cuuint64_t strides[2] = {static_cast<cuuint64_t>(code_pitch), static_cast<cuuint64_t>(code_pitch)};
      const cuuint32_t box[3] = {static_cast<cuuint32_t>(kWgTile[w.wide].k / 2), 64, 1};
      st = api_tensor_map(&p.tm_q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(codes), dims, strides, box,
                          CU_TENSOR_MAP_SWIZZLE_NONE);
      if (st != MUON_OK) return st;
    }
    p.exps = exponents;
    p.grad = grad;
    p.status = static_cast<unsigned int*>(workspace);
    p.partial = reinterpret_cast<float*>(base + 256 + w.staged);
    p.rows = rows;
    p.n = static_cast<int>(n);
    p.k = static_cast<int>(k);
    p.nblk = (p.k + kCkptBlock - 1) / kCkptBlock;
    p.row_blocks = static_cast<int>((rows + 63) / 64);
    p.kblocks = w.kblocks;
    p.tiles_n = static_cast<int>(w.tiles_n);
    p.tiles_k = static_cast<int>(w.tiles_k);
    p.tiles = static_cast<int>(w.tiles);
    p.workers = w.workers;
    p.whole_tiles = w.whole_tiles;
    p.wide = w.wide;
    const int64_t blocks = (w.tiles - w.whole_tiles) * w.kblocks;
    p.run_len = blocks / w.workers;
    p.run_longer = static_cast<int>(blocks % w.workers);
    p.grad_bf16 = grad_dtype == MUON_BF16;
    p.accumulate = accumulate != 0;
    st = launched(api_timed_launch(K_WEIGHT_GRAD, s, [&] { return launch_weight_grad_tc(p, s); }),
                  "weight gradient launch");
    if (st != MUON_OK || !w.shared) return st;
    return launched(api_timed_launch(K_WEIGHT_GRAD, s, [&] { return launch_weight_grad_join(p, s); }),
                    "weight gradient join launch");
  });
}

}  // extern "C"
