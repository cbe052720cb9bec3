// grad_params.cuh -- parameter blocks of the operators that make the
// optimizer's gradients, shared by their kernels and entry points.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace muon {

// ------------------------------------------------------------ embedding
struct EmbedParams {
  const void* table;   // [vocab, dim]
  const void* ids;     // [n] int32 or int64
  void* out;           // [n, dim], row pitch out_ld elements
  long long vocab, n, out_ld;
  int dim;
  int ids64, table_bf16, out_bf16;
  int vec;             // 16-byte accesses allowed
  float scale;
};

constexpr int kEmbedLongRun = 32;      // runs of one token longer than this are cut into
constexpr int kEmbedPiece = 128;       // pieces of this many sorted positions
constexpr uint32_t kEmbedNoSlot = 0xffffffffu;
// Most pieces that n positions can make.
inline long long embed_max_items(long long n) { return n / kEmbedPiece + n / (kEmbedLongRun + 1); }
struct EmbedCounts {
  uint32_t shorts, items, slots, joins;
};

struct EmbedGradParams {
  const void* dout;    // [n, dim], row pitch dout_ld elements
  const void* ids;
  void* grad;          // [vocab, dim]
  long long vocab, n, dout_ld;
  int dim;
  int ids64, dout_bf16, grad_bf16, accumulate;
  int vec;
  float scale;
  // workspace
  unsigned int* status;   // word 0: cleared by every call (muon_query_status)
  uint2* sorted[2];    // [n] sort buffers: (id, vocab for "no token"; position it comes from)
  uint32_t* first;     // [vocab] 1 + first sorted position of each id, 0 where it does not occur
  uint32_t* offset;    // [n] a key's offset within its warp and digit
  EmbedCounts* counts;
  uint4* shorts;       // short runs: (id, first and one past the last sorted position, the last's token)
  uint4* items;        // pieces of long runs: (id, first and one past the last sorted position, slot or kEmbedNoSlot)
  uint4* joins;        // runs of several pieces: (id, first and one past the last slot, -)
  float* partial;      // [slot][dim] sums of the pieces of such runs
  int passes;          // of the radix sort, 9 bits each
  int sms;
};

// ------------------------------------------------------------ layer norm
constexpr int kNormMaxCols = 16384;
struct NormParams {
  const void* x; const void* dy;
  const float* gain; const float* bias;
  void* y;             // forward: y; backward: dx
  float* mean; float* rstd;
  void* dgain; void* dbias;
  float* partial;      // backward: [blocks][2][cols]
  unsigned int* status;   // backward: workspace word 0
  long long rows, x_ld, dy_ld, y_ld;
  int cols;
  int x_bf16, y_bf16, grad_bf16, accumulate;
  int vec;
  int blocks;          // backward: persistent blocks
  int sms;
  float eps;
};

// ------------------------------------------------------------ checkpoints
constexpr int kCkptBlock = 128;        // features sharing one exponent
struct CkptParams {
  const void* x;       // pack: source; unpack: unused
  void* out;           // unpack: destination
  uint8_t* q;          // [rows][q_ld] e4m3 codes
  uint8_t* exps;       // [rows][nblk] exponents (power of two = e - 127; 255: NaN)
  long long rows, x_ld, out_ld, q_ld;
  int cols, nblk;
  int bf16;            // type of x / out
  int vec;
};

// The weight gradient on the tensor cores (k_weight_grad.cu).
struct WgTile {
  int n, k;            // dW rows (columns of dy) and features of a tile
};
constexpr WgTile kWgTile[2] = {{256, 128}, {512, 256}};   // narrow, wide
struct alignas(64) WeightGradTc {
  CUtensorMap tm_dy;   // bf16 dy: (n, rows, planes), or (64, rows, n / 64, planes) when chunked
  CUtensorMap tm_q;    // codes: (k, rows, 1)
  const uint8_t* exps;
  void* grad;          // [n, k]
  float* partial;      // [2 * workers][tile.n][tile.k] sums of parts of tiles
  unsigned int* status;   // workspace word 0
  long long rows;
  int n, k, nblk;
  int chunked;
  int wide;            // tile geometry
  int row_blocks;      // 64-row blocks of one plane
  int kblocks;         // planes * row_blocks
  int tiles_n, tiles_k, tiles;
  int workers;         // CTA pairs
  int whole_tiles;     // dealt out whole, tile i to worker i % workers; the rest by row blocks:
  long long run_len;   // row blocks of a run, and the workers whose run is one longer
  int run_longer;
  int grad_bf16, accumulate;
};

cudaError_t launch_embedding(const EmbedParams& p, cudaStream_t s);
cudaError_t launch_embedding_sort(const EmbedGradParams& p, cudaStream_t s);
cudaError_t launch_embedding_rows(const EmbedGradParams& p, cudaStream_t s);
cudaError_t launch_embedding_join(const EmbedGradParams& p, cudaStream_t s);
cudaError_t launch_layer_norm(const NormParams& p, cudaStream_t s);
cudaError_t launch_layer_norm_grad(const NormParams& p, cudaStream_t s);
cudaError_t launch_layer_norm_columns(const NormParams& p, cudaStream_t s);
int layer_norm_grad_blocks(long long rows, int cols, int sms);
cudaError_t launch_checkpoint_pack(const CkptParams& p, cudaStream_t s);
cudaError_t launch_checkpoint_unpack(const CkptParams& p, cudaStream_t s);
cudaError_t launch_weight_grad_stage(const void* dy, int bf16, int vec, long long dy_ld, void* out, long long rows,
                                     int n, int pitch, cudaStream_t s);
cudaError_t launch_weight_grad_tc(const WeightGradTc& p, cudaStream_t s);
cudaError_t launch_weight_grad_join(const WeightGradTc& p, cudaStream_t s);

}  // namespace muon
