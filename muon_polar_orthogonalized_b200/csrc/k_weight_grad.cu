// k_weight_grad.cu -- a hidden matrix's gradient from an 8-bit checkpoint, on
// the 5th-generation tensor cores.
//
//   dW[n][k] (+)= sum over rows t of dy[t][n] * x[t][k],
//   x[t][k] = code[t][k] * 2^(e[t][k / 128] - 127)
//
// 2 T N K operations on operands of 2 T N + T K bytes: bound by the tensor
// pipe for all but the smallest shapes.  The tensor cores' bf16 product needs
// both operands in bf16, and every restored value is exact in bf16
// (k_checkpoint.cu), so the codes are turned into bf16 on the way through
// shared memory and never exist in memory at 2 bytes: the kernel reads half
// the bytes of x that a product of kept bf16 activations would.
//
// Structure: persistent CTA pairs (cta_group::2) on tiles of 512 columns of dy
// by 256 features.  Both operands are MN-major (their rows are the summed
// index).  Per 64 rows and stage, each CTA brings by TMA 2 x 128 columns of dy
// (bf16, 128-byte swizzle: the MMA operand as it stands) and 128 features of
// codes (exactly one exponent per row), and sixteen warps write the codes'
// bf16 values into the second operand's swizzled layout.  The leader issues
// 256x256x16 MMAs, two per 16 rows (one for each half of the dy columns), into
// one 512-column accumulator: restored codes are used for 512 columns of dy,
// which leaves the sixteen warps 1024 tensor-pipe cycles per stage.  The same
// sixteen warps write the finished tile.  Measured on two boards: 1.48 to 1.53
// PFLOP/s at 16384 x 14336 x 4096 (1.26 to 1.30 ms, 1.09 to 1.13 of the measured
// sustained bf16 product; 1.29 in a long loop, at the power cap), 1.20 to 1.32
// at 16384 x 1024 x 4096.  Where there are few tiles, or few
// rows, a tile's start and drain (11 us) outweigh its product, and tiles of
// 256 by 128 are used, on which two groups of eight warps take the stages in
// turn: 11.5 us against 19.3 at 777 x 1664 x 768 and 16.2 against 22.2 at 4096 x
// 768 x 768, but 139 against 98 at 16384 x 1664 x 1664 and 0.74 PFLOP/s at
// 16384 x 14336 x 4096.  The choice is by the estimated time (grad_api.cu).
//   warp 0: TMA producer   warp 1: MMA issuer (+ TMEM owner)
//   warps 2-17: codes to bf16, then the tile's epilogue
// How codes become bf16 is in e4m3.cuh.  Bytes 1 and 3 of a word of four codes need no move to
// their halves, so features 1 and 2 of every four change places in the
// operand, and with them two registers in the epilogue.
//
// The (tile, row block) space is dealt out in whole tiles while there are
// enough for every pair, and the rest in equal runs of row blocks that may
// start and end inside a tile; a run that does not cover its tile writes fp32
// sums to the workspace, and a second kernel adds the runs of such a tile in
// order.  dy in fp32, or with rows that TMA cannot read, is first staged in
// the workspace as bf16: one plane for bf16, three for fp32 (each value is
// the sum of its three parts, but for what a value under 2^-110 has below bf16's
// smallest number, 2^-133), which the product walks one after another as if the
// rows repeated.  The plane of the lowest bits comes
// first: the tensor cores cut what lies below a step of the running sum at
// every addition, so the two lower planes are added while the sum is 2^-16 and
// 2^-8 of what it will be (777 x 1664 x 768, error against 64 bits relative to
// the gradient, root mean square: 2.2e-7, with the highest plane first 3.8e-6).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "grad_params.cuh"
#include "pdl.cuh"
#include "sm100.cuh"
#include "vec8.cuh"

namespace muon {

namespace {
constexpr int WG_BK = 64;                      // rows (summed index) per stage
constexpr int WG_CHUNK = WG_BK * 128;          // one 64-column chunk of an operand
constexpr int WG_SUB_BYTES = 2 * WG_CHUNK;     // dy: 128 columns of one 256-column half
constexpr int WG_WARPS = 16;                   // restoring and writing
constexpr int WG_THREADS = 32 * (2 + WG_WARPS);
constexpr int WG_BAND = 8;                     // tile columns per raster band

// Tile geometry (kWgTile[wide]): 512 columns of dy by 256 features, or 256 by 128.
template <bool WIDE>
struct WgCfg {
  static constexpr int TN = kWgTile[WIDE].n, TK = kWgTile[WIDE].k;
  static constexpr int SUBS = TN / 256;                    // 256-column halves: MMAs per 16 rows
  static constexpr int A_BYTES = SUBS * WG_SUB_BYTES;
  static constexpr int CODES = TK / 2;                     // features per CTA
  static constexpr int B_BYTES = CODES / 64 * WG_CHUNK;    // restored x
  static constexpr int Q_BYTES = CODES * WG_BK;            // codes
  static constexpr int STAGE = A_BYTES + B_BYTES + Q_BYTES;
  static constexpr int STAGES = WIDE ? 4 : 8;
  // a stage has WG_BK rows of CODES / 16 tasks of 16 codes, one per thread: the
  // sixteen warps form GROUPS that take the stages in turn
  static constexpr int ROW_TASKS = CODES / 16;
  static constexpr int GROUP_WARPS = WG_BK * ROW_TASKS / 32;
  static constexpr int GROUPS = WG_WARPS / GROUP_WARPS;
  static constexpr int TMEM = SUBS * TK;                   // accumulator columns
  static constexpr int BAR_OFF = STAGES * STAGE;
  static constexpr int SMEM = BAR_OFF + 1024 + 1024;
  static_assert(SMEM <= 232448, "shared memory per block");
  static_assert(STAGE % 1024 == 0 && A_BYTES % 1024 == 0, "swizzle atoms");
  static_assert(GROUPS * GROUP_WARPS == WG_WARPS && kCkptBlock % CODES == 0, "one exponent per row");
  // A wait by parity tells a phase from the one next to it alone, so whoever
  // waits for a slot's codes must do so at every use of the slot: each slot
  // belongs to one group.
  static_assert(STAGES % GROUPS == 0, "a group would miss phases of its slots");
};
constexpr uint32_t kTimeout = 1u;              // status word bit (muon_query_status)
}  // namespace

// One piece of a worker's work: row blocks [kb0, kb1) of a tile; slot >= 0
// where they are not the whole tile.
struct WgUnit {
  int n0, k0, kb0, kb1, slot;
};

template <bool WIDE>
__device__ __forceinline__ void wg_tile(const WeightGradTc& p, int tile, int& n0, int& k0) {
  const int band_tiles = p.tiles_n * WG_BAND;
  const int band = tile / band_tiles;
  const int r = tile - band * band_tiles;
  const int width = min(WG_BAND, p.tiles_k - band * WG_BAND);
  const int tn = r / width;
  n0 = tn * kWgTile[WIDE].n;
  k0 = (band * WG_BAND + (r - tn * width)) * kWgTile[WIDE].k;
}

// First (tile, row block) of worker w's run over the dealt-out tiles, counted
// from the first of them: runs differ by one block at most, the longer first.
__device__ __forceinline__ long long wg_run(const WeightGradTc& p, int w) {
  return p.run_len * w + min(w, p.run_longer);
}
// The dealt-out tile a position lies in (a 64-bit division takes as long as
// half a stage's product).
__device__ __forceinline__ int wg_run_tile(const WeightGradTc& p, long long pos) {
  if (pos <= 0xffffffffll) return static_cast<int>(static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.kblocks));
  return static_cast<int>(pos / p.kblocks);
}

// A worker's pieces in order; every role walks the same list.
template <bool WIDE>
struct WgWalk {
  int w, next_tile;
  long long pos, end;
  bool first;
  __device__ __forceinline__ explicit WgWalk(const WeightGradTc& p)
      : w(blockIdx.x >> 1), next_tile(blockIdx.x >> 1), pos(wg_run(p, w)), end(wg_run(p, w + 1)), first(true) {}
  __device__ __forceinline__ bool next(const WeightGradTc& p, WgUnit& u) {
    if (next_tile < p.whole_tiles) {
      wg_tile<WIDE>(p, next_tile, u.n0, u.k0);
      u.kb0 = 0;
      u.kb1 = p.kblocks;
      u.slot = -1;
      next_tile += p.workers;
      return true;
    }
    if (pos >= end) return false;
    const int t = wg_run_tile(p, pos);
    const long long base = static_cast<long long>(t) * p.kblocks;
    wg_tile<WIDE>(p, p.whole_tiles + t, u.n0, u.k0);
    u.kb0 = static_cast<int>(pos - base);
    u.kb1 = static_cast<int>(min(end - base, static_cast<long long>(p.kblocks)));
    u.slot = (u.kb0 == 0 && u.kb1 == p.kblocks) ? -1 : 2 * w + (first ? 0 : 1);
    first = false;
    pos = base + u.kb1;
    return true;
  }
};

// A warp's 32 x 32 block of sums, lane = row, to memory.  Stored from where it
// is, every instruction would touch 32 rows (a drain of 8.8 us for a pair's
// tile); so the 8-column pieces are first transposed among each four lanes
// (two butterfly steps), after which lane l holds piece l % 4 of rows l & ~3
// .. + 3 and an instruction fills whole 128-byte lines of 8 rows (fp32).
__device__ __forceinline__ void transpose_pieces(float (&v)[4][8], int lane) {
#pragma unroll
  for (int b = 1; b <= 2; b <<= 1) {
    const bool up = lane & b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & b) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float send = up ? v[i][k] : v[i | b][k];
        const float recv = __shfl_xor_sync(0xffffffffu, send, b);
        if (up) v[i][k] = recv;
        else v[i | b][k] = recv;
      }
    }
  }
}

// The whole block transposed, lane = column, for rows that whole accesses do not
// fit: single stores then adjoin across the warp (one row per instruction).
__device__ __forceinline__ void transpose_block(float (&v)[32], int lane) {
#pragma unroll
  for (int b = 16; b > 0; b >>= 1) {
    const bool up = lane & b;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i & b) continue;
      const float send = up ? v[i] : v[i | b];
      const float recv = __shfl_xor_sync(0xffffffffu, send, b);
      if (up) v[i] = recv;
      else v[i | b] = recv;
    }
  }
}

// dst <- (dst +) 8 columns of one row, accessed whole.
template <typename G>
__device__ __forceinline__ void store_piece(G* dst, float (&v)[8], bool accumulate) {
  if (accumulate) {
    float o[8];
    load8(dst, o);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += o[k];
  }
  store8(dst, v);
}

__device__ __forceinline__ void wg_timeout(unsigned int* status, volatile int* abort_flag) {
  *abort_flag = 1;
  atomicOr(status, kTimeout);
}

// Arrive on the leader's barrier for shared memory that this warp has written
// and passed to the async proxy.  Release at CTA scope: what the leader's
// product reads are this CTA's own shared-memory writes, in place before the
// arrival is sent.  A release at cluster scope would also wait for the
// thread's accesses to global memory, 0.6 us a stage.
__device__ __forceinline__ void arrive_leader(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

template <typename G, bool WIDE>
__global__ void __launch_bounds__(WG_THREADS, 1) weight_grad_tc_kernel(const __grid_constant__ WeightGradTc p) {
  using C = WgCfg<WIDE>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_a = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);   // leader's: both CTAs' dy
  uint64_t* full_q = full_a + C::STAGES;                               // this CTA's codes
  uint64_t* ready = full_q + C::STAGES;                                // leader's: both CTAs' restored x
  uint64_t* empty = ready + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;                                 // accumulator complete
  uint64_t* tempty = tfull + 1;                                        // leader's: both CTAs' drained
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(sm100::cluster_ctarank());

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      sm100::mbar_init(&full_a[s], 1);
      sm100::mbar_init(&full_q[s], 1);
      sm100::mbar_init(&ready[s], 2 * C::GROUP_WARPS);
      sm100::mbar_init(&empty[s], 1);
    }
    sm100::mbar_init(tfull, 1);
    sm100::mbar_init(tempty, 2 * WG_WARPS);
    *abort_flag = 0;
    sm100::fence_mbar_init();
    sm100::prefetch_tmap(&p.tm_dy);
    sm100::prefetch_tmap(&p.tm_q);
  }
  if (warp == 1) {
    sm100::tmem_alloc_pair(tmem_slot, C::TMEM);
    sm100::tmem_relinquish_pair();
  }
  sm100::tc_fence_before();
  __syncwarp();
  sm100::cluster_sync();
  sm100::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  // a wait that gives up does so seconds after this
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;

  WgWalk<WIDE> walk(p);
  WgUnit u;
  if (warp == 0) {
    // ------------------------------------------------------- TMA producer
    if (lane == 0) {
      const int last_plane = p.kblocks / p.row_blocks - 1;
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      while (ok && walk.next(p, u)) {
        const int nact = C::SUBS == 2 && u.n0 + 256 < p.n ? 2 : 1;   // halves of the tile with columns of dy
        const int kcol = u.k0 + rank * C::CODES;
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          if (!sm100::mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
            wg_timeout(p.status, abort_flag);
            ok = false;
            break;
          }
          const int pass = kb / p.row_blocks, plane = last_plane - pass;
          const int t0 = (kb - pass * p.row_blocks) * WG_BK;
          uint8_t* sa = smem + stage * C::STAGE;
          uint8_t* sq = sa + C::A_BYTES + C::B_BYTES;
          sm100::mbar_arrive_expect_tx(&full_q[stage], C::Q_BYTES);
          if (rank == 0) sm100::mbar_arrive_expect_tx(&full_a[stage], 2 * nact * WG_SUB_BYTES);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          sm100::tma_load_3d(sq, &p.tm_q, &full_q[stage], kcol, t0, 0);
          const uint32_t bar = sm100::mapa_shared(sm100::smem_u32(&full_a[stage]), 0);
          for (int h = 0; h < nact; ++h) {
            const int col = u.n0 + h * 256 + rank * 128;
            uint8_t* dst = sa + h * WG_SUB_BYTES;
            if (p.chunked) {
              sm100::tma_load_4d_pair(dst, &p.tm_dy, bar, 0, t0, col / 64, plane);
            } else {
              sm100::tma_load_3d_pair(dst, &p.tm_dy, bar, col, t0, plane);
              sm100::tma_load_3d_pair(dst + WG_CHUNK, &p.tm_dy, bar, col + 64, t0, plane);
            }
          }
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // let every load issued into this CTA's shared memory land before exit
        for (int s = 0; s < C::STAGES; ++s) {
          if (!((issued >> s) & 1u)) continue;
          const uint64_t t = sm100::globaltimer();
          while ((!sm100::mbar_try_wait(&full_q[s], (issued_phase >> s) & 1u) ||
                  (rank == 0 && !sm100::mbar_try_wait(&full_a[s], (issued_phase >> s) & 1u))) &&
                 sm100::globaltimer() - t < 100000000ull) {
          }
        }
        // the second CTA's dy signals the leader's barriers, which it cannot wait
        // on, in phases that the leader may not have begun: a load takes
        // microseconds, so a millisecond stands for its landing
        const uint64_t t = sm100::globaltimer();
        while (rank != 0 && sm100::globaltimer() - t < 1000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = sm100::make_idesc_bf16(256, C::TK, 1, 1);
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      while (ok && walk.next(p, u)) {
        const int nact = C::SUBS == 2 && u.n0 + 256 < p.n ? 2 : 1;
        if (!sm100::mbar_wait(tempty, acc_phase ^ 1u, abort_flag)) {
          wg_timeout(p.status, abort_flag);
          break;
        }
        sm100::tc_fence_after();
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          if (!sm100::mbar_wait(&full_a[stage], phase, abort_flag) ||
              !sm100::mbar_wait(&ready[stage], phase, abort_flag)) {
            wg_timeout(p.status, abort_flag);
            ok = false;
            break;
          }
          sm100::tc_fence_after();
          const uint32_t sa = sm100::smem_u32(smem + stage * C::STAGE);
          const uint64_t ad = sm100::make_sdesc(sa, WG_CHUNK, 1024);
          const uint64_t bd = sm100::make_sdesc(sa + C::A_BYTES, WG_CHUNK, 1024);
#pragma unroll
          for (int kk = 0; kk < WG_BK / 16; ++kk)
#pragma unroll
            for (int h = 0; h < C::SUBS; ++h)
              if (h < nact)
                sm100::umma_bf16_pair(tmem + static_cast<uint32_t>(h * C::TK),
                                      ad + static_cast<uint64_t>((h * WG_SUB_BYTES + kk * 2048) >> 4),
                                      bd + static_cast<uint64_t>((kk * 2048) >> 4), idesc,
                                      (kb > u.kb0 || kk) ? 1u : 0u);
          sm100::umma_commit_pair_both(&empty[stage]);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        sm100::umma_commit_pair_both(tfull);
        acc_phase ^= 1u;
      }
    }
  } else {
    // ---------------------------------------- codes to bf16, then the tile
    // thread j of a group restores codes 16 (j % ROW_TASKS) .. + 15 of row
    // j / ROW_TASKS of the group's stages
    const int group = (warp - 2) / C::GROUP_WARPS;
    const int j = threadIdx.x - 64 - group * C::GROUP_WARPS * 32;
    const int f = j % C::ROW_TASKS, t = j / C::ROW_TASKS;
    // Their place: chunk f / 4, units 2 (f % 4) and the next.  Where 8 lanes
    // share a row, the upper chunk's write their two units in the other order,
    // so that 8 neighbouring lanes always touch 8 different 16-byte columns
    // (where 4 do, the swizzle of the two rows sees to it).
    const int swap = f >> 2;
    const uint32_t src = C::A_BYTES + C::B_BYTES + t * C::CODES + f * 16;
    const uint32_t dst = C::A_BYTES + (f >> 2) * WG_CHUNK + t * 128;
    const uint32_t dst0 = dst + ((((f & 3) * 2 + swap) ^ (t & 7)) << 4);
    const uint32_t dst1 = dst + ((((f & 3) * 2 + 1 - swap) ^ (t & 7)) << 4);
    const uint32_t ready0 = sm100::mapa_shared(sm100::smem_u32(ready), 0);
    const uint32_t tempty0 = sm100::mapa_shared(sm100::smem_u32(tempty), 0);
    const int quad = warp & 3, slice = (warp - 2) >> 2;
    constexpr int CH = C::TK / 32;
    const bool vec = p.k % 8 == 0 && reinterpret_cast<uintptr_t>(p.grad) % (8 * sizeof(G)) == 0;
    int stage = 0, turn = 0;   // ring position of the unit's first stage, and whose it is
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    while (ok && walk.next(p, u)) {
      const int blk = (u.k0 + rank * C::CODES) / kCkptBlock;
      // Exponents of the group's stages in the order of the unit's row blocks;
      // 127 (any finite one) where the tensor map loads zeros.  Read four
      // stages at a time, four ahead: a register that a load is still filling
      // must not be touched, a copy included, or the stage waits out the load.
      const int lead = (group + C::GROUPS - turn) % C::GROUPS;   // the group's first stage of the unit
      int tb = (u.kb0 + lead) % p.row_blocks;
      auto exponent = [&]() -> int {
        const long long row = static_cast<long long>(tb) * WG_BK + t;
        tb += C::GROUPS;
        while (tb >= p.row_blocks) tb -= p.row_blocks;
        return (row < p.rows && blk < p.nblk) ? p.exps[row * p.nblk + blk] : 127;
      };
      int e[4], e_next[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = exponent();
      auto advance = [&](int by) {   // by <= STAGES
        stage += by;
        if (stage >= C::STAGES) {
          stage -= C::STAGES;
          phase ^= 1u;
        }
      };
      auto retreat = [&](int by) {
        stage -= by;
        if (stage < 0) {
          stage += C::STAGES;
          phase ^= 1u;
        }
      };
      advance(lead);
      int kb = u.kb0 + lead;
      for (; ok && kb < u.kb1;) {
#pragma unroll
        for (int i = 0; i < 4; ++i) e_next[i] = exponent();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (kb >= u.kb1) break;
          if (!__all_sync(0xffffffffu, sm100::mbar_wait(&full_q[stage], phase, abort_flag))) {
            if (lane == 0) wg_timeout(p.status, abort_flag);
            ok = false;
            break;
          }
          uint8_t* base = smem + stage * C::STAGE;
          const uint4 q = *reinterpret_cast<const uint4*>(base + src);
          uint4 lo, hi;
          restore16(q, e[i], lo, hi);
          *reinterpret_cast<uint4*>(base + dst0) = swap ? hi : lo;
          *reinterpret_cast<uint4*>(base + dst1) = swap ? lo : hi;
          sm100::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) arrive_leader(ready0 + stage * 8);
          advance(C::GROUPS);
          kb += C::GROUPS;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = e_next[i];
      }
      // kb is the group's first stage past the unit: back to the unit's end
      retreat(kb - u.kb1);
      turn = (turn + (u.kb1 - u.kb0)) % C::GROUPS;
      if (!ok) break;
      if (!__all_sync(0xffffffffu, sm100::mbar_wait(tfull, acc_phase, abort_flag))) {
        if (lane == 0) wg_timeout(p.status, abort_flag);
        break;
      }
      sm100::tc_fence_after();
      acc_phase ^= 1u;
      const int nact = C::SUBS == 2 && u.n0 + 256 < p.n ? 2 : 1;
#pragma unroll 1
      for (int c = slice; c < CH * nact; c += 4) {   // 32-column chunks of the accumulator columns
        const int col = u.k0 + (c % CH) * 32;
        if (col >= p.k) continue;
        uint32_t r[32];
        sm100::tmem_ld32_async(tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(c * 32), r);
        sm100::tmem_wait_ld(r);
        // features 1 and 2 of every four back in place
        auto sum = [&](int k) { return __uint_as_float(r[(k & 3) == 1 ? k + 1 : (k & 3) == 2 ? k - 1 : k]); };
        const int row0 = u.n0 + (c / CH) * 256 + rank * 128 + quad * 32;
        G* grad = static_cast<G*>(p.grad);
        if (vec || u.slot >= 0) {
          float v[4][8];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k >> 3][k & 7] = sum(k);
          transpose_pieces(v, lane);
          const int c0 = col + (lane & 3) * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = row0 + (lane & ~3) + i;
            if (row >= p.n || c0 >= p.k) continue;
            if (u.slot >= 0)
              store8(p.partial + (static_cast<long long>(u.slot) * C::TN + (row - u.n0)) * C::TK + (c0 - u.k0), v[i]);
            else
              store_piece(grad + static_cast<long long>(row) * p.k + c0, v[i], p.accumulate != 0);
          }
        } else {
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = sum(k);
          transpose_block(v, lane);
          if (col + lane < p.k) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if (row0 + k >= p.n) break;
              G* dst = grad + static_cast<long long>(row0 + k) * p.k + col + lane;
              *dst = from_f32<G>(v[k] + (p.accumulate ? to_f32(*dst) : 0.f));
            }
          }
          __syncwarp();
        }
      }
      sm100::tc_fence_before();
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive_cluster(tempty0);
    }
  }

  sm100::tc_fence_before();
  __syncwarp();
  sm100::cluster_sync();
  sm100::tc_fence_after();
  pdl_launch_dependents();
  if (warp == 1) {
    __syncwarp();
    sm100::tmem_dealloc_pair(tmem, C::TMEM);
  }
}

// grad (+)= the runs' sums of each tile that several workers share, in the
// order of their rows.  Block (b, y): the tile that the start of worker b + 1's
// run lies inside, if it is the first start inside it; 4096 elements, kJoinRows
// rows per thread so that their loads are in flight together.
constexpr int kJoinRows = 4;
template <typename G, bool WIDE>
__global__ void __launch_bounds__(256) weight_grad_join_kernel(const __grid_constant__ WeightGradTc p) {
  using C = WgCfg<WIDE>;
  pdl_launch_dependents();
  pdl_wait();
  const int w1 = blockIdx.x + 1;
  const long long at = wg_run(p, w1);
  const int t = wg_run_tile(p, at);
  const long long t0 = static_cast<long long>(t) * p.kblocks, t1 = t0 + p.kblocks;
  if (at == t0 || wg_run(p, w1 - 1) > t0) return;
  int n0, k0;
  wg_tile<WIDE>(p, p.whole_tiles + t, n0, k0);
  int w_end = w1 + 1;
  while (w_end < p.workers && wg_run(p, w_end) < t1) ++w_end;
  // slot 0 of a worker holds the tile its run starts in: of the first worker
  // here only if its run starts with the tile
  const int first_slot = 2 * (w1 - 1) + (wg_run(p, w1 - 1) >= t0 ? 0 : 1);
  constexpr int QUADS = C::TK / 4;   // threads per row
  constexpr int ROWS = 256 / QUADS;  // rows at a time
  const int c = (threadIdx.x % QUADS) * 4, col = k0 + c;
  if (col >= p.k) return;
  float s[kJoinRows][4] = {};
  const float* part = p.partial + static_cast<long long>(blockIdx.y * kJoinRows * ROWS + threadIdx.x / QUADS) * C::TK + c;
  constexpr long long SLOT = static_cast<long long>(C::TN) * C::TK;
  for (int w = w1 - 1; w < w_end; ++w) {
    const float* src = part + (w == w1 - 1 ? first_slot : 2 * w) * SLOT;
    float4 v[kJoinRows];
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) v[i] = *reinterpret_cast<const float4*>(src + i * ROWS * C::TK);
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) {
      s[i][0] += v[i].x;
      s[i][1] += v[i].y;
      s[i][2] += v[i].z;
      s[i][3] += v[i].w;
    }
  }
#pragma unroll
  for (int i = 0; i < kJoinRows; ++i) {
    const int row = n0 + (blockIdx.y * kJoinRows + i) * ROWS + threadIdx.x / QUADS;
    if (row >= p.n) break;
    G* out = static_cast<G*>(p.grad) + static_cast<long long>(row) * p.k + col;
    if (p.k % 4 == 0) {   // grad is 16-byte aligned
      if constexpr (sizeof(G) == 4) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.accumulate) o = *reinterpret_cast<const float4*>(out);
        *reinterpret_cast<float4*>(out) = make_float4(o.x + s[i][0], o.y + s[i][1], o.z + s[i][2], o.w + s[i][3]);
      } else {
        if (p.accumulate)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i][k] += to_f32(out[k]);
        const __nv_bfloat162 a = __floats2bfloat162_rn(s[i][0], s[i][1]), b = __floats2bfloat162_rn(s[i][2], s[i][3]);
        *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (col + k < p.k) out[k] = from_f32<G>(s[i][k] + (p.accumulate ? to_f32(out[k]) : 0.f));
    }
  }
}

// dy -> bf16 planes [planes][rows][pitch] (pitch a multiple of 64, zeros past
// n).  fp32: v = p0 + p1 + p2, each the 8 leading significant bits of what is
// left (cut, not rounded: nothing overflows, and 3 x 8 bits hold all 24 of a
// value from 2^-110 on; below, what is under 2^-133 is dropped);
// infinities and NaN go to plane 0 alone.
// A lane takes 8 columns, a warp 256 of a row.
template <typename D, int PLANES, bool VEC>
__global__ void __launch_bounds__(256) weight_grad_stage_kernel(const D* dy, long long dy_ld, __nv_bfloat16* out,
                                                                long long rows, int n, int pitch) {
  pdl_launch_dependents();
  pdl_wait();
  const long long t = static_cast<long long>(blockIdx.x) * blockDim.z + threadIdx.z;
  const int c = ((blockIdx.y * blockDim.y + threadIdx.y) * 32 + threadIdx.x) * 8;
  if (t >= rows || c >= pitch) return;
  float v[8] = {};
  if constexpr (VEC) {
    if (c < n) load8(dy + t * dy_ld + c, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + k < n) v[k] = to_f32(dy[t * dy_ld + c + k]);
  }
#pragma unroll
  for (int pl = 0; pl < PLANES; ++pl) {
    uint32_t b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      b[k] = isnan(v[k]) ? 0x7fffu : __float_as_uint(v[k]) >> 16;
      v[k] = isfinite(v[k]) ? v[k] - __uint_as_float(b[k] << 16) : 0.f;
    }
    *reinterpret_cast<uint4*>(out + (static_cast<long long>(pl) * rows + t) * pitch + c) =
        make_uint4(b[0] | (b[1] << 16), b[2] | (b[3] << 16), b[4] | (b[5] << 16), b[6] | (b[7] << 16));
  }
}

// ---------------------------------------------------------------- launchers
template <typename G, bool WIDE>
static cudaError_t tc_launch(const WeightGradTc& p, cudaStream_t s) {
  const auto kern = weight_grad_tc_kernel<G, WIDE>;
  const cudaError_t e = allow_smem(kern, WgCfg<WIDE>::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(WG_THREADS);
  cfg.dynamicSmemBytes = WgCfg<WIDE>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(2 * p.workers);
  return cudaLaunchKernelEx(&cfg, kern, p);
}
template <typename G, bool WIDE>
static cudaError_t join_launch(const WeightGradTc& p, cudaStream_t s) {
  const dim3 grid(p.workers - 1, WgCfg<WIDE>::TN * WgCfg<WIDE>::TK / (1024 * kJoinRows));
  return launch_pdl(weight_grad_join_kernel<G, WIDE>, grid, dim3(256), 0, s, p);
}
cudaError_t launch_weight_grad_tc(const WeightGradTc& p, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (p.wide) return p.grad_bf16 ? tc_launch<B, true>(p, s) : tc_launch<float, true>(p, s);
  return p.grad_bf16 ? tc_launch<B, false>(p, s) : tc_launch<float, false>(p, s);
}
cudaError_t launch_weight_grad_join(const WeightGradTc& p, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (p.wide) return p.grad_bf16 ? join_launch<B, true>(p, s) : join_launch<float, true>(p, s);
  return p.grad_bf16 ? join_launch<B, false>(p, s) : join_launch<float, false>(p, s);
}

cudaError_t launch_weight_grad_stage(const void* dy, int bf16, int vec, long long dy_ld, void* out, long long rows,
                                     int n, int pitch, cudaStream_t s) {
  const unsigned segs = static_cast<unsigned>((pitch + 255) / 256);
  unsigned wx = 1;
  while (wx < 8 && wx < segs) wx *= 2;
  const dim3 block(32, wx, 8 / wx), grid(static_cast<unsigned>((rows + block.z - 1) / block.z), (segs + wx - 1) / wx);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
  if (bf16)   // bf16 is staged because it cannot be read in whole accesses
    return launch_pdl(weight_grad_stage_kernel<__nv_bfloat16, 1, false>, grid, block, 0, s,
                      static_cast<const __nv_bfloat16*>(dy), dy_ld, o, rows, n, pitch);
  return launch_pdl(vec ? weight_grad_stage_kernel<float, 3, true> : weight_grad_stage_kernel<float, 3, false>, grid,
                    block, 0, s, static_cast<const float*>(dy), dy_ld, o, rows, n, pitch);
}

}  // namespace muon
