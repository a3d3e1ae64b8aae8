// dp_mx4mm.cu -- the FSDP forward's parameter all-gather fused into the local
// matmul, with both operands in microscaled 4-bit form, or x in 8 bits (below):
//   y[m, f] = tx * tw * sum_d sx[m, b(d)] x[m, d] * sw[f, b(d)] w[f, d]
// x, w: e2m1 values; sx, sw: their blocks' scales (b(d) = d / 32 for mxfp4,
// d / 16 for nvfp4); tx, tw: the tensors' fp32 scales (nvfp4).  The tensor
// cores multiply the scaled values exactly and accumulate in fp32
// (tcgen05.mma with block_scale, 64 values of d at a time); tx tw multiplies
// the fp32 sum once.  The gathered w is never materialised.
//
// The product runs transposed, y^T = w x^T: the 128 TMEM lanes are weight
// rows f and the columns are tokens.  So a tile always lies inside one shard,
// whatever F_shard is, few tokens make a narrow tile instead of an idle one
// (one token: 16 of the instruction's columns), and a warp's store covers 32
// consecutive f of a token.
//
// One CTA (512 threads) per SM, persistent over tiles of 128 f x BN tokens:
//   warp 0      W producer: 128 rows x 256 values (128 bytes) by TMA
//   warp 2      X producer: BN rows x 256 values; also allocates TMEM
//   warp 3      scales' producer: the rows' 512-byte scale tiles, 16 bytes a lane
//               by cp.async, ahead of the operands
//   warps 12-15 scales into TMEM: lane l of each 32-lane quarter takes row l of a
//               scale tile (16 bytes: four columns), tcgen05.st
//   warp 1      MMA issuer: four MMAs of 64 values a stage
//   warps 4-11  epilogue: a warp takes 32 f and half of the tokens, packs its
//               accumulator columns into registers, releases TMEM and stores
//               while the next tile runs
// TMEM: 256 accumulator columns (one tile) and 4 x 48 scale columns (narrow
// tiles: see Geo): a stage has its own, so they are overwritten only when the
// stage is.  With the scales two accumulators of 256 columns do not fit.
//
// Measured (GB300, launches in a CUDA graph): x[8192,4096] . w[4096,4096]^T
// 50 us in mxfp4 (5.5 PFLOP/s) and 58 us in nvfp4 (4.7); x[8192,8192] .
// w[8192,8192]^T 160 and 187 us (up to 200 on general values, which take more
// power).  What bounds it: the MMAs alone (loads of all
// stages but the first four left out) take 139 us of the 160; the rest is
// operand intake, 48 KiB of values a stage, and between tiles the 1300 clocks
// in which the accumulator is drained.  nvfp4 has twice the scales: reading
// them four times from shared memory, once for each quarter of TMEM, costs 20
// us of its 187.  The steps that led here, on that product:
//   * scales through registers (195 / 167 us, nvfp4 / mxfp4) instead of
//     tcgen05.cp straight from shared memory (269 / 204 us): the copies take
//     their turn with the MMAs, about 100 clocks each;
//   * scales to shared memory by cp.async instead of three bulk copies a stage:
//     233 -> 216 and 225 -> 195 us;
//   * output through 4 KiB of shared memory a half and TMA instead of 4-byte
//     stores, which held the MMA issuer up for half a tile.
//
// With x in 8 bits (e4m3, blocks of 32) and mxfp4 weights the MMA is the 8-bit kind,
// 32 values of d at a time: a stage is 128 values, of the same 128 bytes a row, and
// has a quarter of a scale tile a step.  That kind wants each sixteen 4-bit values in
// the first half of 16 bytes: TMA spreads them so (and counts the bytes that it
// read), where rows are whole 128 values and 32-byte aligned; else warp 0 copies
// them, 8 bytes a lane, and warp 3 hands a landed stage on to the MMA's proxy.
// Measured: x[8192,4096] . w[4096,4096]^T 83-85 us (3.3 PFLOP/s; 76 % of the tensor
// pipe, 62 % of L2), with all loads left out 76; x[8192,8192] . w[8192,8192]^T 360.
// What bounds it is the intake, 40 KiB for the 512 clocks that a stage's MMAs take,
// and the MMAs.  All weights by warp 0's copies: 105 us (their half-used lines do
// not stay in the L1 that is left beside the stages).  One token times
// w[65536,8192] 66 us, and without any load 65: an MMA takes 64 clocks to issue
// however narrow it is, so tiles are not narrower than 64 tokens.
//
// Few tiles: the blocks of d are split over a cluster of 2, 4 or 8 CTAs,
// whose fp32 partial sums meet in shared memory: each CTA adds a share of the
// tokens over the cluster in rank order (no atomics, no workspace).
//
// Every mbarrier wait is bounded; on expiry a role flags the error word and
// unwinds, and the cluster's barriers are still reached by every thread.

#include "dp_early.cuh"
#include "dp_launch.h"
#include "dp_mx4.cuh"
#include "dp_tc.cuh"

#include <algorithm>
#include <cstring>

namespace {

using namespace dpk;

constexpr int BM = 128;          // weight rows of a tile
constexpr int kRowBytes = 128;   // of an operand's row in a stage: one swizzle row
constexpr uint32_t kStageW = BM * kRowBytes;
constexpr uint32_t kStageSW = 4 * kScaleTile;  // 128 rows x 16 blocks (nvfp4)

// The operands: both mxfp4, both nvfp4, or mxfp4 weights with x in 8 bits (mxfp8).
enum { kMx4 = 0, kNv4 = 1, kMx8 = 2 };
template <int KIND>
struct Kind {
  static constexpr bool kPow2 = KIND != kNv4;                       // scales are powers of two
  static constexpr int kBlock = KIND == kNv4 ? kNvBlock : kMxBlock;
  static constexpr int kBK = KIND == kMx8 ? 128 : 256;              // values of d per stage
  static constexpr int kStep = kBK / 4;                             // ... per MMA
};
constexpr int kOutTokens = 16;   // tokens of one staged store of an epilogue half
constexpr uint32_t kStageY = kOutTokens * BM * 2;  // per half
constexpr size_t kBarBytes = 512;

// What follows from the widest tile (in tokens) of a kernel: a narrow tile's
// stages are small, and what bounds it is how many weight bytes are on their
// way.  Measured with 8 and 6 stages against 4 of the widest tile's: one token
// times w[65536,8192] in nvfp4 52.2 us (5.8 TB/s), against 55.7 us; 128 tokens
// times w[4096,4096] 8.9 us, against 9.7 us.
template <int BNMAX>
struct Geo {
  static constexpr int kStages = BNMAX == 256 ? 4 : BNMAX == 128 ? 6 : 8;
  static constexpr uint32_t kStageX = BNMAX * kRowBytes;
  static constexpr int kXTiles = BNMAX > 128 ? 2 : 1;  // 128-row scale tiles of X
  static constexpr uint32_t kStageSX = kXTiles * 4 * kScaleTile;
  static constexpr int kXCols = 4 * kXTiles;           // TMEM columns of a step's X scales
  static constexpr int kScaleCol0 = BNMAX;             // first scale column
  static constexpr int kScaleCols = 16 + 4 * kXCols;   // per stage: W's, then X's
  static constexpr size_t kSmem = 1024 +
                                  (size_t)kStages * (kStageW + kStageX + kStageSW + kStageSX) +
                                  2 * kStageY + kBarBytes;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
  static_assert(kScaleCol0 + kStages * kScaleCols <= 512, "TMEM columns");
  static_assert((uint32_t)BNMAX * BM * 4 <= kStages * (kStageW + kStageX), "partial sums");
  static_assert((4 * kStages + 2) * 8 + 8 <= kBarBytes, "barriers");
};

constexpr int kTmemCols = 512;
constexpr int kThreadsM = 512;
constexpr int kEpiWarps = 8;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kMaxSplit = 8;

struct Mx4mmParams {
  CUtensorMap tmX, tmY;
  CUtensorMap tmW[kMaxK];
  const uint8_t* w[kMaxK];  // codes (8-bit x; the 4-bit forms load them through tmW)
  const uint8_t* sx;
  const uint8_t* sw[kMaxK];
  const float* tx;
  const float* tw[kMaxK];
  void* y;
  unsigned* err;
  int M, D, K, F, F_shard;
  int BN;
  int tiles_m, tiles_f;   // tiles_f: of one shard
  int tile0, tiles;       // this launch's tiles
  int num_kb;
  int col_tiles;          // scale tiles along d
  int x_row_tiles;
  int split;              // CTAs of a cluster that share a tile
  int y_f32;
  int next_early;         // let the next kernel move in before this one's end
  int w_copies;           // 8-bit x: W comes by threads' copies instead of TMA
};

// Tile i of this launch.
struct Tile {
  int shard, f0, m0;
};
__device__ __forceinline__ Tile tile_at(const Mx4mmParams& p, int i) {
  const int tile = p.tile0 + i;
  const int ft = tile / p.tiles_m, mt = tile - ft * p.tiles_m;
  const int shard = ft / p.tiles_f;
  return Tile{shard, (ft - shard * p.tiles_f) * BM, mt * p.BN};
}

// ---- PTX wrappers ------------------------------------------------------------

// 16 bytes from global to shared memory by a thread, past L1; the arrival comes
// when all of the thread's copies so far have landed.
__device__ __forceinline__ void async_copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
// Sixteen 4-bit values to the first half of their 16 bytes.
__device__ __forceinline__ void async_copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void async_copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void async_copy_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Instruction descriptor of the block-scaled kinds: both operands K-major, A
// e2m1, B e2m1 or e4m3 (the 8-bit kind numbers its formats differently); scales
// ue8m0 or e4m3.
template <int KIND>
__device__ __forceinline__ uint32_t idesc_fp4(int n) {
  return ((KIND == kMx8 ? 5u : 1u) << 7)      // A format: e2m1
         | ((KIND == kMx8 ? 0u : 1u) << 10)   // B format: e4m3 / e2m1
         | ((uint32_t)(n >> 3) << 17)         // N >> 3
         | (Kind<KIND>::kPow2 ? 1u << 23 : 0u)  // scale format: ue8m0 / ue4m3
         | ((uint32_t)(BM >> 7) << 27); // M >> 7
}

// The MMA and its commits are run by a whole warp and issued by one elected
// lane: with every operand the same in all lanes the compiler keeps them in
// uniform registers.  Inside an if (lane == 0) each MMA took 73 clocks to
// issue, and a stage 788 clocks for 548 of MMAs (x[8192,8192] .
// w[8192,8192]^T, mxfp4: 194 us, against 166).
template <int KIND>
__device__ __forceinline__ void mma_fp4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t sa_tmem, uint32_t sb_tmem,
                                        uint32_t accumulate) {
  if constexpr (KIND == kMx8)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
  else if constexpr (KIND == kMx4)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void commit_elected(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ float2 ld_peer2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr)
               : "memory");
  return v;
}

// Barrier among the 128 threads of an epilogue half.
__device__ __forceinline__ void half_barrier(int half) {
  asm volatile("bar.sync %0, 128;" ::"r"(half + 1) : "memory");
}

// ... that tells all of them whether one of them has `v`.
__device__ __forceinline__ bool half_any(int half, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.or.pred po, %2, 128, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(half + 1)
      : "memory");
  return r != 0;
}

template <int KIND, int BNMAX>
__global__ void __launch_bounds__(kThreadsM, 1) mx4mm_kernel(const __grid_constant__ Mx4mmParams p) {
  using G = Geo<BNMAX>;
  constexpr int kStages = G::kStages, kXCols = G::kXCols;
  constexpr uint32_t kStageX = G::kStageX, kStageSX = G::kStageSX;
  constexpr int kScaleCol0 = G::kScaleCol0, kScaleCols = G::kScaleCols;
  constexpr int kHalfChunks = BNMAX / 32;  // chunks of 16 tokens of an epilogue half, at most
  constexpr bool X8 = KIND == kMx8;
  constexpr int BK = Kind<KIND>::kBK, kStep = Kind<KIND>::kStep;
  constexpr int kTilesKb = BK / (4 * Kind<KIND>::kBlock);  // scale tiles of a stage along d
  constexpr uint32_t kScaleKb = kTilesKb * kScaleTile;  // bytes, of 128 rows
  const bool copies = X8 && p.w_copies;
  extern __shared__ unsigned char smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sW = smem;
  uint8_t* sX = sW + kStages * kStageW;
  uint8_t* sSW = sX + kStages * kStageX;
  uint8_t* sSX = sSW + kStages * kStageSW;
  uint8_t* sY = sSX + kStages * kStageSX;
  uint64_t* full = reinterpret_cast<uint64_t*>(sY + 2 * kStageY);
  uint64_t* empty = full + kStages;
  uint64_t* sfull = empty + kStages;    // a stage's scales (and W, if by copies) are in shared memory
  uint64_t* sempty = sfull + kStages;   // ... and have been read from it
  uint64_t* tmem_full = sempty + kStages;
  uint64_t* tmem_empty = tmem_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tmem_empty + 1);
  volatile int* aborted = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = p.split > 1 ? cluster_rank() : 0;
  const int first = (int)blockIdx.x / p.split;
  const int stride = p.split > 1 ? p.tiles : (int)gridDim.x;  // a cluster runs one tile
  const int kb_lo = (int)rank * p.num_kb / p.split;
  const int kb_hi = ((int)rank + 1) * p.num_kb / p.split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 6);  // W, X, and the four scale warps
      mbar_init(&empty[s], 1);
      mbar_init(&sempty[s], 4);  // one arrival per scale warp
      mbar_init(&sfull[s], 32);  // each lane of warp 3 (W by copies: 0), when its copies have landed
    }
    mbar_init(tmem_full, 1);
    mbar_init(tmem_empty, kEpiWarps);
    *aborted = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
            smem_u32(tmem_slot)),
        "r"(kTmemCols)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    prefetch_map(&p.tmX);
    if (!p.y_f32) prefetch_map(&p.tmY);
  }
  if (!copies && warp == 0 && lane < p.K) prefetch_map(&p.tmW[lane]);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // the launch may begin while the kernel before it in the stream (the
  // quantisation of x) still runs: nothing of global memory is touched before
  // that one has ended
  wait_stream();

  if (copies && warp == 0) {
    // ------------------------------ W by copies -------------------------------
    // What TMA does for the 8-bit kind where its rules (rows of whole 128 values)
    // do not hold: sixteen 4-bit values go to the first 8 bytes of 16, so each lane
    // copies 8 bytes to where the swizzle puts their 16.  Rows past the shard's end
    // read its last and are dropped; what lies past D belongs to no step.
    int stage = 0;
    uint32_t phase = 0;
    const int c = lane & 7, r0 = lane >> 3;  // chunk of the row, first row of every four
    const size_t row = (size_t)(p.D / 2);
    const uint32_t at = (uint32_t)(r0 * kRowBytes);
    const uint32_t even = at + (uint32_t)((c ^ r0) << 4), odd = at + (uint32_t)((c ^ (r0 + 4)) << 4);
    for (int i = first; i < p.tiles && !__any_sync(0xffffffffu, *aborted); i += stride) {
      const Tile t = tile_at(p, i);
      const uint8_t* tile = p.w[t.shard] + (size_t)t.f0 * row + c * 8;
      const int last = p.F_shard - 1 - t.f0;
      const uint8_t* gw =
          p.sw[t.shard] + (size_t)(t.f0 / kScaleRows) * p.col_tiles * kScaleTile + lane * 16;
      const int x0 = t.m0 / kScaleRows;
      const uint8_t* gx = p.sx + (size_t)x0 * p.col_tiles * kScaleTile + lane * 16;
      const int rows =
          min((t.m0 % kScaleRows + p.BN + kScaleRows - 1) / kScaleRows, p.x_row_tiles - x0);
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        const bool ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, p.err, kTimeoutNs);
        if (!__all_sync(0xffffffffu, ok)) {
          *aborted = 1;
          break;
        }
        if (kb * BK + c * 16 < p.D) {
          const uint32_t to = smem_u32(sW + stage * kStageW);
          const uint8_t* from = tile + kb * (BK / 2);
          if (last >= BM - 1) {
            from += r0 * row;
#pragma unroll
            for (int j = 0; j < BM / 4; ++j, from += 4 * row)
              async_copy8(to + (uint32_t)(j * 4 * kRowBytes) + (j & 1 ? odd : even), from);
          } else {
#pragma unroll 8
            for (int j = 0; j < BM / 4; ++j)
              async_copy8(to + (uint32_t)(j * 4 * kRowBytes) + (j & 1 ? odd : even),
                          from + (size_t)min(4 * j + r0, last) * row);
          }
        }
        // the stage's scales with it: they have been read where the stage is empty
        if (kb < p.col_tiles) {
          async_copy16(sSW + stage * kStageSW + lane * 16, gw + (size_t)kb * kScaleTile);
          async_copy16(sSX + stage * kStageSX + lane * 16, gx + (size_t)kb * kScaleTile);
          if (G::kXTiles > 1 && rows > 1)
            async_copy16(sSX + stage * kStageSX + kScaleKb + lane * 16,
                         gx + ((size_t)p.col_tiles + kb) * kScaleTile);
        }
        async_copy_arrive(&sfull[stage]);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (lane == 0 && p.next_early) let_next_start();
    async_copy_wait_all();  // no copy outlives the CTA
  } else if (warp == 0 || warp == 2) {
    // ------------------------------ producers ---------------------------------
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t armed_phase[kStages];
      bool armed[kStages];
      for (int s = 0; s < kStages; ++s) armed[s] = false;
      for (int i = first; i < p.tiles && !*aborted; i += stride) {
        const Tile t = tile_at(p, i);
        for (int kb = kb_lo; kb < kb_hi; ++kb) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, p.err, kTimeoutNs)) {
            *aborted = 1;
            break;
          }
          if (warp == 0) {
            // (8-bit x: half of the bytes, which TMA spreads over the stage's)
            mbar_arrive_expect_tx(&full[stage], X8 ? kStageW / 2 : kStageW);
            tma_load_2d(&p.tmW[t.shard], &full[stage], sW + stage * kStageW, kb * 128, t.f0);
          } else {
            mbar_arrive_expect_tx(&full[stage], (uint32_t)p.BN * kRowBytes);
            tma_load_2d(&p.tmX, &full[stage], sX + stage * kStageX, kb * kRowBytes, t.m0);
          }
          armed[stage] = true;
          armed_phase[stage] = phase;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // the next kernel's CTAs may move in beside the last tile's end
      if (warp == 0 && p.next_early) let_next_start();
      // Drain: every load this thread issued has landed before the CTA exits.
      for (int s = 0; s < kStages; ++s)
        if (armed[s]) (void)mbar_wait_bounded(&full[s], armed_phase[s], p.err, kTimeoutNs);
    }
  } else if (copies && warp == 3) {
    // ------------------------------ W to the MMA's proxy ----------------------
    // W was written by threads' copies; the MMA sees them after this fence.
    int stage = 0;
    uint32_t phase = 0;
    for (int i = first; i < p.tiles && !__any_sync(0xffffffffu, *aborted); i += stride)
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        const bool ok = mbar_wait_bounded(&sfull[stage], phase, p.err, kTimeoutNs);
        if (!__all_sync(0xffffffffu, ok)) {
          *aborted = 1;
          break;
        }
        if (lane == 0) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          mbar_arrive(&full[stage]);
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
  } else if (warp == 3) {
    // ------------------------------ scales into shared memory -----------------
    int stage = 0;
    uint32_t phase = 0;
    for (int i = first; i < p.tiles && !__any_sync(0xffffffffu, *aborted); i += stride) {
      const Tile t = tile_at(p, i);
      const uint8_t* gw =
          p.sw[t.shard] + (size_t)(t.f0 / kScaleRows) * p.col_tiles * kScaleTile + lane * 16;
      const int r0 = t.m0 / kScaleRows;
      const uint8_t* gx = p.sx + (size_t)r0 * p.col_tiles * kScaleTile + lane * 16;
      const int rows =
          min((t.m0 % kScaleRows + p.BN + kScaleRows - 1) / kScaleRows, p.x_row_tiles - r0);
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        const bool ok = mbar_wait_bounded(&sempty[stage], phase ^ 1u, p.err, kTimeoutNs);
        if (!__all_sync(0xffffffffu, ok)) {
          *aborted = 1;
          break;
        }
        uint8_t* dw = sSW + stage * kStageSW + lane * 16;
        uint8_t* dx = sSX + stage * kStageSX + lane * 16;
#pragma unroll
        for (int j = 0; j < kTilesKb; ++j) {
          const int c = kb * kTilesKb + j;
          if (c < p.col_tiles) {  // the last stage may end early
            async_copy16(dw + j * kScaleTile, gw + (size_t)c * kScaleTile);
            async_copy16(dx + j * kScaleTile, gx + (size_t)c * kScaleTile);
            if (G::kXTiles > 1 && rows > 1)
              async_copy16(dx + kScaleKb + j * kScaleTile,
                           gx + ((size_t)p.col_tiles + c) * kScaleTile);
          }
        }
        async_copy_arrive(&sfull[stage]);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    async_copy_wait_all();  // no copy outlives the CTA
  } else if (warp == 1) {
    // ------------------------------ MMA issuer --------------------------------
    const uint32_t idesc = idesc_fp4<KIND>(p.BN);
    const uint64_t a0 = sw128_kmajor_desc(smem_u32(sW)), b0 = sw128_kmajor_desc(smem_u32(sX));
    int stage = 0, w = 0;
    uint32_t phase = 0;
    bool issued = false;
    for (int i = first; i < p.tiles && !__any_sync(0xffffffffu, *aborted); i += stride, ++w) {
      // the first stage first: it is there long before the accumulator is free
      bool ready = true;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[stage], phase, p.err, kTimeoutNs) &&
                                       mbar_wait_bounded(tmem_empty, ((uint32_t)w & 1u) ^ 1u,
                                                         p.err, kTimeoutNs))) {
        *aborted = 1;
        break;
      }
      tc_fence_after();
      bool ok = true;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        if (!ready && !__all_sync(0xffffffffu, mbar_wait_bounded(&full[stage], phase, p.err,
                                                                 kTimeoutNs))) {
          *aborted = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t a = a0 + (uint32_t)stage * (kStageW >> 4);
        const uint64_t b = b0 + (uint32_t)stage * (kStageX >> 4);
        const uint32_t tw = tmem_base + (uint32_t)(kScaleCol0 + stage * kScaleCols);
        const uint32_t tx = tw + 16u;
        const int steps = (p.D - kb * BK + kStep - 1) / kStep;  // the last stage may end early
        // step k: 32 bytes further along the rows.  nvfp4: its four scales
        // are a tile's; mxfp4: its two are half of a tile's, and with 8-bit x
        // its one a quarter, chosen by the scale ids of the descriptor
        constexpr int kPer = KIND == kNv4 ? 1 : X8 ? 4 : 2;  // steps of a scale tile
#define DP_STEP(k)                                                                          \
  mma_fp4<KIND>(tmem_base, a + 2u * (k), b + 2u * (k),                                      \
                idesc | (uint32_t)((k) % kPer * (4 / kPer)) * ((1u << 4) | (1u << 29)),     \
                tw + 4u * ((k) / kPer), tx + (uint32_t)kXCols * ((k) / kPer),               \
                (k) > 0 || kb > kb_lo ? 1u : 0u)
        if (steps >= 4) {
          DP_STEP(0);
          DP_STEP(1);
          DP_STEP(2);
          DP_STEP(3);
        } else {
          DP_STEP(0);
          if (steps > 1) DP_STEP(1);
          if (steps > 2) DP_STEP(2);
        }
#undef DP_STEP
        commit_elected(&empty[stage]);
        issued = true;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        // the MMAs are issued at about the rate at which they run, so what
        // comes between two stages' must be short: one look at the next one
        ready = __all_sync(0xffffffffu, mbar_test_wait(&full[stage], phase));
      }
      if (!ok) break;
      commit_elected(tmem_full);
    }
    // Drain: every MMA issued has completed before TMEM is freed.
    if (issued) {
      const int last = stage == 0 ? kStages - 1 : stage - 1;
      const uint32_t last_phase = stage == 0 ? phase ^ 1u : phase;
      (void)mbar_wait_bounded(&empty[last], last_phase, p.err, kTimeoutNs);
    }
  } else if (warp >= 12) {
    // ------------------------------ scales into TMEM --------------------------
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    int stage = 0;
    uint32_t phase = 0;
    for (int i = first; i < p.tiles && !__any_sync(0xffffffffu, *aborted); i += stride) {
      const int turn = tile_at(p, i).m0 % kScaleRows / 32;  // 0 unless tiles are 32 or 64 tokens
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        const bool ok = mbar_wait_bounded(&sfull[stage], phase, p.err, kTimeoutNs);
        if (!__all_sync(0xffffffffu, ok)) {
          *aborted = 1;
          break;
        }
        // this quarter's copy of each tile; a tile that the last stage lacks,
        // or a second row tile that X lacks, is stale and belongs to no step or
        // to no token
        const uint8_t* gw = sSW + stage * kStageSW + lane * 16;
        const uint8_t* gx = sSX + stage * kStageSX + lane * 16;
        const uint32_t tw = tmem_base + lanes + (uint32_t)(kScaleCol0 + stage * kScaleCols);
        uint32_t w[4 * kTilesKb], x[kXCols * kTilesKb];
#pragma unroll
        for (int t = 0; t < kTilesKb; ++t) {
          const uint4 a = *reinterpret_cast<const uint4*>(gw + t * kScaleTile);
          w[4 * t] = a.x, w[4 * t + 1] = a.y, w[4 * t + 2] = a.z, w[4 * t + 3] = a.w;
#pragma unroll
          for (int r = 0; r < G::kXTiles; ++r) {
            const uint4 b = *reinterpret_cast<const uint4*>(gx + r * kScaleKb + t * kScaleTile);
            const int o = kXCols * t + 4 * r;
            x[o] = b.x, x[o + 1] = b.y, x[o + 2] = b.z, x[o + 3] = b.w;
          }
        }
        if (G::kXTiles == 1 && turn) {  // a word is a group of 32 tokens: the tile's first one goes first
#pragma unroll
          for (int t = 0; t < kTilesKb; ++t) {
            const int o = kXCols * t;
            uint4 b = make_uint4(x[o], x[o + 1], x[o + 2], x[o + 3]);
            if (turn & 1) b = make_uint4(b.y, b.z, b.w, b.x);
            if (turn & 2) b = make_uint4(b.z, b.w, b.x, b.y);
            x[o] = b.x, x[o + 1] = b.y, x[o + 2] = b.z, x[o + 3] = b.w;
          }
        }
        if (!copies) {  // (else the scales came after the stage was empty)
          __syncwarp();
          if (lane == 0) mbar_arrive(&sempty[stage]);  // the next ones can come while these wait
          const bool free = mbar_wait_bounded(&empty[stage], phase ^ 1u, p.err, kTimeoutNs);
          if (!__all_sync(0xffffffffu, free)) {
            *aborted = 1;
            break;
          }
        }
        tc_fence_after();
        if constexpr (kTilesKb == 1)
          DP_TMEM_ST_X4(tw, w);
        else if constexpr (kTilesKb == 2)
          DP_TMEM_ST_X8(tw, w);
        else
          DP_TMEM_ST_X16(tw, w);
        if constexpr (kXCols * kTilesKb == 4) {
          DP_TMEM_ST_X4(tw + 16u, x);
        } else if constexpr (kXCols * kTilesKb == 8) {
          DP_TMEM_ST_X8(tw + 16u, x);
        } else {
          DP_TMEM_ST_X16(tw + 16u, x);
          if constexpr (kXCols * kTilesKb == 32) {
            const uint32_t* hi = x + 16;
            DP_TMEM_ST_X16(tw + 32u, hi);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[stage]);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    // ------------------------------ epilogue ----------------------------------
    const int quarter = warp & 3;          // the TMEM lanes this warp may read
    const int half = (warp - 4) >> 2;
    const int chunks = p.BN / 16;
    const int c0 = half ? (chunks + 1) / 2 : 0;
    const int cn = half ? chunks / 2 : (chunks + 1) / 2;  // chunks of 16 tokens, at most 8
    const int fl = quarter * 32 + lane;
    int w = 0;
    for (int i = first; i < p.tiles; i += stride, ++w) {
      const Tile t = tile_at(p, i);
      const int shard = t.shard, m0 = t.m0 + c0 * 16;
      float alpha = 1.0f;
      if constexpr (KIND == kNv4) {
        if (p.tx) alpha = *p.tx;
        if (p.tw[shard]) alpha = __fmul_rn(alpha, *p.tw[shard]);
      }
      // A wait that ran out is acted on where the half's threads next meet, so
      // that they leave together; until then nothing depends on what was read.
      const bool ok = mbar_wait_bounded(tmem_full, (uint32_t)w & 1u, p.err, kTimeoutNs);
      __syncwarp();
      tc_fence_after();
      const uint32_t tbase = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(c0 * 16);
      const int f = t.f0 + fl;                     // inside the shard
      const bool f_in = f < p.F_shard;
      if (p.split > 1 || p.y_f32) {
        // 32-bit values leave chunk by chunk: the partial sums of a split tile
        // as [token][128 f] to where the operands were (every MMA of this tile,
        // the CTA's only one, has completed), or y
        float* red = reinterpret_cast<float*>(smem) + c0 * 16 * BM + fl;
        float* y = static_cast<float*>(p.y) + (size_t)shard * p.F_shard + f;
        for (int c = 0; c < cn; ++c) {
          uint32_t r[16];
          DP_TMEM_LD_X16(tbase + (uint32_t)(c * 16), r);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const int m = m0 + c * 16 + q;
            if (p.split > 1)
              red[(c * 16 + q) * BM] = __uint_as_float(r[q]);
            else if (f_in && m < p.M)
              y[(size_t)m * p.F] = __fmul_rn(__uint_as_float(r[q]), alpha);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tmem_empty);
        if (half_any(half, !ok || *aborted)) {
          *aborted = 1;
          break;
        }
        continue;
      }
      // bf16: pairs of tokens are packed into a register as they are read, so
      // the accumulator is free again before the first store
      constexpr int kH = kHalfChunks > 1 ? kHalfChunks : 2;  // read two at a time
      uint32_t h[kH][8];
      const auto pack32 = [&](const uint32_t(&r)[32], int c) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float lo = __uint_as_float(r[e * 16 + 2 * q]);
            const float hi = __uint_as_float(r[e * 16 + 2 * q + 1]);
            h[c + e][q] = KIND != kNv4 ? pack_bf16x2_rn(lo, hi)
                             : pack_bf16x2_rn(__fmul_rn(lo, alpha), __fmul_rn(hi, alpha));
          }
      };
#pragma unroll
      for (int c = 0; c < kH; c += 2) {
        uint32_t r[32];
        if (c < cn) {  // an odd last chunk reads 16 columns too many, which stay unused
          DP_TMEM_LD_X32(tbase + (uint32_t)(c * 16), r);
          tmem_ld_wait();
          pack32(r, c);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tmem_empty);
      // 16 tokens at a time through the half's 4 KiB of shared memory, which
      // one thread stores as a box that ends where the shard and y do
      uint8_t* buf = sY + (uint32_t)half * kStageY;
      const bool leader = quarter == 0 && lane == 0;
      if (half_any(half, !ok || *aborted)) {
        *aborted = 1;
        break;
      }
#pragma unroll
      for (int c = 0; c < kHalfChunks; ++c)
        if (c < cn) {
          if (leader) bulk_wait_read0();  // the previous box has been read
          half_barrier(half);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint16_t* o = reinterpret_cast<uint16_t*>(buf) + (2 * q) * BM + fl;
            o[0] = (uint16_t)h[c][q];
            o[BM] = (uint16_t)(h[c][q] >> 16);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          half_barrier(half);
          if (leader && m0 + c * 16 < p.M) {
            tma_store_3d(&p.tmY, buf, t.f0, shard, m0 + c * 16);
            bulk_commit();
          }
        }
    }
    if (quarter == 0 && lane == 0) bulk_wait_all();  // written before the CTA leaves
  }

  __syncwarp();
  if (p.split > 1) {
    __syncthreads();
    cluster_barrier();  // every CTA's partial sums are in its shared memory
    const Tile t = tile_at(p, first);
    const int shard = t.shard, f0 = t.f0, m0 = t.m0;
    float alpha = 1.0f;
    if constexpr (KIND == kNv4) {
      if (p.tx) alpha = *p.tx;
      if (p.tw[shard]) alpha = __fmul_rn(alpha, *p.tw[shard]);
    }
    const int tokens = min(p.BN, p.M - m0);
    const int share = (tokens + p.split - 1) / p.split;
    const int lo = (int)rank * share, hi = min(tokens, lo + share);
    const uint32_t red = smem_u32(smem);
    for (int i = threadIdx.x; i < (hi - lo) * (BM / 2); i += kThreadsM) {
      const int f = f0 + (i & (BM / 2 - 1)) * 2, m = lo + i / (BM / 2);
      const uint32_t at = red + (uint32_t)(m * BM + (f - f0)) * 4u;
      float2 sum = ld_peer2(peer_addr(at, 0));
      for (int c = 1; c < p.split; ++c) {
        const float2 v = ld_peer2(peer_addr(at, (uint32_t)c));
        sum.x = __fadd_rn(sum.x, v.x);
        sum.y = __fadd_rn(sum.y, v.y);
      }
      if (f < p.F_shard) {
        const size_t o = (size_t)(m0 + m) * p.F + (size_t)shard * p.F_shard + f;
        sum.x = __fmul_rn(sum.x, alpha);
        sum.y = __fmul_rn(sum.y, alpha);
        if (p.y_f32)
          *reinterpret_cast<float2*>(static_cast<float*>(p.y) + o) = sum;
        else
          *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.y) + o) =
              pack_bf16x2_rn(sum.x, sum.y);
      }
    }
    cluster_barrier();  // no CTA leaves while another reads its shared memory
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kTmemCols)
                 : "memory");
  }
}

template <int KIND, int BNMAX>
cudaError_t launch_for(Mx4mmParams p, int tiles, const dph::DeviceInfo& dev, cudaStream_t s) {
  constexpr size_t kSmemBytes = Geo<BNMAX>::kSmem;
  auto kernel = mx4mm_kernel<KIND, BNMAX>;
  if (dph::prepare_kernel(reinterpret_cast<const void*>(kernel), kThreadsM, kSmemBytes,
                          dev.device) < 1)
    return cudaErrorInvalidConfiguration;
  const int limit = dph::gemm_cta_limit();
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreadsM);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  if (p.split == 1) {
    int grid = std::min(tiles, dev.sm_count);
    if (limit > 0) grid = std::min(grid, limit);
    p.tile0 = 0;
    p.tiles = tiles;
    cfg.gridDim = dim3((unsigned)grid);
    return cudaLaunchKernelEx(&cfg, kernel, p);
  }
  // under a CTA limit the clusters go in several launches (one cluster each at least)
  const int per = limit > 0 ? std::max(1, std::min(tiles, limit / p.split)) : tiles;
  for (int t = 0; t < tiles; t += per) {
    p.tile0 = t;
    p.tiles = std::min(per, tiles - t);
    cfg.gridDim = dim3((unsigned)(p.tiles * p.split));
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int KIND>
cudaError_t launch_mx4mm(const Mx4mmParams& p, int tiles, const dph::DeviceInfo& dev,
                         cudaStream_t s) {
  if (p.BN <= 32) return launch_for<KIND, 32>(p, tiles, dev, s);
  if (p.BN <= 128) return launch_for<KIND, 128>(p, tiles, dev, s);
  return launch_for<KIND, 256>(p, tiles, dev, s);
}

using dph::aligned;
using dph::clash;
using dph::Span;
using dph::span_of;

}  // namespace

namespace {

// The product's checks, on the host alone.  x8: x is in 8 bits.
dp_status_t check_args(const dp_mx4_t* x, int M, int D, const dp_mx4_t* w_shards, int K,
                       int F_shard, dp_mx4_format_t format, bool x8, void* y,
                       dp_dtype_t y_dtype) {
  if (!x || !w_shards || K < 1 || K > DP_MAX_K) return DP_ERR_INVALID_ARG;
  if (M < 0 || D < 0 || F_shard < 0) return DP_ERR_INVALID_ARG;
  if (format != DP_MXFP4 && format != DP_NVFP4) return DP_ERR_UNSUPPORTED;
  if (y_dtype != DP_FP32 && y_dtype != DP_BF16) return DP_ERR_UNSUPPORTED;
  if (D % 32 || F_shard % 16) return DP_ERR_UNSUPPORTED;
  if ((long long)K * F_shard > 0x7fffff00ll || M > 0x7fffff00 || D > 0x7fffff00)
    return DP_ERR_UNSUPPORTED;
  if (!aligned(y, 16)) return DP_ERR_UNSUPPORTED;
  const bool mx = format == DP_MXFP4;
  const size_t ysz = (size_t)M * K * F_shard * (y_dtype == DP_FP32 ? 4 : 2);
  if (!y && ysz) return DP_ERR_INVALID_ARG;
  const Span out = span_of(y, ysz);
  const auto check = [&](const dp_mx4_t& a, int rows, size_t row_bytes) -> dp_status_t {
    if (mx && a.tensor_scale) return DP_ERR_INVALID_ARG;
    if ((!a.codes || !a.scales) && rows && D) return DP_ERR_INVALID_ARG;
    if (!aligned(a.codes, 16) || !aligned(a.scales, 16) || !aligned(a.tensor_scale, 4))
      return DP_ERR_UNSUPPORTED;
    size_t sbytes = 0;
    dp_mx4_scales_size(rows, D, format, &sbytes);
    if (clash(out, span_of(a.codes, (size_t)rows * row_bytes)) ||
        clash(out, span_of(a.scales, sbytes)) ||
        (a.tensor_scale && clash(out, span_of(a.tensor_scale, 4))))
      return DP_ERR_ALIAS;
    return DP_OK;
  };
  dp_status_t st = check(*x, M, x8 ? D : D / 2);
  for (int k = 0; k < K && st == DP_OK; ++k) st = check(w_shards[k], F_shard, D / 2);
  return st;
}

// The launch parameters of a checked product; nothing is enqueued.  *tiles is
// 0 where there is nothing to multiply (then *zero_bytes of y are to be zeroed).
dp_status_t prepare(const dp_mx4_t* x, int M, int D, const dp_mx4_t* w_shards, int K, int F_shard,
                    dp_mx4_format_t format, bool x8, void* y, dp_dtype_t y_dtype,
                    dph::DeviceInfo* devp, Mx4mmParams* pp, int* tilesp, size_t* zero_bytes) {
  *tilesp = 0;
  *zero_bytes = 0;
  const int F = K * F_shard, block = mx4_block(format);
  const size_t ysz = (size_t)M * F * (y_dtype == DP_FP32 ? 4 : 2);
  if (M == 0 || F == 0) return DP_OK;
  dph::DeviceInfo& dev = *devp;
  if (!dph::current_device(&dev)) return DP_ERR_CUDA;
  if (D == 0) {
    *zero_bytes = ysz;
    return DP_OK;
  }
  if (dev.cc_major != 10 || dev.cc_minor != 3 || dev.smem_optin < Geo<256>::kSmem)
    return DP_ERR_UNSUPPORTED;

  Mx4mmParams& p = *pp;
  memset(&p, 0, sizeof p);
  p.M = M;
  p.D = D;
  p.K = K;
  p.F = F;
  p.F_shard = F_shard;
  p.tiles_f = (F_shard + BM - 1) / BM;
  const int all_f = K * p.tiles_f;
  // Tokens of a tile: the call's own up to 128, rounded up to the
  // instruction's 16, and beyond that 256; fewer, down to 32, while the tiles
  // would fill at most half of the SMs (a tile starts on one of the 32-row
  // groups of a scale tile).
  p.BN = M <= 128 ? (M + 15) / 16 * 16 : 256;
  const auto tiles_of = [&](int bn) { return (long long)all_f * ((M + bn - 1) / bn); };
  if (M > 128 && tiles_of(256) < dev.sm_count) p.BN = 128;
  // With 8-bit x, 64 at least: a step of d takes as long for 32 tokens (x[64,4096]
  // . w[4096,4096]^T 10.0 -> 8.8 us, 128 tokens 11.4 -> 10.9).
  while (p.BN > (x8 ? 64 : 32) && tiles_of(p.BN) * 2 <= dev.sm_count) p.BN = p.BN > 64 ? 64 : 32;
  p.tiles_m = (M + p.BN - 1) / p.BN;
  const int bk = x8 ? Kind<kMx8>::kBK : Kind<kMx4>::kBK;
  p.num_kb = (D + bk - 1) / bk;
  p.col_tiles = mx4_col_tiles(D, block);
  p.x_row_tiles = (M + kScaleRows - 1) / kScaleRows;
  if ((long long)all_f * p.tiles_m > 0x3fffffffll) return DP_ERR_UNSUPPORTED;
  const int tiles = all_f * p.tiles_m;
  // CTAs of a cluster that share a tile's blocks of d: as many as keep the
  // launch on the SMs and leave each a block.  Clusters of 8 on half of the SMs
  // at most: sixteen of them, 128 CTAs, do not all find eight free SMs that are
  // close enough, and the rest run after them (x[64,4096], 512 f: 13.3 us,
  // against 7.2 us with eight clusters of 8 for x[32,4096]).
  p.split = 1;
  while (p.split < kMaxSplit && p.num_kb >= p.split * 2 &&
         tiles * p.split * 2 <= (p.split == 4 ? dev.sm_count / 2 : dev.sm_count))
    p.split *= 2;
  // A kernel that moves in beside this one's shared memory keeps the little L1
  // that is left: the next product starts about 1 us earlier (128x512x512: 6.3
  // -> 5.0 us each; x[16,4096] 7.3 -> 6.6), but a next quantisation of a large x
  // runs slower by more (linear of x[512,4096]: 10.9 -> 12.0 us, x[8192,4096]:
  // 63 -> 70, x[128,4096]: 8.9 -> 9.3; x[128,512] and x[16,4096] gain as well).
  p.next_early = (size_t)M * (size_t)D <= (128u << 10);
  p.sx = static_cast<const uint8_t*>(x->scales);
  p.tx = x->tensor_scale;
  p.y = y;
  p.y_f32 = y_dtype == DP_FP32;
  p.err = dev.err_word;
  if (!p.y_f32 && !dpl::encode_output_shards(&p.tmY, y, M, K, F_shard, kOutTokens))
    return DP_ERR_UNSUPPORTED;
  if (!dpl::encode_kmajor_bytes(&p.tmX, x->codes, M, x8 ? D : D / 2, p.BN)) return DP_ERR_UNSUPPORTED;
  if (x8) {
    p.w_copies = D % 128 != 0;
    for (int k = 0; k < K; ++k) p.w_copies |= !aligned(w_shards[k].codes, 32);
  }
  for (int k = 0; k < K; ++k) {
    if (x8 ? !p.w_copies && !dpl::encode_kmajor_padded4(&p.tmW[k], w_shards[k].codes, F_shard, D, BM)
           : !dpl::encode_kmajor_bytes(&p.tmW[k], w_shards[k].codes, F_shard, D / 2, BM))
      return DP_ERR_UNSUPPORTED;
    p.w[k] = static_cast<const uint8_t*>(w_shards[k].codes);
    p.sw[k] = static_cast<const uint8_t*>(w_shards[k].scales);
    p.tw[k] = w_shards[k].tensor_scale;
  }
  *tilesp = tiles;
  return DP_OK;
}

dp_status_t enqueue(const Mx4mmParams& p, int tiles, size_t zero_bytes, int kind,
                    const dph::DeviceInfo& dev, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (zero_bytes)
    e = cudaMemsetAsync(p.y, 0, zero_bytes, s);
  else if (tiles)
    e = kind == kMx8   ? launch_mx4mm<kMx8>(p, tiles, dev, s)
        : kind == kMx4 ? launch_mx4mm<kMx4>(p, tiles, dev, s)
                       : launch_mx4mm<kNv4>(p, tiles, dev, s);
  return e == cudaSuccess ? DP_OK : DP_ERR_CUDA;
}

// The scratch of the call that quantises x: its codes, then its scales.
size_t codes_bytes(int M, size_t row_bytes) {
  return ((size_t)M * row_bytes + 255) / 256 * 256;
}

}  // namespace

namespace {

// The product of quantised operands.
dp_status_t product(const dp_mx4_t* x, int M, int D, const dp_mx4_t* w_shards, int K, int F_shard,
                    dp_mx4_format_t format, bool x8, void* y, dp_dtype_t y_dtype,
                    dp_stream_t stream) {
  dph::DeviceInfo dev;
  Mx4mmParams p;
  int tiles;
  size_t zero;
  dp_status_t st = check_args(x, M, D, w_shards, K, F_shard, format, x8, y, y_dtype);
  if (st == DP_OK)
    st = prepare(x, M, D, w_shards, K, F_shard, format, x8, y, y_dtype, &dev, &p, &tiles, &zero);
  if (st != DP_OK) return st;
  p.y = y;
  return enqueue(p, tiles, zero, x8 ? kMx8 : format == DP_MXFP4 ? kMx4 : kNv4, dev,
                 reinterpret_cast<cudaStream_t>(stream));
}

dp_status_t workspace_size(int M, int D, dp_mx4_format_t format, bool x8, size_t* bytes) {
  if (!bytes) return DP_ERR_INVALID_ARG;
  *bytes = 0;
  if (M < 0 || D < 0) return DP_ERR_INVALID_ARG;
  size_t scales = 0;
  const dp_status_t st = dp_mx4_scales_size(M, D, format, &scales);
  if (st != DP_OK) return st;
  *bytes = codes_bytes(M, x8 ? D : D / 2) + scales;
  return DP_OK;
}

// ... with x quantised on the way.
dp_status_t linear(const void* x, int M, int D, long long ld, dp_dtype_t x_dtype,
                   const float* x_scale, const dp_mx4_t* w_shards, int K, int F_shard,
                   dp_mx4_format_t format, bool x8, void* y, dp_dtype_t y_dtype, void* workspace,
                   size_t workspace_bytes, dp_stream_t stream) {
  size_t need = 0;
  dp_status_t st = workspace_size(M, D, format, x8, &need);
  if (st != DP_OK) return st;
  if (workspace_bytes < need || (!workspace && need)) return DP_ERR_INVALID_ARG;
  const dp_mx4_t q{workspace, static_cast<uint8_t*>(workspace) + codes_bytes(M, x8 ? D : D / 2),
                   x_scale};
  // everything is checked before the first launch; the workspace, written by
  // the quantisation, must leave the weights alone too, and y the unquantised x
  st = check_args(&q, M, D, w_shards, K, F_shard, format, x8, y, y_dtype);
  if (st != DP_OK) return st;
  const Span ws = span_of(workspace, need);
  size_t sbytes = 0;
  dp_mx4_scales_size(F_shard, D, format, &sbytes);
  for (int k = 0; k < K; ++k)
    if (clash(ws, span_of(w_shards[k].codes, (size_t)F_shard * (D / 2))) ||
        clash(ws, span_of(w_shards[k].scales, sbytes)) ||
        (w_shards[k].tensor_scale && clash(ws, span_of(w_shards[k].tensor_scale, 4))))
      return DP_ERR_ALIAS;
  if (M > 0 && D > 0 && x && ld >= D &&
      clash(span_of(x, ((size_t)(M - 1) * (size_t)ld + D) * (x_dtype == DP_FP32 ? 4 : 2)),
            span_of(y, (size_t)M * K * F_shard * (y_dtype == DP_FP32 ? 4 : 2))))
    return DP_ERR_ALIAS;
  dph::DeviceInfo dev;
  Mx4mmParams p;
  int tiles;
  size_t zero;
  st = prepare(&q, M, D, w_shards, K, F_shard, format, x8, y, y_dtype, &dev, &p, &tiles, &zero);
  if (st != DP_OK) return st;
  void* scales = const_cast<void*>(q.scales);
  st = x8 ? dp_mx8_quantize(x, M, D, ld, x_dtype, workspace, scales, stream)
          : dp_mx4_quantize(&x, 1, M, D, ld, x_dtype, format, 0, x_scale, workspace, scales, stream);
  if (st != DP_OK) return st;
  p.y = y;
  return enqueue(p, tiles, zero, x8 ? kMx8 : format == DP_MXFP4 ? kMx4 : kNv4, dev,
                 reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

dp_status_t dp_allgather_matmul_mx4(const dp_mx4_t* x, int M, int D, const dp_mx4_t* w_shards,
                                    int K, int F_shard, dp_mx4_format_t format, void* y,
                                    dp_dtype_t y_dtype, dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_allgather_matmul_mx4");
  return product(x, M, D, w_shards, K, F_shard, format, false, y, y_dtype, stream);
}

dp_status_t dp_allgather_linear_mx4_workspace_size(int M, int D, dp_mx4_format_t format,
                                                   size_t* bytes) {
  return workspace_size(M, D, format, false, bytes);
}

dp_status_t dp_allgather_linear_mx4(const void* x, int M, int D, long long ld, dp_dtype_t x_dtype,
                                    const float* x_scale, const dp_mx4_t* w_shards, int K,
                                    int F_shard, dp_mx4_format_t format, void* y,
                                    dp_dtype_t y_dtype, void* workspace, size_t workspace_bytes,
                                    dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_allgather_linear_mx4");
  return linear(x, M, D, ld, x_dtype, x_scale, w_shards, K, F_shard, format, false, y, y_dtype,
                workspace, workspace_bytes, stream);
}

dp_status_t dp_allgather_matmul_mx8(const dp_mx4_t* x, int M, int D, const dp_mx4_t* w_shards,
                                    int K, int F_shard, void* y, dp_dtype_t y_dtype,
                                    dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_allgather_matmul_mx8");
  return product(x, M, D, w_shards, K, F_shard, DP_MXFP4, true, y, y_dtype, stream);
}

dp_status_t dp_allgather_linear_mx8_workspace_size(int M, int D, size_t* bytes) {
  return workspace_size(M, D, DP_MXFP4, true, bytes);
}

dp_status_t dp_allgather_linear_mx8(const void* x, int M, int D, long long ld, dp_dtype_t x_dtype,
                                    const dp_mx4_t* w_shards, int K, int F_shard, void* y,
                                    dp_dtype_t y_dtype, void* workspace, size_t workspace_bytes,
                                    dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_allgather_linear_mx8");
  return linear(x, M, D, ld, x_dtype, nullptr, w_shards, K, F_shard, DP_MXFP4, true, y, y_dtype,
                workspace, workspace_bytes, stream);
}

}  // extern "C"
