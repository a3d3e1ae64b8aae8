// dp_w4.cu -- few tokens times gathered 4-bit weight shards, the tokens as they
// are (bf16):  y[m, f] = tw sum_d x[m, d] s[f, b(d)] w[f, d]
// with b(d) = d / 32 (mxfp4) or d / 16 (nvfp4) and tw the shard's fp32 scale (nvfp4).
//
// With one token, or a few, the product is bound by the weights' bytes, so they
// go from memory to the tensor core with as little in between as possible:
//   * A warp takes 32 weight rows and d, or its share of it, 128 values at a time.
//     A lane copies 16 bytes (32 values: whole blocks) of each of its four rows to
//     its own place in shared memory (cp.async, two steps ahead) and later reads the
//     same bytes back: no barrier, and no register waits for memory.
//   * Eight codes become four pairs of f16 (one conversion each), which one
//     multiplication by the block's scale makes the exact weight: e2m1 has two
//     significant bits, e4m3 four.  As bf16 the decoding takes 23 instructions
//     for eight codes instead of 8, more than the SM issues at the rate at which
//     they arrive (measured in registers: 4.7 against 10.6 words a clock; 5.1
//     arrive).
//   * mma.sync m16n8k16 with the weights as the 16 rows: one to eight tokens are
//     one instruction's eight columns (2.15 clocks each on an SM).  Which d a lane's
//     values stand for does not matter as long as x comes in the same order.
//   * The rows of a lane are g, g + 32, g + 64, g + 96 of a 128-row scale tile:
//     their scales are one 16-byte word.
//   * x is staged as f16 for all warps of a CTA, a slab of d at a time.  More than
//     eight tokens are made f16 by a small kernel beforehand, and come by bulk
//     copies: made by every CTA, they took more instructions than the weights.
// f16 has less range than bf16 and 2^k scales.  So x is multiplied by a power of
// two that takes its largest magnitude (up to eight tokens: the largest so far) to
// about 2^10, and mxfp4's scales are taken relative to the largest of the row so
// far; where a larger one comes by more than the headroom, the sums are multiplied
// down first.  A value of x loses bits only below 2^-27 of that token's largest (and
// is then off by at most 2^-35 of it), an mxfp4 weight only where its block's scale is
// below 2^-27 of its row's largest (by at most 2^-25 of that).  Sums are fp32.
//
// Few rows: d is split over the warps of a CTA, whose partial sums meet in shared
// memory and are added in order.
//
// Measured (GB300, launches in a CUDA graph), w[65536,8192]: one token 57 us in
// either form (5.3 TB/s of weights in nvfp4), eight 62 us, 16 71 us in mxfp4, 32 116
// us; 4096 x 4096: one token 6.9 us, 16 8.6 us.  What bounds it: one token's bytes
// alone (no decoding, no products) take 52 us and its instructions alone (the same
// codes again and again) 50.  16 tokens' instructions alone take 66, with nothing full
// (53 % of the issue slots, 51 % of DRAM, 44 % of the tensor pipe): 2048 units are 14
// warps on each of 147 SMs, four on half of the schedulers and three on the others,
// and all wait for four.  32 tokens: MMAs, 138 clocks of a step against the 87 in which
// its bytes arrive; there 128 registers do not suffice (-Xptxas -v, bytes of spill
// stores a thread: nvfp4 76, mxfp4 48; 16 tokens in nvfp4 16).  Rows past a shard's
// end are decoded and multiplied like the others, so shards of fewer than 128 rows
// cost as much as ones of 128.  Neither rings of 4 or 5 steps
// nor 28 warps of 72 registers gained anything.  The steps that led here: x
// converted by each warp for itself 83 us (one token, nvfp4) and 138 us (16, mxfp4);
// rings half as large, twice the warps 69 and 128; x staged for the CTA 59 and 91; x
// prepared beforehand 70 (16); divisions and ldexpf around the steps by shifts and
// products, one token of 4096 x 4096 7.5 -> 6.9.

#include "dp_early.cuh"
#include "dp_launch.h"
#include "dp_mx4.cuh"
#include "dp_mx4q.cuh"
#include "dp_w4_plan.h"

#include <algorithm>
#include <cstring>
#include <mutex>

namespace {

using namespace dpk;
using w4::kMaxSmem;
using w4::kMaxWarps;
using w4::kRows;  // two instructions' 16
using w4::kStep;
using w4::x_row_bytes;

constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kXRoom = 5;        // exponents that x may grow by before the sums are scaled down
constexpr int kSRoom = 9;        // ... and mxfp4's scales
constexpr int kSBelow = 18;      // exponents below the reference that f16 holds as they are

struct W4Params {
  const uint16_t* x;   // or what prepare_kernel made of it, ld elements (f16) apart
  const int* xexp;     // ... and the exponents of its tokens
  long long ld;
  const uint8_t* codes[kMaxK];
  const uint8_t* scales[kMaxK];
  const float* tw[kMaxK];
  void* y;
  int M, D, F, F_shard;
  int tiles_f;     // 128-row scale tiles of a shard
  int col_tiles;
  int units;       // of 32 rows, of all shards
  int split, split_bits, slab, slabs;  // (w4::Plan)
  int x_vec;       // x's rows start on 16-byte boundaries
  int y_f32;
  unsigned* err;
};

// Shared memory: each warp's ring of codes and scales, and two slabs of x (one, if
// there is no other) for each share and token.
template <bool MX, int NT>
struct W4Ring {
  static constexpr int kStages = w4::ring_steps(NT);
  static constexpr uint32_t kCodes = kRows * (kStep / 2);
  static constexpr uint32_t kStage = w4::step_bytes(MX);
  static constexpr uint32_t kWarp = kStages * kStage;
  static_assert(kRows * 8 * NT * 4 <= kWarp, "partial sums");
};
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The largest exponent (biased) of eight bf16 values.
__device__ __forceinline__ int top_exponent(uint4 v) {
  uint32_t t = max_abs2(max_abs2(max_abs2(v.x & 0x7fff7fffu, v.y), v.z), v.w);
  t = max(t >> 16, t & 0xffffu);
  return (int)(t >> 7);
}
// 2^e as fp32, for e in [-126, 127]; 0 below.
__device__ __forceinline__ float pow2(int e) {
  return __uint_as_float(e < -126 ? 0u : (uint32_t)(e + 127) << 23);
}

// v 2^e, in two steps, for e in [-258, 250]: what pow2 makes 0 of is far below fp32's
// smallest (an infinite v may become NaN).
__device__ __forceinline__ float scaled(float v, int e) {
  return __fmul_rn(__fmul_rn(v, pow2(e >> 1)), pow2(e - (e >> 1)));
}

// Eight e2m1 codes to four pairs of f16.
__device__ __forceinline__ void decode8(uint32_t c, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The place of 16 bytes (eight values from k on) in a slab's row: a step's sixteen
// pieces are kept so that the four lanes of a token read 64 consecutive bytes.
__device__ __forceinline__ uint32_t x_place(int k) {
  const int piece = k / 8 % 16;
  return (uint32_t)(k / kStep * 256 + piece % 4 * 64 + piece / 4 * 16);
}

// x as the products of more than eight tokens take it: f16 relative to the token's
// largest, 2^(137 - exponent) times its values, in steps of 128 (zero past D) whose
// pieces are in x_place's order.  A CTA for each token.
struct XParams {
  const uint16_t* x;
  long long ld;
  int D, steps;
  int x_vec;
  uint16_t* out;
  int* xexp;
};
__device__ __forceinline__ uint4 load8(const uint16_t* x, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(x);
  return make_uint4((uint32_t)x[0] | (uint32_t)x[1] << 16, (uint32_t)x[2] | (uint32_t)x[3] << 16,
                    (uint32_t)x[4] | (uint32_t)x[5] << 16, (uint32_t)x[6] | (uint32_t)x[7] << 16);
}
__device__ __forceinline__ uint4 to_f16(uint4 v, float f) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float lo, hi;
    unpair(mul2(pair(bf16lo(w[q]), bf16hi(w[q])), pair(f, f)), lo, hi);
    w[q] = pack_f16x2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
constexpr int kXThreads = 512;
__global__ void __launch_bounds__(kXThreads) prepare_kernel(const __grid_constant__ XParams p) {
  __shared__ int tops[kXThreads / 32];
  stream_order();
  const uint16_t* x = p.x + (long long)blockIdx.x * p.ld;
  uint8_t* out = reinterpret_cast<uint8_t*>(p.out) + (size_t)blockIdx.x * p.steps * 256;
  int e = 0;
  for (int i = threadIdx.x; i < p.D / 8; i += kXThreads) {
    const uint4 v = load8(x + 8ll * i, p.x_vec);
    e = max(e, top_exponent(v));
  }
  e = __reduce_max_sync(0xffffffffu, e);
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = e;
  __syncthreads();
  e = __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < kXThreads / 32 ? tops[threadIdx.x & 31] : 0);
  e = max(e, 10);
  const float f = __uint_as_float((uint32_t)(264 - e) << 23);
  if (threadIdx.x == 0) p.xexp[blockIdx.x] = e;
  for (int i = threadIdx.x; i < p.steps * 16; i += kXThreads) {
    const uint4 v = i < p.D / 8 ? to_f16(load8(x + 8ll * i, p.x_vec), f) : make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(out + (size_t)(i / 16) * 256 + x_place(i % 16 * 8)) = v;
  }
}

template <bool MX, int NT, bool kReady>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) w4_kernel(const __grid_constant__ W4Params p) {
  using G = W4Ring<MX, NT>;
  constexpr int kStages = G::kStages;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t xfull[2], xfree[2];  // (x prepared: a slab has landed, has been read)
  __shared__ int xexp[kReady ? 1 : 2][kReady ? 1 : kMaxWarps][8 * NT];  // slab, share, token
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int share = warp & (p.split - 1);
  const int unit = (int)blockIdx.x * (warps >> p.split_bits) + (warp >> p.split_bits);
  const int m0 = (int)blockIdx.y * 8 * NT;
  const int tokens = min(p.M - m0, 8 * NT);
  const uint32_t mine = smem_u32(smem) + (uint32_t)warp * G::kWarp;
  const uint32_t ring = mine + (uint32_t)lane * 16;
  // the scales of the lane's rows: one copy for the lanes that share them
  const uint32_t srow = mine + G::kCodes + (uint32_t)(MX ? 0 : (t >> 1) * 128) + (uint32_t)g * 16;
  const uint32_t xrow = x_row_bytes(p.slab);
  const uint32_t xs = smem_u32(smem) + (uint32_t)warps * G::kWarp;
  const auto x_at = [&](int buf, int s, int m) {
    return xs + ((uint32_t)((buf * p.split + s) * tokens + m)) * xrow;
  };
  if constexpr (!kReady) {
    for (int i = threadIdx.x; i < 2 * kMaxWarps * 8 * NT; i += blockDim.x)
      (&xexp[0][0][0])[i] = -1000;
    stream_order();
  }

  const bool live_unit = unit < p.units;
  const int u = live_unit ? unit : 0;
  int tile = u / 4, shard = 0;
  while (tile >= p.tiles_f) tile -= p.tiles_f, ++shard;
  const int row0 = tile * 128 + u % 4 * 8;  // rows g, + 32, + 64, + 96
  const uint8_t* code[4];
#pragma unroll
  for (int r = 0; r < 4; ++r)  // rows past the shard's end read its last, and are dropped
    code[r] = p.codes[shard] + (size_t)min(row0 + g + 32 * r, p.F_shard - 1) * (p.D / 2) + t * 16;
  const uint8_t* scale =
      p.scales[shard] + (size_t)(row0 / 128) * p.col_tiles * kScaleTile + (row0 % 32 + g) * 16;

  // this share's steps of d
  const int steps = (p.D + kStep - 1) / kStep, per = p.slabs * p.slab;
  const int c_lo = min(share * per, steps);
  const int c_hi = live_unit ? min(c_lo + per, steps) : c_lo;

  int slot = 0;  // of the ring, for the next copy
  const auto fetch = [&](int c) {
    if (c < c_hi) {
      const uint32_t at = ring + (uint32_t)slot * G::kStage;
      if (c * kStep + t * 32 < p.D) {
#pragma unroll
        for (int r = 0; r < 4; ++r) copy16(at + r * 512, code[r] + (size_t)c * (kStep / 2));
      }
      const int ct = min(MX ? c : 2 * c + (t >> 1), p.col_tiles - 1);
      if (t == 0 || (!MX && t == 2)) copy16(srow + (at - ring), scale + (size_t)ct * kScaleTile);
    }
    copy_commit();
    if (++slot == kStages) slot = 0;
  };

  // x of one slab, a warp for each share and token: first its values as they are
  // come to their place (cp.async), later they become f16 there, relative to the
  // token's largest so far.  A lane takes eight values of every other step, both times.
  const int half = lane >> 4;
  const uint32_t piece = (uint32_t)half * 256 + x_place((lane & 15) * 8);
  // q / tokens for q below 1024: 2^16 / tokens rounded up is off by less than 1 / q of it
  const int per_token = kReady ? 0 : 65536 / tokens + 1;
  const auto each_job = [&](auto f) {
    for (int q = warp; q < tokens * p.split; q += warps) {
      const int s = (q * per_token) >> 16;
      f(s, q - s * tokens);
    }
  };
  const auto x_copy = [&](int slab) {
    if constexpr (kReady) {
      // whole slabs lie as they are to lie: a lane has one copied (what the share has
      // of it, which is all that is read)
      const int q = warp + lane * warps, s = q / tokens, m = q - s * tokens;
      const int step = s * per + slab * p.slab;
      const uint32_t n =
          s < p.split ? (uint32_t)max(0, min(p.slab, steps - step)) * 256u : 0u;
      const uint32_t all = __reduce_add_sync(0xffffffffu, n);
      uint64_t* bar = &xfull[slab & 1];
      if (lane == 0) mbar_arrive_expect_tx(bar, all);
      __syncwarp();
      if (n)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
                "r"(x_at(slab & 1, s, m)),
            "l"(reinterpret_cast<const uint8_t*>(p.x) + ((size_t)(m0 + m) * steps + step) * 256),
            "r"(n), "r"(smem_u32(bar))
            : "memory");
      return;
    }
    each_job([&](int s, int m) {
      uint32_t to = x_at(slab & 1, s, m);
      const int first = (s * per + slab * p.slab + half) * kStep + (lane & 15) * 8;
      const uint16_t* x = p.x + (long long)(m0 + m) * p.ld + first;
      to += piece;
      for (int i = half, k = first; i < p.slab; i += 2, k += 2 * kStep, x += 2 * kStep, to += 512) {
        if (k >= p.D)
          sts16(to, make_uint4(0u, 0u, 0u, 0u));
        else if (p.x_vec)
          copy16(to, x);
        else
          sts16(to, load8(x, false));
      }
    });
  };
  const auto x_convert = [&](int slab) {
    if constexpr (!kReady) {
      const int buf = slab & 1;
      each_job([&](int s, int m) {
        const uint32_t row = x_at(buf, s, m) + piece;
        int e = 0;
        for (int i = half, o = 0; i < p.slab; i += 2, o += 512) e = max(e, top_exponent(lds16(row + o)));
        __syncwarp();
        e = __reduce_max_sync(0xffffffffu, e);
        const int was = xexp[buf ^ 1][s][m];
        const int to = e > was + kXRoom ? max(e, 10) : was;
        const float f = __uint_as_float((uint32_t)(264 - to) << 23);  // 2^(137 - to)
        for (int i = half, o = 0; i < p.slab; i += 2, o += 512)
          sts16(row + o, to_f16(lds16(row + o), f));
        __syncwarp();
        if (lane == 0) xexp[buf][s][m] = to;
      });
    }
  };

  float acc[2][NT][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.0f;
  int xref[NT][2];  // the exponents (biased) of tokens 2t, 2t + 1 of each eight that go to 2^10
  int sbase[4];     // mxfp4: the scale byte of each row that goes to 2^4, less kSBelow
#pragma unroll
  for (int n = 0; n < NT; ++n) xref[n][0] = xref[n][1] = -1000;
#pragma unroll
  for (int r = 0; r < 4; ++r) sbase[r] = -kSBelow;
  // which bytes of the 16 rows' word of four are this lane's
  const uint32_t take = MX ? 0x4440u + (uint32_t)t : t & 1 ? 0x4432u : 0x4410u;
  const int last_step = steps - 1;

  if constexpr (kReady) {
    // The kernel before this one is prepare_kernel, which let this one start when all
    // before it had ended: the weights may be read already, x not yet.  The call's lock
    // keeps this library's kernels of other threads from between the two; one of another
    // kind that is put there has ended when this one starts.
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(c_lo + s);
    stream_order();
    for (int i = threadIdx.x; i < 8 * NT; i += blockDim.x)
      xexp[0][0][i] = i < tokens ? p.xexp[m0 + i] : 0;
    if (threadIdx.x == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&xfull[i], warps);
        mbar_init(&xfree[i], warps);
      }
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    x_copy(0);
  } else {
    __syncthreads();  // xexp
    x_copy(0);
    copy_commit();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(c_lo + s);
    copy_wait<kStages - 1>();
    x_convert(0);
    __syncthreads();
  }
  if constexpr (kReady) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      xref[n][0] = xexp[0][0][n * 8 + 2 * t];
      xref[n][1] = xexp[0][0][n * 8 + 2 * t + 1];
    }
  }
  int c = c_lo, read = 0;
  for (int slab = 0; slab < p.slabs; ++slab) {
    // the next slab's x is on its way while this one is worked on: its copies belong
    // to the group of the first step's fetch, which the kStages-th step waits for
    if (!kReady && slab + 1 < p.slabs) x_copy(slab + 1);
    const int buf = slab & 1;
    if constexpr (kReady)
      (void)mbar_wait_bounded(&xfull[buf], (uint32_t)(slab >> 1) & 1u, p.err, kTimeoutNs);
    uint32_t xtok[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      xtok[n] = x_at(buf, share, min(n * 8 + g, tokens - 1));
      if constexpr (kReady) continue;
      const int e0 = xexp[kReady ? 0 : buf][kReady ? 0 : share][n * 8 + 2 * t], e1 = xexp[kReady ? 0 : buf][kReady ? 0 : share][n * 8 + 2 * t + 1];
      if (__any_sync(0xffffffffu, e0 != xref[n][0] || e1 != xref[n][1])) {
        const float d0 = pow2(xref[n][0] - e0), d1 = pow2(xref[n][1] - e1);
        xref[n][0] = e0;
        xref[n][1] = e1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc[i][n][0] = __fmul_rn(acc[i][n][0], d0);
          acc[i][n][1] = __fmul_rn(acc[i][n][1], d1);
          acc[i][n][2] = __fmul_rn(acc[i][n][2], d0);
          acc[i][n][3] = __fmul_rn(acc[i][n][3], d1);
        }
      }
    }
    for (int k = 0; k < p.slab; ++k, ++c) {
      copy_wait<kStages - 2>();
      __syncwarp();  // the scales are other lanes' copies, too
      fetch(c + kStages - 1);  // to where the step before this one was
      if (kReady && k == p.slab / 2 && slab + 1 < p.slabs) {
        // every warp is done with the slab before this one: the next takes its place
        if (slab > 0)
          (void)mbar_wait_bounded(&xfree[buf ^ 1], (uint32_t)((slab - 1) >> 1) & 1u, p.err,
                                  kTimeoutNs);
        __syncwarp();
        x_copy(slab + 1);
      }
      if (c >= c_hi) continue;  // past this share's end: only the groups go on
      const uint32_t at = ring + (uint32_t)read * G::kStage;
      if (++read == kStages) read = 0;
      // the rows' scales as pairs of f16: one block (mxfp4) or two (nvfp4)
      uint32_t s[4][MX ? 1 : 2];
      {
        const uint4 v = lds16(srow + (at - ring));
        uint32_t word[4] = {v.x, v.y, v.z, v.w};
        if (c == last_step && c * kStep + t * 32 >= p.D)  // a lane past the end: any finite ones
          word[0] = word[1] = word[2] = word[3] = 0u;
        if constexpr (MX) {
          // A scale relative to the row's: exponent byte - sref + 4, as f16 bits.  What
          // f16 cannot hold takes the long way, but for byte 0: that is most often a block
          // of zeros, and counts as one where its row's reference is 28 or more.
          int d[4];
          bool far = false;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int byte = (int)__byte_perm(word[r], 0u, take);
            d[r] = byte - sbase[r];
            far |= (uint32_t)d[r] > (uint32_t)(kSRoom + kSBelow) && byte != 0;
            s[r][0] = (uint32_t)(max(d[r], -1) + 1) * 0x04000400u;
          }
          if (__any_sync(0xffffffffu, far)) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int byte = d[r] + sbase[r], sref = sbase[r] + kSBelow;
              int e = byte == 255 ? 0 : byte;
              e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
              e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
              // (not between, where byte 0 would count as nothing too early, see above, and
              // no higher than where byte 255, NaN, is out of the room for good)
              const int up = e <= kSBelow + kSRoom ? kSBelow : min(e, 254 - kSRoom);
              const int to = e > sref + kSRoom ? up : sref;
              const float down = pow2(sref - to);
              sbase[r] = to - kSBelow;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float* a = &acc[r / 2][n][(r % 2) * 2];
                a[0] = __fmul_rn(a[0], down);
                a[1] = __fmul_rn(a[1], down);
              }
              // 2^(byte - sref + 4): at most 2^13, below f16's smallest 0
              const float f = __uint_as_float((uint32_t)max(byte - to + 131, 0) << 23);
              s[r][0] = byte == 255 ? 0x7fff7fffu : pack_f16x2(f, f);
            }
          }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            uint32_t f;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"((uint16_t)__byte_perm(word[r], 0u, take)));
            s[r][0] = __byte_perm(f, f, 0x1010);
            s[r][1] = __byte_perm(f, f, 0x3232);
          }
        }
      }

      uint32_t w[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint4 v = lds16(at + r * 512);
        w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
      }
      const uint32_t xk = (uint32_t)(k * 256 + t * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          decode8(w[r][j], h[r]);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[r][e] = mul_f16x2(h[r][e], s[r][MX ? 0 : j / 2]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          // (columns past the last token hold the last one's, and are dropped)
          const uint4 b = lds16(xtok[n] + xk + j * 64);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mma16816(acc[i][n], h[2 * i][0], h[2 * i + 1][0], h[2 * i][1], h[2 * i + 1][1], b.x, b.y);
            mma16816(acc[i][n], h[2 * i][2], h[2 * i + 1][2], h[2 * i][3], h[2 * i + 1][3], b.z, b.w);
          }
        }
      }
    }
    if (slab + 1 < p.slabs) {
      if constexpr (kReady) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&xfree[buf]);
      } else {
        if (p.slab < kStages) copy_wait<1>();  // (a longer slab's steps have waited for it)
        x_convert(slab + 1);
        __syncthreads();
      }
    }
  }
  copy_wait<0>();

  // the sums as they are: back from the powers of two
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int to = xref[n][e & 1] - 137;
        if (MX) to += sbase[2 * i + e / 2] + kSBelow - 131;
        acc[i][n][e] = scaled(acc[i][n][e], to);
      }
  float alpha = 1.0f;
  if constexpr (!MX)
    if (p.tw[shard]) alpha = *p.tw[shard];
  const auto store = [&](int f, int col, float v) {  // f of the shard
    const int m = m0 + col;
    if (f < p.F_shard && m < p.M) {
      const size_t o = (size_t)m * p.F + (size_t)shard * p.F_shard + f;
      v = __fmul_rn(v, alpha);
      if (p.y_f32)
        static_cast<float*>(p.y)[o] = v;
      else
        static_cast<uint16_t*>(p.y)[o] = bf16_rn(v);
    }
  };
  if (p.split == 1) {
    if (!live_unit) return;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          store(row0 + g + 32 * (2 * i + e / 2), n * 8 + 2 * t + (e & 1), acc[i][n][e]);
    return;
  }
  // partial sums [token][row of the unit], row r * 8 + g, each warp in its own ring
  float* part = reinterpret_cast<float*>(smem + (size_t)warp * G::kWarp);
  __syncwarp();
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        part[(n * 8 + 2 * t + (e & 1)) * kRows + (2 * i + e / 2) * 8 + g] = acc[i][n][e];
  __syncthreads();
  if (!live_unit) return;
  const float* first = reinterpret_cast<const float*>(smem + (size_t)(warp - share) * G::kWarp);
  for (int i = share * 32 + lane; i < kRows * tokens; i += p.split * 32) {
    float v = first[i];
    for (int k = 1; k < p.split; ++k) v = __fadd_rn(v, first[(size_t)k * (G::kWarp / 4) + i]);
    store(row0 + i % 8 + i % kRows / 8 * 32, i / kRows, v);
  }
}

constexpr int kMaxTokens = 65535 * 8;  // the grid's second dimension
constexpr int kMaxD = 1 << 30;         // a share's last slab, past D, still has int positions
constexpr int kOwnTokens = 8;          // of a call whose kernel makes f16 of x itself

template <bool MX, int NT, bool READY>
cudaError_t launch_for(W4Params p, const dph::DeviceInfo& dev, cudaStream_t s) {
  const w4::Plan plan = w4::plan(std::min(p.M, 8 * NT), p.D, p.units, MX, NT, READY);
  p.split = plan.split, p.split_bits = plan.split_bits;
  p.slab = plan.slab, p.slabs = plan.slabs;
  auto kernel = w4_kernel<MX, NT, READY>;
  if (dph::prepare_kernel(reinterpret_cast<const void*>(kernel), kMaxWarps * 32, kMaxSmem,
                          dev.device) < 1)
    return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((p.units + plan.per - 1) / plan.per),
                     (unsigned)((p.M + 8 * NT - 1) / (8 * NT)));
  cfg.blockDim = dim3((unsigned)plan.warps * 32);
  cfg.dynamicSmemBytes = plan.smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool MX>
cudaError_t launch_w4(const W4Params& p, const dph::DeviceInfo& dev, cudaStream_t s) {
  if (p.M <= kOwnTokens) return launch_for<MX, 1, false>(p, dev, s);
  if (p.M <= 16) return launch_for<MX, 2, true>(p, dev, s);
  return launch_for<MX, 4, true>(p, dev, s);
}

using dph::aligned;
using dph::clash;
using dph::Span;
using dph::span_of;

size_t prepared_bytes(int M, int D) { return (size_t)M * (((size_t)D + kStep - 1) / kStep) * 256; }

}  // namespace

extern "C" {

dp_status_t dp_allgather_linear_w4_workspace_size(int M, int D, size_t* bytes) {
  if (!bytes) return DP_ERR_INVALID_ARG;
  *bytes = 0;
  if (M < 0 || D < 0) return DP_ERR_INVALID_ARG;
  if (M > kMaxTokens || D > kMaxD) return DP_ERR_UNSUPPORTED;
  if (M > kOwnTokens && D) *bytes = prepared_bytes(M, D) + (size_t)M * sizeof(int);
  return DP_OK;
}

dp_status_t dp_allgather_linear_w4(const void* x, int M, int D, long long ld,
                                   const dp_mx4_t* w_shards, int K, int F_shard,
                                   dp_mx4_format_t format, void* y, dp_dtype_t y_dtype,
                                   void* workspace, size_t workspace_bytes, dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_allgather_linear_w4");
  if (!w_shards || K < 1 || K > DP_MAX_K) return DP_ERR_INVALID_ARG;
  if (M < 0 || D < 0 || F_shard < 0 || ld < D) return DP_ERR_INVALID_ARG;
  if (format != DP_MXFP4 && format != DP_NVFP4) return DP_ERR_UNSUPPORTED;
  if (y_dtype != DP_FP32 && y_dtype != DP_BF16) return DP_ERR_UNSUPPORTED;
  if (D % 32 || F_shard % 16) return DP_ERR_UNSUPPORTED;
  if ((long long)K * F_shard > 0x7fffff00ll || M > kMaxTokens || D > kMaxD)
    return DP_ERR_UNSUPPORTED;
  const size_t ysz = y_dtype == DP_FP32 ? 4 : 2;
  if (!aligned(x, 2) || !aligned(y, ysz)) return DP_ERR_UNSUPPORTED;
  const int F = K * F_shard;
  if (M == 0 || F == 0) return DP_OK;
  if (!y || (!x && D)) return DP_ERR_INVALID_ARG;
  size_t need = 0;
  dp_allgather_linear_w4_workspace_size(M, D, &need);
  if (need && (!workspace || workspace_bytes < need)) return DP_ERR_INVALID_ARG;
  if (need && !aligned(workspace, 16)) return DP_ERR_UNSUPPORTED;
  const Span ws = span_of(workspace, need);
  const Span out = span_of(y, (size_t)M * F * ysz);
  const Span xs = span_of(x, D ? ((size_t)(M - 1) * (size_t)ld + (size_t)D) * 2 : 0);
  if (clash(out, xs) || clash(ws, xs) || clash(ws, out)) return DP_ERR_ALIAS;
  size_t sbytes = 0;
  dp_mx4_scales_size(F_shard, D, format, &sbytes);
  W4Params p;
  memset(&p, 0, sizeof p);
  for (int k = 0; k < K; ++k) {
    const dp_mx4_t& w = w_shards[k];
    if (format == DP_MXFP4 && w.tensor_scale) return DP_ERR_INVALID_ARG;
    if ((!w.codes || !w.scales) && D) return DP_ERR_INVALID_ARG;
    if (!aligned(w.codes, 16) || !aligned(w.scales, 16) || !aligned(w.tensor_scale, 4))
      return DP_ERR_UNSUPPORTED;
    const Span of[3] = {span_of(w.codes, (size_t)F_shard * (D / 2)), span_of(w.scales, sbytes),
                        span_of(w.tensor_scale, w.tensor_scale ? 4 : 0)};
    for (const Span& o : of)
      if (clash(out, o) || clash(ws, o)) return DP_ERR_ALIAS;
    p.codes[k] = static_cast<const uint8_t*>(w.codes);
    p.scales[k] = static_cast<const uint8_t*>(w.scales);
    p.tw[k] = w.tensor_scale;
  }
  dph::DeviceInfo dev;
  if (!dph::current_device(&dev)) return DP_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (D == 0)
    return cudaMemsetAsync(y, 0, (size_t)M * F * ysz, s) == cudaSuccess ? DP_OK : DP_ERR_CUDA;
  p.x = static_cast<const uint16_t*>(x);
  p.ld = ld;
  p.y = y;
  p.M = M, p.D = D, p.F = F, p.F_shard = F_shard;
  p.tiles_f = (F_shard + kScaleRows - 1) / kScaleRows;
  p.col_tiles = mx4_col_tiles(D, mx4_block(format));
  p.x_vec = aligned(x, 16) && ld % 8 == 0;
  p.y_f32 = y_dtype == DP_FP32;
  p.err = dev.err_word;
  p.units = (int)((long long)K * p.tiles_f * 4);
  cudaError_t e = cudaSuccess;
  std::unique_lock<std::mutex> pair(dph::early_launches(), std::defer_lock);
  if (need) {
    pair.lock();  // (the product reads weights on the strength of prepare_kernel's wait)
    XParams q{p.x, ld, D, (D + kStep - 1) / kStep, p.x_vec, static_cast<uint16_t*>(workspace),
              reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + prepared_bytes(M, D))};
    e = dph::launch_early_held(prepare_kernel, q, (unsigned)M, kXThreads, s);
    p.x = q.out;
    p.xexp = q.xexp;
  }
  if (e == cudaSuccess)
    e = format == DP_MXFP4 ? launch_w4<true>(p, dev, s) : launch_w4<false>(p, dev, s);
  return e == cudaSuccess ? DP_OK : DP_ERR_CUDA;
}

}  // extern "C"
