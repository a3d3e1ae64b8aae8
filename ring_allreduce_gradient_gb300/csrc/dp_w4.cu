// dp_w4.cu -- few tokens times gathered 4-bit weight shards, the tokens as they
// are (bf16):  y[m, f] = tw sum_d x[m, d] s[f, b(d)] w[f, d]
// with b(d) = d / 32 (mxfp4) or d / 16 (nvfp4) and tw the shard's fp32 scale (nvfp4).
//
// With one token, or a few, the product is bound by the weights' bytes, so they
// go from memory to the tensor core with as little in between as possible:
//   * A warp takes 16 MT weight rows and its share of d, 128 at a time.  A lane
//     copies 16 bytes (32 values: whole blocks) of each of its 2 MT rows to its
//     own place in shared memory (cp.async, several steps ahead) and later reads
//     the same bytes back: no barrier, and no register waits for memory.
//   * Eight codes become four pairs of f16 (one conversion each), which one
//     multiplication by the block's scale makes the exact weight: e2m1 has two
//     significant bits, e4m3 four.  As bf16 the decoding takes 23 instructions
//     for eight codes instead of 8, more than the SM issues at the rate at which
//     they arrive (measured in registers: 4.7 against 10.6 words a clock; 5.1
//     arrive).
//   * mma.sync m16n8k16 with the weights as the 16 rows: one to eight tokens are
//     one instruction's eight columns.  Which d a lane's values stand for does not
//     matter as long as x comes in the same order, so both stay as they lie.
//   * The rows of a warp are g, g + 32, g + 64, g + 96 of a 128-row scale tile (g
//     of eight neighbours): their scales are one 16-byte word.
// f16 has less range than bf16 and 2^k scales.  So x is multiplied by a power of
// two that takes its largest magnitude seen so far to about 2^10, and mxfp4's
// scales are taken relative to the largest of the row so far; where a larger one
// comes by more than the headroom, the sums are multiplied down first.  A value
// of x loses bits only below 2^-27 of that token's largest (and is then off by at
// most 2^-35 of it), a weight below 2^-27 of its row's.  Sums are fp32.
//
// Few rows: d is split over the warps of a CTA, whose partial sums meet in shared
// memory and are added in order.

#include "dp_early.cuh"
#include "dp_launch.h"
#include "dp_mx4.cuh"
#include "dp_mx4q.cuh"

#include <algorithm>
#include <cstring>

namespace {

using namespace dpk;

constexpr int kStep = 128;       // values of d a warp takes at once: 32 a lane
constexpr int kXRoom = 5;        // exponents that x may grow by before the sums are scaled down
constexpr int kSRoom = 9;        // ... and mxfp4's scales

struct W4Params {
  const uint16_t* x;
  long long ld;
  const uint8_t* codes[kMaxK];
  const uint8_t* scales[kMaxK];
  const float* tw[kMaxK];
  void* y;
  int M, D, F, F_shard;
  int tiles_f;     // 128-row scale tiles of a shard
  int col_tiles;
  int units;       // of all shards
  int split;       // warps that share a unit's d
  int x_vec;       // x's rows start on 16-byte boundaries
  int y_f32;
};

template <bool MX, int MT, int NT>
struct W4Geo {
  static constexpr int kStages = NT == 4 || MT == 4 ? 2 : 3;
  static constexpr int kWarps = MT == 4 ? 4 : 8;              // of a CTA, at most
  static constexpr uint32_t kCodes = 2 * MT * 512;            // bytes of a stage, for a warp
  static constexpr uint32_t kScaleSet = MX ? 128 : 256;       // of eight neighbouring rows
  static constexpr uint32_t kScales = (MT / 2) * kScaleSet;
  static constexpr uint32_t kX = NT * 2048;
  static constexpr uint32_t kStage = kCodes + kScales + kX;
  static constexpr uint32_t kWarp = kStages * kStage;
  static_assert(16 * MT * 8 * NT * 4 <= kWarp, "partial sums");
  static_assert(kWarps * kWarp <= 232448, "shared memory of a CTA");
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
               : "r"(a)
               : "memory");
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
// The larger magnitude of each half (with a sign that means nothing).
__device__ __forceinline__ uint32_t max_mag2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 2^e as fp32, for e in [-126, 127]; 0 below.
__device__ __forceinline__ float pow2(int e) {
  return __uint_as_float(e < -126 ? 0u : (uint32_t)(e + 127) << 23);
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
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool MX, int MT, int NT>
__global__ void __launch_bounds__((W4Geo<MX, MT, NT>::kWarps * 32)) w4_kernel(const __grid_constant__ W4Params p) {
  using G = W4Geo<MX, MT, NT>;
  constexpr int R = 2 * MT;                 // rows of a lane
  constexpr int kUnits = 128 / (16 * MT);   // units of a scale tile
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int kw = warp % p.split;
  const int unit = (int)(blockIdx.x * ((blockDim.x >> 5) / p.split)) + warp / p.split;
  const int m0 = (int)blockIdx.y * 8 * NT;
  const uint32_t mine = smem_u32(smem) + (uint32_t)warp * G::kWarp;
  const uint32_t ring = mine + (uint32_t)lane * 16;
  // the scales of the lane's rows: one copy for the lanes that share them
  const uint32_t srow = mine + G::kCodes + (uint32_t)(MX ? 0 : (t >> 1) * 128) + (uint32_t)g * 16;
  stream_order();

  const bool live_unit = unit < p.units;
  const int u = live_unit ? unit : 0;
  const int tile = u / kUnits, shard = tile / p.tiles_f;
  const int row0 = (tile - shard * p.tiles_f) * 128 + (u % kUnits) * (4 * MT);
  const auto row_of = [&](int r) { return row0 + g + (r / 4) * 8 + (r % 4) * 32; };
  const uint8_t* code[R];
#pragma unroll
  for (int r = 0; r < R; ++r)  // rows past the shard's end read its last, and are dropped
    code[r] = p.codes[shard] + (size_t)min(row_of(r), p.F_shard - 1) * (p.D / 2) + t * 16;
  const uint8_t* scale =
      p.scales[shard] + (size_t)(row0 / 128) * p.col_tiles * kScaleTile + (row0 % 32 + g) * 16;

  const int chunks = (p.D + kStep - 1) / kStep;
  const int c_lo = live_unit ? (int)((long long)kw * chunks / p.split) : 0;
  const int c_hi = live_unit ? (int)((long long)(kw + 1) * chunks / p.split) : 0;

  const auto fetch = [&](int c) {
    if (c < c_hi) {
      const uint32_t at = ring + (uint32_t)((c - c_lo) % G::kStages) * G::kStage;
      const bool live = c * kStep + t * 32 < p.D;
      const int k = live ? c * kStep : 0;  // a lane past the end reads its place at the start
      if (live || p.D > t * 32) {
#pragma unroll
        for (int r = 0; r < R; ++r) copy16(at + r * 512, code[r] + k / 2);
      }
      const int ct = min(MX ? c : 2 * c + (t >> 1), p.col_tiles - 1);
      if (t == 0 || (!MX && t == 2))
#pragma unroll
        for (int h = 0; h < MT / 2; ++h)
          copy16(srow + (at - ring) + h * G::kScaleSet, scale + (size_t)ct * kScaleTile + h * 128);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int m = m0 + n * 8 + g;
        if (live && m < p.M) {
          const uint16_t* x = p.x + (long long)m * p.ld + c * kStep + t * 32;
          const uint32_t to = at + G::kCodes + G::kScales + n * 2048;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (p.x_vec) {
              copy16(to + i * 512, x + 8 * i);
            } else {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = (uint32_t)x[8 * i + 2 * e] | (uint32_t)x[8 * i + 2 * e + 1] << 16;
              sts16(to + i * 512, make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
        }
      }
    }
    copy_commit();
  };

  float acc[MT][NT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.0f;
  int xref[NT];   // the exponent (biased) of token g of each eight that goes to 2^10
  int sref[R];    // mxfp4: the scale byte of each row that goes to 2^4
#pragma unroll
  for (int n = 0; n < NT; ++n) xref[n] = -1000;
#pragma unroll
  for (int r = 0; r < R; ++r) sref[r] = -1000;

#pragma unroll
  for (int s = 0; s < G::kStages - 1; ++s) fetch(c_lo + s);
  for (int c = c_lo; c < c_hi; ++c) {
    copy_wait<G::kStages - 2>();
    __syncwarp();  // the scales are other lanes' copies, too
    fetch(c + G::kStages - 1);  // to where the step before this one was
    const uint32_t at = ring + (uint32_t)((c - c_lo) % G::kStages) * G::kStage;
    const bool live = c * kStep + t * 32 < p.D;

    // x: 32 values of a token, as f16 relative to the token's largest so far
    uint32_t b[NT][16];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool have = live && m0 + n * 8 + g < p.M;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (have) v = lds16(at + G::kCodes + G::kScales + n * 2048 + i * 512);
        b[n][4 * i] = v.x, b[n][4 * i + 1] = v.y, b[n][4 * i + 2] = v.z, b[n][4 * i + 3] = v.w;
      }
      uint32_t top = b[n][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = max_mag2(top, b[n][i]);
      int e = max((int)(top >> 23) & 255, (int)(top >> 7) & 255);
      if (__any_sync(0xffffffffu, e > xref[n] + kXRoom)) {
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
        const int to = e > xref[n] + kXRoom ? max(e, 10) : xref[n];
        const float down = pow2(xref[n] - to);
        xref[n] = to;
        const float d0 = __shfl_sync(0xffffffffu, down, 8 * t);
        const float d1 = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          acc[i][n][0] = __fmul_rn(acc[i][n][0], d0);
          acc[i][n][1] = __fmul_rn(acc[i][n][1], d1);
          acc[i][n][2] = __fmul_rn(acc[i][n][2], d0);
          acc[i][n][3] = __fmul_rn(acc[i][n][3], d1);
        }
      }
      const float f = __uint_as_float((uint32_t)(264 - xref[n]) << 23);  // 2^(137 - xref)
      const uint64_t ff = pair(f, f);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float lo, hi;
        unpair(mul2(pair(bf16lo(b[n][i]), bf16hi(b[n][i])), ff), lo, hi);
        b[n][i] = pack_f16x2(lo, hi);
      }
    }

    // the rows' scales as pairs of f16: one block (mxfp4) or two (nvfp4)
    uint32_t s[R][MX ? 1 : 2];
#pragma unroll
    for (int h = 0; h < MT / 2; ++h) {
      const uint4 v = lds16(srow + (at - ring) + h * G::kScaleSet);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 4 * h + j;
        if constexpr (MX) {
          s[r][0] = live ? (w[j] >> (8 * t)) & 255u : 0u;
        } else {
          const uint16_t two = live ? (uint16_t)(w[j] >> (16 * (t & 1))) : (uint16_t)0;
          uint32_t f;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(two));
          s[r][0] = __byte_perm(f, f, 0x1010);
          s[r][1] = __byte_perm(f, f, 0x3232);
        }
      }
    }
    if constexpr (MX) {
      bool above = false;
#pragma unroll
      for (int r = 0; r < R; ++r) above |= s[r][0] != 255u && (int)s[r][0] > sref[r] + kSRoom;
      if (__any_sync(0xffffffffu, above)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          int e = s[r][0] == 255u ? 0 : (int)s[r][0];
          e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
          e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
          const int to = e > sref[r] + kSRoom ? e : sref[r];
          const float down = pow2(sref[r] - to);
          sref[r] = to;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float* a = &acc[r / 2][n][(r % 2) * 2];
            a[0] = __fmul_rn(a[0], down);
            a[1] = __fmul_rn(a[1], down);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        // 2^(byte - sref + 4): at most 2^13, below f16's smallest 0
        const float f = __uint_as_float((uint32_t)max((int)s[r][0] - sref[r] + 131, 0) << 23);
        const uint32_t v = pack_f16x2(f, f);
        s[r][0] = s[r][0] == 255u ? 0x7fff7fffu : live ? v : 0u;
      }
    }

#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const uint4 va = lds16(at + (2 * i) * 512), vb = lds16(at + (2 * i + 1) * 512);
      const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t ha[4], hb[4];
        decode8(wa[j], ha);
        decode8(wb[j], hb);
        const uint32_t sa = s[2 * i][MX ? 0 : j / 2], sb = s[2 * i + 1][MX ? 0 : j / 2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ha[e] = mul_f16x2(ha[e], sa);
          hb[e] = mul_f16x2(hb[e], sb);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816(acc[i][n], ha[0], hb[0], ha[1], hb[1], b[n][4 * j], b[n][4 * j + 1]);
          mma16816(acc[i][n], ha[2], hb[2], ha[3], hb[3], b[n][4 * j + 2], b[n][4 * j + 3]);
        }
      }
    }
  }
  copy_wait<0>();

  // the sums as they are: back from the powers of two
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int x0 = __shfl_sync(0xffffffffu, xref[n], 8 * t);
    const int x1 = __shfl_sync(0xffffffffu, xref[n], 8 * t + 4);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int to = (e & 1 ? x1 : x0) - 137;
        if (MX) to += sref[2 * i + e / 2] - 131;
        acc[i][n][e] = ldexpf(acc[i][n][e], to);
      }
  }
  float alpha = 1.0f;
  if constexpr (!MX)
    if (p.tw[shard]) alpha = *p.tw[shard];
  const auto store = [&](int r, int col, float v) {  // row r of lane row g: f of the shard
    const int m = m0 + col;
    if (r < p.F_shard && m < p.M) {
      const size_t o = (size_t)m * p.F + (size_t)shard * p.F_shard + r;
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
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          store(row_of(2 * i + e / 2), n * 8 + 2 * t + (e & 1), acc[i][n][e]);
    return;
  }
  // partial sums [token][row of the unit], row r * 8 + g, each warp in its own ring
  float* part = reinterpret_cast<float*>(smem + (size_t)warp * G::kWarp);
  __syncwarp();
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        part[(n * 8 + 2 * t + (e & 1)) * (16 * MT) + (2 * i + e / 2) * 8 + g] = acc[i][n][e];
  __syncthreads();
  if (!live_unit) return;
  const float* first = reinterpret_cast<const float*>(smem + (size_t)(warp - kw) * G::kWarp);
  for (int i = kw * 32 + lane; i < 16 * MT * 8 * NT; i += p.split * 32) {
    float v = first[i];
    for (int k = 1; k < p.split; ++k) v = __fadd_rn(v, first[(size_t)k * (G::kWarp / 4) + i]);
    const int r = i % (16 * MT);
    store(row0 + r % 8 + (r / 32) * 8 + (r / 8 % 4) * 32, i / (16 * MT), v);
  }
}

template <bool MX, int MT, int NT>
cudaError_t launch_for(const W4Params& p, int warps, const dph::DeviceInfo& dev, cudaStream_t s) {
  auto kernel = w4_kernel<MX, MT, NT>;
  using G = W4Geo<MX, MT, NT>;
  if (dph::prepare_kernel(reinterpret_cast<const void*>(kernel), G::kWarps * 32,
                          (size_t)G::kWarps * G::kWarp, dev.device) < 1)
    return cudaErrorInvalidConfiguration;
  const int per = warps / p.split;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((p.units + per - 1) / per), (unsigned)((p.M + 8 * NT - 1) / (8 * NT)));
  cfg.blockDim = dim3((unsigned)warps * 32);
  cfg.dynamicSmemBytes = (size_t)warps * G::kWarp;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool MX, int MT>
cudaError_t launch_w4(const W4Params& p, int warps, const dph::DeviceInfo& dev, cudaStream_t s) {
  if (p.M <= 8) return launch_for<MX, MT, 1>(p, warps, dev, s);
  if (p.M <= 16) return launch_for<MX, MT, 2>(p, warps, dev, s);
  return launch_for<MX, MT, 4>(p, warps, dev, s);
}

using dph::aligned;
using dph::clash;
using dph::Span;
using dph::span_of;

constexpr int kMaxTokens = 65535 * 8;  // the grid's second dimension

}  // namespace

extern "C" {

dp_status_t dp_allgather_linear_w4(const void* x, int M, int D, long long ld,
                                   const dp_mx4_t* w_shards, int K, int F_shard,
                                   dp_mx4_format_t format, void* y, dp_dtype_t y_dtype,
                                   dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_allgather_linear_w4");
  if (!w_shards || K < 1 || K > DP_MAX_K) return DP_ERR_INVALID_ARG;
  if (M < 0 || D < 0 || F_shard < 0 || ld < D) return DP_ERR_INVALID_ARG;
  if (format != DP_MXFP4 && format != DP_NVFP4) return DP_ERR_UNSUPPORTED;
  if (y_dtype != DP_FP32 && y_dtype != DP_BF16) return DP_ERR_UNSUPPORTED;
  if (D % 32 || F_shard % 16) return DP_ERR_UNSUPPORTED;
  if ((long long)K * F_shard > 0x7fffff00ll || M > kMaxTokens || D > 0x7fffff00)
    return DP_ERR_UNSUPPORTED;
  const size_t ysz = y_dtype == DP_FP32 ? 4 : 2;
  if (!aligned(x, 2) || !aligned(y, ysz)) return DP_ERR_UNSUPPORTED;
  const int F = K * F_shard;
  if (M == 0 || F == 0) return DP_OK;
  if (!y || (!x && D)) return DP_ERR_INVALID_ARG;
  const Span out = span_of(y, (size_t)M * F * ysz);
  if (D && clash(out, span_of(x, ((size_t)(M - 1) * (size_t)ld + (size_t)D) * 2)))
    return DP_ERR_ALIAS;
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
    if (clash(out, span_of(w.codes, (size_t)F_shard * (D / 2))) ||
        clash(out, span_of(w.scales, sbytes)) ||
        (w.tensor_scale && clash(out, span_of(w.tensor_scale, 4))))
      return DP_ERR_ALIAS;
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
  // Rows of a warp and the warps that share them: 64 rows (x is converted once
  // for all of them) while they make 8 warps an SM with d in four shares, else 32;
  // d in as many shares, up to a CTA's warps, as have a step each.
  const int chunks = (D + kStep - 1) / kStep;
  const long long tiles = (long long)K * p.tiles_f;
  const bool wide = tiles * 2 * 4 >= 8ll * dev.sm_count;
  p.units = (int)std::min<long long>(tiles * (wide ? 2 : 4), 0x7fffffffll);
  p.split = wide ? 4 : 8;
  while (p.split > chunks) p.split /= 2;
  const int warps = p.split < 4 ? 4 : p.split;
  cudaError_t e;
  if (format == DP_MXFP4)
    e = wide ? launch_w4<true, 4>(p, warps, dev, s) : launch_w4<true, 2>(p, warps, dev, s);
  else
    e = wide ? launch_w4<false, 4>(p, warps, dev, s) : launch_w4<false, 2>(p, warps, dev, s);
  return e == cudaSuccess ? DP_OK : DP_ERR_CUDA;
}

}  // extern "C"
