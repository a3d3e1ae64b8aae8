// dp_mx4.cu -- quantisation of row shards to microscaled 4-bit matrices, as
// they are or transposed, and their decoding.
//
// mxfp4: a block's scale is 2^(floor(log2(amax)) - 2), which puts its largest
// magnitude in [4, 8); what lies above 6 saturates.  The quotient by a power
// of two is exact, so each value is rounded once.
// nvfp4: with t the tensor's scale, a block's scale is s = e4m3(amax / 6 / t)
// and its values are e2m1(x / (s t)): the tensor's scale takes the largest
// block's s to the top of e4m3, s takes the block's largest value to 6; what
// lies above saturates.  Quotients are rounded once in fp32 (Divisor): bf16
// inputs often fall exactly between two values, and a product with a rounded
// reciprocal would break such ties to either side.
// A block of zeros has scale 0 (mxfp4: 2^-127); a block that holds a NaN or
// an infinity has a NaN scale.
//
// Bound by memory: 2 bytes read and 0.53 / 0.56 written for each bf16 value.
// Rows form: a warp takes up to 2048 columns of a row with all its loads
// issued first, a lane sixteen columns of each 512, so a block is one lane
// (nvfp4) or two.  Transposed form: blocks run down the columns, so a lane
// takes two neighbouring columns and reads 64 rows of them (a warp reads 128
// contiguous bytes of each bf16 row): a block's largest value needs no
// exchange, a lane ends with 32 contiguous bytes of each of its two output
// rows, and the four warps of a CTA, one below the other, with a 128-byte
// line.  Neither goes through shared memory.  Measured on 8192 x 4096 bf16
// (GB300, launches in a CUDA graph): rows 13.9 us to nvfp4 and 10.8 to mxfp4
// (6.2 and 7.9 TB/s, part of it from L2), transposed 16.3 and 11.9, decoding
// 11.7.  The nvfp4 forms have two divisors a block more to compute, and no unit
// at its limit: 60 % of the SM and 70 % of DRAM for rows, 46 and 59 % transposed
// with a third of the warps resident, whose loads and arithmetic alternate.

#include "dp_early.cuh"
#include "dp_launch.h"
#include "dp_mx4.cuh"

#include <algorithm>
#include <cstring>

namespace {

using namespace dpk;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// Rows or columns of a matrix: the end of the widest share (2048 columns) that
// starts inside one has to be an int.
constexpr int kMaxSize = 0x7fff0000;

struct QuantParams {
  const void* x[kMaxK];
  int rows;        // of one shard
  long long ld;    // elements between rows of a shard
  int vec_ok;      // the loads of several elements are aligned
  int whole;       // each 32 concatenated rows lie in one shard
  int R, L;        // the output: R rows of L values (blocks run along L)
  int col_tiles;
  const float* tscale;
  uint8_t* codes;
  uint8_t* scales;
};

template <typename T>
__device__ __forceinline__ const T* row_at(const QuantParams& p, int r) {
  const int k = r < p.rows ? 0 : r / p.rows;
  return static_cast<const T*>(p.x[k]) + (long long)(r - k * p.rows) * p.ld;
}

// Eight fp32 values to eight e2m1 codes, the first in the lowest half byte.
__device__ __forceinline__ uint32_t pack_e2m1(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

__device__ __forceinline__ void widen_f16x2(uint32_t h, float& lo, float& hi) {
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}
__device__ __forceinline__ void unpack_e2m1(uint32_t c, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int i = 0; i < 4; ++i) widen_f16x2(h[i], v[2 * i], v[2 * i + 1]);
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)byte));
  float lo, hi;
  widen_f16x2(h, lo, hi);
  return lo;
}

// Division by a value that many others are divided by, as a product with its
// reciprocal in two words: hi is within e < 2^-22 of it (relative), lo takes up
// what hi misses and leaves e^2, so hi + lo is within 2^-44.  x hi is rounded
// once, together with x lo, so the result is the rounded quotient unless the
// quotient lies within 2^-44 of a midpoint between two fp32 values; a quotient
// that is an fp32 value, a tie between two codes among them, comes out exactly.
// (8192 x 4096 bf16 to nvfp4, in the kernel's first form: 43.9 us with
// __fdiv_rn for every value, 23.5 us with this and the loads issued first.)
// Divisors too far from 1 for the two words take the division, and so do values
// above 1e30 divisors: x lo would overflow by itself and give the quotient the
// sign of lo.
struct Divisor {
  float d, hi, lo, far;
  bool near;
  __device__ __forceinline__ explicit Divisor(float v) : d(v) {
    near = v > 1e-30f && v < 1e30f;
    far = __fmul_rn(v, 1e30f);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(hi) : "f"(v));
    lo = __fmul_rn(__fmaf_rn(-hi, v, 1.0f), hi);
  }
  // Whether the two words serve for magnitudes up to x.
  __device__ __forceinline__ bool fits(float x) const { return near && x <= far; }
  __device__ __forceinline__ float of(float x) const {
    return fits(x) ? __fmaf_rn(x, hi, __fmul_rn(x, lo)) : __fdiv_rn(x, d);
  }
};

// Two fp32 operations in one instruction, each lane of the pair rounded by itself.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The tensor's scale, and a block's: its byte from the block's largest
// magnitude, and eight of its values to codes.
template <int BLOCK>
struct Scale;

template <>
struct Scale<kMxBlock> {
  uint32_t byte;
  float f;
  bool zero;
  __device__ __forceinline__ Scale(float amax, float, const Divisor&) {
    const uint32_t bits = __float_as_uint(amax);
    zero = bits >= 0x7f800000u;
    byte = zero ? 255u : (uint32_t)max((int)(bits >> 23) - 2, 0);
    f = __uint_as_float((254u - byte) << 23);
  }
  __device__ __forceinline__ uint32_t codes(const float (&v)[8]) const {
    float w[8];
    const uint64_t ff = pair(f, f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) unpair(mul2(pair(v[i], v[i + 1]), ff), w[i], w[i + 1]);
    return zero ? 0u : pack_e2m1(w);
  }
};

template <>
struct Scale<kNvBlock> {
  uint32_t byte;
  float step;
  Divisor by;
  bool fits;
  __device__ __forceinline__ Scale(float amax, float t, const Divisor& by_t) : by(1.0f) {
    uint16_t c;
    const float s = amax > 0.0f ? by_t.of(__fmul_rn(amax, 1.0f / 6.0f)) : 0.0f;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.0f), "f"(s));
    byte = __float_as_uint(amax) < 0x7f800000u ? (uint32_t)c & 0xffu : 0x7fu;
    step = __fmul_rn(e4m3_value(byte), t);
    by = Divisor(step);
    fits = by.fits(amax);
  }
  __device__ __forceinline__ uint32_t codes(const float (&v)[8]) const {
    if (!(step > 0.0f)) return 0u;  // a block of zeros, or a NaN step
    float w[8];
    if (fits) {
      const uint64_t hi = pair(by.hi, by.hi), lo = pair(by.lo, by.lo);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint64_t x = pair(v[i], v[i + 1]);
        unpair(fma2(x, hi, mul2(x, lo)), w[i], w[i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __fdiv_rn(v[i], step);
    }
    return pack_e2m1(w);
  }
};

// Sixteen consecutive elements as they were loaded, from a 32-byte boundary:
// bf16 ones stay in pairs until they are needed, for their registers' sake.
// Magnitudes order as their bits, NaN above all.
template <typename T>
struct Sixteen;

template <>
struct Sixteen<float> {
  float v[16];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int h = 0; h < 16; h += 8)
      asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=f"(v[h]), "=f"(v[h + 1]), "=f"(v[h + 2]), "=f"(v[h + 3]), "=f"(v[h + 4]),
                     "=f"(v[h + 5]), "=f"(v[h + 6]), "=f"(v[h + 7])
                   : "l"(p + h));
  }
  __device__ __forceinline__ void each(const float* p, bool in) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = in ? p[i] : 0.0f;
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) t = max(t, __float_as_uint(v[i]) & 0x7fffffffu);
    return t;
  }
  __device__ __forceinline__ void widen(int half, float (&w)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[8 * half + i];
  }
};

// The larger magnitude of each half of two pairs of bf16.
__device__ __forceinline__ uint32_t max_abs2(uint32_t t, uint32_t v) {
  return __vmaxu2(t, v & 0x7fff7fffu);
}

template <>
struct Sixteen<uint16_t> {
  uint32_t r[8];
  __device__ __forceinline__ void load(const uint16_t* p) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
  }
  __device__ __forceinline__ void each(const uint16_t* p, bool in) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      r[i] = in ? (uint32_t)p[2 * i] | (uint32_t)p[2 * i + 1] << 16 : 0u;
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max_abs2(t, r[i]);
    return max(t & 0xffff0000u, t << 16);
  }
  __device__ __forceinline__ void widen(int half, float (&w)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[2 * i] = bf16lo(r[4 * half + i]);
      w[2 * i + 1] = bf16hi(r[4 * half + i]);
    }
  }
};

// Where the four scales of (row, column tile) lie.
__device__ __forceinline__ size_t scale_at(int row, int tile, int col_tiles) {
  return ((size_t)(row / kScaleRows) * col_tiles + tile) * kScaleTile + (row % 32) * 16 +
         (row % kScaleRows) / 32 * 4;
}

// ---- rows form ---------------------------------------------------------------

// One row's G x 512 columns from e0 on, by a warp.
template <typename T, int BLOCK, int G>
__device__ __forceinline__ void quant_row(const QuantParams& p, int r, int e0, bool vec, float t,
                                          const Divisor& by_t) {
  const int lane = threadIdx.x & 31;
  Sixteen<T> v[G];
  const T* x = r < p.R ? row_at<T>(p, r) : nullptr;
  if (x && vec && e0 + G * 512 <= p.L) {
#pragma unroll
    for (int g = 0; g < G; ++g) v[g].load(x + e0 + g * 512 + lane * 16);
  } else {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int e = e0 + g * 512 + lane * 16;
      v[g].each(x + e, x && e < p.L);  // L is a multiple of 32: all sixteen are inside or none
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int e = e0 + g * 512 + lane * 16;
    const bool in = x && e < p.L;
    uint32_t top = v[g].top();
    if (BLOCK == kMxBlock) top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const Scale<BLOCK> s(__uint_as_float(top), t, by_t);
    if (in) {
      uint32_t c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float w[8];
        v[g].widen(h, w);
        c[h] = s.codes(w);
      }
      *reinterpret_cast<uint2*>(p.codes + (size_t)r * (p.L / 2) + e / 2) = make_uint2(c[0], c[1]);
    }
    const int b = e / BLOCK;
    if (b / 4 < p.col_tiles && (BLOCK == kNvBlock || lane % 2 == 0))
      p.scales[scale_at(r, b / 4, p.col_tiles) + b % 4] = in ? (uint8_t)s.byte : (uint8_t)0;
  }
}

template <typename T, int BLOCK, int G>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(const __grid_constant__ QuantParams p) {
  stream_order();
  const unsigned groups = ((unsigned)p.col_tiles * 4 * BLOCK + G * 512 - 1) / (G * 512);
  const unsigned blocks = ((unsigned)p.R + kScaleRows - 1) / kScaleRows * (kScaleRows / kWarps) * groups;
  const float t = BLOCK == kNvBlock && p.tscale ? *p.tscale : 1.0f;
  const Divisor by_t(t);
  for (unsigned b = blockIdx.x; b < blocks; b += gridDim.x) {
    const unsigned q = b / groups;
    quant_row<T, BLOCK, G>(p, (int)(q * kWarps + (threadIdx.x >> 5)), (int)((b - q * groups) * G * 512),
                           p.vec_ok, t, by_t);
  }
}

// ---- transposed form ----------------------------------------------------------

// Two neighbouring columns of a row.
template <bool FAST>
__device__ __forceinline__ float2 load2(const float* x, int c, int last) {
  if constexpr (FAST) return *reinterpret_cast<const float2*>(x + c);
  return make_float2(x[c], x[min(c + 1, last)]);
}
template <bool FAST>
__device__ __forceinline__ uint32_t load2(const uint16_t* x, int c, int last) {
  if constexpr (FAST) return *reinterpret_cast<const uint32_t*>(x + c);
  return (uint32_t)x[c] | (uint32_t)x[min(c + 1, last)] << 16;
}
__device__ __forceinline__ float part(float2 v, int j) { return j ? v.y : v.x; }
__device__ __forceinline__ float part(uint32_t v, int j) { return j ? bf16hi(v) : bf16lo(v); }

// The two columns' largest magnitudes over N rows.
template <int N>
__device__ __forceinline__ void tops(const float2* v, uint32_t (&t)[2]) {
  t[0] = t[1] = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    t[0] = max(t[0], __float_as_uint(v[i].x) & 0x7fffffffu);
    t[1] = max(t[1], __float_as_uint(v[i].y) & 0x7fffffffu);
  }
}
template <int N>
__device__ __forceinline__ void tops(const uint32_t* v, uint32_t (&t)[2]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max_abs2(m, v[i]);
  t[0] = m << 16;
  t[1] = m & 0xffff0000u;
}

template <typename T>
struct Pair;
template <>
struct Pair<float> {
  using type = float2;
};
template <>
struct Pair<uint16_t> {
  using type = uint32_t;
};

constexpr int kTRows = 64;  // input rows a warp takes at once: 32 bytes of each output row

// FAST: two columns are one aligned load, R is even and 32 rows lie in one
// shard.  Otherwise columns past the last are read as the last (and dropped),
// so that no load hangs on a branch.
template <typename T, int BLOCK, bool FAST>
__global__ void __launch_bounds__(kThreads) quant_cols_kernel(const __grid_constant__ QuantParams p) {
  constexpr int kBlocks = kTRows / BLOCK;
  stream_order();
  const int lane = threadIdx.x & 31;
  const unsigned cgroups = ((unsigned)p.R + kScaleRows - 1) / kScaleRows * 2;  // 64 columns each
  const unsigned rgroups = ((unsigned)p.col_tiles * 4 * BLOCK + kTRows * kWarps - 1) / (kTRows * kWarps);
  const float t = BLOCK == kNvBlock && p.tscale ? *p.tscale : 1.0f;
  const Divisor by_t(t);
  for (unsigned u = blockIdx.x; u < cgroups * rgroups; u += gridDim.x) {
    const unsigned q = u / cgroups;
    const int c = (int)(u - q * cgroups) * 64 + lane * 2;  // input column = output row
    const int l0 = (int)(q * kWarps + (threadIdx.x >> 5)) * kTRows;
    if (l0 >= p.col_tiles * 4 * BLOCK) continue;
    const int cl = min(c, FAST ? p.R - 2 : p.R - 1);
    uint32_t code[2][kTRows / 8];
    uint32_t sc[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int l = l0 + 32 * h;
      if (l >= p.L) continue;  // L is a multiple of 32
      typename Pair<T>::type v[32];
      const T* x = row_at<T>(p, l);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (!FAST && !p.whole && i) x = row_at<T>(p, l + i);
        v[i] = load2<FAST>(x, cl, p.R - 1);
        if (FAST || p.whole) x += p.ld;
      }
#pragma unroll
      for (int b = 0; b < 32 / BLOCK; ++b) {
        uint32_t top[2];
        tops<BLOCK>(v + b * BLOCK, top);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const Scale<BLOCK> s(__uint_as_float(top[j]), t, by_t);
          if (c + j < p.R) sc[j] |= s.byte << (8 * (h * (32 / BLOCK) + b));
#pragma unroll
          for (int i = 0; i < BLOCK / 8; ++i) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = part(v[b * BLOCK + 8 * i + e], j);
            code[j][4 * h + b * (BLOCK / 8) + i] = s.codes(w);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (c + j < p.R) {
        uint8_t* out = p.codes + (size_t)(c + j) * (p.L / 2) + l0 / 2;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (l0 + 32 * h < p.L)
            *reinterpret_cast<uint4*>(out + 16 * h) = make_uint4(
                code[j][4 * h], code[j][4 * h + 1], code[j][4 * h + 2], code[j][4 * h + 3]);
      }
      // the scales of 64 rows: a tile's four (nvfp4) or half of them (mxfp4)
      uint8_t* s = p.scales + scale_at(c + j, l0 / (4 * BLOCK), p.col_tiles);
      if constexpr (kBlocks == 4)
        *reinterpret_cast<uint32_t*>(s) = sc[j];
      else
        *reinterpret_cast<uint16_t*>(s + (l0 / BLOCK) % 4) = (uint16_t)sc[j];
    }
  }
}

// ---- decoding ------------------------------------------------------------------

struct DecodeParams {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* tscale;
  void* out;
  int R, L, col_tiles;
};

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) { store8_f32(p, v); }
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) { store8_bf16(p, v); }

template <int BLOCK>
__device__ __forceinline__ float step_of(uint32_t byte, float t) {
  if constexpr (BLOCK == kNvBlock) return __fmul_rn(e4m3_value(byte), t);
  if (byte == 255u) return __uint_as_float(0x7fffffffu);
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);  // 2^-127 is subnormal
}

// A warp takes G x 256 columns of a row, a lane eight of each 256.
template <typename T, int BLOCK, int G>
__global__ void __launch_bounds__(kThreads) decode_kernel(const __grid_constant__ DecodeParams p) {
  stream_order();
  const float t = BLOCK == kNvBlock && p.tscale ? *p.tscale : 1.0f;
  const int lane = threadIdx.x & 31;
  const unsigned groups = ((unsigned)p.L + G * 256 - 1) / (G * 256);
  const unsigned blocks = ((unsigned)p.R + kWarps - 1) / kWarps * groups;
  for (unsigned u = blockIdx.x; u < blocks; u += gridDim.x) {
    const unsigned q = u / groups;
    const int r = (int)(q * kWarps + (threadIdx.x >> 5));
    const int e0 = (int)((u - q * groups) * G * 256) + lane * 8;
    if (r >= p.R) continue;
    const uint8_t* codes = p.codes + (size_t)r * (p.L / 2);
    uint32_t c[G], byte[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int e = min(e0 + g * 256, p.L - 8);  // past the end: the last, and dropped
      const int b = e / BLOCK;
      c[g] = *reinterpret_cast<const uint32_t*>(codes + e / 2);
      byte[g] = p.scales[scale_at(r, b / 4, p.col_tiles) + b % 4];
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int e = e0 + g * 256;
      const float step = step_of<BLOCK>(byte[g], t);
      float v[8];
      unpack_e2m1(c[g], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], step);
      if (e < p.L) store8(static_cast<T*>(p.out) + (size_t)r * p.L + e, v);
    }
  }
}

// One CTA for each share of the work, which the hardware hands out as SMs
// become free; under a CTA limit the CTAs go over the shares.
template <typename P>
cudaError_t launch(void (*kernel)(P), const P& p, long long blocks, cudaStream_t s) {
  const int limit = dph::stream_cta_limit();
  if (limit > 0) blocks = std::min<long long>(blocks, limit);
  return dph::launch_early(kernel, p, (unsigned)std::min<long long>(blocks, 0x7fffffffll), kThreads,
                           s);
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Whether there is work enough to fill the GPU with warps that take `span`
// columns of a row at once.  All loads of a warp are in flight together: 8192 x
// 4096 bf16 to nvfp4 18.8 us with 512 columns, 15.7 with 1024, 14.1 with 2048;
// short calls spread wider instead.
bool wide(long long rows, long long cols, int span) {
  return cols >= span && rows * cols >= (1ll << 11) * span;
}

template <typename T, int BLOCK>
cudaError_t quantize(const QuantParams& p, bool transpose, cudaStream_t s) {
  const long long rows = ceil_div(p.R, kScaleRows) * kScaleRows;
  const long long cols = (long long)p.col_tiles * 4 * BLOCK;
  if (transpose) {
    const long long blocks = rows / 64 * ceil_div(cols, kTRows * kWarps);
    if (p.vec_ok && p.whole && p.R % 2 == 0)
      return launch(quant_cols_kernel<T, BLOCK, true>, p, blocks, s);
    return launch(quant_cols_kernel<T, BLOCK, false>, p, blocks, s);
  }
  if (wide(p.R, p.L, 2048))
    return launch(quant_rows_kernel<T, BLOCK, 4>, p, rows / kWarps * ceil_div(cols, 2048), s);
  if (wide(p.R, p.L, 1024))
    return launch(quant_rows_kernel<T, BLOCK, 2>, p, rows / kWarps * ceil_div(cols, 1024), s);
  return launch(quant_rows_kernel<T, BLOCK, 1>, p, rows / kWarps * ceil_div(cols, 512), s);
}

template <typename T, int BLOCK>
cudaError_t decode(const DecodeParams& p, cudaStream_t s) {
  if (wide(p.R, p.L, 1024))
    return launch(decode_kernel<T, BLOCK, 4>, p, ceil_div(p.R, kWarps) * ceil_div(p.L, 1024), s);
  return launch(decode_kernel<T, BLOCK, 1>, p, ceil_div(p.R, kWarps) * ceil_div(p.L, 256), s);
}

using dph::aligned;
using dph::clash;
using dph::Span;
using dph::span_of;

}  // namespace

extern "C" {

dp_status_t dp_mx4_scales_size(int rows, int cols, dp_mx4_format_t format, size_t* bytes) {
  if (!bytes) return DP_ERR_INVALID_ARG;
  *bytes = 0;
  if (rows < 0 || cols < 0) return DP_ERR_INVALID_ARG;
  if (format != DP_MXFP4 && format != DP_NVFP4) return DP_ERR_UNSUPPORTED;
  *bytes = ((size_t)rows + kScaleRows - 1) / kScaleRows *
           (((size_t)cols + 4 * mx4_block(format) - 1) / (4 * mx4_block(format))) * kScaleTile;
  return DP_OK;
}

dp_status_t dp_mx4_quantize(const void* const* x, int K, int rows, int cols, long long ld,
                            dp_dtype_t x_dtype, dp_mx4_format_t format, int transpose,
                            const float* tensor_scale, void* codes, void* scales,
                            dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_mx4_quantize");
  if (!x || K < 1 || K > DP_MAX_K) return DP_ERR_INVALID_ARG;
  if (rows < 0 || cols < 0 || ld < cols) return DP_ERR_INVALID_ARG;
  if (x_dtype != DP_FP32 && x_dtype != DP_BF16) return DP_ERR_UNSUPPORTED;
  if (format != DP_MXFP4 && format != DP_NVFP4) return DP_ERR_UNSUPPORTED;
  if (tensor_scale && format != DP_NVFP4) return DP_ERR_INVALID_ARG;
  const size_t esz = x_dtype == DP_FP32 ? 4 : 2;
  const long long all = (long long)K * rows;
  if (all > kMaxSize || cols > kMaxSize) return DP_ERR_UNSUPPORTED;
  const int R = transpose ? cols : (int)all, L = transpose ? (int)all : cols;
  if (L % 32) return DP_ERR_UNSUPPORTED;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(tensor_scale, 4))
    return DP_ERR_UNSUPPORTED;
  if (R == 0 || L == 0) return DP_OK;  // an empty matrix has no buffers
  if (!codes || !scales) return DP_ERR_INVALID_ARG;
  size_t sbytes = 0;
  dp_mx4_scales_size(R, L, format, &sbytes);
  const Span out[2] = {span_of(codes, (size_t)R * (L / 2)), span_of(scales, sbytes)};
  if (clash(out[0], out[1])) return DP_ERR_ALIAS;
  QuantParams p{};
  bool vec = true;
  for (int k = 0; k < K; ++k) {
    if (!x[k]) return DP_ERR_INVALID_ARG;
    if (!aligned(x[k], esz)) return DP_ERR_UNSUPPORTED;
    const Span in = span_of(x[k], ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * esz);
    if (clash(in, out[0]) || clash(in, out[1])) return DP_ERR_ALIAS;
    vec = vec && aligned(x[k], transpose ? 2 * esz : 32);
    p.x[k] = x[k];
  }
  if (tensor_scale) {
    const Span in = span_of(tensor_scale, 4);
    if (clash(in, out[0]) || clash(in, out[1])) return DP_ERR_ALIAS;
  }
  p.rows = rows;
  p.whole = K == 1 || rows % 32 == 0;
  p.ld = ld;
  p.vec_ok = vec && ld % (transpose ? 2 : 16) == 0;
  p.R = R;
  p.L = L;
  p.col_tiles = mx4_col_tiles(L, mx4_block(format));
  p.tscale = tensor_scale;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  dph::DeviceInfo dev;
  if (!dph::current_device(&dev)) return DP_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (x_dtype == DP_FP32)
    e = format == DP_NVFP4 ? quantize<float, kNvBlock>(p, transpose, s)
                           : quantize<float, kMxBlock>(p, transpose, s);
  else
    e = format == DP_NVFP4 ? quantize<uint16_t, kNvBlock>(p, transpose, s)
                           : quantize<uint16_t, kMxBlock>(p, transpose, s);
  return e == cudaSuccess ? DP_OK : DP_ERR_CUDA;
}

dp_status_t dp_mx4_dequantize(const void* codes, const void* scales, int rows, int cols,
                              dp_mx4_format_t format, const float* tensor_scale, void* out,
                              dp_dtype_t out_dtype, dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_mx4_dequantize");
  if (rows < 0 || cols < 0) return DP_ERR_INVALID_ARG;
  if (out_dtype != DP_FP32 && out_dtype != DP_BF16) return DP_ERR_UNSUPPORTED;
  if (format != DP_MXFP4 && format != DP_NVFP4) return DP_ERR_UNSUPPORTED;
  if (tensor_scale && format != DP_NVFP4) return DP_ERR_INVALID_ARG;
  if (cols % 32 || cols > kMaxSize || rows > kMaxSize) return DP_ERR_UNSUPPORTED;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 16) || !aligned(tensor_scale, 4))
    return DP_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return DP_OK;
  if (!codes || !scales || !out) return DP_ERR_INVALID_ARG;
  size_t sbytes = 0;
  dp_mx4_scales_size(rows, cols, format, &sbytes);
  const Span w = span_of(out, (size_t)rows * cols * (out_dtype == DP_FP32 ? 4 : 2));
  if (clash(w, span_of(codes, (size_t)rows * (cols / 2))) || clash(w, span_of(scales, sbytes)) ||
      (tensor_scale && clash(w, span_of(tensor_scale, 4))))
    return DP_ERR_ALIAS;
  DecodeParams p{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales),
                 tensor_scale, out, rows, cols, mx4_col_tiles(cols, mx4_block(format))};
  dph::DeviceInfo dev;
  if (!dph::current_device(&dev)) return DP_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (out_dtype == DP_FP32)
    e = format == DP_NVFP4 ? decode<float, kNvBlock>(p, s)
                           : decode<float, kMxBlock>(p, s);
  else
    e = format == DP_NVFP4 ? decode<uint16_t, kNvBlock>(p, s)
                           : decode<uint16_t, kMxBlock>(p, s);
  return e == cudaSuccess ? DP_OK : DP_ERR_CUDA;
}

}  // extern "C"
