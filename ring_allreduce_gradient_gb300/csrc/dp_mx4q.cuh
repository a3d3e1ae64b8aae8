// dp_mx4q.cuh -- the arithmetic of microscaled quantisation: values to codes and
// back, a block's scale from its largest magnitude, and sixteen elements of a
// row as a lane holds them.  Shared by the kernels that quantise (dp_mx4.cu,
// dp_mx8.cu, dp_norm.cu).
#pragma once

#include "dp_mx4.cuh"

namespace dpk {

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

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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

// The 8-bit form (mxfp8): a block of 32 has the smallest power of two, 2^-127 at
// least, that keeps its largest magnitude within e4m3's 448, so nothing saturates.
// Multiplying by a power of two is exact: each value is rounded once, by at most
// 2^-4 of itself where it is 2^-6 or more of the scale, 2^-10 of the scale below.
struct Scale8 {
  uint32_t byte;
  float f;
  bool bad;
  __device__ __forceinline__ explicit Scale8(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    bad = bits >= 0x7f800000u;
    const int e = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    byte = bad ? 255u : (uint32_t)max(e, 0);
    f = __uint_as_float((254u - byte) << 23);
  }
  // Four values, in pairs, to four codes, the first in the lowest byte.
  __device__ __forceinline__ uint32_t codes(uint64_t ab, uint64_t cd) const {
    float a, b, c, d;
    unpair(mul2(ab, pair(f, f)), a, b);
    unpair(mul2(cd, pair(f, f)), c, d);
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return bad ? 0u : r;
  }
};

// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float power_of(uint32_t byte) {
  if (byte == 255u) return __uint_as_float(0x7fffffffu);
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);  // 2^-127 is subnormal
}

// Where the four scales of (row, column tile) lie.
__device__ __forceinline__ size_t scale_at(int row, int tile, int col_tiles) {
  return ((size_t)(row / kScaleRows) * col_tiles + tile) * kScaleTile + (row % 32) * 16 +
         (row % kScaleRows) / 32 * 4;
}

}  // namespace dpk
