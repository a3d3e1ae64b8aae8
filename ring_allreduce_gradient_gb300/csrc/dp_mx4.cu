// dp_mx4.cu -- quantisation of row shards to microscaled 4-bit matrices, as
// they are or transposed, and their decoding.
//
// mxfp4: a block's scale is 2^(floor(log2(amax)) - 2), which puts its largest
// magnitude in [4, 8); what lies above 6 saturates.  The quotient by a power
// of two is exact, so each value is rounded once.
// nvfp4: with t the tensor's scale, a block's scale is s = e4m3(amax / 6 / t)
// and its values are e2m1(x / (s t)): the tensor's scale takes the largest
// block's s to the top of e4m3, s takes the block's largest value to 6.  The
// quotient is a true division (rounded once in fp32): bf16 inputs often fall
// exactly between two values, and a product with a rounded reciprocal would
// break such ties to either side.
// A block of zeros has scale 0 (mxfp4: 2^-127); a block that holds a NaN or
// an infinity has a NaN scale.
//
// Bound by memory: 2 bytes read and 0.53 / 0.56 written for each bf16 value.
// Rows form: a warp takes 256 columns of a row, a lane eight of them, so a
// block is 2 or 4 neighbouring lanes.  Transposed form: blocks run down the
// columns, so a lane takes two neighbouring columns and reads 64 rows of
// them (a warp reads 128 contiguous bytes of each bf16 row): a block's
// largest value needs no exchange, and a lane ends with 32 contiguous bytes
// of each of its two output rows.  Neither goes through shared memory.

#include "dp_launch.h"
#include "dp_mx4.cuh"

#include <algorithm>
#include <cstring>

namespace {

using namespace dpk;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

struct QuantParams {
  const void* x[kMaxK];
  int rows;        // of one shard
  int in_rows;     // of all
  int cols;
  long long ld;    // elements between rows of a shard
  int vec_ok;
  int R, L;        // the output: R rows of L values (blocks run along L)
  int col_tiles;
  const float* tscale;
  uint8_t* codes;
  uint8_t* scales;
};

__device__ __forceinline__ const void* row_at(const QuantParams& p, int r, int esz) {
  const int k = r < p.rows ? 0 : r / p.rows;
  return static_cast<const uint8_t*>(p.x[k]) +
         (long long)(r - k * p.rows) * p.ld * esz;
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

// A block's scale byte from its largest magnitude, and what its values are
// divided by (nvfp4) or multiplied by (mxfp4); `zero`: every code is zero.
template <int BLOCK>
__device__ __forceinline__ uint32_t block_scale(float amax, float t, float& f, bool& zero) {
  const uint32_t bits = __float_as_uint(amax);
  const bool finite = bits < 0x7f800000u;
  if constexpr (BLOCK == kMxBlock) {
    const int e = (int)(bits >> 23) - 2;
    const uint32_t byte = finite ? (uint32_t)max(e, 0) : 255u;
    f = __uint_as_float((254u - byte) << 23);
    zero = !finite;
    return byte;
  } else {
    uint16_t c;
    const float s = amax > 0.0f ? __fdiv_rn(__fmul_rn(amax, 1.0f / 6.0f), t) : 0.0f;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.0f), "f"(s));
    const uint32_t byte = finite ? (uint32_t)c & 0xffu : 0x7fu;
    f = __fmul_rn(e4m3_value(byte), t);
    zero = !(f > 0.0f);
    return byte;
  }
}

template <int BLOCK>
__device__ __forceinline__ float scaled(float x, float f, bool zero) {
  if (zero) return 0.0f;
  return BLOCK == kMxBlock ? __fmul_rn(x, f) : __fdiv_rn(x, f);
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                 "=f"(v[6]), "=f"(v[7])
               : "l"(p));
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  uint4 raw[1];
  Vec8<uint16_t>::load(p, raw);
  Vec8<uint16_t>::widen(raw, v);
}

// Where the four scales of (row, column tile) lie.
__device__ __forceinline__ size_t scale_at(int row, int tile, int col_tiles) {
  return ((size_t)(row / kScaleRows) * col_tiles + tile) * kScaleTile + (row % 32) * 16 +
         (row % kScaleRows) / 32 * 4;
}

// ---- rows form ---------------------------------------------------------------

template <typename T, int BLOCK>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(const __grid_constant__ QuantParams p) {
  constexpr int kLanes = BLOCK / 8;  // lanes of a block
  const int lane = threadIdx.x & 31;
  const int segs = (p.col_tiles * 4 * BLOCK + 255) / 256;
  const long long units = (long long)((p.R + kScaleRows - 1) / kScaleRows * kScaleRows) * segs;
  const float t = BLOCK == kNvBlock && p.tscale ? __ldg(p.tscale) : 1.0f;
  for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units;
       u += (long long)gridDim.x * kWarps) {
    const int r = (int)(u / segs);
    const int e = (int)(u - (long long)r * segs) * 256 + lane * 8;
    const bool in = r < p.R && e < p.L;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (in) {
      const T* x = static_cast<const T*>(row_at(p, r, sizeof(T))) + e;
      if (p.vec_ok) {
        load8(x, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = widen_scalar(x, i);
      }
    }
    uint32_t top = 0;  // magnitudes order as their bits, NaN above all
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < kLanes; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    float f;
    bool zero;
    uint32_t byte = block_scale<BLOCK>(__uint_as_float(top), t, f, zero);
    if (!in) byte = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = scaled<BLOCK>(v[i], f, zero);
    if (in)
      *reinterpret_cast<uint32_t*>(p.codes + (size_t)r * (p.L / 2) + e / 2) = pack_e2m1(v);
    uint32_t four = byte;
#pragma unroll
    for (int i = 1; i < 4; ++i)
      four |= __shfl_down_sync(0xffffffffu, byte, i * kLanes) << (8 * i);
    const int tile = e / (4 * BLOCK);
    if (lane % (4 * kLanes) == 0 && tile < p.col_tiles)
      *reinterpret_cast<uint32_t*>(p.scales + scale_at(r, tile, p.col_tiles)) = four;
  }
}

// ---- transposed form ----------------------------------------------------------

__device__ __forceinline__ void load2(const float* p, bool vec, bool two, float& a, float& b) {
  if (vec) {
    const float2 v = __ldg(reinterpret_cast<const float2*>(p));
    a = v.x;
    b = v.y;
  } else {
    a = __ldg(p);
    b = two ? __ldg(p + 1) : 0.0f;
  }
}
__device__ __forceinline__ void load2(const uint16_t* p, bool vec, bool two, float& a, float& b) {
  if (vec) {
    const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(p));
    a = bf16lo(v);
    b = bf16hi(v);
  } else {
    a = widen_scalar(p, 0);
    b = two ? widen_scalar(p, 1) : 0.0f;
  }
}

constexpr int kTRows = 64;  // input rows a warp takes at once: 32 bytes of each output row

template <typename T, int BLOCK>
__global__ void __launch_bounds__(kThreads) quant_cols_kernel(const __grid_constant__ QuantParams p) {
  constexpr int kBlocks = kTRows / BLOCK;
  const int lane = threadIdx.x & 31;
  const int cgroups = (p.R + kScaleRows - 1) / kScaleRows * 2;  // 64 columns each
  const long long units = (long long)cgroups * ((p.col_tiles * 4 * BLOCK + kTRows - 1) / kTRows);
  const float t = BLOCK == kNvBlock && p.tscale ? __ldg(p.tscale) : 1.0f;
  for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units;
       u += (long long)gridDim.x * kWarps) {
    const int g = (int)(u / cgroups);
    const int c = (int)(u - (long long)g * cgroups) * 64 + lane * 2;  // input column = output row
    const int l0 = g * kTRows;
    const bool in = c < p.R, two = c + 1 < p.R;
    uint32_t code[2][kTRows / 8];
    uint32_t sc[2] = {0, 0};
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const int l = l0 + b * BLOCK;  // L is a multiple of 32: a block is inside or outside
      float v[2][BLOCK];
      const bool inside = in && l < p.L;
#pragma unroll
      for (int i = 0; i < BLOCK; ++i) {
        v[0][i] = v[1][i] = 0.0f;
        if (inside)
          load2(static_cast<const T*>(row_at(p, l + i, sizeof(T))) + c, p.vec_ok && two, two,
                v[0][i], v[1][i]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < BLOCK; ++i) top = max(top, __float_as_uint(v[j][i]) & 0x7fffffffu);
        float f;
        bool zero;
        const uint32_t byte = block_scale<BLOCK>(__uint_as_float(top), t, f, zero);
        if (inside && (j == 0 || two)) sc[j] |= byte << (8 * b);
#pragma unroll
        for (int i = 0; i < BLOCK / 8; ++i) {
          float w[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) w[q] = scaled<BLOCK>(v[j][8 * i + q], f, zero);
          code[j][b * (BLOCK / 8) + i] = pack_e2m1(w);
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
      const int tile = l0 / (4 * BLOCK);
      uint8_t* s = p.scales + scale_at(c + j, tile, p.col_tiles);
      if (tile < p.col_tiles) {
        if constexpr (kBlocks == 4)
          *reinterpret_cast<uint32_t*>(s) = sc[j];
        else
          *reinterpret_cast<uint16_t*>(s + (l0 / BLOCK) % 4) = (uint16_t)sc[j];
      }
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

template <typename T, int BLOCK>
__global__ void __launch_bounds__(kThreads) decode_kernel(const __grid_constant__ DecodeParams p) {
  const float t = BLOCK == kNvBlock && p.tscale ? __ldg(p.tscale) : 1.0f;
  const int lane = threadIdx.x & 31;
  const int segs = (p.L + 255) / 256;
  const long long units = (long long)p.R * segs;
  for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units;
       u += (long long)gridDim.x * kWarps) {
    const int r = (int)(u / segs);
    const int e = (int)(u - (long long)r * segs) * 256 + lane * 8;
    if (e >= p.L) continue;
    const int b = e / BLOCK;
    const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(p.codes + (size_t)r * (p.L / 2) + e / 2));
    const uint32_t byte = __ldg(p.scales + scale_at(r, b / 4, p.col_tiles) + b % 4);
    float step;
    if constexpr (BLOCK == kMxBlock)  // 2^(byte - 127): a subnormal at 0
      step = byte == 255 ? __uint_as_float(0x7fffffffu)
                         : (byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u));
    else
      step = __fmul_rn(e4m3_value(byte), t);
    float v[8];
    unpack_e2m1(c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], step);
    store8(static_cast<T*>(p.out) + (size_t)r * p.L + e, v);
  }
}

template <typename KernelT, typename P>
cudaError_t launch(KernelT kernel, const P& p, long long units, const dph::DeviceInfo& dev,
                   cudaStream_t s) {
  const int b = dph::prepare_kernel(reinterpret_cast<const void*>(kernel), kThreads, 0, dev.device);
  long long resident = (long long)dev.sm_count * (b < 1 ? 1 : b);
  const int limit = dph::stream_cta_limit();
  if (limit > 0 && resident > limit) resident = limit;
  const long long grid = std::max(1LL, std::min(resident, (units + kWarps - 1) / kWarps));
  kernel<<<(unsigned)grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int BLOCK>
cudaError_t quantize(const QuantParams& p, bool transpose, const dph::DeviceInfo& dev,
                     cudaStream_t s) {
  const long long rows = (p.R + kScaleRows - 1) / kScaleRows * kScaleRows;
  const long long cols = (long long)p.col_tiles * 4 * BLOCK;
  if (transpose)
    return launch(quant_cols_kernel<T, BLOCK>, p, rows / 64 * ((cols + kTRows - 1) / kTRows), dev, s);
  return launch(quant_rows_kernel<T, BLOCK>, p, rows * ((cols + 255) / 256), dev, s);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Span {
  uintptr_t lo, hi;
};
Span span_of(const void* p, size_t n) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + n};
}
bool clash(const Span& a, const Span& b) {
  return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo;
}

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
  if (all > 0x7fffff00ll || cols > 0x7fffff00) return DP_ERR_UNSUPPORTED;
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
    vec = vec && aligned(x[k], transpose ? 2 * esz : 8 * esz);
    p.x[k] = x[k];
  }
  if (tensor_scale) {
    const Span in = span_of(tensor_scale, 4);
    if (clash(in, out[0]) || clash(in, out[1])) return DP_ERR_ALIAS;
  }
  p.rows = rows;
  p.in_rows = (int)all;
  p.cols = cols;
  p.ld = ld;
  p.vec_ok = vec && ld % (transpose ? 2 : 8) == 0;
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
    e = format == DP_NVFP4 ? quantize<float, kNvBlock>(p, transpose, dev, s)
                           : quantize<float, kMxBlock>(p, transpose, dev, s);
  else
    e = format == DP_NVFP4 ? quantize<uint16_t, kNvBlock>(p, transpose, dev, s)
                           : quantize<uint16_t, kMxBlock>(p, transpose, dev, s);
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
  if (cols % 32 || cols > 0x7fffff00 || rows > 0x7fffff00) return DP_ERR_UNSUPPORTED;
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
  const long long units = (long long)rows * ((cols + 255) / 256);
  cudaError_t e;
  if (out_dtype == DP_FP32)
    e = format == DP_NVFP4 ? launch(decode_kernel<float, kNvBlock>, p, units, dev, s)
                           : launch(decode_kernel<float, kMxBlock>, p, units, dev, s);
  else
    e = format == DP_NVFP4 ? launch(decode_kernel<uint16_t, kNvBlock>, p, units, dev, s)
                           : launch(decode_kernel<uint16_t, kMxBlock>, p, units, dev, s);
  return e == cudaSuccess ? DP_OK : DP_ERR_CUDA;
}

}  // extern "C"
