// dp_mx8.cu -- quantisation of a matrix to the 8-bit microscaled form, and its
// decoding: e4m3 codes, one to a byte, with a power of two for each 32
// consecutive columns (the arithmetic: Scale8; the scales' tiles: dp_mx4.cuh).
//
// Bound by memory: 2 bytes read and 1.03 written for each bf16 value, and back.
// A warp takes G x 512 columns of a row with all its loads issued first, a lane
// sixteen columns of each 512, so a block is two lanes.  Measured on 8192 x 4096 bf16
// (GB300, launches in a CUDA graph): quantisation 16.5 us (102 MB: 6.2 TB/s),
// decoding 13.0 (7.8 TB/s, part of it from L2).

#include "dp_early.cuh"
#include "dp_launch.h"
#include "dp_mx4.cuh"
#include "dp_mx4q.cuh"

#include <algorithm>

namespace {

using namespace dpk;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSize = 0x7fff0000;  // the end of a share that starts inside a row is an int

struct Quant8Params {
  const void* x;
  long long ld;
  int R, L, col_tiles;
  int vec_ok;
  uint8_t* codes;
  uint8_t* scales;
};

template <typename T, int G>
__global__ void __launch_bounds__(kThreads) quant8_kernel(const __grid_constant__ Quant8Params p) {
  stream_order();
  const int lane = threadIdx.x & 31;
  const unsigned groups = ((unsigned)p.col_tiles * 128 + G * 512 - 1) / (G * 512);
  const unsigned blocks =
      ((unsigned)p.R + kScaleRows - 1) / kScaleRows * (kScaleRows / kWarps) * groups;
  for (unsigned u = blockIdx.x; u < blocks; u += gridDim.x) {
    const unsigned q = u / groups;
    const int r = (int)(q * kWarps + (threadIdx.x >> 5));
    const int e0 = (int)((u - q * groups) * G * 512) + lane * 16;
    Sixteen<T> v[G];
    const T* x = r < p.R ? static_cast<const T*>(p.x) + (long long)r * p.ld : nullptr;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int e = e0 + g * 512;
      if (x && p.vec_ok && e < p.L)
        v[g].load(x + e);
      else
        v[g].each(x + e, x && e < p.L);
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int e = e0 + g * 512;
      const bool in = x && e < p.L;
      uint32_t top = v[g].top();
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      const Scale8 s(__uint_as_float(top));
      if (in) {
        uint32_t c[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[8];
          v[g].widen(h, w);
          c[2 * h] = s.codes(pair(w[0], w[1]), pair(w[2], w[3]));
          c[2 * h + 1] = s.codes(pair(w[4], w[5]), pair(w[6], w[7]));
        }
        *reinterpret_cast<uint4*>(p.codes + (size_t)r * p.L + e) = make_uint4(c[0], c[1], c[2], c[3]);
      }
      const int b = e / kMxBlock;
      if (b / 4 < p.col_tiles && lane % 2 == 0)
        p.scales[scale_at(r, b / 4, p.col_tiles) + b % 4] = in ? (uint8_t)s.byte : (uint8_t)0;
    }
  }
}

struct Decode8Params {
  const uint8_t* codes;
  const uint8_t* scales;
  void* out;
  int R, L, col_tiles;
};

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) { store8_f32(p, v); }
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) { store8_bf16(p, v); }

// A warp takes G x 256 columns of a row, a lane eight of each 256.
template <typename T, int G>
__global__ void __launch_bounds__(kThreads) decode8_kernel(const __grid_constant__ Decode8Params p) {
  stream_order();
  const int lane = threadIdx.x & 31;
  const unsigned groups = ((unsigned)p.L + G * 256 - 1) / (G * 256);
  const unsigned blocks = ((unsigned)p.R + kWarps - 1) / kWarps * groups;
  for (unsigned u = blockIdx.x; u < blocks; u += gridDim.x) {
    const unsigned q = u / groups;
    const int r = (int)(q * kWarps + (threadIdx.x >> 5));
    const int e0 = (int)((u - q * groups) * G * 256) + lane * 8;
    if (r >= p.R) continue;
    const uint8_t* codes = p.codes + (size_t)r * p.L;
    uint2 c[G];
    uint32_t byte[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int e = min(e0 + g * 256, p.L - 8);  // past the end: the last, and dropped
      const int b = e / kMxBlock;
      c[g] = *reinterpret_cast<const uint2*>(codes + e);
      byte[g] = p.scales[scale_at(r, b / 4, p.col_tiles) + b % 4];
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int e = e0 + g * 256;
      const float step = power_of(byte[g]);
      const uint32_t w[2] = {c[g].x, c[g].y};
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i / 2] >> (16 * (i % 2)))));
        widen_f16x2(h, v[2 * i], v[2 * i + 1]);
        v[2 * i] = __fmul_rn(v[2 * i], step);
        v[2 * i + 1] = __fmul_rn(v[2 * i + 1], step);
      }
      if (e < p.L) store8(static_cast<T*>(p.out) + (size_t)r * p.L + e, v);
    }
  }
}

// One CTA for each share of the work; under a CTA limit the CTAs go over the shares.
template <typename P>
cudaError_t launch(void (*kernel)(P), const P& p, long long blocks, cudaStream_t s) {
  const int limit = dph::stream_cta_limit();
  if (limit > 0) blocks = std::min<long long>(blocks, limit);
  return dph::launch_early(kernel, p, (unsigned)std::min<long long>(blocks, 0x7fffffffll), kThreads,
                           s);
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Whether there is work enough to fill the GPU with warps that take `span`
// columns of a row at once (the same rule as the 4-bit forms').
bool wide(long long rows, long long cols, int span) {
  return cols >= span && rows * cols >= (1ll << 11) * span;
}

template <typename T>
cudaError_t quantize(const Quant8Params& p, cudaStream_t s) {
  const long long quads = ceil_div(p.R, kScaleRows) * (kScaleRows / kWarps);
  const long long cols = (long long)p.col_tiles * 128;
  if (wide(p.R, p.L, 2048)) return launch(quant8_kernel<T, 4>, p, quads * ceil_div(cols, 2048), s);
  if (wide(p.R, p.L, 1024)) return launch(quant8_kernel<T, 2>, p, quads * ceil_div(cols, 1024), s);
  return launch(quant8_kernel<T, 1>, p, quads * ceil_div(cols, 512), s);
}

template <typename T>
cudaError_t decode(const Decode8Params& p, cudaStream_t s) {
  if (wide(p.R, p.L, 1024))
    return launch(decode8_kernel<T, 4>, p, ceil_div(p.R, kWarps) * ceil_div(p.L, 1024), s);
  return launch(decode8_kernel<T, 1>, p, ceil_div(p.R, kWarps) * ceil_div(p.L, 256), s);
}

using dph::aligned;
using dph::clash;
using dph::Span;
using dph::span_of;

}  // namespace

extern "C" {

dp_status_t dp_mx8_quantize(const void* x, int rows, int cols, long long ld, dp_dtype_t x_dtype,
                            void* codes, void* scales, dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_mx8_quantize");
  if (rows < 0 || cols < 0 || ld < cols) return DP_ERR_INVALID_ARG;
  if (x_dtype != DP_FP32 && x_dtype != DP_BF16) return DP_ERR_UNSUPPORTED;
  if (rows > kMaxSize || cols > kMaxSize || cols % 32) return DP_ERR_UNSUPPORTED;
  const size_t esz = x_dtype == DP_FP32 ? 4 : 2;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(x, esz)) return DP_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return DP_OK;  // an empty matrix has no buffers
  if (!x || !codes || !scales) return DP_ERR_INVALID_ARG;
  size_t sbytes = 0;
  dp_mx4_scales_size(rows, cols, DP_MXFP4, &sbytes);
  const Span in = span_of(x, ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * esz);
  const Span out[2] = {span_of(codes, (size_t)rows * cols), span_of(scales, sbytes)};
  if (clash(out[0], out[1]) || clash(in, out[0]) || clash(in, out[1])) return DP_ERR_ALIAS;
  Quant8Params p{x, ld, rows, cols, mx4_col_tiles(cols, kMxBlock),
                 aligned(x, 32) && ld % 16 == 0, static_cast<uint8_t*>(codes),
                 static_cast<uint8_t*>(scales)};
  dph::DeviceInfo dev;
  if (!dph::current_device(&dev)) return DP_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = x_dtype == DP_FP32 ? quantize<float>(p, s) : quantize<uint16_t>(p, s);
  return e == cudaSuccess ? DP_OK : DP_ERR_CUDA;
}

dp_status_t dp_mx8_dequantize(const void* codes, const void* scales, int rows, int cols, void* out,
                              dp_dtype_t out_dtype, dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_mx8_dequantize");
  if (rows < 0 || cols < 0) return DP_ERR_INVALID_ARG;
  if (out_dtype != DP_FP32 && out_dtype != DP_BF16) return DP_ERR_UNSUPPORTED;
  if (rows > kMaxSize || cols > kMaxSize || cols % 32) return DP_ERR_UNSUPPORTED;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 16)) return DP_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return DP_OK;
  if (!codes || !scales || !out) return DP_ERR_INVALID_ARG;
  size_t sbytes = 0;
  dp_mx4_scales_size(rows, cols, DP_MXFP4, &sbytes);
  const Span w = span_of(out, (size_t)rows * cols * (out_dtype == DP_FP32 ? 4 : 2));
  if (clash(w, span_of(codes, (size_t)rows * cols)) || clash(w, span_of(scales, sbytes)))
    return DP_ERR_ALIAS;
  Decode8Params p{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), out,
                  rows, cols, mx4_col_tiles(cols, kMxBlock)};
  dph::DeviceInfo dev;
  if (!dph::current_device(&dev)) return DP_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = out_dtype == DP_FP32 ? decode<float>(p, s) : decode<uint16_t>(p, s);
  return e == cudaSuccess ? DP_OK : DP_ERR_CUDA;
}

}  // extern "C"
