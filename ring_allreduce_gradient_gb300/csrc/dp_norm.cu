// dp_norm.cu -- the root-mean-square norm in front of a layer's products, with
// the residual's addition and the quantised form of its output in the same
// pass, and its backward pass.
//
// Forward, for every row (D elements of type T):
//   h = round_T(x + residual)          (no residual: h = x, not written)
//   r = 1 / sqrt(mean(h^2) + eps)
//   y = (h r) w                        fp32; stored as T, or quantised as it is
// The norm is of h as it is stored, so the backward pass sees the same values.
// Backward, with xh = h r and g = dy w:
//   dx = r (g - xh mean(g xh)) + dh
//   dw = sum over rows of dy xh
//
// Both are bound by memory (bf16, residual, 8-bit output: 7.03 bytes an element
// for about 10 operations; backward with dh: 8 bytes).  A row is held in
// registers by TPR threads, 16 G elements each, from its load to its store, so
// it crosses memory once; a thread's sixteen consecutive elements are one or two
// 32-byte loads and half a block of 32 (the other half is its neighbour lane's).

#include "dp_early.cuh"
#include "dp_launch.h"
#include "dp_mx4.cuh"
#include "dp_mx4q.cuh"

#include <algorithm>

namespace {

using namespace dpk;

constexpr int kMaxCols = 32768;  // 1024 threads hold 32 elements each
constexpr int kMaxRows = 0x7fff0000;

// What the forward pass writes y as.
enum { kPlain = 0, kToMx4 = 1, kToNv4 = 2, kToMx8 = 3 };

struct NormFwdParams {
  const void* x;
  const void* res;
  const void* w;
  void* h;
  void* y;       // or NULL
  float* rstd;
  uint8_t* codes;
  uint8_t* scales;
  const float* tscale;
  long long ldx, ldr;
  int M, D, col_tiles;
  int rows;      // M, up to a whole scale tile where there are scales
  float eps;
  int vec;       // every row of every buffer starts on a 32-byte boundary and D is a multiple of 16
  int w_f32;
};

// The elements that a thread holds of a row.  Where rows are aligned (or
// blocks of 32 are needed) they are G groups of sixteen consecutive ones;
// else every TPR-th element, so that a warp's scalar accesses are consecutive.
template <int TPR>
__device__ __forceinline__ int element(bool chunks, int t, int i) {
  return chunks ? (i / 16 * TPR + t) * 16 + i % 16 : i * TPR + t;
}

template <typename T>
__device__ __forceinline__ float value_at(const T* p) {
  return widen_scalar(p, 0);
}
__device__ __forceinline__ void put_at(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_at(uint16_t* p, float v) { *p = bf16_rn(v); }

template <typename T>
__device__ __forceinline__ float rounded(float v) {
  if constexpr (sizeof(T) == 2) return bf16lo(pack_bf16x2_rn(v, 0.0f));
  return v;
}

// Sixteen elements from a 32-byte boundary, widened.
template <typename T>
__device__ __forceinline__ void load16(const T* p, float* v) {
  Sixteen<T> s;
  s.load(p);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float w[8];
    s.widen(h, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * h + i] = w[i];
  }
}
__device__ __forceinline__ void store16(float* p, const float* v) {
#pragma unroll
  for (int h = 0; h < 16; h += 8)
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p + h), "f"(v[h]),
                 "f"(v[h + 1]), "f"(v[h + 2]), "f"(v[h + 3]), "f"(v[h + 4]), "f"(v[h + 5]),
                 "f"(v[h + 6]), "f"(v[h + 7])
                 : "memory");
}
__device__ __forceinline__ void store16(uint16_t* p, const float* v) {
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = pack_bf16x2_rn(v[2 * i], v[2 * i + 1]);
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// A thread's elements of a row; zero past its end.
template <typename T, int TPR, int G>
__device__ __forceinline__ void load_row(const T* p, bool in, bool vec, bool chunks, int t, int D,
                                         float (&v)[16 * G]) {
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int e = element<TPR>(true, t, 16 * g);
    if (in && vec && e < D) {
      load16(p + e, v + 16 * g);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int o = element<TPR>(chunks, t, 16 * g + i);
        v[16 * g + i] = in && !vec && o < D ? value_at(p + o) : 0.0f;
      }
    }
  }
}
template <typename T, int TPR, int G>
__device__ __forceinline__ void store_row(T* p, bool vec, bool chunks, int t, int D,
                                          const float (&v)[16 * G]) {
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int e = element<TPR>(true, t, 16 * g);
    if (vec) {
      if (e < D) store16(p + e, v + 16 * g);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int o = element<TPR>(chunks, t, 16 * g + i);
        if (o < D) put_at(p + o, v[16 * g + i]);
      }
    }
  }
}
template <int TPR, int G>
__device__ __forceinline__ void load_weight(const void* w, bool f32, bool in, bool vec, bool chunks,
                                            int t, int D, float (&v)[16 * G]) {
  if (f32)
    load_row<float, TPR, G>(static_cast<const float*>(w), in, vec, chunks, t, D, v);
  else
    load_row<uint16_t, TPR, G>(static_cast<const uint16_t*>(w), in, vec, chunks, t, D, v);
}

// The sum over a row's TPR threads, in all of them and in a fixed order.  part:
// a word for each warp; a call's words are not reused before the call after the
// next, so one barrier a call is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (TPR > 32) {
    constexpr int kWarpsRow = TPR / 32;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float p[kWarpsRow];
#pragma unroll
    for (int i = 0; i < kWarpsRow; ++i) p[i] = part[(threadIdx.x / TPR) * kWarpsRow + i];
#pragma unroll
    for (int s = 1; s < kWarpsRow; s *= 2)
#pragma unroll
      for (int i = 0; i + s < kWarpsRow; i += 2 * s) p[i] = __fadd_rn(p[i], p[i + s]);
    v = p[0];
  }
  return v;
}

template <int TPR>
constexpr int kThreadsOf = TPR < 128 ? 128 : TPR;  // of a CTA

// A thread's quantised elements and their scales.  Every lane comes here: a
// block of 32 is two lanes'.
template <int FMT, int TPR, int G>
__device__ __forceinline__ void quantise_row(const NormFwdParams& p, int r, int t, float tscale,
                                             const Divisor& by_t, const float (&y)[16 * G]) {
  constexpr int BLOCK = FMT == kToNv4 ? kNvBlock : kMxBlock;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int e = element<TPR>(true, t, 16 * g);
    const float* v = y + 16 * g;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    if constexpr (BLOCK == kMxBlock) top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const bool in = r < p.M && e < p.D;
    uint32_t byte;
    if constexpr (FMT == kToMx8) {
      const Scale8 s(__uint_as_float(top));
      byte = s.byte;
      if (in) {
        uint4 c;
        c.x = s.codes(v[0], v[1], v[2], v[3]);
        c.y = s.codes(v[4], v[5], v[6], v[7]);
        c.z = s.codes(v[8], v[9], v[10], v[11]);
        c.w = s.codes(v[12], v[13], v[14], v[15]);
        *reinterpret_cast<uint4*>(p.codes + (size_t)r * p.D + e) = c;
      }
    } else {
      const Scale<BLOCK> s(__uint_as_float(top), tscale, by_t);
      byte = s.byte;
      if (in) {
        uint32_t c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = v[8 * h + i];
          c[h] = s.codes(w);
        }
        *reinterpret_cast<uint2*>(p.codes + (size_t)r * (p.D / 2) + e / 2) =
            make_uint2(c[0], c[1]);
      }
    }
    const int b = e / BLOCK;
    if (b / 4 < p.col_tiles && (BLOCK == kNvBlock || t % 2 == 0))
      p.scales[scale_at(r, b / 4, p.col_tiles) + b % 4] = in ? (uint8_t)byte : (uint8_t)0;
  }
}

template <typename T, int FMT, int TPR, int G>
__global__ void __launch_bounds__(kThreadsOf<TPR>)
    norm_fwd_kernel(const __grid_constant__ NormFwdParams p) {
  constexpr int RPC = kThreadsOf<TPR> / TPR;  // rows of a CTA
  __shared__ float part[2][kThreadsOf<TPR> / 32];
  stream_order();
  const int t = threadIdx.x % TPR;
  const bool vec = p.vec, chunks = FMT != kPlain || p.vec;
  const float tscale = FMT == kToNv4 && p.tscale ? *p.tscale : 1.0f;
  const Divisor by_t(tscale);
  int turn = 0;
  for (int r0 = blockIdx.x * RPC; r0 < p.rows; r0 += gridDim.x * RPC, turn ^= 1) {
    const int r = r0 + threadIdx.x / TPR;
    const bool in = r < p.M;
    float v[16 * G], w[16 * G];
    load_row<T, TPR, G>(static_cast<const T*>(p.x) + (long long)r * p.ldx, in, vec, chunks, t, p.D,
                        v);
    if (p.res) {
      load_row<T, TPR, G>(static_cast<const T*>(p.res) + (long long)r * p.ldr, in, vec, chunks, t,
                          p.D, w);
#pragma unroll
      for (int i = 0; i < 16 * G; ++i) v[i] = rounded<T>(__fadd_rn(v[i], w[i]));
      if (in) store_row<T, TPR, G>(static_cast<T*>(p.h) + (size_t)r * p.D, vec, chunks, t, p.D, v);
    }
    load_weight<TPR, G>(p.w, p.w_f32, in, vec, chunks, t, p.D, w);
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 16 * G; ++i) s[i % 4] = __fmaf_rn(v[i], v[i], s[i % 4]);
    const float ss = row_sum<TPR>(__fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3])), part[turn]);
    const float rstd =
        __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)p.D), p.eps)));
    if (in && t == 0 && p.rstd) p.rstd[r] = rstd;
#pragma unroll
    for (int i = 0; i < 16 * G; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], rstd), w[i]);
    if (in && p.y)
      store_row<T, TPR, G>(static_cast<T*>(p.y) + (size_t)r * p.D, vec, chunks, t, p.D, v);
    if constexpr (FMT != kPlain) quantise_row<FMT, TPR, G>(p, r, t, tscale, by_t, v);
  }
}

// ---- backward -----------------------------------------------------------------

struct NormBwdParams {
  const void* dy;
  const void* h;
  const void* dh;  // or NULL
  const void* w;
  const float* rstd;
  void* dx;
  float* part;     // [groups][D]: a group's sum of dy xh over its rows
  long long ldy, ldh, ldd;
  int M, D;
  int groups;      // sets of rows: every groups-th RPC rows
  int vec;
  int w_f32;
};

// A group's rows and the order of its sums follow from M and D alone, whatever
// CTA takes it, so dw has the same bits under any grid.
template <typename T, int TPR, int G>
__global__ void __launch_bounds__(kThreadsOf<TPR>)
    norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  constexpr int RPC = kThreadsOf<TPR> / TPR;
  __shared__ float part[2][kThreadsOf<TPR> / 32];
  stream_order();
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const bool vec = p.vec;
  float w[16 * G];
  load_weight<TPR, G>(p.w, p.w_f32, true, vec, vec, t, p.D, w);
  int turn = 0;
  for (int q = blockIdx.x; q < p.groups; q += gridDim.x) {
    float dw[16 * G];
#pragma unroll
    for (int i = 0; i < 16 * G; ++i) dw[i] = 0.0f;
    for (long long r0 = (long long)q * RPC; r0 < p.M; r0 += (long long)p.groups * RPC, turn ^= 1) {
      const long long r = r0 + sub;
      const bool in = r < p.M;
      float h[16 * G], g[16 * G], d[16 * G];
      load_row<T, TPR, G>(static_cast<const T*>(p.h) + r * p.ldh, in, vec, vec, t, p.D, h);
      load_row<T, TPR, G>(static_cast<const T*>(p.dy) + r * p.ldy, in, vec, vec, t, p.D, g);
      if (p.dh)
        load_row<T, TPR, G>(static_cast<const T*>(p.dh) + r * p.ldd, in, vec, vec, t, p.D, d);
      const float rstd = in ? p.rstd[r] : 0.0f;
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 16 * G; ++i) {
        h[i] = __fmul_rn(h[i], rstd);
        dw[i] = __fmaf_rn(g[i], h[i], dw[i]);
        g[i] = __fmul_rn(g[i], w[i]);
        s[i % 4] = __fmaf_rn(g[i], h[i], s[i % 4]);
      }
      const float sum =
          row_sum<TPR>(__fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3])), part[turn]);
      const float c = __fdiv_rn(sum, (float)p.D);
#pragma unroll
      for (int i = 0; i < 16 * G; ++i) {
        const float v = __fmul_rn(__fmaf_rn(-h[i], c, g[i]), rstd);
        g[i] = p.dh ? __fadd_rn(v, d[i]) : v;
      }
      if (in) store_row<T, TPR, G>(static_cast<T*>(p.dx) + (size_t)r * p.D, vec, vec, t, p.D, g);
    }
    store_row<float, TPR, G>(p.part + ((size_t)q * RPC + sub) * p.D, vec, vec, t, p.D, dw);
  }
}

// dw = the sum of the groups' sums, in order: a CTA takes 32 columns, each of
// its warps every 32nd row of part.
struct NormSumParams {
  const float* part;
  float* dw;
  int rows, D;
};
__global__ void __launch_bounds__(1024) norm_sum_kernel(const __grid_constant__ NormSumParams p) {
  __shared__ float sums[32][33];
  stream_order();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int c0 = blockIdx.x * 32; c0 < p.D; c0 += gridDim.x * 32) {
    const int c = c0 + lane;
    float s = 0.0f;
#pragma unroll 4
    for (int r = warp; r < p.rows; r += 32)
      s = __fadd_rn(s, c < p.D ? p.part[(size_t)r * p.D + c] : 0.0f);
    sums[warp][lane] = s;
    __syncthreads();
    float v = sums[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (lane == 0 && c0 + warp < p.D) p.dw[c0 + warp] = v;
    __syncthreads();
  }
}

// ---- host ---------------------------------------------------------------------

template <typename P>
cudaError_t launch(void (*kernel)(P), const P& p, long long blocks, int threads, cudaStream_t s) {
  const int limit = dph::stream_cta_limit();
  if (limit > 0) blocks = std::min<long long>(blocks, limit);
  return dph::launch_early(kernel, p, (unsigned)std::min<long long>(blocks, 0x7fffffffll),
                           (unsigned)threads, s);
}

// Threads of a row and groups of sixteen elements of a thread, by the row's length.
template <typename F>
cudaError_t by_length(int D, const F& f) {
  if (D <= 512) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  if (D <= 1024) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 2>());
  if (D <= 2048) return f(std::integral_constant<int, 128>(), std::integral_constant<int, 1>());
  if (D <= 4096) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 1>());
  if (D <= 8192) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 1>());
  if (D <= 16384) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 2>());
  return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 2>());
}

// Rows of a CTA in the backward pass.
int rows_per_cta(int D) { return D <= 1024 ? 4 : 1; }
// Sets of rows whose sums of dy xh are kept apart: a constant, so that the bits
// do not follow the GPU's size.
int groups_of(int M, int D) {
  const int per = rows_per_cta(D);
  return (int)std::min<long long>(((long long)M + per - 1) / per, 456 / per);
}

using dph::aligned;
using dph::Span;
using dph::span_of;
using dph::any_clash;

size_t esize(dp_dtype_t t) { return t == DP_FP32 ? 4 : 2; }
bool dtype_ok(dp_dtype_t t) { return t == DP_FP32 || t == DP_BF16; }
Span rows_span(const void* p, int M, int D, long long ld, size_t esz, bool written) {
  return span_of(p, p && M && D ? ((size_t)(M - 1) * (size_t)ld + (size_t)D) * esz : 0, written);
}

}  // namespace

extern "C" {

dp_status_t dp_rms_norm(const void* x, long long ldx, const void* residual, long long ldr, int M,
                        int D, dp_dtype_t dtype, const void* weight, dp_dtype_t weight_dtype,
                        float eps, void* h, void* y, float* rstd, dp_norm_format_t format,
                        const float* tensor_scale, void* codes, void* scales, dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_rms_norm");
  if (M < 0 || D < 0 || ldx < D || (residual && ldr < D)) return DP_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return DP_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype)) return DP_ERR_UNSUPPORTED;
  if (format < DP_NORM_PLAIN || format > DP_NORM_MXFP8) return DP_ERR_UNSUPPORTED;
  const bool q = format != DP_NORM_PLAIN;
  if (M > kMaxRows || D > kMaxCols || (q && D % 32)) return DP_ERR_UNSUPPORTED;
  if (tensor_scale && format != DP_NORM_NVFP4) return DP_ERR_INVALID_ARG;
  const size_t esz = esize(dtype), wsz = esize(weight_dtype);
  if (!aligned(x, esz) || !aligned(residual, esz) || !aligned(weight, wsz) || !aligned(h, esz) ||
      !aligned(y, esz) || !aligned(rstd, 4) || !aligned(tensor_scale, 4))
    return DP_ERR_UNSUPPORTED;
  if (q && (!aligned(codes, 16) || !aligned(scales, 16))) return DP_ERR_UNSUPPORTED;
  if (!q && (codes || scales)) return DP_ERR_INVALID_ARG;
  if ((residual != nullptr) != (h != nullptr) && M && D) return DP_ERR_INVALID_ARG;
  if (M == 0 || D == 0) return DP_OK;
  if (!x || !weight || (q ? !codes || !scales : !y)) return DP_ERR_INVALID_ARG;
  const int block = format == DP_NORM_NVFP4 ? kNvBlock : kMxBlock;
  size_t sbytes = 0;
  if (q) dp_mx4_scales_size(M, D, format == DP_NORM_NVFP4 ? DP_NVFP4 : DP_MXFP4, &sbytes);
  const size_t n = (size_t)M * D;
  const Span spans[] = {
      rows_span(x, M, D, ldx, esz, false),
      rows_span(residual, M, D, ldr, esz, false),
      span_of(weight, (size_t)D * wsz),
      span_of(tensor_scale, tensor_scale ? 4 : 0),
      span_of(h, h ? n * esz : 0, true),
      span_of(y, y ? n * esz : 0, true),
      span_of(rstd, rstd ? (size_t)M * 4 : 0, true),
      span_of(codes, q ? (format == DP_NORM_MXFP8 ? n : n / 2) : 0, true),
      span_of(scales, sbytes, true)};
  if (any_clash(spans)) return DP_ERR_ALIAS;
  NormFwdParams p{};
  p.x = x, p.res = residual, p.w = weight, p.h = h, p.y = y, p.rstd = rstd;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  p.tscale = tensor_scale;
  p.ldx = ldx, p.ldr = ldr, p.M = M, p.D = D, p.eps = eps;
  p.w_f32 = weight_dtype == DP_FP32;
  p.col_tiles = q ? mx4_col_tiles(D, block) : 0;
  p.rows = q ? (M + kScaleRows - 1) / kScaleRows * kScaleRows : M;
  p.vec = D % 16 == 0 && aligned(x, 32) && ldx % 16 == 0 && aligned(weight, 32) &&
          (!residual || (aligned(residual, 32) && ldr % 16 == 0 && aligned(h, 32))) &&
          aligned(y, 32);
  dph::DeviceInfo dev;
  if (!dph::current_device(&dev)) return DP_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = by_length(D, [&](auto tpr, auto g) {
    constexpr int TPR = decltype(tpr)::value, G = decltype(g)::value;
    const auto go = [&](auto kernel) {
      const int threads = kThreadsOf<TPR>;
      return launch(kernel, p, ((long long)p.rows * TPR + threads - 1) / threads, threads, s);
    };
    if (dtype == DP_FP32) {
      if (format == DP_NORM_MXFP4) return go(norm_fwd_kernel<float, kToMx4, TPR, G>);
      if (format == DP_NORM_NVFP4) return go(norm_fwd_kernel<float, kToNv4, TPR, G>);
      if (format == DP_NORM_MXFP8) return go(norm_fwd_kernel<float, kToMx8, TPR, G>);
      return go(norm_fwd_kernel<float, kPlain, TPR, G>);
    }
    if (format == DP_NORM_MXFP4) return go(norm_fwd_kernel<uint16_t, kToMx4, TPR, G>);
    if (format == DP_NORM_NVFP4) return go(norm_fwd_kernel<uint16_t, kToNv4, TPR, G>);
    if (format == DP_NORM_MXFP8) return go(norm_fwd_kernel<uint16_t, kToMx8, TPR, G>);
    return go(norm_fwd_kernel<uint16_t, kPlain, TPR, G>);
  });
  return e == cudaSuccess ? DP_OK : DP_ERR_CUDA;
}

dp_status_t dp_rms_norm_backward_workspace_size(int M, int D, size_t* bytes) {
  if (!bytes) return DP_ERR_INVALID_ARG;
  *bytes = 0;
  if (M < 0 || D < 0) return DP_ERR_INVALID_ARG;
  if (M > kMaxRows || D > kMaxCols) return DP_ERR_UNSUPPORTED;
  *bytes = (size_t)groups_of(M, D) * rows_per_cta(D) * D * sizeof(float);
  return DP_OK;
}

dp_status_t dp_rms_norm_backward(const void* dy, long long ldy, const void* h, long long ldh,
                                 const void* dh, long long ldd, int M, int D, dp_dtype_t dtype,
                                 const void* weight, dp_dtype_t weight_dtype, const float* rstd,
                                 void* dx, float* dweight, void* workspace, size_t workspace_bytes,
                                 dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_rms_norm_backward");
  size_t need = 0;
  const dp_status_t st = dp_rms_norm_backward_workspace_size(M, D, &need);
  if (st != DP_OK) return st;
  if (ldy < D || ldh < D || (dh && ldd < D)) return DP_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype)) return DP_ERR_UNSUPPORTED;
  const size_t esz = esize(dtype), wsz = esize(weight_dtype);
  if (!aligned(dy, esz) || !aligned(h, esz) || !aligned(dh, esz) || !aligned(dx, esz) ||
      !aligned(weight, wsz) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(workspace, 32))
    return DP_ERR_UNSUPPORTED;
  if (D == 0) return DP_OK;
  if (!dweight) return DP_ERR_INVALID_ARG;
  if (M && (!dy || !h || !dx || !weight || !rstd || !workspace || workspace_bytes < need))
    return DP_ERR_INVALID_ARG;
  const size_t n = (size_t)M * D;
  const Span spans[] = {rows_span(dy, M, D, ldy, esz, false),
                             rows_span(h, M, D, ldh, esz, false),
                             rows_span(dh, M, D, ldd, esz, false),
                             span_of(weight, (size_t)D * wsz),
                             span_of(rstd, (size_t)M * 4),
                             span_of(dx, n * esz, true),
                             span_of(dweight, (size_t)D * 4, true),
                             span_of(workspace, need, true)};
  if (any_clash(spans)) return DP_ERR_ALIAS;
  dph::DeviceInfo dev;
  if (!dph::current_device(&dev)) return DP_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0)
    return cudaMemsetAsync(dweight, 0, (size_t)D * 4, s) == cudaSuccess ? DP_OK : DP_ERR_CUDA;
  NormBwdParams p{};
  p.dy = dy, p.h = h, p.dh = dh, p.w = weight, p.rstd = rstd, p.dx = dx;
  p.part = static_cast<float*>(workspace);
  p.ldy = ldy, p.ldh = ldh, p.ldd = ldd, p.M = M, p.D = D;
  p.groups = groups_of(M, D);
  p.w_f32 = weight_dtype == DP_FP32;
  p.vec = D % 16 == 0 && aligned(dy, 32) && ldy % 16 == 0 && aligned(h, 32) && ldh % 16 == 0 &&
          (!dh || (aligned(dh, 32) && ldd % 16 == 0)) && aligned(dx, 32) && aligned(weight, 32);
  cudaError_t e = by_length(D, [&](auto tpr, auto g) {
    constexpr int TPR = decltype(tpr)::value, G = decltype(g)::value;
    if (dtype == DP_FP32)
      return launch(norm_bwd_kernel<float, TPR, G>, p, p.groups, kThreadsOf<TPR>, s);
    return launch(norm_bwd_kernel<uint16_t, TPR, G>, p, p.groups, kThreadsOf<TPR>, s);
  });
  if (e == cudaSuccess) {
    const NormSumParams q{p.part, dweight, p.groups * rows_per_cta(D), D};
    e = launch(norm_sum_kernel, q, (D + 31) / 32, 1024, s);
  }
  return e == cudaSuccess ? DP_OK : DP_ERR_CUDA;
}

}  // extern "C"
