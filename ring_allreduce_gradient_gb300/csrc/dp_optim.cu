// dp_optim.cu -- the optimizer step on the reduced gradients: the global
// gradient norm with its clip coefficient, and AdamW over a list of tensors
// with 32-bit or 8-bit states.
//
// The mathematics (decoupled weight decay; t counts steps from 1):
//   g' = c g                    c: the clip coefficient, min(1, max / (||g|| + 1e-6))
//   m' = b1 m + (1 - b1) g'
//   v' = b2 v + (1 - b2) g'^2
//   p' = p (1 - lr wd) - lr / (1 - b1^t) * m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
// in fp32, one rounding per operation (no contraction; with bf16 parameters or
// 8-bit states the root and the quotient to 2^-22); the factors that depend on t
// alone formed in double on the host.
//
// 8-bit states: m and r = sqrt(v) are e4m3 codes with one fp32 scale for each
// 256 consecutive elements, the block's largest magnitude at e4m3's largest
// value (448).  The root of v is stored because the step divides by it: e4m3
// spans 2^17.8 between its smallest and largest value, so the stored v spans
// 2^35.  A root that would round to zero while v > 0 takes the smallest code
// instead (a zero root under a nonzero m would make the next steps
// unbounded).  The step itself uses the unrounded m' and v' of this step.
//
// Both kernels are bound by memory: AdamW moves 30 bytes an element (fp32
// parameters, gradients and states, bf16 copy) for about 15 operations, the
// 8-bit form 18, the norm 4.  A warp takes 256 consecutive elements of one
// tensor at a time (an 8-bit block), each lane eight of them as one 32-byte
// load per fp32 array, so every array's load is issued before any is used.
// Tensors whose pointers are not aligned for that, and the last elements of a
// tensor, go lane by lane over consecutive elements with the same arithmetic.

#include "dp_early.cuh"
#include "dp_launch.h"

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>
#include <type_traits>
#include <vector>

namespace {

using namespace dpk;

constexpr int kThreads = 128;      // AdamW
constexpr int kWarps = kThreads / 32;
constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kUnit = 256;         // elements a warp takes at once = an 8-bit block
// The norm: 2048 elements, eight loads of each lane in flight together, and
// three CTAs an SM (measured against 512 and 1024 elements and two to eight
// CTAs: one layer's fp32 gradients 8.0 us, against 8.4 to 11.3 us).
constexpr int kNormUnit = 2048;
constexpr int kNormLoads = kNormUnit / 256;
constexpr int kNormSlots = 456;    // partial sums of one norm launch: three CTAs on each of 152 SMs
constexpr float kE4m3Max = 448.0f;
constexpr float kTopFp4 = 1.0f / 2688.0f;     // e2m1's largest value (6) times e4m3's
constexpr float kE4m3Min = 0.001953125f;      // 2^-9, the smallest e4m3 value above zero
constexpr float kTiny = 7.703719777548943e-34f;  // 2^-110: below it a block's reciprocal is left out

// ---- eight consecutive elements --------------------------------------------

__device__ __forceinline__ void ld8(const float* p, float (&v)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                 "=f"(v[6]), "=f"(v[7])
               : "l"(p));
}
__device__ __forceinline__ void st8(float* p, const float (&v)[8]) {
  asm volatile("st.global.cs.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void ld8(const uint16_t* p, float (&v)[8]) {
  uint4 raw[1] = {ld_v4(p)};
  Vec8<uint16_t>::widen(raw, v);
}
__device__ __forceinline__ void st8(uint16_t* p, const float (&v)[8]) { store8_bf16(p, v); }

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// e4m3 -> fp32 through fp16, which holds every e4m3 value.
__device__ __forceinline__ void widen_e4m3x2(uint16_t c, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}
__device__ __forceinline__ void ld8_codes(const uint8_t* p, uint32_t (&c)[2]) {
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(c[0]), "=r"(c[1]) : "l"(p));
}
__device__ __forceinline__ void st8_codes(uint8_t* p, const uint32_t (&c)[2]) {
  asm volatile("st.global.cs.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(c[0]), "r"(c[1]) : "memory");
}
__device__ __forceinline__ void widen_codes(const uint32_t (&c)[2], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    widen_e4m3x2((uint16_t)(c[i >> 1] >> (16 * (i & 1))), v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void pack_codes(const float (&v)[8], uint32_t (&c)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    c[i] = (uint32_t)e4m3x2(v[4 * i], v[4 * i + 1]) |
           ((uint32_t)e4m3x2(v[4 * i + 2], v[4 * i + 3]) << 16);
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = bf16_rn(v); }

// ---- AdamW -------------------------------------------------------------------

// One tensor of a list; what a warp needs of it lies together.
struct alignas(16) AdamwTensor {
  void* param;
  const void* grad;
  uint16_t* copy;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  unsigned long long numel;
  double decay;
  int vec_ok;
};

template <int CAP>
struct AdamwParams {
  AdamwTensor tensor[CAP];
  unsigned ustart[CAP + 1];  // prefix sums of units (kUnit elements) per tensor
  int n;
  double lr;
  float beta1, omb1, beta2, omb2, eps, step_size, inv_root;
  const float* grad_scale;
  const float* schedule;
  unsigned* skips;           // NULL, or the steps left out so far
  unsigned step;             // counts those too
  int counts;                // 1: this launch adds a step that is left out
  float log_beta1, log_beta2;
};

struct Hyper {
  float coef, beta1, omb1, beta2, omb2, eps, step_size, inv_root;
};

// Root and quotient.  EXACT, correctly rounded: fp32 parameters with 32-bit
// states, whose traffic hides them (GPT-2-small-shaped step 524 us with and
// without, one layer 29.7 and 29.2 us, 98 vectors 2.9 and 2.3 us on the GPU).
// Otherwise to 2^-22 of the step, which is itself far below a parameter that is
// rounded to 2^-8 (bf16) or comes from states that are (8-bit ones, 2^-4): the
// rounded forms take about 20 instructions each and a call for every zero
// (parameters that have had no gradient yet), which bound those kernels: eight 8
// Mi shards with 8-bit states take 194 us with them, and 267 us where the
// gradients are zero, against 172 and 171; a layer's bf16 parameters with 32-bit
// states 17.9 us, against 14.2.  The root is the one that knows v below the
// normal range (1 us of the 172): a v flushed to 0 would make the step
// lr m / eps.  The divisor is at least eps, which is in the normal range.
template <bool EXACT>
__device__ __forceinline__ float root_of(float v) {
  if constexpr (EXACT) return __fsqrt_rn(v);
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
template <bool EXACT>
__device__ __forceinline__ float quotient(float a, float b) {
  if constexpr (EXACT) return __fdiv_rn(a, b);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b));
  return __fmul_rn(a, r);
}

// One element: the new m, v and root of v, and the parameter's step.
template <bool EXACT>
__device__ __forceinline__ float adamw_one(float p, float g, float& m, float& v, float& root,
                                           float keep, const Hyper& h) {
  g = __fmul_rn(g, h.coef);
  m = __fadd_rn(__fmul_rn(m, h.beta1), __fmul_rn(g, h.omb1));
  v = __fadd_rn(__fmul_rn(v, h.beta2), __fmul_rn(__fmul_rn(g, g), h.omb2));
  root = root_of<EXACT>(v);
  const float denom = __fadd_rn(__fmul_rn(root, h.inv_root), h.eps);
  return __fsub_rn(__fmul_rn(p, keep), __fmul_rn(h.step_size, quotient<EXACT>(m, denom)));
}

// The factors of step t where steps have been left out: 1 - b^t is -expm1(t
// log b), within 2^-21 in fp32 (the host's are formed in double; they are for a
// count that knows of no step left out).
__device__ __forceinline__ void correct_for(float t, float lr, float log_beta1, float log_beta2,
                                            Hyper& h) {
  h.step_size = __fdiv_rn(lr, -expm1f(__fmul_rn(t, log_beta1)));
  h.inv_root = __frcp_rn(__fsqrt_rn(-expm1f(__fmul_rn(t, log_beta2))));
}

// A block's largest magnitude over the warp.  Magnitudes order as their bit
// patterns; a NaN's is above every other, so it reaches the scale.
__device__ __forceinline__ float warp_max_abs(const float (&v)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  return __uint_as_float(__reduce_max_sync(0xffffffffu, top));
}

__device__ __forceinline__ float code_factor(float top) {
  return top > kTiny ? __fmul_rn(__frcp_rn(top), kE4m3Max) : (top <= kTiny ? 0.0f : top);
}

// Eight CTAs of four warps on an SM, which is 64 registers: eight 8 Mi shards
// with 8-bit states 174 us, against 192 us at the 80 registers the kernel would
// take; ragged bf16 parameters with 8-bit states 97 us, against 108 us.
constexpr int kAdamwCtas = 8;

template <typename PT, typename GT, bool S8, int CAP>
__global__ void __launch_bounds__(kThreads, kAdamwCtas) adamw_kernel(const __grid_constant__ AdamwParams<CAP> a) {
  constexpr bool kExact = !S8 && std::is_same<PT, float>::value;
  const int lane = threadIdx.x & 31;
  const unsigned units = a.ustart[a.n];
  stream_order();
  Hyper h{1.0f, a.beta1, a.omb1, a.beta2, a.omb2, a.eps, a.step_size, a.inv_root};
  double lr = a.lr;
  if (a.grad_scale) h.coef = *a.grad_scale;
  if (a.schedule) {
    lr = (double)a.schedule[0];
    h.step_size = (float)(lr / (double)a.schedule[1]);
    h.inv_root = (float)(1.0 / sqrt((double)a.schedule[2]));
  }
  for (unsigned u = blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kWarps) {
    // the unit's tensor: the last t with ustart[t] <= u
    int t = 0;
    for (int hi = a.n - 1; t < hi;) {
      const int mid = (t + hi + 1) >> 1;
      if (a.ustart[mid] <= u) t = mid;
      else hi = mid - 1;
    }
    const AdamwTensor& x = a.tensor[t];
    const unsigned b = u - a.ustart[t];  // block of this tensor
    const unsigned long long e0 = (unsigned long long)b * kUnit;
    const unsigned long long left = x.numel - e0;
    PT* pp = static_cast<PT*>(x.param) + e0;
    const GT* gp = static_cast<const GT*>(x.grad) + e0;
    uint16_t* cp = x.copy ? x.copy + e0 : nullptr;
    const bool vec = x.vec_ok && left >= kUnit;
    const int len = left < kUnit ? (int)left : kUnit;
    // on its way ahead of the unit's loads (read before the loop it stays in a
    // register across it: eight 8 Mi shards 181 us, against 174; without a count 172)
    const unsigned skipped = a.skips ? *a.skips : 0u;
    float p[8], g[8], m[8], v[8], root[8];
    uint32_t mc[2], rc[2];
    float ms = 0.0f, rs = 0.0f;
    float* mp = static_cast<float*>(x.m) + (S8 ? 0 : e0);
    float* vp = static_cast<float*>(x.v) + (S8 ? 0 : e0);
    uint8_t* m8 = static_cast<uint8_t*>(x.m) + e0;
    uint8_t* r8 = static_cast<uint8_t*>(x.v) + e0;
    if (vec) {
      const int o = lane * 8;
      ld8(pp + o, p);
      ld8(gp + o, g);
      if constexpr (S8) {
        ld8_codes(m8 + o, mc);
        ld8_codes(r8 + o, rc);
        ms = x.m_scale[b];
        rs = x.v_scale[b];
        widen_codes(mc, m);
        widen_codes(rc, v);
      } else {
        ld8(mp + o, m);
        ld8(vp + o, v);
      }
    } else {
      const auto load = [&](auto whole) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int o = i * 32 + lane;
          const bool in = whole.value || o < len;
          p[i] = in ? widen_scalar(pp, o) : 0.0f;
          g[i] = in ? widen_scalar(gp, o) : 0.0f;
          if constexpr (S8) {
            float none;
            widen_e4m3x2(in ? (uint16_t)m8[o] : (uint16_t)0, m[i], none);
            widen_e4m3x2(in ? (uint16_t)r8[o] : (uint16_t)0, v[i], none);
          } else {
            m[i] = in ? mp[o] : 0.0f;
            v[i] = in ? vp[o] : 0.0f;
          }
        }
      };
      // without bounds where there are none to keep: 61 ragged bf16 tensors 109
      // us, against 119 us
      if (len == kUnit) load(std::true_type{});
      else load(std::false_type{});
      if constexpr (S8) {
        ms = x.m_scale[b];
        rs = x.v_scale[b];
      }
    }
    // one branch for both: the norm was not finite and nothing is changed (a warp
    // that reads the count after this step's is added comes here too), or steps
    // have been left out before
    if ((h.coef != h.coef) | (skipped != 0)) {
      if (h.coef != h.coef) {
        if (a.counts && u == 0 && lane == 0) *a.skips = skipped + 1u;
        return;
      }
      if (!a.schedule)
        correct_for((float)max(1, (int)(a.step - skipped)), (float)lr, a.log_beta1, a.log_beta2, h);
    }
    const float keep = (float)(1.0 - lr * x.decay);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (S8) {
        m[i] = __fmul_rn(m[i], ms);
        v[i] = __fmul_rn(v[i], rs);
        v[i] = __fmul_rn(v[i], v[i]);
      }
      p[i] = adamw_one<kExact>(p[i], g[i], m[i], v[i], root[i], keep, h);
    }
    if constexpr (S8) {
      if (!vec) {  // lanes past the end take no part in the block's largest value
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i * 32 + lane >= len) m[i] = v[i] = root[i] = 0.0f;
      }
      const float mt = warp_max_abs(m), rt = warp_max_abs(root);
      const float mf = code_factor(mt), rf = code_factor(rt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m[i] = __fmul_rn(m[i], mf);
        root[i] = __fmul_rn(root[i], rf);
        if (v[i] > 0.0f && root[i] < kE4m3Min) root[i] = kE4m3Min;
      }
      if (lane == 0) {
        x.m_scale[b] = __fmul_rn(mt, 1.0f / kE4m3Max);
        x.v_scale[b] = __fmul_rn(rt, 1.0f / kE4m3Max);
      }
    }
    if (vec) {
      const int o = lane * 8;
      st8(pp + o, p);
      if (cp) store8_bf16(cp + o, p);
      if constexpr (S8) {
        pack_codes(m, mc);
        pack_codes(root, rc);
        st8_codes(m8 + o, mc);
        st8_codes(r8 + o, rc);
      } else {
        st8(mp + o, m);
        st8(vp + o, v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int o = i * 32 + lane;
        if (o >= len) continue;
        put(pp + o, p[i]);
        if (cp) cp[o] = bf16_rn(p[i]);
        if constexpr (S8) {
          m8[o] = (uint8_t)e4m3x2(m[i], 0.0f);
          r8[o] = (uint8_t)e4m3x2(root[i], 0.0f);
        } else {
          mp[o] = m[i];
          vp[o] = v[i];
        }
      }
    }
  }
}

template <typename KernelT>
int resident_blocks(KernelT kernel, const dph::DeviceInfo& dev) {
  const int b = dph::prepare_kernel(reinterpret_cast<const void*>(kernel), kNormThreads, 0, dev.device);
  long long r = (long long)dev.sm_count * (b < 1 ? 1 : b);
  const int limit = dph::stream_cta_limit();
  if (limit > 0 && r > limit) r = limit;
  return (int)r;
}

// A warp for each unit: the hardware hands out CTAs as SMs become free, which
// the two dies do at different rates (GPT-2-small-shaped step, fp32 states: 524
// us, against 590 with a resident grid over the units).  Under a CTA limit the
// CTAs go over the units.
unsigned blocks_for(unsigned units) {
  const unsigned want = (units - 1) / kWarps + 1;
  const int limit = dph::stream_cta_limit();
  return limit > 0 ? std::min(want, (unsigned)limit) : want;
}

// ---- the global norm -----------------------------------------------------------

template <int CAP>
struct NormParams {
  const void* grad[CAP];
  unsigned long long numel[CAP];
  unsigned ustart[CAP + 1];  // prefix sums of units (kNormUnit elements)
  uint8_t vec_ok[CAP];
  int n;
  int slots;         // this launch's partial sums
  int slots_before;  // earlier launches' of the same call
  int last;          // 1: this launch forms the norm
  float max_norm;
  unsigned* ticket;
  double* part;
  float* norm;
  float* coef;
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
  return v;
}

// What is gathered over a list: the sum of squares, or the largest magnitude
// (kept as its bit pattern, which orders as the magnitude does with NaN above
// all, and is exact in fp32's and double's place alike).
enum { kSumSquares = 0, kMaxAbs = 1 };

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_down_sync(0xffffffffu, v, o));
  return v;
}
template <int OP>
__device__ __forceinline__ double joined(double a, double b) {
  return OP == kSumSquares ? a + b : fmax(a, b);
}
template <int OP>
__device__ __forceinline__ double warp_joined(double v) {
  return OP == kSumSquares ? warp_sum(v) : warp_max(v);
}
// The whole CTA's, in thread 0.
template <int OP>
__device__ __forceinline__ double block_joined(double v, double* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_joined<OP>(v);
  if (lane == 0) sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    v = lane < kNormWarps ? sums[lane] : 0.0;
#pragma unroll
    for (int o = kNormWarps / 2; o > 0; o >>= 1)
      v = joined<OP>(v, __shfl_down_sync(0xffffffffu, v, o));
  }
  return v;
}

// Squares are summed in fp32 over 32 elements of a lane, two such sums are
// added in fp32, and the rest is in double.  Partial sum s covers the units of
// virtual CTA s (s, s + slots, ... by warps), whatever CTA computes it, and the
// last CTA to finish adds the partial sums in order: the result depends neither
// on the grid nor on the order in which CTAs finish.
template <typename GT, int OP, int CAP>
__global__ void __launch_bounds__(kNormThreads, 3) norm_kernel(const __grid_constant__ NormParams<CAP> a) {
  __shared__ double sums[kNormWarps];
  __shared__ bool is_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned units = a.ustart[a.n];
  stream_order();
  for (int s = blockIdx.x; s < a.slots; s += gridDim.x) {
    unsigned u = (unsigned)s * kNormWarps + warp;
    double sum = 0.0;
    int t = 0;
    for (int hi = a.n - 1; t < hi;) {
      const int mid = (t + hi + 1) >> 1;
      if (a.ustart[mid] <= u) t = mid;
      else hi = mid - 1;
    }
    for (; u < units; u += (unsigned)a.slots * kNormWarps) {
      while (a.ustart[t + 1] <= u) ++t;
      const unsigned long long e0 = (unsigned long long)(u - a.ustart[t]) * kNormUnit;
      const unsigned long long left = a.numel[t] - e0;
      const GT* gp = static_cast<const GT*>(a.grad[t]) + e0;
      float acc[2] = {0.0f, 0.0f};
      uint32_t top = 0;
      const auto take = [&](float g, int half) {
        if constexpr (OP == kSumSquares)
          acc[half] = __fadd_rn(acc[half], __fmul_rn(g, g));
        else
          top = max(top, __float_as_uint(g) & 0x7fffffffu);
      };
      if (a.vec_ok[t] && left >= kNormUnit) {
        float g[kNormLoads][8];
#pragma unroll
        for (int j = 0; j < kNormLoads; ++j) ld8(gp + j * 256 + lane * 8, g[j]);
#pragma unroll
        for (int j = 0; j < kNormLoads; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) take(g[j][i], j & 1);
      } else {
        const int len = left < kNormUnit ? (int)left : kNormUnit;
#pragma unroll 8
        for (int i = 0; i < kNormUnit / 32; ++i) {
          const int o = i * 32 + lane;
          take(o < len ? widen_scalar(gp, o) : 0.0f, i & 1);
        }
      }
      sum = joined<OP>(sum, OP == kSumSquares ? (double)__fadd_rn(acc[0], acc[1]) : (double)top);
    }
    sum = block_joined<OP>(sum, sums);
    if (threadIdx.x == 0) a.part[a.slots_before + s] = sum;
    __syncthreads();
  }
  if (!a.last) return;
  if (threadIdx.x == 0) {
    __threadfence();
    is_last = atomicInc(a.ticket, gridDim.x - 1) == gridDim.x - 1;  // wraps to 0 for the next call
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  const int total = a.slots_before + a.slots;
  double sum = 0.0;
  for (int i = threadIdx.x; i < total; i += kNormThreads) sum = joined<OP>(sum, __ldcg(a.part + i));
  const double all = block_joined<OP>(sum, sums);
  if (threadIdx.x == 0) {
    if constexpr (OP == kMaxAbs) {
      *a.norm = __fmul_rn(__uint_as_float((uint32_t)all), kTopFp4);
      return;
    }
    const float norm = (float)sqrt(all);
    const float c = __fdiv_rn(a.max_norm, __fadd_rn(norm, 1e-6f));
    if (a.norm) *a.norm = norm;
    if (a.coef)
      *a.coef = isfinite(norm) ? fminf(c, 1.0f) : __uint_as_float(0x7fffffffu);
  }
}

size_t esize(dp_dtype_t t) { return t == DP_FP32 ? 4u : 2u; }
bool dtype_ok(dp_dtype_t t) { return t == DP_FP32 || t == DP_BF16; }
using dph::aligned;
using dph::Span;
using dph::span_of;
using dph::spans_clash;

constexpr int kNormCap = 768;      // tensors per norm launch: 19 KB of kernel parameters
constexpr int kNormCapSmall = 32;

template <typename GT, int OP, int CAP>
cudaError_t norm_launch(const void* const* grads, const size_t* numels, const std::vector<int>& at,
                        size_t first, size_t count, int slots_before, int* slots, bool last,
                        float max_norm, unsigned* ticket, double* part, float* norm, float* coef,
                        const dph::DeviceInfo& dev, cudaStream_t s) {
  NormParams<CAP> p;
  unsigned units = 0;
  for (size_t i = 0; i < count; ++i) {
    const int t = at[first + i];
    p.grad[i] = grads[t];
    p.numel[i] = numels[t];
    p.vec_ok[i] = aligned(grads[t], sizeof(GT) * 8);
    p.ustart[i] = units;
    units += (unsigned)((numels[t] + kNormUnit - 1) / kNormUnit);
  }
  p.n = (int)count;
  p.ustart[count] = units;
  *slots = (int)std::min<unsigned>(kNormSlots, std::max(1u, (units + kNormWarps - 1) / kNormWarps));
  p.slots = *slots;
  p.slots_before = slots_before;
  p.last = last;
  p.max_norm = max_norm;
  p.ticket = ticket;
  p.part = part;
  p.norm = norm;
  p.coef = coef;
  const int grid = std::min(*slots, resident_blocks(norm_kernel<GT, OP, CAP>, dev));
  return dph::launch_early(norm_kernel<GT, OP, CAP>, p, (unsigned)grid, kNormThreads, s);
}

constexpr size_t kNormHead = 256;  // the ticket, ahead of the partial sums

}  // namespace

// ---- the AdamW object ----------------------------------------------------------

struct dp_adamw {
  static constexpr int kCap = 384;      // tensors per launch (32 KB of kernel parameters)
  static constexpr int kCapSmall = 32;  // short lists: less to pass with each launch
  dp_dtype_t param_dtype, grad_dtype;
  dp_state_t state;
  std::vector<AdamwParams<kCap>> tables;
  std::vector<dph::Span> spans;         // the list's buffers
  unsigned* skips = nullptr;
  std::mutex mu;
};

namespace {

template <typename PT, typename GT, bool S8>
cudaError_t adamw_launch(const AdamwParams<dp_adamw::kCap>& table, cudaStream_t s) {
  const unsigned units = table.ustart[table.n];
  if (table.n > dp_adamw::kCapSmall) {
    return dph::launch_early(adamw_kernel<PT, GT, S8, dp_adamw::kCap>, table, blocks_for(units),
                             kThreads, s);
  }
  AdamwParams<dp_adamw::kCapSmall> p;
  const size_t n = (size_t)table.n;
  memcpy(p.tensor, table.tensor, n * sizeof(AdamwTensor));
  memcpy(p.ustart, table.ustart, (n + 1) * sizeof(unsigned));
  p.n = table.n;
  p.lr = table.lr;
  p.beta1 = table.beta1;
  p.omb1 = table.omb1;
  p.beta2 = table.beta2;
  p.omb2 = table.omb2;
  p.eps = table.eps;
  p.step_size = table.step_size;
  p.inv_root = table.inv_root;
  p.grad_scale = table.grad_scale;
  p.schedule = table.schedule;
  p.skips = table.skips;
  p.step = table.step;
  p.counts = table.counts;
  p.log_beta1 = table.log_beta1;
  p.log_beta2 = table.log_beta2;
  return dph::launch_early(adamw_kernel<PT, GT, S8, dp_adamw::kCapSmall>, p, blocks_for(units),
                           kThreads, s);
}

template <typename PT, typename GT>
cudaError_t adamw_launch_s(const dp_adamw& o, const AdamwParams<dp_adamw::kCap>& table,
                           cudaStream_t s) {
  return o.state == DP_STATE_8BIT ? adamw_launch<PT, GT, true>(table, s)
                                  : adamw_launch<PT, GT, false>(table, s);
}

cudaError_t adamw_dispatch(const dp_adamw& o, const AdamwParams<dp_adamw::kCap>& table,
                           cudaStream_t s) {
  if (o.param_dtype == DP_FP32)
    return o.grad_dtype == DP_FP32 ? adamw_launch_s<float, float>(o, table, s)
                                   : adamw_launch_s<float, uint16_t>(o, table, s);
  return o.grad_dtype == DP_FP32 ? adamw_launch_s<uint16_t, float>(o, table, s)
                                 : adamw_launch_s<uint16_t, uint16_t>(o, table, s);
}

// One pass over a list: the checks, and as many launches as the list needs.
template <int OP>
dp_status_t gather_list(const void* const* grads, const size_t* numels, int n,
                        dp_dtype_t grad_dtype, float max_norm, float* norm, float* coef,
                        void* workspace, size_t workspace_bytes, cudaStream_t s) {
  if (n < 0 || (n > 0 && (!grads || !numels)) || !workspace) return DP_ERR_INVALID_ARG;
  if (!dtype_ok(grad_dtype)) return DP_ERR_UNSUPPORTED;
  size_t need = 0;
  dp_grad_norm_workspace_size(n, &need);
  if (workspace_bytes < need) return DP_ERR_INVALID_ARG;
  const size_t es = esize(grad_dtype);
  if (!aligned(workspace, 16) || (norm && !aligned(norm, 4)) || (coef && !aligned(coef, 4)))
    return DP_ERR_UNSUPPORTED;
  try {
    std::vector<int> at;  // tensors with elements
    std::vector<Span> spans;
    unsigned long long units = 0;
    at.reserve((size_t)n);
    spans.reserve((size_t)n + 3);
    for (int t = 0; t < n; ++t) {
      if (numels[t] == 0) continue;
      if (!grads[t]) return DP_ERR_INVALID_ARG;
      units += (numels[t] - 1) / kNormUnit + 1;
      if (!aligned(grads[t], es) || units > 0x7fffffffull) return DP_ERR_UNSUPPORTED;
      spans.push_back(span_of(grads[t], numels[t] * es));
      at.push_back(t);
    }
    const auto out = [&](const void* p, size_t b) {
      if (p) spans.push_back(span_of(p, b, true));
    };
    out(norm, 4);
    out(coef, 4);
    out(workspace, need);
    if (spans_clash(spans)) return DP_ERR_ALIAS;
    dph::DeviceInfo dev;
    if (!dph::current_device(&dev)) return DP_ERR_CUDA;
    unsigned* ticket = static_cast<unsigned*>(workspace);
    double* part = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + kNormHead);
    int slots_before = 0;
    size_t first = 0;
    do {  // one launch at least: an empty list has norm 0
      const size_t count = std::min<size_t>(at.size() - first, kNormCap);
      const bool last = first + count == at.size();
      int slots = 0;
      cudaError_t e;
      const bool small = count <= kNormCapSmall;
#define DP_NORM(GT, CAP)                                                                        \
  norm_launch<GT, OP, CAP>(grads, numels, at, first, count, slots_before, &slots, last, max_norm,   \
                       ticket, part, norm, coef, dev, s)
      if (grad_dtype == DP_FP32)
        e = small ? DP_NORM(float, kNormCapSmall) : DP_NORM(float, kNormCap);
      else
        e = small ? DP_NORM(uint16_t, kNormCapSmall) : DP_NORM(uint16_t, kNormCap);
#undef DP_NORM
      if (e != cudaSuccess) return DP_ERR_CUDA;
      slots_before += slots;
      first += count;
    } while (first < at.size());
  } catch (const std::bad_alloc&) {
    return DP_ERR_INVALID_ARG;
  }
  return DP_OK;
}

}  // namespace

extern "C" {

dp_status_t dp_grad_norm_workspace_size(int n, size_t* bytes) {
  if (!bytes) return DP_ERR_INVALID_ARG;
  *bytes = 0;
  if (n < 0) return DP_ERR_INVALID_ARG;
  const size_t launches = ((size_t)n + kNormCap - 1) / kNormCap;
  *bytes = kNormHead + std::max<size_t>(1, launches) * kNormSlots * sizeof(double);
  return DP_OK;
}

dp_status_t dp_grad_norm(const void* const* grads, const size_t* numels, int n,
                         dp_dtype_t grad_dtype, float max_norm, float* norm, float* coef,
                         void* workspace, size_t workspace_bytes, dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_grad_norm");
  if ((!norm && !coef) || !(max_norm > 0.0f)) return DP_ERR_INVALID_ARG;
  return gather_list<kSumSquares>(grads, numels, n, grad_dtype, max_norm, norm, coef, workspace,
                                  workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dp_status_t dp_mx4_tensor_scale(const void* const* x, const size_t* numels, int n,
                                dp_dtype_t x_dtype, float* scale, void* workspace,
                                size_t workspace_bytes, dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_mx4_tensor_scale");
  if (!scale) return DP_ERR_INVALID_ARG;
  return gather_list<kMaxAbs>(x, numels, n, x_dtype, 1.0f, scale, nullptr, workspace,
                              workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dp_status_t dp_adamw_create(const dp_adamw_tensor_t* tensors, int n, dp_dtype_t param_dtype,
                            dp_dtype_t grad_dtype, dp_state_t state, dp_adamw_t** out) {
  if (!out) return DP_ERR_INVALID_ARG;
  *out = nullptr;
  if (n < 0 || (n > 0 && !tensors)) return DP_ERR_INVALID_ARG;
  if (!dtype_ok(param_dtype) || !dtype_ok(grad_dtype)) return DP_ERR_UNSUPPORTED;
  if (state != DP_STATE_FP32 && state != DP_STATE_8BIT) return DP_ERR_UNSUPPORTED;
  const bool s8 = state == DP_STATE_8BIT;
  const size_t ps = esize(param_dtype), gs = esize(grad_dtype), ss = s8 ? 1 : 4;
  dp_adamw* o = nullptr;
  try {
    o = new dp_adamw;
    o->param_dtype = param_dtype;
    o->grad_dtype = grad_dtype;
    o->state = state;
    std::vector<Span>& spans = o->spans;
    spans.reserve((size_t)n * 7);
    dp_status_t bad = DP_OK;
    unsigned long long units = 0;
    for (int t = 0; t < n && bad == DP_OK; ++t) {
      const dp_adamw_tensor_t& x = tensors[t];
      if (x.numel == 0) continue;
      if (!x.param || !x.grad || !x.exp_avg || !x.exp_avg_sq ||
          (s8 && (!x.exp_avg_scale || !x.exp_avg_sq_scale)) || !(x.weight_decay >= 0.0f) ||
          std::isinf(x.weight_decay)) {
        bad = DP_ERR_INVALID_ARG;
        break;
      }
      const unsigned long long u = (x.numel - 1) / kUnit + 1;
      if (!aligned(x.param, ps) || !aligned(x.grad, gs) || !aligned(x.copy, 2) ||
          !aligned(x.exp_avg, ss) || !aligned(x.exp_avg_sq, ss) ||
          (s8 && (!aligned(x.exp_avg_scale, 4) || !aligned(x.exp_avg_sq_scale, 4))) ||
          u > 0x7fffffffull) {
        bad = DP_ERR_UNSUPPORTED;
        break;
      }
      const auto span = [&](const void* p, size_t bytes, bool written) {
        if (p) spans.push_back(span_of(p, bytes, written));
      };
      span(x.param, x.numel * ps, true);
      span(x.grad, x.numel * gs, false);
      span(x.copy, x.numel * 2, true);
      span(x.exp_avg, x.numel * ss, true);
      span(x.exp_avg_sq, x.numel * ss, true);
      if (s8) {
        span(x.exp_avg_scale, (size_t)u * 4, true);
        span(x.exp_avg_sq_scale, (size_t)u * 4, true);
      }
      if (o->tables.empty() || o->tables.back().n == dp_adamw::kCap || units + u > 0x7fffffffull) {
        o->tables.emplace_back();
        memset(&o->tables.back(), 0, sizeof o->tables.back());
        units = 0;
      }
      auto& p = o->tables.back();
      const int i = p.n++;
      AdamwTensor& y = p.tensor[i];
      y.param = x.param;
      y.grad = x.grad;
      y.copy = static_cast<uint16_t*>(x.copy);
      y.m = x.exp_avg;
      y.v = x.exp_avg_sq;
      y.m_scale = s8 ? x.exp_avg_scale : nullptr;
      y.v_scale = s8 ? x.exp_avg_sq_scale : nullptr;
      y.numel = x.numel;
      y.decay = x.weight_decay;
      // eight elements of every array from an address that one load or store takes
      y.vec_ok = aligned(x.param, ps * 8) && aligned(x.grad, gs * 8) && aligned(x.copy, 16) &&
                 aligned(x.exp_avg, ss * 8) && aligned(x.exp_avg_sq, ss * 8);
      units += u;
      p.ustart[i + 1] = (unsigned)units;
    }
    if (bad == DP_OK && spans_clash(spans)) bad = DP_ERR_ALIAS;
    if (bad != DP_OK) {
      delete o;
      return bad;
    }
  } catch (const std::bad_alloc&) {
    delete o;
    return DP_ERR_INVALID_ARG;
  }
  *out = o;
  return DP_OK;
}

void dp_adamw_destroy(dp_adamw_t* o) { delete o; }

dp_status_t dp_adamw_count_skips(dp_adamw_t* o, unsigned int* skips) {
  if (!o) return DP_ERR_INVALID_ARG;
  if (!aligned(skips, 4)) return DP_ERR_UNSUPPORTED;
  if (skips)
    for (const Span& x : o->spans)
      if (dph::clash(x, span_of(skips, 4))) return DP_ERR_ALIAS;
  std::lock_guard<std::mutex> lock(o->mu);
  o->skips = skips;
  return DP_OK;
}

dp_status_t dp_adamw_step(dp_adamw_t* o, double lr, double beta1, double beta2, double eps,
                          long long step, const float* grad_scale, const float* schedule,
                          dp_stream_t stream) {
  dph::NvtxRange nvtx_range("dp_adamw_step");
  if (!o || step < 1 || !std::isfinite(lr)) return DP_ERR_INVALID_ARG;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return DP_ERR_INVALID_ARG;
  if (!((float)eps >= FLT_MIN) || std::isinf((float)eps)) return DP_ERR_INVALID_ARG;
  if (!aligned(grad_scale, 4) || !aligned(schedule, 4)) return DP_ERR_UNSUPPORTED;
  if (o->tables.empty()) return DP_OK;
  dph::DeviceInfo dev;
  if (!dph::current_device(&dev)) return DP_ERR_CUDA;
  const double fix1 = 1.0 - std::pow(beta1, (double)step);
  const double fix2 = 1.0 - std::pow(beta2, (double)step);
  std::lock_guard<std::mutex> lock(o->mu);
  for (auto& table : o->tables) {
    table.lr = lr;
    table.beta1 = (float)beta1;
    table.omb1 = (float)(1.0 - beta1);
    table.beta2 = (float)beta2;
    table.omb2 = (float)(1.0 - beta2);
    table.eps = (float)eps;
    table.step_size = (float)(lr / fix1);
    table.inv_root = (float)(1.0 / std::sqrt(fix2));
    table.grad_scale = grad_scale;
    table.schedule = schedule;
    table.skips = o->skips;
    table.step = (unsigned)std::min<long long>(step, 0x7fffffffll);
    table.counts = o->skips && &table == &o->tables.front();
    table.log_beta1 = (float)std::log(beta1);
    table.log_beta2 = (float)std::log(beta2);
    if (adamw_dispatch(*o, table, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
      return DP_ERR_CUDA;
  }
  return DP_OK;
}

}  // extern "C"
