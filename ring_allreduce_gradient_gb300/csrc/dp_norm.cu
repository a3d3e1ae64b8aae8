// dp_norm.cu -- the root-mean-square norm in front of a layer's products, with
// the residual's addition and the quantised form of its output in the same
// pass, and its backward pass.
//
// Forward, for every row (D elements of type T):
//   h = round_T(x + residual)          (no residual: h = x, not written)
//   r = 1 / sqrt(mean(h^2) + eps)
//   y = (h w) r                        fp32; stored as T, or quantised as it is
// The norm is of h as it is stored, so the backward pass sees the same values.
// Backward, with xh = h r and g = dy w:
//   dx = r (g - xh mean(g xh)) + dh
//   dw = sum over rows of dy xh
//
// Both are bound by memory (bf16, residual, 8-bit output: 7.03 bytes an element
// for about 10 operations; backward with dh: 8 bytes).  A row is held in
// registers by its warps, 16 G elements a thread, from its load to its store, so
// it crosses memory once (where they suffice, see below); a thread's sixteen consecutive elements are one or two
// 32-byte loads and half a block of 32 (the other half is its neighbour lane's).
// Where a CTA takes several rows, the next ones are on their way to shared memory
// by bulk copies.  Arithmetic is in pairs of fp32, one instruction each.
//
// Measured (GB300, launches in a CUDA graph, inputs larger than L2), 8192 x 4096
// bf16: forward with residual to 8 bits 39.5 us (236 MB: 6.0 TB/s; 58 % of the
// issue slots), to mxfp4 38, to nvfp4 41.5, plain 28 (134 MB; 44 with the residual),
// backward with dh 45.5 us with the sum over 304 sets of rows (268 MB: 5.9 TB/s, 75 %
// of DRAM under the profiler); fp32: 69, 68, 76, 44 (90) and 83 us.  One row of 4096: 2.1 us, 1000 x 768
// fp32 4.8, 2050 x 1120 to nvfp4 8.7 (first loads, and the two divisors of each block
// of 16), backward of 1031 x 1601 fp32 11 us (scalar accesses).  What led there: a CTA
// for each row with scalar fp32 arithmetic 49 and 101 us; pairs of fp32 and
// add.bf16x2 took the forward from 34 to 25 instructions an element; a thread's own
// 16-byte cp.async pieces touched every sector twice (61 and 87 us); rows ahead in
// registers spilled (backward 72 us); bulk copies with 2 stages and turns of 6 sets
// forward (3 stages 41 us, the whole share of the GPU in one turn 40.4), 3 stages and
// 128 registers backward (80 registers, three CTAs an SM, spill: 60; 456 sets of rows
// 55.7).
//
// Long rows do not fit the registers.  Above D = 8192 a thread has 32 elements (G = 2),
// in 128 registers, and above 16384 in 64: what does not fit is spilled to local memory
// (-Xptxas -v, bytes of stores a thread: backward up to 16384 444-1140, above that
// 1584-2188; forward above 16384 584-1436, below it 108 at most), next to 64 or 128
// bytes of an array that the thread's share of the row has.  Forward with residual to 8
// bits / backward with dh, bf16: 8192 x 8192 91 / 93 us (5.2 / 5.8 TB/s), 4096 x 12288
// 66 / 110 (5.3 / 3.7), 4096 x 16384 81 / 145 (5.8 / 3.7), 2048 x 24576 112 / 299 (3.2 /
// 1.4), 2048 x 32768 156 / 462 (3.0 / 1.2); fp32: 150 / 160 (5.9 / 6.7), 133 / 195 (4.9 /
// 4.1), 134 / 259 (6.5 / 4.2), 213 / 455 (3.1 / 1.8), 296 / 634 (3.0 / 1.7).

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

// How a row is laid over threads: `warps` of them hold it, rows_cta rows at once
// in a CTA.  vec: every row of every buffer starts on a 32-byte boundary and D is a
// multiple of 16.  It is one flag for all of them, and without it every access is of one
// element and no row comes ahead: 8192 x 4096 to 8 bits takes 228 us with the weight alone
// off a boundary, against 39.5 (a flag for each buffer has not been built).  stages: sets of rows that are on their way to shared memory.
struct RowPlan {
  int warps, rows_cta, vec, stages;
};

struct NormFwdParams {
  RowPlan plan;
  unsigned* err;
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
  int span;      // sets of rows_cta rows that a CTA takes one after another
  float down;    // a power of two, one over a row's threads or less
  float eps, inv_d;  // inv_d: 1 / (D down)
  int w_f32;
};

struct NormBwdParams {
  RowPlan plan;
  unsigned* err;
  const void* dy;
  const void* h;
  const void* dh;  // or NULL
  const void* w;
  const float* rstd;
  void* dx;
  float* part;     // [groups][D]: a group's sum of dy xh over its rows
  long long ldy, ldh, ldd;
  int M, D;
  int groups;      // a group's rows: every groups-th set of rows_cta
  float inv_d;
  int w_f32;
};

__device__ __forceinline__ void put_at(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_at(uint16_t* p, float v) { *p = bf16_rn(v); }

// A thread's 16 G elements of a row as they are stored, bf16 ones in pairs; taken
// out and put in two at a time (fp32 pairs are one instruction's operands).
template <typename T, int G>
struct Held;
template <int G>
struct Held<float, G> {
  uint32_t r[16 * G];
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(r[i]); }
  __device__ __forceinline__ uint64_t two(int j) const { return pair(at(2 * j), at(2 * j + 1)); }
  __device__ __forceinline__ void put(int j, uint64_t v) {
    float a, b;
    unpair(v, a, b);
    r[2 * j] = __float_as_uint(a);
    r[2 * j + 1] = __float_as_uint(b);
  }
  __device__ __forceinline__ void add(int j, const Held& o) { put(j, add2(two(j), o.two(j))); }
};
template <int G>
struct Held<uint16_t, G> {
  uint32_t r[8 * G];
  __device__ __forceinline__ float at(int i) const {
    return i & 1 ? bf16hi(r[i / 2]) : bf16lo(r[i / 2]);
  }
  __device__ __forceinline__ uint64_t two(int j) const { return pair(bf16lo(r[j]), bf16hi(r[j])); }
  __device__ __forceinline__ void put(int j, uint64_t v) {
    float a, b;
    unpair(v, a, b);
    r[j] = pack_bf16x2_rn(a, b);
  }
  // Rounded once.  That is also the fp32 sum rounded: where fp32 cannot hold the
  // sum of two bf16 values, the smaller is below half a step of the larger.
  __device__ __forceinline__ void add(int j, const Held& o) {
    asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(r[j]) : "r"(o.r[j]));
  }
};

// A thread's place in its row.  Element i of the thread is sixteen to a group,
// groups a row's threads apart, where rows are aligned (or blocks are quantised);
// else every threads-th element, so that a warp's scalar accesses are consecutive.
struct Place {
  int t, threads, sub, D;  // sub: which of the CTA's rows
  bool vec, chunks;
  __device__ __forceinline__ int group(int g) const { return (g * threads + t) * 16; }
  __device__ __forceinline__ int element(int i) const {
    return chunks ? group(i / 16) + i % 16 : i * threads + t;
  }
};

template <typename T, int G>
__device__ __forceinline__ void load_row(const T* p, bool in, const Place& at, Held<T, G>& v) {
  constexpr int kWords = sizeof(v.r) / 4 / G;  // of a group
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int e = at.group(g);
    uint32_t* r = v.r + g * kWords;
    if (at.vec) {  // (lanes past the row's end only take zeros, not the other way round)
#pragma unroll
      for (int h = 0; h < kWords; ++h) r[h] = 0u;
      if (in && e < at.D) {
#pragma unroll
        for (int h = 0; h < kWords; h += 8)
          asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                       : "=r"(r[h]), "=r"(r[h + 1]), "=r"(r[h + 2]), "=r"(r[h + 3]), "=r"(r[h + 4]),
                         "=r"(r[h + 5]), "=r"(r[h + 6]), "=r"(r[h + 7])
                       : "l"(reinterpret_cast<const uint32_t*>(p + e) + h));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const int a = at.element(16 * g + i), b = at.element(16 * g + i + 1);
        v.put(8 * g + i / 2, pair(in && a < at.D ? widen_scalar(p, a) : 0.0f,
                                  in && b < at.D ? widen_scalar(p, b) : 0.0f));
      }
    }
  }
}

template <typename T, int G>
__device__ __forceinline__ void store_row(T* p, const Place& at, const Held<T, G>& v) {
  constexpr int kWords = sizeof(v.r) / 4 / G;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int e = at.group(g);
    const uint32_t* r = v.r + g * kWords;
    if (at.vec) {
      if (e < at.D) {
#pragma unroll
        for (int h = 0; h < kWords; h += 8)
          asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(
                           reinterpret_cast<uint32_t*>(p + e) + h),
                       "r"(r[h]), "r"(r[h + 1]), "r"(r[h + 2]), "r"(r[h + 3]), "r"(r[h + 4]),
                       "r"(r[h + 5]), "r"(r[h + 6]), "r"(r[h + 7])
                       : "memory");
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int o = at.element(16 * g + i);
        if (o < at.D) put_at(p + o, v.at(16 * g + i));
      }
    }
  }
}

template <int G>
__device__ __forceinline__ void load_weight(const void* w, bool f32, const Place& at,
                                            uint64_t (&v)[8 * G]) {
  if (f32) {
    Held<float, G> h;
    load_row(static_cast<const float*>(w), true, at, h);
#pragma unroll
    for (int j = 0; j < 8 * G; ++j) v[j] = h.two(j);
  } else {
    Held<uint16_t, G> h;
    load_row(static_cast<const uint16_t*>(w), true, at, h);
#pragma unroll
    for (int j = 0; j < 8 * G; ++j) v[j] = h.two(j);
  }
}
// The four sums that two pairs hold.
__device__ __forceinline__ float sum4(uint64_t p, uint64_t q) {
  float a, b;
  unpair(add2(p, q), a, b);
  return __fadd_rn(a, b);
}

// Rows on their way to shared memory, a ring of them for each row that the CTA
// takes at once: its first thread copies whole rows (cp.async.bulk), so what is in
// flight takes no registers and comes in whole lines.
constexpr int kMaxStages = 3;
constexpr uint64_t kTimeoutNs = 2000000000ull;
template <typename T, int G, int ARRAYS>
struct Ring {
  uint8_t* base;      // of this row
  int arrays;         // that there are
  uint64_t* full;     // a barrier for each stage
  uint32_t bytes;     // of a row
  int stages, slot;   // the stage to read next
  uint32_t phase;
  unsigned* err;
  __device__ __forceinline__ void init(uint8_t* smem, uint64_t* bars, const RowPlan& plan, int sub,
                                       int D, int n, unsigned* e) {
    bytes = (uint32_t)D * sizeof(T);
    arrays = n;
    stages = plan.stages;
    base = smem + (size_t)sub * stages * arrays * bytes;
    full = bars + sub * kMaxStages;
    slot = 0;
    phase = 0;
    err = e;
    if (threadIdx.x == 0) {
      for (int i = 0; i < plan.rows_cta * kMaxStages; ++i) mbar_init(&bars[i], 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
  }
  // By the row's first thread: the arrays' rows (NULL: none) into a stage.
  __device__ __forceinline__ void copy(int stage, const T* const (&from)[ARRAYS]) const {
    uint32_t n = 0;
#pragma unroll
    for (int a = 0; a < ARRAYS; ++a) n += from[a] ? bytes : 0u;
    mbar_arrive_expect_tx(&full[stage], n);
#pragma unroll
    for (int a = 0; a < ARRAYS; ++a)
      if (from[a])
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
            "[%3];" ::"r"(smem_u32(base + (size_t)(stage * arrays + a) * bytes)),
            "l"(from[a]), "r"(bytes), "r"(smem_u32(&full[stage]))
            : "memory");
  }
  // Until the stage to read has landed (or the error word says that it did not).
  __device__ __forceinline__ void wait() const {
    (void)mbar_wait_bounded(&full[slot], phase, err, kTimeoutNs);
  }
  __device__ __forceinline__ void read(int array, bool in, const Place& at, Held<T, G>& v) const {
    constexpr int kPieces = (int)sizeof(T);  // of 16 bytes, of a group
    const uint8_t* row = base + (size_t)(slot * arrays + array) * bytes;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const bool have = in && at.group(g) < at.D;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (have)
          q = *reinterpret_cast<const uint4*>(row + (size_t)at.group(g) * sizeof(T) + i * 16);
        uint32_t* r = v.r + (g * kPieces + i) * 4;
        r[0] = q.x, r[1] = q.y, r[2] = q.z, r[3] = q.w;
      }
    }
  }
  __device__ __forceinline__ void next() {
    if (++slot == stages) slot = 0, phase ^= 1u;
  }
};

// The sum over a row's threads, in all of them and in a fixed order.  part: 32
// words for each row of the CTA; a call's words are not reused before the call
// after the next, so one barrier a call (of the row's warps alone; barrier 0 is the
// whole CTA's) is enough.
__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float row_sum(float v, float* part, const Place& at) {
  v = warp_total(v);
  if (at.threads > 32) {
    if ((at.t & 31) == 0) part[at.t >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(at.sub + 1), "r"(at.threads) : "memory");
    v = warp_total((at.t & 31) * 32 < at.threads ? part[at.t & 31] : 0.0f);
  } else {
    __syncwarp();
  }
  return v;
}

// 1 / sqrt(m): the approximate one, corrected by what its square misses; 0 for
// infinity, infinity for 0.
__device__ __forceinline__ float inverse_root(float m) {
  const float r = rsqrtf(m);
  const float miss = __fmaf_rn(-__fmul_rn(m, r), r, 1.0f);
  const float better = __fmaf_rn(__fmul_rn(0.5f, r), miss, r);
  return m > 0.0f && m < 3.0e38f ? better : r;
}

// The largest magnitude of three; NaN if one is.
__device__ __forceinline__ float max_mag3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A thread's quantised elements and their scales.  Every lane comes here: a
// block of 32 is two lanes'.
template <int FMT, int G>
__device__ __forceinline__ void quantise_row(const NormFwdParams& p, int r, const Place& at,
                                             float tscale, const Divisor& by_t,
                                             const uint64_t (&y)[8 * G]) {
  constexpr int BLOCK = FMT == kToNv4 ? kNvBlock : kMxBlock;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int e = at.group(g);
    const uint64_t* v = y + 8 * g;
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float a, b;
      unpair(v[j], a, b);
      top = max_mag3(top, a, b);
    }
    if constexpr (BLOCK == kMxBlock) {
      const float other = __shfl_xor_sync(0xffffffffu, top, 1);
      top = max_mag3(top, other, other);
    }
    const bool in = r < p.M && e < p.D;
    uint32_t byte;
    if constexpr (FMT == kToMx8) {
      const Scale8 s(top);
      byte = s.byte;
      if (in)
        *reinterpret_cast<uint4*>(p.codes + (size_t)r * p.D + e) =
            make_uint4(s.codes(v[0], v[1]), s.codes(v[2], v[3]), s.codes(v[4], v[5]),
                       s.codes(v[6], v[7]));
    } else {
      const Scale<BLOCK> s(top, tscale, by_t);
      byte = s.byte;
      if (in) {
        uint32_t c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) unpair(v[4 * h + j], w[2 * j], w[2 * j + 1]);
          c[h] = s.codes(w);
        }
        *reinterpret_cast<uint2*>(p.codes + (size_t)r * (p.D / 2) + e / 2) =
            make_uint2(c[0], c[1]);
      }
    }
    const int b = e / BLOCK;
    if (b / 4 < p.col_tiles && (BLOCK == kNvBlock || at.t % 2 == 0))
      p.scales[scale_at(r, b / 4, p.col_tiles) + b % 4] = in ? (uint8_t)byte : (uint8_t)0;
  }
}

template <typename T, int FMT, int THREADS, int G, bool BULK>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? (BULK ? 3 : 4) : 1)
    norm_fwd_kernel(const __grid_constant__ NormFwdParams p) {
  __shared__ float part[2][THREADS / 32];
  stream_order();
  const int threads = p.plan.warps * 32, sub = (int)threadIdx.x / threads;
  const Place at{(int)threadIdx.x - sub * threads, threads, sub, p.D, p.plan.vec != 0,
                 FMT != kPlain || p.plan.vec != 0};
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t bars[BULK ? 8 * kMaxStages : 1];
  Ring<T, G, 2> ring;
  if constexpr (BULK) ring.init(smem, bars, p.plan, sub, p.D, p.res ? 2 : 1, p.err);
  // What all rows share.  It is asked for after the first row: unpacking it would
  // hold the row's loads up for as long as it takes to come (2050 x 1120 to nvfp4 9.5
  // -> 8.7 us).
  uint64_t w[8 * G];
  float tscale = 1.0f;
  Divisor by_t(1.0f);
  bool ready = false;

  // This CTA's sets of rows, in turns of `span` sets one after another.
  struct Walk {
    long long row;  // of this thread's row
    int left;       // sets of the turn after this one
  };
  const long long skip = (long long)(gridDim.x - 1) * p.span * p.plan.rows_cta;
  const auto next = [&](Walk& k) {
    k.row += p.plan.rows_cta;
    if (k.left-- == 0) k.left = p.span - 1, k.row += skip;
  };
  Walk now{(long long)blockIdx.x * p.span * p.plan.rows_cta + sub, p.span - 1}, ahead = now;
  const auto fetch = [&](int stage) {
    if (ahead.row < p.M) {
      const T* const from[2] = {
          static_cast<const T*>(p.x) + ahead.row * p.ldx,
          p.res ? static_cast<const T*>(p.res) + ahead.row * p.ldr : nullptr};
      ring.copy(stage, from);
    }
    next(ahead);
  };
  if (BULK && at.t == 0)
    for (int i = 0; i < ring.stages; ++i) fetch(i);
  int turn = 0;
  for (; now.row - sub < p.rows; next(now), turn ^= 1) {
    const int r = (int)now.row;
    const bool in = r < p.M;
    Held<T, G> v, d;
    if constexpr (BULK) {
      if (in) ring.wait();
      ring.read(0, in, at, v);
      if (p.res) ring.read(1, in, at, d);
    } else {
      load_row(static_cast<const T*>(p.x) + now.row * p.ldx, in, at, v);
      if (p.res) load_row(static_cast<const T*>(p.res) + now.row * p.ldr, in, at, d);
    }
    if (!ready) {
      load_weight<G>(p.w, p.w_f32, at, w);
      if (FMT == kToNv4 && p.tscale) {
        tscale = *p.tscale;
        by_t = Divisor(tscale);
      }
      ready = true;
    }
    if (p.res) {
#pragma unroll
      for (int j = 0; j < 8 * G; ++j) v.add(j, d);
      if (in) store_row(static_cast<T*>(p.h) + (size_t)r * p.D, at, v);
    }
    uint64_t s[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8 * G; ++j) s[j % 2] = fma2(v.two(j), v.two(j), s[j % 2]);
    // A thread's own 16 G squares have to fit fp32; times `down` the row's then do, too.
    const float ss =
        row_sum(__fmul_rn(sum4(s[0], s[1]), p.down), part[turn] + sub * p.plan.warps, at);
    if constexpr (BULK) {  // every thread of the row has read its stage
      if (at.t == 0) fetch(ring.slot);
      ring.next();
    }
    const float rstd = inverse_root(__fadd_rn(__fmul_rn(ss, p.inv_d), p.eps));
    if (in && at.t == 0 && p.rstd) p.rstd[r] = rstd;
    // h w first: of bf16 values it is exact, and the product with rstd rounds once
    uint64_t y[8 * G];
#pragma unroll
    for (int j = 0; j < 8 * G; ++j) y[j] = mul2(mul2(v.two(j), w[j]), pair(rstd, rstd));
    if (in && p.y) {
#pragma unroll
      for (int j = 0; j < 8 * G; ++j) d.put(j, y[j]);
      store_row(static_cast<T*>(p.y) + (size_t)r * p.D, at, d);
    }
    if constexpr (FMT != kPlain) quantise_row<FMT, G>(p, r, at, tscale, by_t, y);
  }
}

// ---- backward -----------------------------------------------------------------

// A group's rows and the order of its sums follow from M and D alone, whatever
// CTA takes it, so dw has the same bits under any grid.
template <typename T, int THREADS, int G, bool BULK>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 2 : 1)
    norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float part[2][THREADS / 32];
  __shared__ uint64_t sums[THREADS == 256 ? 8 * 256 : 1];
  stream_order();
  const int threads = p.plan.warps * 32, sub = (int)threadIdx.x / threads;
  const Place at{(int)threadIdx.x - sub * threads, threads, sub, p.D, p.plan.vec != 0, p.plan.vec != 0};
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t bars[BULK ? 8 * kMaxStages : 1];
  Ring<T, G, 3> ring;
  if constexpr (BULK) ring.init(smem, bars, p.plan, sub, p.D, p.dh ? 3 : 2, p.err);
  uint64_t w[8 * G];  // (after the first row's loads, as in the forward pass)
  bool ready = false;

  const long long stride = (long long)p.groups * p.plan.rows_cta;
  int turn = 0;
  for (int q = blockIdx.x; q < p.groups; q += gridDim.x) {
    const long long first = (long long)q * p.plan.rows_cta;
    uint64_t dw[8 * G];
#pragma unroll
    for (int j = 0; j < 8 * G; ++j) dw[j] = 0;
    long long ahead = first + sub;
    const auto fetch = [&](int stage) {
      if (ahead < p.M) {
        const T* const from[3] = {
            static_cast<const T*>(p.h) + ahead * p.ldh, static_cast<const T*>(p.dy) + ahead * p.ldy,
            p.dh ? static_cast<const T*>(p.dh) + ahead * p.ldd : nullptr};
        ring.copy(stage, from);
      }
      ahead += stride;
    };
    if (BULK && at.t == 0)
      for (int i = 0, k = ring.slot; i < ring.stages; ++i, k = k + 1 == ring.stages ? 0 : k + 1)
        fetch(k);
    float rstd_next = first + sub < p.M ? p.rstd[first + sub] : 0.0f;
    for (long long r0 = first; r0 < p.M; r0 += stride, turn ^= 1) {
      const long long r = r0 + sub;
      const bool in = r < p.M;
      const float rstd = rstd_next;
      rstd_next = r + stride < p.M ? p.rstd[r + stride] : 0.0f;
      Held<T, G> h, g, d;
      if constexpr (BULK) {
        if (in) ring.wait();
        ring.read(0, in, at, h);
        ring.read(1, in, at, g);
        if (p.dh) ring.read(2, in, at, d);
      } else {
        load_row(static_cast<const T*>(p.h) + r * p.ldh, in, at, h);
        load_row(static_cast<const T*>(p.dy) + r * p.ldy, in, at, g);
        if (p.dh) load_row(static_cast<const T*>(p.dh) + r * p.ldd, in, at, d);
      }
      if (!ready) {
        load_weight<G>(p.w, p.w_f32, at, w);
        ready = true;
      }
      const uint64_t rr = pair(rstd, rstd);
      uint64_t s[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8 * G; ++j) {
        const uint64_t xh = mul2(h.two(j), rr);
        dw[j] = fma2(g.two(j), xh, dw[j]);
        s[j % 2] = fma2(mul2(g.two(j), w[j]), xh, s[j % 2]);
      }
      const float sum = row_sum(sum4(s[0], s[1]), part[turn] + sub * p.plan.warps, at);
      if constexpr (BULK) {  // every thread of the row has read its stage
        if (at.t == 0) fetch(ring.slot);
        if (in) ring.next();
      }
      const float c = -__fmul_rn(sum, p.inv_d);
      const uint64_t cc = pair(c, c);
#pragma unroll
      for (int j = 0; j < 8 * G; ++j) {
        const uint64_t xh = mul2(h.two(j), rr);
        uint64_t v = mul2(fma2(xh, cc, mul2(g.two(j), w[j])), rr);
        if (p.dh) v = add2(v, d.two(j));
        h.put(j, v);
      }
      if (in) store_row(static_cast<T*>(p.dx) + (size_t)r * p.D, at, h);
    }
    // the rows that a CTA takes at once have their sums added in order
    if (p.plan.rows_cta > 1) {
      uint64_t* mine = sums + threadIdx.x;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8 * G; ++j) mine[j * blockDim.x] = dw[j];
      __syncthreads();
      if (sub == 0)
        for (int k = 1; k < p.plan.rows_cta; ++k)
#pragma unroll
          for (int j = 0; j < 8 * G; ++j)
            dw[j] = add2(dw[j], mine[j * blockDim.x + k * threads]);
      __syncthreads();
    }
    if (sub == 0) {
      Held<float, G> o;
#pragma unroll
      for (int j = 0; j < 8 * G; ++j) o.put(j, dw[j]);
      store_row(p.part + (size_t)q * p.D, at, o);
    }
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

// Threads of a CTA at most, and groups of sixteen elements of a thread, by the
// row's length.
template <typename F>
cudaError_t by_length(int D, const F& f) {
  if (D <= 4096) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 1>());
  if (D <= 8192) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 1>());
  if (D <= 16384) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 2>());
  return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 2>());
}

RowPlan plan_for(int D, bool vec) {
  const int per = D <= 8192 ? 512 : 1024;  // elements of a warp
  const int warps = (D + per - 1) / per;
  return RowPlan{warps, warps <= 8 ? 8 / warps : 1, vec, 0};
}

// Bytes of a ring, and its stages in *p: `most` at most, in `room` bytes of shared
// memory (200 KB where one row is too long for that); 0 where two do not fit.
size_t plan_ring(RowPlan* p, int D, size_t esz, int arrays, int most, size_t room) {
  const size_t stage = (size_t)p->rows_cta * arrays * D * esz;
  if (stage * 2 > room) room = 200u << 10;
  p->stages = p->vec ? (int)std::min<size_t>(most, room / stage) : 0;
  if (p->stages < 2) p->stages = 0;
  return p->stages * stage;
}

template <typename P>
cudaError_t launch(void (*kernel)(P), const P& p, long long blocks, int threads, size_t smem,
                   cudaStream_t s) {
  const int limit = dph::stream_cta_limit();
  if (limit > 0) blocks = std::min<long long>(blocks, limit);
  return dph::launch_early(kernel, p, (unsigned)std::min<long long>(blocks, 0x7fffffffll),
                           (unsigned)threads, s, smem);
}

// Rows of a CTA at once, and sets of rows whose sums of dy xh are kept apart: by
// the sizes alone, so that the bits do not follow the GPU's size.
int rows_per_cta(int D) { return D <= 4096 ? 8 / std::max(1, (D + 511) / 512) : 1; }
int groups_of(int M, int D) {
  const int per = rows_per_cta(D);
  return (int)std::min<long long>(((long long)M + per - 1) / per, D <= 4096 ? 304 : 152);
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
  const bool vec = D % 16 == 0 && aligned(x, 32) && ldx % 16 == 0 && aligned(weight, 32) &&
                   (!residual || (aligned(residual, 32) && ldr % 16 == 0 && aligned(h, 32))) &&
                   aligned(y, 32);
  p.plan = plan_for(D, vec);
  int shares = 32;
  while (shares < p.plan.warps * 32) shares *= 2;
  p.down = 1.0f / (float)shares;
  p.inv_d = 1.0f / (float)D * (float)shares;
  dph::DeviceInfo dev;
  if (!dph::current_device(&dev)) return DP_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const long long sets = ((long long)p.rows + p.plan.rows_cta - 1) / p.plan.rows_cta;
  // A CTA keeps the weights and has rows ahead over a turn of several sets, as long
  // as there are CTAs enough to even out (8192 x 4096: 48.4 us with turns of one,
  // 41.3 of four, 39.4 of six, 39.5 of nine; 4000 x 768 bf16: 10.6 of one, 8.4 of two).
  // What that measured is also how full the last round of CTAs is: 456 of them fit at
  // once, and six make 3.00 rounds of 8192 rows, four 4.49, nine 2.00.  Elsewhere, to 8
  // bits with residual: 4096 rows of 4096 (1.50 rounds) 4.8 TB/s, 5000 5.4, 6000 (2.20)
  // 5.1, 10000 5.9, 8192 of 2048 (1.50) 4.6; the turn of 8192 x 4096 has 5.9.
  p.span = (int)std::max(1ll, std::min(6ll, sets / (dev.sm_count * 3)));
  p.err = dev.err_word;
  const int threads = p.plan.warps * p.plan.rows_cta * 32;
  size_t smem = p.span > 1 ? plan_ring(&p.plan, D, esz, residual ? 2 : 1, 2, 72u << 10) : 0;
  const cudaError_t e = by_length(D, [&](auto most, auto groups) {
    constexpr int N = decltype(most)::value, G = decltype(groups)::value;
    const auto go = [&](auto kernel, auto bulk_kernel) {
      if (smem && dph::prepare_kernel(reinterpret_cast<const void*>(bulk_kernel), N, 200 << 10,
                                      dev.device) < 1)
        return cudaErrorInvalidConfiguration;
      return launch(smem ? bulk_kernel : kernel, p, (sets + p.span - 1) / p.span, threads, smem, s);
    };
#define DP_NORM_FWD(T, F) go(norm_fwd_kernel<T, F, N, G, false>, norm_fwd_kernel<T, F, N, G, true>)
    if (dtype == DP_FP32) {
      if (format == DP_NORM_MXFP4) return DP_NORM_FWD(float, kToMx4);
      if (format == DP_NORM_NVFP4) return DP_NORM_FWD(float, kToNv4);
      if (format == DP_NORM_MXFP8) return DP_NORM_FWD(float, kToMx8);
      return DP_NORM_FWD(float, kPlain);
    }
    if (format == DP_NORM_MXFP4) return DP_NORM_FWD(uint16_t, kToMx4);
    if (format == DP_NORM_NVFP4) return DP_NORM_FWD(uint16_t, kToNv4);
    if (format == DP_NORM_MXFP8) return DP_NORM_FWD(uint16_t, kToMx8);
    return DP_NORM_FWD(uint16_t, kPlain);
#undef DP_NORM_FWD
  });
  return e == cudaSuccess ? DP_OK : DP_ERR_CUDA;
}

dp_status_t dp_rms_norm_backward_workspace_size(int M, int D, size_t* bytes) {
  if (!bytes) return DP_ERR_INVALID_ARG;
  *bytes = 0;
  if (M < 0 || D < 0) return DP_ERR_INVALID_ARG;
  if (M > kMaxRows || D > kMaxCols) return DP_ERR_UNSUPPORTED;
  *bytes = (size_t)groups_of(M, D) * D * sizeof(float);
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
  p.ldy = ldy, p.ldh = ldh, p.ldd = ldd, p.M = M, p.D = D, p.inv_d = 1.0f / (float)D;
  p.groups = groups_of(M, D);
  p.w_f32 = weight_dtype == DP_FP32;
  const bool vec = D % 16 == 0 && aligned(dy, 32) && ldy % 16 == 0 && aligned(h, 32) &&
                   ldh % 16 == 0 && (!dh || (aligned(dh, 32) && ldd % 16 == 0)) &&
                   aligned(dx, 32) && aligned(weight, 32);
  p.plan = plan_for(D, vec);
  p.err = dev.err_word;
  const int threads = p.plan.warps * p.plan.rows_cta * 32;
  const bool several = (M + p.plan.rows_cta - 1) / p.plan.rows_cta > p.groups;
  size_t smem = several ? plan_ring(&p.plan, D, esz, dh ? 3 : 2, 3, 96u << 10) : 0;
  cudaError_t e = by_length(D, [&](auto most, auto groups) {
    constexpr int N = decltype(most)::value, G = decltype(groups)::value;
    const auto go = [&](auto kernel, auto bulk_kernel) {
      if (smem && dph::prepare_kernel(reinterpret_cast<const void*>(bulk_kernel), N, 200 << 10,
                                      dev.device) < 1)
        return cudaErrorInvalidConfiguration;
      return launch(smem ? bulk_kernel : kernel, p, p.groups, threads, smem, s);
    };
    if (dtype == DP_FP32)
      return go(norm_bwd_kernel<float, N, G, false>, norm_bwd_kernel<float, N, G, true>);
    return go(norm_bwd_kernel<uint16_t, N, G, false>, norm_bwd_kernel<uint16_t, N, G, true>);
  });
  if (e == cudaSuccess) {
    const NormSumParams q{p.part, dweight, p.groups, D};
    e = launch(norm_sum_kernel, q, (D + 31) / 32, 1024, 0, s);
  }
  return e == cudaSuccess ? DP_OK : DP_ERR_CUDA;
}

}  // extern "C"
