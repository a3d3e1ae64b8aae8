// dp_w4_plan.h -- how a product of a few tokens with 4-bit weights (dp_w4.cu) is laid
// over CTAs and warps.  Plain host C++.  It follows from the call's sizes alone, and
// with it the order in which products are summed: the SM count that it is made for is
// a constant, so a part of the GPU, or another GPU, gives the same bits.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace w4 {

constexpr int kStep = 128;       // values of d a warp takes at once: 32 a lane
constexpr int kRows = 32;        // weight rows of a unit, a warp's
constexpr int kMaxWarps = 16;    // of a CTA
constexpr int kSms = 152;        // that the work is spread over
constexpr size_t kMaxSmem = 220 << 10;

// A warp's ring of codes and scales: steps of it, and their bytes, for nt groups of
// eight tokens.
constexpr int ring_steps(int nt) { return nt == 4 ? 2 : 3; }
constexpr uint32_t step_bytes(bool mx) { return kRows * (kStep / 2) + (mx ? 128 : 256); }
// x of one token and share of d for `slab` steps (padded: neighbouring tokens fall into
// other banks).
#ifdef __CUDACC__
__host__ __device__
#endif
constexpr uint32_t x_row_bytes(int slab) { return (uint32_t)slab * kStep * 2 + 64; }

struct Plan {
  int split;      // warps that share a unit's d: a power of two, 2^split_bits
  int split_bits;
  int per;        // units of a CTA
  int warps;      // of a CTA: per x split
  int slab;       // steps of d whose x is in shared memory at once, for each share
  int slabs;      // slabs of a share
  size_t smem;
};

// tokens: of a CTA.  ready: x was made f16 beforehand.
// Many units: one CTA an SM (or as many rounds of them as it takes), each warp its own
// unit, x shared by all.  Few: d is split over warps, up to 16 an SM, while each share
// has a step and x fits.
inline Plan plan(int tokens, int D, int units, bool mx, int nt, bool ready) {
  Plan p{};
  const int steps = (int)(((long long)D + kStep - 1) / kStep);
  const long long full = (long long)kMaxWarps * kSms;
  for (p.split = kMaxWarps; p.split >= 1; p.split /= 2) {
    const long long all = (long long)units * p.split;
    if (p.split > 1 && (p.split > steps || all > full)) continue;
    const long long ctas = (all + full - 1) / full * kSms;
    p.per = (int)((units + ctas - 1) / ctas);
    p.per = std::max(1, std::min(p.per, kMaxWarps / p.split));
    p.warps = p.per * p.split;
    const int share = (steps + p.split - 1) / p.split;
    // Slabs as long as fit; where the kernel makes f16 of x itself, 64 steps of all
    // tokens at most (longer ones are staged too long before the first step).
    const size_t ring = (size_t)p.warps * ring_steps(nt) * step_bytes(mx);
    const auto fits = [&](int slabs, int slab) {
      p.smem = ring + (size_t)(slabs > 1 ? 2 : 1) * p.split * tokens * x_row_bytes(slab);
      return p.smem <= kMaxSmem && (ready || slabs == share || slab <= std::max(16, 64 / tokens));
    };
    for (p.slabs = 1;; ++p.slabs) {
      p.slab = (share + p.slabs - 1) / p.slabs;
      if (fits(p.slabs, p.slab) || p.slab <= 2) break;
    }
    p.slabs = (share + p.slab - 1) / p.slab;
    if (p.smem <= kMaxSmem) break;
  }
  while ((1 << p.split_bits) < p.split) ++p.split_bits;
  return p;
}

}  // namespace w4
