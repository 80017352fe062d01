// score_math.cuh — score rules on the tensor-core kernels' accumulators: the
// cap's tanh, the distance bias and the tiles that documents leave.
//
// A capped score in units of log2, cap log2e tanh(s scale / cap), is odd in the
// raw product s: with u = s^2 it is s (c0 + c1 u + c2 u^2 + ...). The
// polynomials are minimax fits (relative error, computed by Remez exchange) of
// tanh(x) / x in x^2: kPoly3 on |x| <= 1/2 (5.4e-7), kPoly6 on |x| <= 1
// (5.0e-8); the host folds cap, log2 e and (scale / cap)^(2k+1) into the
// coefficients. Beyond |x| = 1 the exact form 1 - 2 / (1 + e^2x) is taken: two
// more results of the special-function unit a score, which is what the softmax
// is short of (16 a cycle and multiprocessor against 128 FMAs).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "cp_ptx.cuh"
#include "cp_score.h"

namespace cp {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

// Coefficients and limits of a launch's cap (host: make_cap_coef).
struct CapCoef {
  float p3[4], u3;  // for s^2 <= u3
  float p6[7], u6;  // for s^2 <= u6
  float a0, capl2;  // exact: capl2 (1 - 2 / (1 + 2^(s a0)))
};

inline CapCoef make_cap_coef(float scale, float cap) {
  static const double t3[4] = {0.9999994558, -0.3332631794, 0.131902966, -0.04440222613};
  static const double t6[7] = {0.9999999502,  -0.3333283915,  0.1332520408, -0.05345702957,
                               0.02028998042, -0.006203379104, 0.001041022634};
  CapCoef c{};
  if (!(cap > 0.f)) return c;
  const double l2e = 1.4426950408889634, r = static_cast<double>(scale) / cap;
  double pw = r;
  // a coefficient that fp32 cannot hold to full precision rules its polynomial out
  bool ok3 = true, ok6 = true;
  for (int k = 0; k < 7; ++k, pw *= r * r) {
    const double x = cap * l2e * pw;
    if (k < 4) {
      c.p3[k] = static_cast<float>(x * t3[k]);
      ok3 = ok3 && (pw == 0.0 || (x * t3[k] > 1e-30 || x * t3[k] < -1e-30)) && x < 1e30 && x > -1e30;
    }
    c.p6[k] = static_cast<float>(x * t6[k]);
    ok6 = ok6 && (pw == 0.0 || (x * t6[k] > 1e-30 || x * t6[k] < -1e-30)) && x < 1e30 && x > -1e30;
  }
  const double lim = r != 0.0 ? 1.0 / (r * r) : 3e38;
  c.u3 = ok3 ? static_cast<float>(lim * 0.25 < 3e38 ? lim * 0.25 : 3e38) : -1.f;
  c.u6 = ok6 ? static_cast<float>(lim < 3e38 ? lim : 3e38) : -1.f;
  c.a0 = static_cast<float>(2.0 * l2e * r);
  c.capl2 = static_cast<float>(cap * l2e);
  return c;
}

// The polynomials' factor of s, for a pair of scores with u = s^2.
template <int kDeg>
__device__ __forceinline__ void cap_poly(const CapCoef& c, float u0, float u1, float& f0, float& f1) {
  if constexpr (kDeg == 3) {
    f0 = f1 = c.p3[3];
#pragma unroll
    for (int k = 2; k >= 0; --k) fma2(f0, f1, f0, f1, u0, u1, c.p3[k], c.p3[k]);
  } else {
    f0 = f1 = c.p6[6];
#pragma unroll
    for (int k = 5; k >= 0; --k) fma2(f0, f1, f0, f1, u0, u1, c.p6[k], c.p6[k]);
  }
}

__device__ __forceinline__ float cap_exact(const CapCoef& c, float s) {
  return c.capl2 * (1.f - __fdividef(2.f, 1.f + ex2_approx(s * c.a0)));
}

// The row of document ranges of 64-row blocks, and the range of n consecutive
// blocks (those past the row's end left out).
__device__ __forceinline__ DocRange doc_span(const DocRange* row, int nblk, int blk, int n) {
  DocRange r = blk < nblk ? row[blk] : DocRange{INT_MAX, -1, 0, 0};
  for (int i = 1; i < n; ++i)
    if (blk + i < nblk) r = docs_join(r, row[blk + i]);
  return r;
}

// The tiles of a launch that meet a CTA's rows, as a bitmap in shared memory:
// bit t of act, and whether the tile holds a pair of different documents.
// Without documents every tile of [t0, t1) is taken.
struct TileWalk {
  const uint32_t* act;  // nullptr: all of [t0, t1)
  int t, t1;
  __device__ __forceinline__ TileWalk(const uint32_t* bits, int t0, int end) : act(bits), t(t0 - 1), t1(end) { next(); }
  __device__ __forceinline__ void next() {
    ++t;
    if (act == nullptr || t >= t1) return;
    uint32_t w = act[t >> 5] >> (t & 31);
    if (w) {
      t += __ffs(w) - 1;
      return;
    }
    int i = (t >> 5) + 1;
    const int ni = (t1 + 31) >> 5;
    while (i < ni && (w = act[i]) == 0) ++i;
    t = i < ni ? i * 32 + __ffs(w) - 1 : t1;
  }
};

}  // namespace cp
