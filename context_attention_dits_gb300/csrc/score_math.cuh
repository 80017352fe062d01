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
// is short of (16 a cycle and multiprocessor against 128 FMAs). The derivative
// 1 - tanh^2 is formed from the tanh only below |x| = 1: beyond, where it
// cancels (2e-3 of it lost at 6.5, all at 9), it is 4 e / (1 + e)^2 with
// e = e^-2|x|, by the same two results.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "cp_ptx.cuh"
#include "cp_score.h"

namespace cp {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

// Bounded wait that ignores the abort flag, for a CTA that gives up and lets its
// copies and products end.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
    if ((n & 255u) == 0 && global_timer_ns() - t0 > timeout_ns) return;
  }
}

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }

// Holds the uses of loaded registers behind the wait that precedes it.
template <int N>
__device__ __forceinline__ void tmem_pin(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                 "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// Pairs of fp32 values in a 64-bit register pair, for the packed instructions
// (one issue slot a pair). Coefficients are kept as pairs of equal values, so
// that they are operands as they stand and no register pair is built for them.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f32x2 pair_u(uint32_t lo, uint32_t hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void split(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma_x2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul_x2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add_x2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Coefficients and limits of a launch's cap (host: make_cap_coef).
struct CapCoef {
  f32x2 p3[4], p6[7];  // pairs of equal values
  float u3, u6;        // the polynomials serve s^2 <= u3, u6
  float a0, capl2;     // exact: capl2 (1 - 2 / (1 + 2^(s a0)))
};

// unit: the coefficients give tanh itself, without cap log2e.
inline CapCoef make_cap_coef(float scale, float cap, bool unit) {
  static const double t3[4] = {0.9999994558, -0.3332631794, 0.131902966, -0.04440222613};
  static const double t6[7] = {0.9999999502,  -0.3333283915,  0.1332520408, -0.05345702957,
                               0.02028998042, -0.006203379104, 0.001041022634};
  CapCoef c{};
  if (!(cap > 0.f)) return c;
  const double l2e = 1.4426950408889634, r = static_cast<double>(scale) / cap;
  auto twice = [](double x) {
    const float f = static_cast<float>(x);
    uint32_t u;
    std::memcpy(&u, &f, 4);
    return static_cast<f32x2>(u) << 32 | u;
  };
  // Coefficients below fp32's normal numbers (a wide cap) become 0, and their
  // polynomial then serves only the x for which they do not count; one above its
  // range (a narrow cap) rules its polynomial out. x3, x6: the largest x^2.
  double x3 = 0.25, x6 = 1.0, pw = r;
  for (int k = 0; k < 7; ++k, pw *= r * r) {
    const double x = (unit ? 1.0 : cap * l2e) * pw;
    auto put = [&](const double* t, int deg, f32x2* p, double* most) {
      if (k > deg) return;
      double v = x * t[k];
      const double av = v < 0 ? -v : v;
      if (av < 2e-38 && r != 0.0 && k > 0) {
        v = 0.0;
        const double only = std::pow(1e-7 / std::fabs(t[k]), 1.0 / k);
        if (only < *most) *most = only;
      }
      if (av > 1e38) *most = -1.0;
      p[k] = twice(v);
    };
    put(t3, 3, c.p3, &x3);
    put(t6, 6, c.p6, &x6);
  }
  auto limit = [&](double most) {
    if (most < 0) return -1.f;
    const double u = r != 0.0 ? most / (r * r) : 3e38;
    return static_cast<float>(u < 3e38 ? u : 3e38);
  };
  c.u3 = limit(x3);
  c.u6 = limit(x6);
  c.a0 = static_cast<float>(2.0 * l2e * r);
  c.capl2 = unit ? 1.f : static_cast<float>(cap * l2e);
  return c;
}

// The polynomials' factor of s, for a pair of scores with u = s^2.
template <int kDeg>
__device__ __forceinline__ f32x2 cap_poly(const CapCoef& c, f32x2 u) {
  const f32x2* p = kDeg == 3 ? c.p3 : c.p6;
  f32x2 f = fma_x2(p[kDeg], u, p[kDeg - 1]);
#pragma unroll
  for (int k = kDeg - 2; k >= 0; --k) f = fma_x2(f, u, p[k]);
  return f;
}

__device__ __forceinline__ float cap_exact(const CapCoef& c, float s) {
  return c.capl2 * (1.f - __fdividef(2.f, 1.f + ex2_approx(s * c.a0)));
}

// tanh and tanh^2 - 1 (coefficients with unit set). One score at a time: in pairs
// the constants' register pairs cost the polynomials' passes 1.5%.
__device__ __forceinline__ void tanh_exact(const CapCoef& c, float s, float& th, float& neg_d) {
  const float x2 = s * c.a0, e = ex2_approx(-fabsf(x2)), r = rcp_approx(1.f + e), er = e * r;
  th = copysignf(fmaf(-2.f, er, 1.f), x2);
  neg_d = -4.f * er * r;
}

// 0 .. 127 in pairs: the columns of a tile, for biases linear in the column.
__constant__ float kColumn[128] = {
    0.f, 1.f, 2.f, 3.f, 4.f, 5.f, 6.f, 7.f, 8.f, 9.f, 10.f, 11.f, 12.f, 13.f, 14.f, 15.f,
    16.f, 17.f, 18.f, 19.f, 20.f, 21.f, 22.f, 23.f, 24.f, 25.f, 26.f, 27.f, 28.f, 29.f, 30.f, 31.f,
    32.f, 33.f, 34.f, 35.f, 36.f, 37.f, 38.f, 39.f, 40.f, 41.f, 42.f, 43.f, 44.f, 45.f, 46.f, 47.f,
    48.f, 49.f, 50.f, 51.f, 52.f, 53.f, 54.f, 55.f, 56.f, 57.f, 58.f, 59.f, 60.f, 61.f, 62.f, 63.f,
    64.f, 65.f, 66.f, 67.f, 68.f, 69.f, 70.f, 71.f, 72.f, 73.f, 74.f, 75.f, 76.f, 77.f, 78.f, 79.f,
    80.f, 81.f, 82.f, 83.f, 84.f, 85.f, 86.f, 87.f, 88.f, 89.f, 90.f, 91.f, 92.f, 93.f, 94.f, 95.f,
    96.f, 97.f, 98.f, 99.f, 100.f, 101.f, 102.f, 103.f, 104.f, 105.f, 106.f, 107.f, 108.f, 109.f, 110.f, 111.f,
    112.f, 113.f, 114.f, 115.f, 116.f, 117.f, 118.f, 119.f, 120.f, 121.f, 122.f, 123.f, 124.f, 125.f, 126.f, 127.f};
__device__ __forceinline__ f32x2 columns(int c) { return *reinterpret_cast<const f32x2*>(kColumn + c); }

// The row of document ranges of 64-row blocks, and the range of n consecutive
// blocks (those past the row's end left out).
__device__ __forceinline__ DocRange doc_span(const DocRange* row, int nblk, int blk, int n) {
  DocRange r = blk < nblk ? row[blk] : DocRange{INT_MAX, -1, 0, 0};
  for (int i = 1; i < n; ++i)
    if (blk + i < nblk) r = docs_join(r, row[blk + i]);
  return r;
}

// Which of kWords x 32 document ids (lane c of word w holds id 32 w + c) are the
// lane's own: a bit each; none for a negative one. One pass for each document
// among the warp's own ids, which are rarely more than two.
template <int kWords>
__device__ __forceinline__ void same_docs(int own, const int (&ids)[kWords], uint32_t (&same)[kWords]) {
#pragma unroll
  for (int w = 0; w < kWords; ++w) same[w] = 0u;
  uint32_t todo = __ballot_sync(0xffffffffu, own >= 0);
  while (todo) {
    const int d = __shfl_sync(0xffffffffu, own, __ffs(todo) - 1);
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const uint32_t b = __ballot_sync(0xffffffffu, ids[w] == d);
      if (own == d) same[w] = b;
    }
    todo &= ~__ballot_sync(0xffffffffu, own == d);
  }
}

// The tiles of [lo, hi) that a CTA walks: all, or those whose bit is set in act
// (a bitmap in shared memory, a bit for a tile, or for 2^shift where kGroups).
// First from `start` down to lo, then from start + 1 up; start < lo
// walks upwards only.
template <bool kGroups = false>
struct TileWalk {
  const uint32_t* act;
  int t, lo, hi, start, shift;
  bool down;
  __device__ __forceinline__ TileWalk(const uint32_t* bits, int lo_, int hi_, int start_, int shift_ = 0)
      : act(bits), t(start_), lo(lo_), hi(hi_), start(start_ < lo_ ? lo_ - 1 : start_), shift(kGroups ? shift_ : 0),
        down(start_ >= lo_) {
    if (down) {
      find_down();
    } else {
      t = lo - 1;
      next();
    }
  }
  __device__ __forceinline__ bool done() const { return t >= hi; }
  // whether the tile's bit is set in another bitmap of the same kind
  __device__ __forceinline__ bool in(const uint32_t* map) const {
    const int g = t >> shift;
    return (map[g >> 5] >> (g & 31)) & 1u;
  }
  __device__ __forceinline__ void next() {
    if (down) {
      --t;
      find_down();
      return;
    }
    ++t;
    if (act == nullptr || t >= hi) return;
    const int g = t >> shift;
    uint32_t w = act[g >> 5] >> (g & 31);
    if (w & 1u) return;
    if (w) {
      t = (g + __ffs(w) - 1) << shift;
      return;
    }
    int i = (g >> 5) + 1;
    const int ni = (((hi - 1) >> shift) >> 5) + 1;
    while (i < ni && (w = act[i]) == 0) ++i;
    t = i < ni ? (i * 32 + __ffs(w) - 1) << shift : hi;
  }
  // the last set tile at or below t, else on to the upward part
  __device__ __forceinline__ void find_down() {
    if (act != nullptr && t >= lo) {
      const int g = t >> shift;
      uint32_t w = act[g >> 5] << (31 - (g & 31));
      if (w >> 31) return;
      auto last = [&](int group) { return kGroups ? ((group + 1) << shift) - 1 : group; };
      if (w) {
        t = last(g - __clz(w));
        return;
      }
      int i = (g >> 5) - 1;
      const int i0 = (lo >> shift) >> 5;
      while (i >= i0 && (w = act[i]) == 0) --i;
      if (i >= i0) {
        t = last(i * 32 + 31 - __clz(w));
        return;
      }
      t = lo - 1;
    }
    if (t < lo) {
      down = false;
      t = start;
      next();
    }
  }
};

}  // namespace cp
