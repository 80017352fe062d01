// score_attn_f32.cu — attention with a score rule on the CUDA cores, fp32
// throughout: forward and backward.
//
// With x_ij = scale q_i.k_j, capped to cap tanh(x / cap) if there is a cap,
// less slope_h |i - j| if there are slopes, -inf where a mask rules the pair
// out:
//   out_i = sum_j softmax_j(x_ij) v_j,  lse_i = ln sum_j exp(x_ij)
//   p_ij  = exp(x_ij - lse_i),  t_ij = p_ij (dout_i.v_j - delta_i),
//   ds_ij = t_ij (1 - tanh^2),  dq_i = scale sum_j ds_ij k_j,
//   dk_j  = scale sum_{h, i} ds_ij q_i,  dv_j = sum_{h, i} p_ij dout_i
// where h runs over the query heads that share the key/value head.
//
// Tiles: a CTA owns 32 rows (queries; keys for dk, dv) and walks 64-row tiles
// of the other side. 128 threads; a thread forms a 4 x 4 block of scores (rows
// 4 ti .. 4 ti + 3, columns tj + 16 c), then 4 rows x D/16 columns of the
// second product. Every tile is kept row-major with D + 4 floats a row: a
// float4 column of 16 neighbouring rows then takes two wavefronts (the least
// for 256 bytes), so one copy of K serves both Q K^T and dS K and nothing is
// transposed. A 4 x 4 block costs 8 16-byte loads per 64 FMAs.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "cp_score.h"

namespace cp {
namespace {

constexpr int kThr = 128;
constexpr int kR = 32;        // rows of the owned tile
constexpr int kC = 64;        // rows of a streamed tile
constexpr int kPT = kR + 4;   // row of the transposed probability tile
constexpr float kL2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

__device__ __forceinline__ void store4(void* base, int64_t i, float4 x) {
  *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = x;
}

// Rows row0 .. row0 + n - 1 (of `rows`; the others zero) of a [., S, heads, D]
// tensor's head into dst, D + 4 floats a row.
template <int D>
__device__ __forceinline__ void load_rows(float* dst, const float* src, int64_t stride, int n, int rows) {
  for (int e = threadIdx.x; e < rows * (D / 4); e += kThr) {
    const int r = e / (D / 4), d = (e % (D / 4)) * 4;
    const float4 x = r < n ? load4(src + r * stride + d) : make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4*>(dst + r * (D + 4) + d) = x;
  }
}

// s[i][c] = row (4 ti + i) of a . row (tj + 16 c) of b
template <int D>
__device__ __forceinline__ void dots(float (&s)[4][4], const float* a, const float* b, int ti, int tj) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[i][c] = 0.f;
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (4 * ti + i) * (D + 4) + d);
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = *reinterpret_cast<const float4*>(b + (tj + 16 * c) * (D + 4) + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        s[i][c] = fmaf(x[i].w, y[c].w, fmaf(x[i].z, y[c].z, fmaf(x[i].y, y[c].y, fmaf(x[i].x, y[c].x, s[i][c]))));
  }
}

// acc[i][.] += sum over the streamed tile's rows j of pt[j][4 ti + i] * b[j][columns of tj]
// (columns 4 tj + 64 u, u < D / 64)
template <int D>
__device__ __forceinline__ void second(float4 (&acc)[4][D / 64], const float* pt, const float* b, int ti, int tj) {
#pragma unroll 4
  for (int j = 0; j < kC; ++j) {
    const float4 p = *reinterpret_cast<const float4*>(pt + j * kPT + 4 * ti);
    const float w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
      const float4 y = *reinterpret_cast<const float4*>(b + j * (D + 4) + 4 * tj + 64 * u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i][u].x = fmaf(w[i], y.x, acc[i][u].x);
        acc[i][u].y = fmaf(w[i], y.y, acc[i][u].y);
        acc[i][u].z = fmaf(w[i], y.z, acc[i][u].z);
        acc[i][u].w = fmaf(w[i], y.w, acc[i][u].w);
      }
    }
  }
}

// The score of a pair in units of log2, before the mask, and the derivative of
// the cap. dist = |position of the query - position of the key|.
struct Scorer {
  float scale, cap, inv_cap, slope2;
  bool capped;
  __device__ Scorer(const ScoreArgs& a, int h)
      : scale(a.scale), cap(a.cap), inv_cap(a.cap > 0.f ? 1.f / a.cap : 0.f),
        slope2(a.slopes ? a.slopes[h] * kL2e : 0.f), capped(a.cap > 0.f) {}
  __device__ __forceinline__ float operator()(float dot, int dist, float& dcap) const {
    float x = dot * scale;
    dcap = 1.f;
    if (capped) {
      const float t = tanhf(x * inv_cap);
      x = cap * t;
      dcap = 1.f - t * t;
    }
    return fmaf(x, kL2e, -slope2 * static_cast<float>(abs(dist)));
  }
};

// Document ranges of the owned tile [row0, row0 + 32) (one 64-row block) and
// of a streamed 64-row tile starting at a multiple of 64.
__device__ __forceinline__ DocRange doc_range(const DocRange* r, int b, int S, int row) {
  return r[static_cast<int64_t>(b) * ((S + kDocBlock - 1) / kDocBlock) + row / kDocBlock];
}

template <int D>
constexpr int fwd_floats() {
  return (kR + 2 * kC) * (D + 4) + kC * kPT;
}

template <int D>
__global__ void __launch_bounds__(kThr) score_fwd_f32_kernel(const __grid_constant__ ScoreArgs a) {
  extern __shared__ __align__(16) float sm[];
  float* Q = sm;
  float* K = Q + kR * (D + 4);
  float* V = K + kC * (D + 4);
  float* Pt = V + kC * (D + 4);
  const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  const int h = blockIdx.y, b = blockIdx.z, hk = h / a.G;
  const int row0 = (gridDim.x - 1 - blockIdx.x) * kR;  // longest causal rows first
  const int nrows = min(kR, a.Sq - row0);
  const int64_t qs = static_cast<int64_t>(a.H) * D, ks = static_cast<int64_t>(a.Hkv) * D;
  const int64_t qo = (static_cast<int64_t>(b) * a.Sq + row0) * qs + static_cast<int64_t>(h) * D;
  const int64_t ko = static_cast<int64_t>(b) * a.Skv * ks + static_cast<int64_t>(hk) * D;
  load_rows<D>(Q, static_cast<const float*>(a.q) + qo, qs, nrows, kR);
  const Scorer score(a, h);
  const int plim = prefix_limit(a, b);
  int lim[4], qd[4];
  float m[4], l[4];
  float4 acc[4][D / 64];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ti + i;
    lim[i] = min(a.Skv, key_limit(a, plim, row0 + r));
    qd[i] = a.qdoc && r < nrows ? a.qdoc[static_cast<int64_t>(b) * a.Sq + row0 + r] : -1;
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int u = 0; u < D / 64; ++u) acc[i][u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int last = min(a.Skv, key_limit(a, plim, row0 + nrows - 1));
  DocRange qr{};
  if (a.qdoc) qr = doc_range(a.qrange, b, a.Sq, row0);
  for (int k0 = 0; k0 < last; k0 += kC) {
    if (a.qdoc && !docs_meet(qr, doc_range(a.krange, b, a.Skv, k0))) continue;
    const int nk = min(kC, a.Skv - k0);
    __syncthreads();  // the last tile's readers are done
    load_rows<D>(K, static_cast<const float*>(a.k) + ko + k0 * ks, ks, nk, kC);
    load_rows<D>(V, static_cast<const float*>(a.v) + ko + k0 * ks, ks, nk, kC);
    __syncthreads();
    float s[4][4];
    dots<D>(s, Q, K, ti, tj);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int j = k0 + tj + 16 * c;
      const int kd = a.qdoc && j < a.Skv ? a.kdoc[static_cast<int64_t>(b) * a.Skv + j] : -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float unused;
        const bool on = j < lim[i] && (!a.qdoc || (qd[i] == kd && kd >= 0));
        s[i][c] = on ? score(s[i][c], a.rel + row0 + 4 * ti + i - j, unused) : -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[i] - base);  // 0 while m is -inf
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[i][c] = exp2f(s[i][c] - base);
        sum += s[i][c];
      }
      l[i] = l[i] * f + sum;
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
        acc[i][u].x *= f;
        acc[i][u].y *= f;
        acc[i][u].z *= f;
        acc[i][u].w *= f;
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<float4*>(Pt + (tj + 16 * c) * kPT + 4 * ti) = make_float4(s[0][c], s[1][c], s[2][c], s[3][c]);
    __syncthreads();
    second<D>(acc, Pt, V, ti, tj);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
    const int r = 4 * ti + i;
    if (r >= nrows) continue;
    const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
#pragma unroll
    for (int u = 0; u < D / 64; ++u)
      store4(a.out, qo + r * qs + 4 * tj + 64 * u,
             make_float4(acc[i][u].x * inv, acc[i][u].y * inv, acc[i][u].z * inv, acc[i][u].w * inv));
    if (tj == 0)
      a.lse[(static_cast<int64_t>(b) * a.H + h) * a.Sq + row0 + r] =
          l[i] > 0.f ? (m[i] + log2f(l[i])) * kLn2 : -INFINITY;
  }
}

// delta[b, h, i] = out_i . dout_i, a warp per row of [B, Sq, H, D]
template <int D>
__global__ void __launch_bounds__(256) score_delta_kernel(const __grid_constant__ ScoreArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.B) * a.Sq * a.H) return;
  const int64_t h = row % a.H, bs = row / a.H, s = bs % a.Sq, b = bs / a.Sq;
  float sum = 0.f;
  if (lane * 4 < D) {
    const float4 g = load4(static_cast<const float*>(a.dout) + row * D + lane * 4);
    const float4 o = load4(static_cast<const float*>(a.o) + row * D + lane * 4);
    sum = fmaf(g.x, o.x, fmaf(g.y, o.y, fmaf(g.z, o.z, g.w * o.w)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) a.delta[(b * a.H + h) * a.Sq + s] = sum;
}

// lse in units of log2 for the recomputed probabilities; a row that saw no
// key, or lies past the end, gets +inf, so that p = 0.
__device__ __forceinline__ float lse2_of(const ScoreArgs& a, int64_t o, bool valid) {
  if (!valid) return INFINITY;
  const float x = a.lse[o];
  return x == -INFINITY ? INFINITY : x * kL2e;
}

template <int D>
constexpr int bwd_floats() {
  return (2 * kR + 2 * kC) * (D + 4) + kC * kPT + 2 * kC;
}

template <int D>
__global__ void __launch_bounds__(kThr) score_dq_f32_kernel(const __grid_constant__ ScoreArgs a) {
  extern __shared__ __align__(16) float sm[];
  float* Q = sm;
  float* dO = Q + kR * (D + 4);
  float* K = dO + kR * (D + 4);
  float* V = K + kC * (D + 4);
  float* Pt = V + kC * (D + 4);
  const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  const int h = blockIdx.y, b = blockIdx.z, hk = h / a.G;
  const int row0 = (gridDim.x - 1 - blockIdx.x) * kR;
  const int nrows = min(kR, a.Sq - row0);
  const int64_t qs = static_cast<int64_t>(a.H) * D, ks = static_cast<int64_t>(a.Hkv) * D;
  const int64_t qo = (static_cast<int64_t>(b) * a.Sq + row0) * qs + static_cast<int64_t>(h) * D;
  const int64_t ko = static_cast<int64_t>(b) * a.Skv * ks + static_cast<int64_t>(hk) * D;
  load_rows<D>(Q, static_cast<const float*>(a.q) + qo, qs, nrows, kR);
  load_rows<D>(dO, static_cast<const float*>(a.dout) + qo, qs, nrows, kR);
  const Scorer score(a, h);
  const int plim = prefix_limit(a, b);
  int lim[4], qd[4];
  float lse2[4], dlt[4];
  float4 acc[4][D / 64];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ti + i;
    const int64_t o = (static_cast<int64_t>(b) * a.H + h) * a.Sq + row0 + r;
    lim[i] = min(a.Skv, key_limit(a, plim, row0 + r));
    qd[i] = a.qdoc && r < nrows ? a.qdoc[static_cast<int64_t>(b) * a.Sq + row0 + r] : -1;
    lse2[i] = lse2_of(a, o, r < nrows);
    dlt[i] = r < nrows ? a.delta[o] : 0.f;
#pragma unroll
    for (int u = 0; u < D / 64; ++u) acc[i][u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int last = min(a.Skv, key_limit(a, plim, row0 + nrows - 1));
  DocRange qr{};
  if (a.qdoc) qr = doc_range(a.qrange, b, a.Sq, row0);
  for (int k0 = 0; k0 < last; k0 += kC) {
    if (a.qdoc && !docs_meet(qr, doc_range(a.krange, b, a.Skv, k0))) continue;
    const int nk = min(kC, a.Skv - k0);
    __syncthreads();
    load_rows<D>(K, static_cast<const float*>(a.k) + ko + k0 * ks, ks, nk, kC);
    load_rows<D>(V, static_cast<const float*>(a.v) + ko + k0 * ks, ks, nk, kC);
    __syncthreads();
    float s[4][4], dp[4][4];
    dots<D>(s, Q, K, ti, tj);
    dots<D>(dp, dO, V, ti, tj);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int j = k0 + tj + 16 * c;
      const int kd = a.qdoc && j < a.Skv ? a.kdoc[static_cast<int64_t>(b) * a.Skv + j] : -1;
      float ds[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float dcap;
        const bool on = j < lim[i] && (!a.qdoc || (qd[i] == kd && kd >= 0));
        const float p = exp2f(score(s[i][c], a.rel + row0 + 4 * ti + i - j, dcap) - lse2[i]);
        ds[i] = on ? p * (dp[i][c] - dlt[i]) * dcap : 0.f;
      }
      *reinterpret_cast<float4*>(Pt + (tj + 16 * c) * kPT + 4 * ti) = make_float4(ds[0], ds[1], ds[2], ds[3]);
    }
    __syncthreads();
    second<D>(acc, Pt, K, ti, tj);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ti + i;
    if (r >= nrows) continue;
#pragma unroll
    for (int u = 0; u < D / 64; ++u)
      store4(a.dq, qo + r * qs + 4 * tj + 64 * u,
             make_float4(acc[i][u].x * a.scale, acc[i][u].y * a.scale, acc[i][u].z * a.scale, acc[i][u].w * a.scale));
  }
}

// dk, dv of 32 keys: the streamed tiles are 64 query rows of each head that
// shares the key/value head, head by head. Scores are formed transposed (rows
// are keys), and P^T and then dS^T pass through one buffer.
template <int D>
__global__ void __launch_bounds__(kThr) score_dkdv_f32_kernel(const __grid_constant__ ScoreArgs a) {
  extern __shared__ __align__(16) float sm[];
  float* K = sm;
  float* V = K + kR * (D + 4);
  float* Q = V + kR * (D + 4);
  float* dO = Q + kC * (D + 4);
  float* Pt = dO + kC * (D + 4);
  float* lse2 = Pt + kC * kPT;
  float* dlt = lse2 + kC;
  const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int key0 = blockIdx.x * kR;  // the first keys meet the most causal rows
  const int nk = min(kR, a.Skv - key0);
  const int64_t qs = static_cast<int64_t>(a.H) * D, ks = static_cast<int64_t>(a.Hkv) * D;
  const int64_t ko = (static_cast<int64_t>(b) * a.Skv + key0) * ks + static_cast<int64_t>(hk) * D;
  load_rows<D>(K, static_cast<const float*>(a.k) + ko, ks, nk, kR);
  load_rows<D>(V, static_cast<const float*>(a.v) + ko, ks, nk, kR);
  const int plim = prefix_limit(a, b);
  int kd[4];
  float4 dk[4][D / 64], dv[4][D / 64];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ti + i;
    kd[i] = a.qdoc && r < nk ? a.kdoc[static_cast<int64_t>(b) * a.Skv + key0 + r] : -1;
#pragma unroll
    for (int u = 0; u < D / 64; ++u) dk[i][u] = dv[i][u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // the first query row that reaches any key of the tile, down to a tile start
  int first = 0;
  if (a.causal && key0 >= plim) first = max(0, key0 - a.rel) / kC * kC;
  DocRange kr{};
  if (a.qdoc) kr = doc_range(a.krange, b, a.Skv, key0);
  for (int h = hk * a.G; h < (hk + 1) * a.G; ++h) {
    const Scorer score(a, h);
    for (int q0 = first; q0 < a.Sq; q0 += kC) {
      if (a.qdoc && !docs_meet(doc_range(a.qrange, b, a.Sq, q0), kr)) continue;
      const int nq = min(kC, a.Sq - q0);
      const int64_t qo = (static_cast<int64_t>(b) * a.Sq + q0) * qs + static_cast<int64_t>(h) * D;
      const int64_t lo = (static_cast<int64_t>(b) * a.H + h) * a.Sq + q0;
      __syncthreads();
      load_rows<D>(Q, static_cast<const float*>(a.q) + qo, qs, nq, kC);
      load_rows<D>(dO, static_cast<const float*>(a.dout) + qo, qs, nq, kC);
      if (threadIdx.x < kC) {
        const int r = threadIdx.x;
        lse2[r] = lse2_of(a, lo + r, r < nq);
        dlt[r] = r < nq ? a.delta[lo + r] : 0.f;
      }
      __syncthreads();
      float s[4][4], dp[4][4];
      dots<D>(s, K, Q, ti, tj);
      dots<D>(dp, V, dO, ti, tj);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int r = tj + 16 * c, i = q0 + r;
        const int lim = key_limit(a, plim, i);
        const int qd = a.qdoc && r < nq ? a.qdoc[static_cast<int64_t>(b) * a.Sq + i] : -1;
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = key0 + 4 * ti + e;
          float dcap;
          const bool on = r < nq && j < lim && (!a.qdoc || (qd == kd[e] && qd >= 0));
          const float x = exp2f(score(s[e][c], a.rel + i - j, dcap) - lse2[r]);
          p[e] = on ? x : 0.f;
          dp[e][c] = on ? x * (dp[e][c] - dlt[r]) * dcap : 0.f;
        }
        *reinterpret_cast<float4*>(Pt + r * kPT + 4 * ti) = make_float4(p[0], p[1], p[2], p[3]);
      }
      __syncthreads();
      second<D>(dv, Pt, dO, ti, tj);
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<float4*>(Pt + (tj + 16 * c) * kPT + 4 * ti) =
            make_float4(dp[0][c], dp[1][c], dp[2][c], dp[3][c]);
      __syncthreads();
      second<D>(dk, Pt, Q, ti, tj);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ti + i;
    if (r >= nk) continue;
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
      store4(a.dk, ko + r * ks + 4 * tj + 64 * u,
             make_float4(dk[i][u].x * a.scale, dk[i][u].y * a.scale, dk[i][u].z * a.scale, dk[i][u].w * a.scale));
      store4(a.dv, ko + r * ks + 4 * tj + 64 * u, dv[i][u]);
    }
  }
}

// A warp per 64-row block of the document ids of q (the first nq blocks of a
// batch entry) and k.
__global__ void __launch_bounds__(256) doc_ranges_kernel(const __grid_constant__ ScoreArgs a, int nq, int nk) {
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(a.B) * (nq + nk)) return;
  const int64_t b = w / (nq + nk);
  const int t = static_cast<int>(w % (nq + nk));
  const bool isq = t < nq;
  const int blk = isq ? t : t - nq, S = isq ? a.Sq : a.Skv;
  const int* ids = (isq ? a.qdoc : a.kdoc) + b * S;
  int lo = INT_MAX, hi = -1, neg = 0;
#pragma unroll
  for (int u = 0; u < kDocBlock / 32; ++u) {
    const int i = blk * kDocBlock + u * 32 + lane;
    if (i < S) {
      const int id = ids[i];
      if (id >= 0) {
        lo = min(lo, id);
        hi = max(hi, id);
      } else {
        neg = 1;
      }
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  neg = __reduce_or_sync(0xffffffffu, neg);
  if (lane == 0) {
    DocRange* dst = const_cast<DocRange*>(isq ? a.qrange : a.krange) + b * (isq ? nq : nk) + blk;
    *dst = DocRange{lo, hi, neg, 0};
  }
}

template <int D>
cudaError_t fwd_d(const ScoreArgs& a, cudaStream_t s) {
  constexpr int bytes = fwd_floats<D>() * 4;
  cudaError_t e = allow_smem<score_fwd_f32_kernel<D>>(bytes);
  if (e != cudaSuccess) return e;
  score_fwd_f32_kernel<D><<<dim3((a.Sq + kR - 1) / kR, a.H, a.B), kThr, bytes, s>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t bwd_d(const ScoreArgs& a, cudaStream_t s) {
  constexpr int bytes = bwd_floats<D>() * 4;
  cudaError_t e = allow_smem<score_dq_f32_kernel<D>>(bytes);
  if (e == cudaSuccess) e = allow_smem<score_dkdv_f32_kernel<D>>(bytes);
  if (e != cudaSuccess) return e;
  if (a.Sq > 0) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.Sq * a.H;
    score_delta_kernel<D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    score_dq_f32_kernel<D><<<dim3((a.Sq + kR - 1) / kR, a.H, a.B), kThr, bytes, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (a.Skv > 0) {
    score_dkdv_f32_kernel<D><<<dim3((a.Skv + kR - 1) / kR, a.Hkv, a.B), kThr, bytes, s>>>(a);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace

cudaError_t launch_doc_ranges(const ScoreArgs& a, cudaStream_t s) {
  const int nq = (a.Sq + kDocBlock - 1) / kDocBlock, nk = (a.Skv + kDocBlock - 1) / kDocBlock;
  const int64_t warps = static_cast<int64_t>(a.B) * (nq + nk);
  if (warps == 0) return cudaSuccess;
  doc_ranges_kernel<<<static_cast<unsigned>((warps + 7) / 8), 256, 0, s>>>(a, nq, nk);
  return cudaGetLastError();
}

cudaError_t launch_score_fwd_f32(const ScoreArgs& a, int D, cudaStream_t s) {
  return D == 64 ? fwd_d<64>(a, s) : fwd_d<128>(a, s);
}

cudaError_t launch_score_bwd_f32(const ScoreArgs& a, int D, cudaStream_t s) {
  return D == 64 ? bwd_d<64>(a, s) : bwd_d<128>(a, s);
}

}  // namespace cp
