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
// of the other side. 128 threads form a group; a thread forms a 4 x 4 block of
// scores (rows 4 ti .. 4 ti + 3, columns tj + 16 c), then 4 rows x D/16 columns
// of the second product. Every tile is kept row-major with D + 4 floats a row: a
// float4 column of 16 neighbouring rows then takes two wavefronts (the least
// for 256 bytes), so one copy of K serves both Q K^T and dS K and nothing is
// transposed. A 4 x 4 block costs 8 16-byte loads per 64 FMAs.
// What bounds these kernels at the sizes fp32 is used for (a few hundred rows:
// less than a CTA per multiprocessor) is the latency of a tile's chain of
// copies, loads and barriers, so a CTA holds kGroups groups (as many as shared
// memory holds tiles for: 4 at D = 64, 2 at D = 128) that take the tiles in
// turn, each with its own buffers, barrier and running state, joined once at
// the end; and a buffer's next tile is copied (16-byte asynchronous copies) as
// soon as its last reader is through. Where that still leaves multiprocessors
// idle, a cluster of 2, 4 or 8 CTAs shares the tiles of one item in the same way
// and joins through distributed shared memory (see cluster_for).
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "cp_ptx.cuh"
#include "cp_score.h"

namespace cp {
namespace {

constexpr int kGrp = 128;     // threads of a group
constexpr int kR = 32;        // rows of the owned tile
constexpr int kC = 64;        // rows of a streamed tile
constexpr int kPT = kR + 4;   // row of the transposed probability tile
constexpr float kL2e = 1.4426950408889634f;
constexpr float kLn2f = 0.69314718055994531f;

template <int D>
struct Cfg {
  static constexpr int kGroups = 256 / D;
  static constexpr int kThreads = kGroups * kGrp;
  static constexpr int kRow = D + 4;                           // floats of a row
  static constexpr int kOwn = kR * kRow, kTile = kC * kRow;    // floats of a tile
  static constexpr int kP = kC * kPT;
  static constexpr int kFwd = kOwn + kGroups * (2 * kTile + kP);
  static constexpr int kBwd = 2 * kOwn + kGroups * (2 * kTile + kP + 2 * kC);
  static_assert(2 * kOwn + 2 * kR <= 2 * kTile + kP, "a group's buffers hold its results at the end");
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(void* base, int64_t i, float4 x) {
  *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = x;
}
__device__ __forceinline__ float4 scaled(float4 x, float f) { return make_float4(x.x * f, x.y * f, x.z * f, x.w * f); }
__device__ __forceinline__ void add4(float4& x, float4 y) {
  x.x += y.x;
  x.y += y.y;
  x.z += y.z;
  x.w += y.w;
}

// Barrier of the caller's group.
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(kGrp) : "memory"); }

__device__ __forceinline__ void copy16(float* dst, const float* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// `rows` rows of a [., S, heads, D] tensor's head (the first n exist, the
// others become zero) into dst, by threads t of nt.
template <int D>
__device__ __forceinline__ void copy_rows(float* dst, const float* src, int64_t stride, int n, int rows, int t, int nt) {
  for (int e = t; e < rows * (D / 4); e += nt) {
    const int r = e / (D / 4), d = (e % (D / 4)) * 4;
    copy16(dst + r * (D + 4) + d, src + (r < n ? r * stride + d : 0), r < n);
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
    for (int i = 0; i < 4; ++i) x[i] = load4(a + (4 * ti + i) * (D + 4) + d);
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = load4(b + (tj + 16 * c) * (D + 4) + d);
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
    const float4 p = load4(pt + j * kPT + 4 * ti);
    const float w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
      const float4 y = load4(b + j * (D + 4) + 4 * tj + 64 * u);
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

template <int D>
__device__ __forceinline__ void clear(float4 (&acc)[4][D / 64]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < D / 64; ++u) acc[i][u] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// acc as a [kR][D] tile (rows of D + 4) in shared memory
template <int D>
__device__ __forceinline__ void put(const float4 (&acc)[4][D / 64], float* dst, int ti, int tj) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < D / 64; ++u)
      *reinterpret_cast<float4*>(dst + (4 * ti + i) * (D + 4) + 4 * tj + 64 * u) = acc[i][u];
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

// The document range of the 64-row block that holds row `row`.
__device__ __forceinline__ DocRange doc_range(const DocRange* r, int b, int S, int row) {
  return r[static_cast<int64_t>(b) * ((S + kDocBlock - 1) / kDocBlock) + row / kDocBlock];
}

// The tiles (64 rows, from tile t0 to t1) of a walk that meet the owned rows'
// documents; a group takes every kGroups-th of them.
struct Walk {
  const DocRange* r;  // of the batch entry; nullptr: no documents
  DocRange own;
  int t, t1;
  __device__ __forceinline__ void skip() {
    while (t < t1 && r != nullptr && !docs_meet(r[t], own)) ++t;
  }
  __device__ __forceinline__ void step(int n) {
    for (int i = 0; i < n && t < t1; ++i) {
      ++t;
      skip();
    }
  }
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1) score_fwd_f32_kernel(const __grid_constant__ ScoreArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(16) float sm[];
  const int g = threadIdx.x / kGrp, tid = threadIdx.x % kGrp;
  float* Q = sm;
  float* K = sm + C::kOwn + g * (2 * C::kTile + C::kP);
  float* V = K + C::kTile;
  float* Pt = V + C::kTile;
  const int ti = tid / 16, tj = tid % 16;
  const int cs = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int item = blockIdx.x / cs, nrt = (a.Sq + kR - 1) / kR;
  const int h = item % a.H, b = item / a.H % a.B, hk = h / a.G;
  const int row0 = (nrt - 1 - item / (a.H * a.B)) * kR;  // longest causal rows first
  const int nrows = min(kR, a.Sq - row0);
  const int64_t qs = static_cast<int64_t>(a.H) * D, ks = static_cast<int64_t>(a.Hkv) * D;
  const int64_t qo = (static_cast<int64_t>(b) * a.Sq + row0) * qs + static_cast<int64_t>(h) * D;
  const int64_t ko = static_cast<int64_t>(b) * a.Skv * ks + static_cast<int64_t>(hk) * D;
  const int plim = prefix_limit(a, b);
  const int last = min(a.Skv, key_limit(a, plim, row0 + nrows - 1));
  Walk cur{};
  cur.t1 = (max(last, 0) + kC - 1) / kC;
  if (a.qdoc) {
    cur.r = a.krange + static_cast<int64_t>(b) * ((a.Skv + kDocBlock - 1) / kDocBlock);
    cur.own = doc_range(a.qrange, b, a.Sq, row0);
  }
  cur.skip();
  cur.step(rank * C::kGroups + g);
  auto copy = [&](float* dst, const void* src, int t) {
    if (t < cur.t1)
      copy_rows<D>(dst, static_cast<const float*>(src) + ko + t * kC * ks, ks, min(kC, a.Skv - t * kC), kC, tid, kGrp);
    copy_commit();
  };
  copy_rows<D>(Q, static_cast<const float*>(a.q) + qo, qs, nrows, kR, threadIdx.x, C::kThreads);
  copy(K, a.k, cur.t);  // with Q
  copy(V, a.v, cur.t);
  const Scorer score(a, h);
  int lim[4], qd[4];
  float m[4], l[4];
  float4 acc[4][D / 64];
  clear<D>(acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ti + i;
    lim[i] = min(a.Skv, key_limit(a, plim, row0 + r));
    qd[i] = a.qdoc && r < nrows ? a.qdoc[static_cast<int64_t>(b) * a.Sq + row0 + r] : -1;
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  copy_wait<1>();
  __syncthreads();  // Q is every thread's
  while (cur.t < cur.t1) {
    const int k0 = cur.t * kC;
    cur.step(cs * C::kGroups);
    copy_wait<1>();  // K
    group_sync(g);
    float s[4][4];
    dots<D>(s, Q, K, ti, tj);
    group_sync(g);
    copy(K, a.k, cur.t);
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
      for (int u = 0; u < D / 64; ++u) acc[i][u] = scaled(acc[i][u], f);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<float4*>(Pt + (tj + 16 * c) * kPT + 4 * ti) = make_float4(s[0][c], s[1][c], s[2][c], s[3][c]);
    copy_wait<1>();  // V
    group_sync(g);
    second<D>(acc, Pt, V, ti, tj);
    group_sync(g);
    copy(V, a.v, cur.t);
  }
  copy_wait<0>();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
  // ---- the states of every CTA's groups joined: a CTA stores the rows of its share ----
  group_sync(g);
  put<D>(acc, K, ti, tj);
  if (tj == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(K + C::kOwn + 2 * (4 * ti + i)) = make_float2(m[i], l[i]);
  cluster_sync();
  const uint32_t st0 = smem_addr(sm + C::kOwn);
  constexpr int kStep = (2 * C::kTile + C::kP) * 4;  // bytes from a group's buffers to the next's
  const int share = kR / cs;
  for (int e = threadIdx.x; e < share * (D / 4); e += C::kThreads) {
    const int r = rank * share + e / (D / 4), d = (e % (D / 4)) * 4;
    if (r >= nrows) break;
    float mx = -INFINITY;
    for (int x = 0; x < cs; ++x)
#pragma unroll
      for (int y = 0; y < C::kGroups; ++y)
        mx = fmaxf(mx, ld_peer2(cluster_peer(st0 + y * kStep + (C::kOwn + 2 * r) * 4, x)).x);
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 0; x < cs; ++x)
#pragma unroll
      for (int y = 0; y < C::kGroups; ++y) {
        const uint32_t st = cluster_peer(st0 + y * kStep, x);
        const float2 ml = ld_peer2(st + (C::kOwn + 2 * r) * 4);
        const float f = exp2f(ml.x - base);
        sum = fmaf(ml.y, f, sum);
        add4(o, scaled(ld_peer4(st + (r * (D + 4) + d) * 4), f));
      }
    store4(a.out, qo + r * qs + d, scaled(o, sum != 0.f ? 1.f / sum : 0.f));
    if (d == 0)
      a.lse[(static_cast<int64_t>(b) * a.H + h) * a.Sq + row0 + r] = sum != 0.f ? (mx + log2f(sum)) * kLn2f : -INFINITY;
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
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
    const float4 x = load4(static_cast<const float*>(a.dout) + row * D + lane * 4);
    const float4 o = load4(static_cast<const float*>(a.o) + row * D + lane * 4);
    sum = fmaf(x.x, o.x, fmaf(x.y, o.y, fmaf(x.z, o.z, x.w * o.w)));
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

// dq of 32 query rows: key tiles stream by.
template <int D>
__device__ __forceinline__ void dq_cta(const ScoreArgs& a, float* sm, int cs, int rank, int bx, int h, int b) {
  using C = Cfg<D>;
  constexpr int kStep = 2 * C::kTile + C::kP + 2 * kC;
  const int g = threadIdx.x / kGrp, tid = threadIdx.x % kGrp;
  float* Q = sm;
  float* dO = Q + C::kOwn;
  float* K = dO + C::kOwn + g * kStep;
  float* V = K + C::kTile;
  float* Pt = V + C::kTile;
  const int ti = tid / 16, tj = tid % 16, hk = h / a.G;
  const int row0 = bx * kR;
  const int nrows = min(kR, a.Sq - row0);
  const int64_t qs = static_cast<int64_t>(a.H) * D, ks = static_cast<int64_t>(a.Hkv) * D;
  const int64_t qo = (static_cast<int64_t>(b) * a.Sq + row0) * qs + static_cast<int64_t>(h) * D;
  const int64_t ko = static_cast<int64_t>(b) * a.Skv * ks + static_cast<int64_t>(hk) * D;
  const int plim = prefix_limit(a, b);
  const int last = min(a.Skv, key_limit(a, plim, row0 + nrows - 1));
  Walk cur{};
  cur.t1 = (max(last, 0) + kC - 1) / kC;
  if (a.qdoc) {
    cur.r = a.krange + static_cast<int64_t>(b) * ((a.Skv + kDocBlock - 1) / kDocBlock);
    cur.own = doc_range(a.qrange, b, a.Sq, row0);
  }
  cur.skip();
  cur.step(rank * C::kGroups + g);
  auto copy = [&](float* dst, const void* src, int t) {
    if (t < cur.t1)
      copy_rows<D>(dst, static_cast<const float*>(src) + ko + t * kC * ks, ks, min(kC, a.Skv - t * kC), kC, tid, kGrp);
    copy_commit();
  };
  copy_rows<D>(Q, static_cast<const float*>(a.q) + qo, qs, nrows, kR, threadIdx.x, C::kThreads);
  copy_rows<D>(dO, static_cast<const float*>(a.dout) + qo, qs, nrows, kR, threadIdx.x, C::kThreads);
  copy(V, a.v, cur.t);
  copy(K, a.k, cur.t);
  const Scorer score(a, h);
  int lim[4], qd[4];
  float lse2[4], dlt[4];
  float4 acc[4][D / 64];
  clear<D>(acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ti + i;
    const int64_t o = (static_cast<int64_t>(b) * a.H + h) * a.Sq + row0 + r;
    lim[i] = min(a.Skv, key_limit(a, plim, row0 + r));
    qd[i] = a.qdoc && r < nrows ? a.qdoc[static_cast<int64_t>(b) * a.Sq + row0 + r] : -1;
    lse2[i] = lse2_of(a, o, r < nrows);
    dlt[i] = r < nrows ? a.delta[o] : 0.f;
  }
  copy_wait<0>();
  __syncthreads();
  while (cur.t < cur.t1) {
    const int k0 = cur.t * kC;
    cur.step(cs * C::kGroups);
    copy_wait<0>();
    group_sync(g);
    float s[4][4], dp[4][4];
    dots<D>(dp, dO, V, ti, tj);
    dots<D>(s, Q, K, ti, tj);
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
    group_sync(g);
    copy(V, a.v, cur.t);
    second<D>(acc, Pt, K, ti, tj);
    group_sync(g);
    copy(K, a.k, cur.t);
  }
  copy_wait<0>();
  group_sync(g);
  put<D>(acc, K, ti, tj);
  cluster_sync();
  const uint32_t st0 = smem_addr(sm + 2 * C::kOwn);
  const int share = kR / cs;
  for (int e = threadIdx.x; e < share * (D / 4); e += C::kThreads) {
    const int r = rank * share + e / (D / 4), d = (e % (D / 4)) * 4;
    if (r >= nrows) break;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < cs; ++c)
#pragma unroll
      for (int y = 0; y < C::kGroups; ++y) add4(x, ld_peer4(cluster_peer(st0 + (y * kStep + r * (D + 4) + d) * 4, c)));
    store4(a.dq, qo + r * qs + d, scaled(x, a.scale));
  }
}

// dk, dv of 32 keys: the streamed tiles are 64 query rows of each head that
// shares the key/value head, head by head. Scores are formed transposed (rows
// are keys), and P^T and then dS^T pass through one buffer.
template <int D>
__device__ __forceinline__ void dkdv_cta(const ScoreArgs& a, float* sm, int cs, int rank, int bx, int hk, int b) {
  using C = Cfg<D>;
  constexpr int kStep = 2 * C::kTile + C::kP + 2 * kC;
  const int g = threadIdx.x / kGrp, tid = threadIdx.x % kGrp;
  float* K = sm;
  float* V = K + C::kOwn;
  float* Q = V + C::kOwn + g * kStep;
  float* dO = Q + C::kTile;
  float* Pt = dO + C::kTile;
  float* lse2 = Pt + C::kP;
  float* dlt = lse2 + kC;
  const int ti = tid / 16, tj = tid % 16;
  const int key0 = bx * kR;
  const int nk = min(kR, a.Skv - key0);
  const int64_t qs = static_cast<int64_t>(a.H) * D, ks = static_cast<int64_t>(a.Hkv) * D;
  const int64_t ko = (static_cast<int64_t>(b) * a.Skv + key0) * ks + static_cast<int64_t>(hk) * D;
  copy_rows<D>(K, static_cast<const float*>(a.k) + ko, ks, nk, kR, threadIdx.x, C::kThreads);
  copy_rows<D>(V, static_cast<const float*>(a.v) + ko, ks, nk, kR, threadIdx.x, C::kThreads);
  copy_commit();
  const int plim = prefix_limit(a, b);
  int kd[4];
  float4 dk[4][D / 64], dv[4][D / 64];
  clear<D>(dk);
  clear<D>(dv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ti + i;
    kd[i] = a.qdoc && r < nk ? a.kdoc[static_cast<int64_t>(b) * a.Skv + key0 + r] : -1;
  }
  // query tiles from the first row that reaches a key of the tile
  const int ntq = (a.Sq + kC - 1) / kC;
  const int t0 = a.causal && key0 >= plim ? min(ntq, max(0, key0 - a.rel) / kC) : 0;
  Walk first{};
  first.t = t0;
  first.t1 = ntq;
  if (a.qdoc) {
    first.r = a.qrange + static_cast<int64_t>(b) * ((a.Sq + kDocBlock - 1) / kDocBlock);
    first.own = doc_range(a.krange, b, a.Skv, key0);
  }
  first.skip();
  // (tile, head) pairs in turn: the next one is `n` further
  Walk cur = first;
  int h = hk * a.G;
  const int h1 = h + a.G;
  auto step = [&](int n) {
    while (n > 0 && h < h1) {
      if (cur.t < cur.t1) {
        cur.step(1);
        --n;
      }
      if (cur.t >= cur.t1) {
        cur = first;
        ++h;
        if (first.t >= first.t1) h = h1;
      }
    }
  };
  if (first.t >= first.t1) h = h1;
  step(rank * C::kGroups + g);
  auto copy = [&](float* dst, const void* src) {
    if (h < h1) {
      const int64_t qo = (static_cast<int64_t>(b) * a.Sq + cur.t * kC) * qs + static_cast<int64_t>(h) * D;
      copy_rows<D>(dst, static_cast<const float*>(src) + qo, qs, min(kC, a.Sq - cur.t * kC), kC, tid, kGrp);
    }
    copy_commit();
  };
  copy(dO, a.dout);
  copy(Q, a.q);
  copy_wait<0>();
  __syncthreads();
  while (h < h1) {
    const Scorer score(a, h);
    const int q0 = cur.t * kC, nq = min(kC, a.Sq - q0);
    const int64_t lo = (static_cast<int64_t>(b) * a.H + h) * a.Sq + q0;
    if (tid < kC) {
      lse2[tid] = lse2_of(a, lo + tid, tid < nq);
      dlt[tid] = tid < nq ? a.delta[lo + tid] : 0.f;
    }
    step(cs * C::kGroups);
    copy_wait<0>();
    group_sync(g);
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
    group_sync(g);
    second<D>(dv, Pt, dO, ti, tj);
    group_sync(g);
    copy(dO, a.dout);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<float4*>(Pt + (tj + 16 * c) * kPT + 4 * ti) =
          make_float4(dp[0][c], dp[1][c], dp[2][c], dp[3][c]);
    group_sync(g);
    second<D>(dk, Pt, Q, ti, tj);
    group_sync(g);
    copy(Q, a.q);
  }
  copy_wait<0>();
  group_sync(g);
  put<D>(dk, Q, ti, tj);
  put<D>(dv, Q + C::kOwn, ti, tj);
  cluster_sync();
  const uint32_t st0 = smem_addr(sm + 2 * C::kOwn);
  const int share = kR / cs;
  for (int e = threadIdx.x; e < share * (D / 4); e += C::kThreads) {
    const int r = rank * share + e / (D / 4), d = (e % (D / 4)) * 4;
    if (r >= nk) break;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    for (int c = 0; c < cs; ++c)
#pragma unroll
      for (int z = 0; z < C::kGroups; ++z) {
        const uint32_t st = cluster_peer(st0 + (z * kStep + r * (D + 4) + d) * 4, c);
        add4(x, ld_peer4(st));
        add4(y, ld_peer4(st + C::kOwn * 4));
      }
    store4(a.dk, ko + r * ks + d, scaled(x, a.scale));
    store4(a.dv, ko + r * ks + d, y);
  }
}

// Both kinds of CTA in one launch: dk/dv CTAs (the first keys, which the most
// causal rows reach, first), then dq CTAs (the last rows first).
template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1) score_bwd_f32_kernel(const __grid_constant__ ScoreArgs a) {
  extern __shared__ __align__(16) float sm[];
  const int cs = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int kv_items = (a.Skv + kR - 1) / kR * a.Hkv * a.B, nq = (a.Sq + kR - 1) / kR;
  const int id = static_cast<int>(blockIdx.x) / cs;
  if (id < kv_items) {
    const int bh = id % (a.Hkv * a.B);
    dkdv_cta<D>(a, sm, cs, rank, id / (a.Hkv * a.B), bh % a.Hkv, bh / a.Hkv);
  } else {
    const int i = id - kv_items, bh = i % (a.H * a.B);
    dq_cta<D>(a, sm, cs, rank, nq - 1 - i / (a.H * a.B), bh % a.H, bh / a.H);
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
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

// CTAs that share an item, 1 to 8: the size with the least estimated time, in
// steps (tiles taken by every group at once): the longest item's, or all items'
// over 152 multiprocessors, with kOver steps of an item's own for its start and
// join. A cluster pays where a few items are long (one key/value head under 32
// query heads: ...) and costs where the items fill a wave (...).
inline int cluster_for(int groups, int64_t items_a, int64_t tiles_a, int64_t items_b = 0, int64_t tiles_b = 0) {
  constexpr double kOver = 1.5;
  int best = 1;
  double least = 0;
  for (int cs = 1; cs <= 8; cs *= 2) {
    const int64_t per = static_cast<int64_t>(cs) * groups;
    const double ta = static_cast<double>((tiles_a + per - 1) / per) + kOver, tb = static_cast<double>((tiles_b + per - 1) / per) + kOver;
    const double all = cs * (items_a * ta + items_b * tb) / 152.0;
    const double t = std::max(std::max(items_a > 0 ? ta : 0.0, items_b > 0 ? tb : 0.0), all);
    if (cs == 1 || t < 0.9 * least) {
      best = cs;
      least = t;
    }
  }
  return best;
}

template <int D>
cudaError_t fwd_d(const ScoreArgs& a, cudaStream_t s) {
  constexpr int bytes = Cfg<D>::kFwd * 4;
  static_assert(bytes <= 227 * 1024, "shared memory budget");
  cudaError_t e = allow_smem<score_fwd_f32_kernel<D>>(bytes);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>((a.Sq + kR - 1) / kR) * a.H * a.B;
  return launch_clusters(score_fwd_f32_kernel<D>, items, cluster_for(Cfg<D>::kGroups, items, (a.Skv + kC - 1) / kC),
                         Cfg<D>::kThreads, bytes, s, a);
}

template <int D>
cudaError_t bwd_d(const ScoreArgs& a, cudaStream_t s) {
  constexpr int bytes = Cfg<D>::kBwd * 4;
  static_assert(bytes <= 227 * 1024, "shared memory budget");
  cudaError_t e = allow_smem<score_bwd_f32_kernel<D>>(bytes);
  if (e != cudaSuccess) return e;
  if (a.Sq > 0) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.Sq * a.H;
    if ((rows + 7) / 8 > 0x7fffffff) return cudaErrorInvalidValue;
    score_delta_kernel<D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const int64_t kv_items = static_cast<int64_t>((a.Skv + kR - 1) / kR) * a.Hkv * a.B;
  const int64_t q_items = static_cast<int64_t>((a.Sq + kR - 1) / kR) * a.H * a.B;
  const int cs = cluster_for(Cfg<D>::kGroups, kv_items, static_cast<int64_t>((a.Sq + kC - 1) / kC) * a.G, q_items,
                             (a.Skv + kC - 1) / kC);
  return launch_clusters(score_bwd_f32_kernel<D>, kv_items + q_items, cs, Cfg<D>::kThreads, bytes, s, a);
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
