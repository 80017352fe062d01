// score_attn_f32.cu — attention with a score rule, fp32 inputs, results and
// sums: forward and backward.
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
// The products run on the tensor cores in three passes of tf32 (m16n8k8): with
// x = hi + lo, hi its upper 11 bits, hi hi' + hi lo' + lo hi' leaves out 2^-22
// of a product, and all sums are fp32. (As FMAs from shared memory the same
// tiles were bound by its 128 bytes a cycle: a 4 x 4 block a thread needs half a
// float an FMA where a quarter is the balance. 2048 tokens, 16 heads on 4, D =
// 128, causal: forward 527 -> 444 us, backward 1611 -> 1283 us; the error
// against 64 bits is below that of fp32 library products.)
// Tiles: a CTA owns 32 rows (queries; keys for dk, dv) and walks 64-row tiles
// of the other side. Four warps form a group; a warp takes 16 of the rows
// against 32 rows of the tile, and keeps its own running state, so that the
// weights never leave registers: accumulator columns 2t, 2t + 1 of a lane are
// the A operand's columns t, t + 4 of the second product once the tile's rows
// are taken in that order. Every tile is row-major with D + 4 floats a row, which
// serves both products without bank conflicts and without a transposed copy.
// A CTA holds kGroups groups (4 at D = 64, 2 at D = 128) that take the tiles in
// turn, each with its own buffers and barrier, joined once at the end; a
// buffer's next tile is copied (16-byte asynchronous copies) as soon as its last
// reader is through. Where that still leaves multiprocessors idle, a cluster of
// 2, 4 or 8 CTAs shares the tiles of one item in the same way and joins through
// distributed shared memory (see cluster_for). At D = 64 four groups leave 128
// registers a thread; the backward spills 356 bytes there.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "cp_ptx.cuh"
#include "cp_score.h"
#include "tf32.cuh"

namespace cp {
namespace {

constexpr int kGrp = 128;     // threads of a group
constexpr int kR = 32;        // rows of the owned tile
constexpr int kC = 64;        // rows of a streamed tile
constexpr float kL2e = 1.4426950408889634f;
constexpr float kLn2f = 0.69314718055994531f;

template <int D>
struct Cfg {
  static constexpr int kGroups = 256 / D;
  static constexpr int kThreads = kGroups * kGrp;
  static constexpr int kRow = D + 4;                           // floats of a row
  static constexpr int kOwn = kR * kRow, kTile = kC * kRow;    // floats of a tile
  static constexpr int kStep = 2 * kTile + 4 * kC;             // a group's: two tiles, then row statistics
  static constexpr int kFwd = kOwn + kGroups * kStep;
  static constexpr int kBwd = 2 * kOwn + kGroups * kStep;
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

// Barrier of the caller's group, whose warps converge for it (and for the matrix
// instructions behind it).
__device__ __forceinline__ void group_sync(int g) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(kGrp) : "memory");
}

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

__device__ __forceinline__ void mma3(float (&big)[4], float (&small)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                     float b0, float b1) {
  uint32_t bh[2], bl[2];
  split_tf32(b0, bh[0], bl[0]);
  split_tf32(b1, bh[1], bl[1]);
  mma3_tf32(big, small, ah, al, bh, bl);
}

// s[n][.] = 16 rows of a . rows 8 n .. 8 n + 7 of b, as accumulator fragments:
// elements 0, 1 are row g, columns 2 t, 2 t + 1; 2, 3 row g + 8 (g = lane / 4, t = lane % 4)
template <int D>
__device__ __forceinline__ void dots(float (&s)[4][4], const float* a, const float* b, int g, int t) {
  float small[4][4];
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[n][e] = small[n][e] = 0.f;
#pragma unroll 1
  for (int k0 = 0; k0 < D; k0 += 32) {
    float big[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) big[n][e] = 0.f;
#pragma unroll
    for (int k = k0; k < k0 + 32; k += 8) {
      uint32_t ah[4], al[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split_tf32(a[(g + (e & 1) * 8) * (D + 4) + k + t + (e >> 1) * 4], ah[e], al[e]);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float* r = b + (8 * n + g) * (D + 4) + k + t;
        mma3(big[n], small[n], ah, al, r[0], r[4]);
      }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] += big[n][e];
  }
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[n][e] += small[n][e];
}

// acc += w b: w the 16 x 32 weights as the fragments of dots, b the tile's 32
// rows; acc[n] columns 8 n .. 8 n + 7
template <int D>
__device__ __forceinline__ void second(float (&acc)[D / 8][4], const float (&w)[4][4], const float* b, int g, int t) {
  uint32_t ah[4][4], al[4][4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) split_tf32(w[k][(e & 1) * 2 + (e >> 1)], ah[k][e], al[k][e]);
  b += 2 * t * (D + 4) + g;
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    float big[4] = {0.f, 0.f, 0.f, 0.f}, small[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float* r = b + 8 * k * (D + 4) + 8 * n;
      mma3(big, small, ah[k], al[k], r[0], r[D + 4]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] += big[e] + small[e];
  }
}

template <int D>
__device__ __forceinline__ void clear(float (&acc)[D / 8][4]) {
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
}

// acc as 16 rows of D + 4 floats in shared memory
template <int D>
__device__ __forceinline__ void put(const float (&acc)[D / 8][4], float* dst, int g, int t) {
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    *reinterpret_cast<float2*>(dst + g * (D + 4) + 8 * n + 2 * t) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(dst + (g + 8) * (D + 4) + 8 * n + 2 * t) = make_float2(acc[n][2], acc[n][3]);
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
      const float y = x * inv_cap;
      x = cap * tanhf(y);
      // 1 - tanh^2 without its cancellation
      const float e = ex2_approx(-2.f * kL2e * fabsf(y)), r = rcp_approx(1.f + e);
      dcap = 4.f * e * r * r;
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
  const int grp = threadIdx.x / kGrp, tid = threadIdx.x % kGrp;
  const int r16 = (tid >> 5 & 1) * 16, c32 = (tid >> 6) * 32;  // the warp's rows and columns
  const int g = (tid & 31) >> 2, t = tid & 3;
  float* Q = sm;
  float* K = sm + C::kOwn + grp * C::kStep;
  float* V = K + C::kTile;
  grid_wait();  // the document ranges
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
  cur.step(rank * C::kGroups + grp);
  auto copy = [&](float* dst, const void* src, int at) {
    if (at < cur.t1)
      copy_rows<D>(dst, static_cast<const float*>(src) + ko + at * kC * ks, ks, min(kC, a.Skv - at * kC), kC, tid, kGrp);
    copy_commit();
  };
  copy_rows<D>(Q, static_cast<const float*>(a.q) + qo, qs, nrows, kR, threadIdx.x, C::kThreads);
  copy(K, a.k, cur.t);  // with Q
  copy(V, a.v, cur.t);
  const Scorer score(a, h);
  int lim[2], qd[2];
  float m[2], l[2];
  float acc[D / 8][4];
  clear<D>(acc);
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // rows g and g + 8 of the warp's
    const int r = r16 + g + 8 * i;
    lim[i] = min(a.Skv, key_limit(a, plim, row0 + r));
    qd[i] = a.qdoc && r < nrows ? a.qdoc[static_cast<int64_t>(b) * a.Sq + row0 + r] : -1;
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  copy_wait<1>();
  __syncthreads();  // Q is every thread's
  while (cur.t < cur.t1) {
    const int j0 = cur.t * kC + c32 + 2 * t;
    cur.step(cs * C::kGroups);
    copy_wait<1>();  // K
    group_sync(grp);
    float s[4][4];
    dots<D>(s, Q + r16 * C::kRow, K + c32 * C::kRow, g, t);
    group_sync(grp);
    copy(K, a.k, cur.t);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int j = j0 + 8 * n + c;
        const int kd = a.qdoc && j < a.Skv ? a.kdoc[static_cast<int64_t>(b) * a.Skv + j] : -1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float unused;
          const bool on = j < lim[i] && (!a.qdoc || (qd[i] == kd && kd >= 0));
          float& x = s[n][2 * i + c];
          x = on ? score(x, a.rel + row0 + r16 + g + 8 * i - j, unused) : -INFINITY;
        }
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int n = 0; n < 4; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * i], s[n][2 * i + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[i] - base);  // 0 while m is -inf
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          s[n][2 * i + c] = exp2f(s[n][2 * i + c] - base);
          sum += s[n][2 * i + c];
        }
      l[i] = l[i] * f + sum;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        acc[n][2 * i] *= f;
        acc[n][2 * i + 1] *= f;
      }
    }
    copy_wait<1>();  // V
    group_sync(grp);
    second<D>(acc, s, V + c32 * C::kRow, g, t);
    group_sync(grp);
    copy(V, a.v, cur.t);
  }
  copy_wait<0>();
  // ---- the states of every CTA's warps joined: a CTA stores the rows of its
  // share. K holds O of the two column halves, [2][32 rows]; then m, l ----
  group_sync(grp);
  put<D>(acc, K + (c32 + r16) * C::kRow, g, t);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (t == 0) *reinterpret_cast<float2*>(K + 2 * C::kTile + 2 * (c32 + r16 + g + 8 * i)) = make_float2(m[i], l[i]);
  }
  cluster_sync();
  const uint32_t st0 = smem_addr(sm + C::kOwn);
  const int share = kR / cs;
  for (int e = threadIdx.x; e < share * (D / 4); e += C::kThreads) {
    const int r = rank * share + e / (D / 4), d = (e % (D / 4)) * 4;
    if (r >= nrows) break;
    float mx = -INFINITY;
    for (int x = 0; x < cs; ++x)
#pragma unroll
      for (int y = 0; y < 2 * C::kGroups; ++y)
        mx = fmaxf(mx, ld_peer2(cluster_peer(st0 + ((y >> 1) * C::kStep + 2 * C::kTile + 2 * ((y & 1) * kR + r)) * 4, x)).x);
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 0; x < cs; ++x)
#pragma unroll
      for (int y = 0; y < 2 * C::kGroups; ++y) {
        const uint32_t st = cluster_peer(st0 + (y >> 1) * C::kStep * 4, x);
        const int rr = (y & 1) * kR + r;
        const float2 ml = ld_peer2(st + (2 * C::kTile + 2 * rr) * 4);
        const float f = exp2f(ml.x - base);
        sum = fmaf(ml.y, f, sum);
        add4(o, scaled(ld_peer4(st + (rr * C::kRow + d) * 4), f));
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
  grid_release();
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

// Sum over every CTA's warps of the 32 x D results that put has left at `at`
// floats into each group's buffers, times mul, to dst (row r at r * stride).
template <int D>
__device__ __forceinline__ void join(const float* sm, int at, int cs, int rank, int n, float mul, void* dst, int64_t to,
                                     int64_t stride) {
  using C = Cfg<D>;
  const uint32_t st0 = smem_addr(sm + 2 * C::kOwn + at);
  const int share = kR / cs;
  for (int e = threadIdx.x; e < share * (D / 4); e += C::kThreads) {
    const int r = rank * share + e / (D / 4), d = (e % (D / 4)) * 4;
    if (r >= n) break;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < cs; ++c)
#pragma unroll
      for (int y = 0; y < 2 * C::kGroups; ++y)
        add4(x, ld_peer4(cluster_peer(st0 + ((y >> 1) * C::kStep + ((y & 1) * kR + r) * C::kRow + d) * 4, c)));
    store4(dst, to + r * stride + d, scaled(x, mul));
  }
}

// dq of 32 query rows: key tiles stream by.
template <int D>
__device__ __forceinline__ void dq_cta(const ScoreArgs& a, float* sm, int cs, int rank, int bx, int h, int b) {
  using C = Cfg<D>;
  const int grp = threadIdx.x / kGrp, tid = threadIdx.x % kGrp;
  const int r16 = (tid >> 5 & 1) * 16, c32 = (tid >> 6) * 32;
  const int g = (tid & 31) >> 2, t = tid & 3;
  float* Q = sm;
  float* dO = Q + C::kOwn;
  float* K = dO + C::kOwn + grp * C::kStep;
  float* V = K + C::kTile;
  const int hk = h / a.G;
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
  cur.step(rank * C::kGroups + grp);
  auto copy = [&](float* dst, const void* src, int at) {
    if (at < cur.t1)
      copy_rows<D>(dst, static_cast<const float*>(src) + ko + at * kC * ks, ks, min(kC, a.Skv - at * kC), kC, tid, kGrp);
    copy_commit();
  };
  copy_rows<D>(Q, static_cast<const float*>(a.q) + qo, qs, nrows, kR, threadIdx.x, C::kThreads);
  copy_rows<D>(dO, static_cast<const float*>(a.dout) + qo, qs, nrows, kR, threadIdx.x, C::kThreads);
  copy(V, a.v, cur.t);
  copy(K, a.k, cur.t);
  const Scorer score(a, h);
  int lim[2], qd[2];
  float lse2[2], dlt[2];
  float acc[D / 8][4];
  clear<D>(acc);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r16 + g + 8 * i;
    const int64_t o = (static_cast<int64_t>(b) * a.H + h) * a.Sq + row0 + r;
    lim[i] = min(a.Skv, key_limit(a, plim, row0 + r));
    qd[i] = a.qdoc && r < nrows ? a.qdoc[static_cast<int64_t>(b) * a.Sq + row0 + r] : -1;
    lse2[i] = lse2_of(a, o, r < nrows);
    dlt[i] = r < nrows ? a.delta[o] : 0.f;
  }
  copy_wait<0>();
  __syncthreads();
  while (cur.t < cur.t1) {
    const int j0 = cur.t * kC + c32 + 2 * t;
    cur.step(cs * C::kGroups);
    copy_wait<0>();
    group_sync(grp);
    float s[4][4], dp[4][4];
    dots<D>(dp, dO + r16 * C::kRow, V + c32 * C::kRow, g, t);
    dots<D>(s, Q + r16 * C::kRow, K + c32 * C::kRow, g, t);
    group_sync(grp);
    copy(V, a.v, cur.t);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int j = j0 + 8 * n + c;
        const int kd = a.qdoc && j < a.Skv ? a.kdoc[static_cast<int64_t>(b) * a.Skv + j] : -1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float dcap;
          const bool on = j < lim[i] && (!a.qdoc || (qd[i] == kd && kd >= 0));
          const int e = 2 * i + c;
          const float p = exp2f(score(s[n][e], a.rel + row0 + r16 + g + 8 * i - j, dcap) - lse2[i]);
          s[n][e] = on ? p * (dp[n][e] - dlt[i]) * dcap : 0.f;
        }
      }
    __syncwarp();  // lanes may have parted over masks and the cap; matrix instructions want the warp converged
    second<D>(acc, s, K + c32 * C::kRow, g, t);
    group_sync(grp);
    copy(K, a.k, cur.t);
  }
  copy_wait<0>();
  group_sync(grp);
  put<D>(acc, K + (c32 + r16) * C::kRow, g, t);
  cluster_sync();
  join<D>(sm, 0, cs, rank, nrows, a.scale, a.dq, qo, qs);
}

// dk, dv of 32 keys: the streamed tiles are 64 query rows of each head that
// shares the key/value head, head by head. Scores are formed transposed (rows
// are keys).
template <int D>
__device__ __forceinline__ void dkdv_cta(const ScoreArgs& a, float* sm, int cs, int rank, int bx, int hk, int b) {
  using C = Cfg<D>;
  const int grp = threadIdx.x / kGrp, tid = threadIdx.x % kGrp;
  const int r16 = (tid >> 5 & 1) * 16, c32 = (tid >> 6) * 32;
  const int g = (tid & 31) >> 2, t = tid & 3;
  float* K = sm;
  float* V = K + C::kOwn;
  float* Q = V + C::kOwn + grp * C::kStep;
  float* dO = Q + C::kTile;
  float* lse2 = dO + C::kTile;
  float* dlt = lse2 + kC;
  const int key0 = bx * kR;
  const int nk = min(kR, a.Skv - key0);
  const int64_t qs = static_cast<int64_t>(a.H) * D, ks = static_cast<int64_t>(a.Hkv) * D;
  const int64_t ko = (static_cast<int64_t>(b) * a.Skv + key0) * ks + static_cast<int64_t>(hk) * D;
  copy_rows<D>(K, static_cast<const float*>(a.k) + ko, ks, nk, kR, threadIdx.x, C::kThreads);
  copy_rows<D>(V, static_cast<const float*>(a.v) + ko, ks, nk, kR, threadIdx.x, C::kThreads);
  copy_commit();
  const int plim = prefix_limit(a, b);
  int kd[2];
  float dk[D / 8][4], dv[D / 8][4];
  clear<D>(dk);
  clear<D>(dv);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r16 + g + 8 * i;
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
      }
    }
  };
  if (first.t >= first.t1) h = h1;
  step(rank * C::kGroups + grp);
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
    group_sync(grp);
    float s[4][4], dp[4][4];
    dots<D>(s, K + r16 * C::kRow, Q + c32 * C::kRow, g, t);
    dots<D>(dp, V + r16 * C::kRow, dO + c32 * C::kRow, g, t);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = c32 + 8 * n + 2 * t + c, i = q0 + r;
        const int lim = key_limit(a, plim, i);
        const int qd = a.qdoc && r < nq ? a.qdoc[static_cast<int64_t>(b) * a.Sq + i] : -1;
        const float l2 = lse2[r], dl = dlt[r];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j = key0 + r16 + g + 8 * u, e = 2 * u + c;
          float dcap;
          const bool on = r < nq && j < lim && (!a.qdoc || (qd == kd[u] && qd >= 0));
          const float p = exp2f(score(s[n][e], a.rel + i - j, dcap) - l2);
          s[n][e] = on ? p : 0.f;
          dp[n][e] = on ? p * (dp[n][e] - dl) * dcap : 0.f;
        }
      }
    __syncwarp();
    second<D>(dv, s, dO + c32 * C::kRow, g, t);
    group_sync(grp);
    copy(dO, a.dout);
    second<D>(dk, dp, Q + c32 * C::kRow, g, t);
    group_sync(grp);
    copy(Q, a.q);
  }
  copy_wait<0>();
  group_sync(grp);
  put<D>(dk, Q + (c32 + r16) * C::kRow, g, t);
  put<D>(dv, dO + (c32 + r16) * C::kRow, g, t);
  cluster_sync();
  join<D>(sm, 0, cs, rank, nk, a.scale, a.dk, ko, ks);
  join<D>(sm, C::kTile, cs, rank, nk, 1.f, a.dv, ko, ks);
}

// Both kinds of CTA in one launch: dk/dv CTAs (the first keys, which the most
// causal rows reach, first), then dq CTAs (the last rows first).
template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1) score_bwd_f32_kernel(const __grid_constant__ ScoreArgs a) {
  extern __shared__ __align__(16) float sm[];
  const int cs = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  grid_wait();  // the delta kernel's results
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
  grid_release();
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
  constexpr int bytes = Cfg<D>::kFwd * 4;
  static_assert(bytes <= 227 * 1024, "shared memory budget");
  cudaError_t e = allow_smem<score_fwd_f32_kernel<D>>(bytes);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>((a.Sq + kR - 1) / kR) * a.H * a.B;
  // steps: tiles taken by every group at once
  const int64_t steps = ((a.Skv + kC - 1) / kC + Cfg<D>::kGroups - 1) / Cfg<D>::kGroups;
  const int cs = cluster_for(1.5, items, steps, 0, 0, a.causal ? 0.5 : 1.0, true, a.sms);
  return launch_clusters(score_fwd_f32_kernel<D>, items, 1, 1, cs, Cfg<D>::kThreads, bytes, a.qdoc != nullptr, s, a);
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
  constexpr int G = Cfg<D>::kGroups;
  const int cs = cluster_for(1.5, kv_items, (static_cast<int64_t>((a.Sq + kC - 1) / kC) * a.G + G - 1) / G, q_items,
                             ((a.Skv + kC - 1) / kC + G - 1) / G, a.causal ? 0.5 : 1.0, true, a.sms);
  return launch_clusters(score_bwd_f32_kernel<D>, kv_items + q_items, 1, 1, cs, Cfg<D>::kThreads, bytes, a.Sq > 0, s, a);
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
