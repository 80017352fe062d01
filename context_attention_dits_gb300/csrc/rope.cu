// rope.cu — queries and keys normalised for each head and rotated by their
// positions in one pass, and the gradients.
//
// A row is one head of one token, x of D values, r = 1 / sqrt(mean x^2 + eps):
//   y = x r w                                          (without a norm: y = x)
//   pair p = (u, v) of y at angle t = position[axis of p] freqs[p]:
//   (u, v) -> (u cos t - v sin t, u sin t + v cos t);  values behind the pairs stay
// and with g the gradient of the result rotated back (by -t):
//   dw = sum over rows of g x r,  dx = r (g w - x r mean(g w x r))
//
// Every value is read once and written once and costs some ten operations, so HBM
// bounds the long calls (2 or 3 streams; 32768 tokens of 24 + 24 heads of 128, bf16,
// take 127 us forward, 6.3 TB/s, and 4608 take 22.2, some 4 of them start and end) and
// the launch the short ones. A row lies in D / 8 lanes, 8 values each: its sums take 3
// or 4 shuffles, and a lane holds both members of its four pairs, by one 16-byte piece
// where pairs are neighbours and two pieces of 8 where they are the row's halves. A
// warp walks the heads of one token, so an angle is formed once for all of them, each
// pair by one lane and handed round by shuffles.
//
// An angle of radians in fp32 is worth nothing far out (half a radian at position
// 2^23). It is kept in turns instead, as 64-bit fixed point: u = f 2^64 / 2 pi,
// whole turns dropped, and position u is exact but for what u itself is off: less
// than (1 + f / 200) 2^-64 of a turn (bits dropped, and those of the constant), times
// the position.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "cp_ptx.cuh"
#include "cp_rope.h"
#include "cp_score.h"
#include "packed.cuh"

namespace cp {
namespace {

constexpr int kThreads = kRopeWarps * 32;
constexpr int kFwdCtas = 3, kBwdCtas = 2;  // on a multiprocessor
constexpr int kRopeSteps = 16;             // row steps of a part at most, while tokens are many

// f 2^64 / 2 pi, whole turns dropped; f as m 2^(e - 1075), m its 53 bits. 2^66 / 2 pi
// rounded to 64 bits is off by 2^-65 of itself. Subnormal and not finite: 0.
__device__ __forceinline__ uint64_t turn_step(double f) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
  const int e = static_cast<int>(bits >> 52) & 0x7ff;
  if (e == 0 || e == 0x7ff) return 0;
  const uint64_t m = (bits & ((1ull << 52) - 1)) | 1ull << 52;
  constexpr uint64_t kC = 11743562013128004906ull;
  const uint64_t lo = m * kC, hi = __umul64hi(m, kC);
  const int sh = 1077 - e;  // m kC 2^(e - 1075) 2^-66 2^64
  uint64_t u = 0;
  if (sh >= 64)
    u = sh < 128 ? hi >> (sh - 64) : 0;
  else if (sh > 0)
    u = lo >> sh | hi << (64 - sh);
  else if (sh > -64)
    u = lo << -sh;
  return bits >> 63 ? 0 - u : u;
}

// cos and sin at position pos. The angle's upper 32 bits name the quarter turn
// (rounded) and the rest, within an eighth turn to either side, where the Taylor
// series' next terms are below 3e-8 (cos) and 2e-9 (sin).
__device__ __forceinline__ void cos_sin(uint64_t step, int pos, float& c, float& s) {
  const uint64_t t = step * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const uint32_t at = static_cast<uint32_t>((t + 0x80000000ull) >> 32);
  const uint32_t quarter = (at + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(at - (quarter << 30))) * 1.46291807926715968e-9f;  // 2 pi 2^-32
  const float xx = x * x;
  const float cs = fmaf(xx, fmaf(xx, fmaf(xx, fmaf(xx, 1.f / 40320, -1.f / 720), 1.f / 24), -0.5f), 1.f);
  const float sn = x * fmaf(xx, fmaf(xx, fmaf(xx, fmaf(xx, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), 1.f);
  c = quarter & 1 ? sn : cs;
  s = quarter & 1 ? cs : sn;
  if (quarter == 1 || quarter == 2) c = -c;
  if (quarter == 2 || quarter == 3) s = -s;
}

// 8 values of a row as the first and the second members of four pairs: neighbours,
// or the two fours against each other; and back.
template <bool kNext>
__device__ __forceinline__ void apart(const float (&x)[8], float2 (&u)[2], float2 (&v)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    u[i] = kNext ? make_float2(x[4 * i], x[4 * i + 2]) : make_float2(x[2 * i], x[2 * i + 1]);
    v[i] = kNext ? make_float2(x[4 * i + 1], x[4 * i + 3]) : make_float2(x[4 + 2 * i], x[4 + 2 * i + 1]);
  }
}
template <bool kNext>
__device__ __forceinline__ void together(const float2 (&u)[2], const float2 (&v)[2], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[kNext ? 4 * i : 2 * i] = u[i].x;
    x[kNext ? 4 * i + 2 : 2 * i + 1] = u[i].y;
    x[kNext ? 4 * i + 1 : 4 + 2 * i] = v[i].x;
    x[kNext ? 4 * i + 3 : 4 + 2 * i + 1] = v[i].y;
  }
}

// A lane's 8 values of a row as they lie in memory: 4 from element e0, 4 from e1.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int e0, int e1, bool one) {
    if (one) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + e0);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(row + e0), y = *reinterpret_cast<const uint2*>(row + e1);
      w[0] = x.x, w[1] = x.y, w[2] = y.x, w[3] = y.y;
    }
  }
  template <bool kNext>
  __device__ __forceinline__ void get(float2 (&u)[2], float2 (&v)[2]) const {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    apart<kNext>(x, u, v);
  }
  template <bool kNext>
  static __device__ __forceinline__ void store(__nv_bfloat16* row, int e0, int e1, const float2 (&u)[2], const float2 (&v)[2]) {
    float x[8];
    together<kNext>(u, v, x);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    if (kNext) {
      *reinterpret_cast<uint4*>(row + e0) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(row + e0) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + e1) = make_uint2(w[2], w[3]);
    }
  }
};
template <>
struct Raw<float> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const float* row, int e0, int e1, bool) {
    const uint4 x = *reinterpret_cast<const uint4*>(row + e0), y = *reinterpret_cast<const uint4*>(row + e1);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
  }
  template <bool kNext>
  __device__ __forceinline__ void get(float2 (&u)[2], float2 (&v)[2]) const {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    apart<kNext>(x, u, v);
  }
  template <bool kNext>
  static __device__ __forceinline__ void store(float* row, int e0, int e1, const float2 (&u)[2], const float2 (&v)[2]) {
    float x[8];
    together<kNext>(u, v, x);
    *reinterpret_cast<float4*>(row + e0) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(row + e1) = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// What a lane is: its place in its row, its values, its weights and its own pairs' steps.
template <int D, typename T, bool kNext>
struct Lane {
  static constexpr int kLanes = D / 8;           // of a row
  static constexpr int kRows = 32 / kLanes;      // of a warp
  static constexpr int kOwn = 4 / kRows;         // pairs whose angle this lane forms
  int l, r, e0, e1;
  bool some_stay, stays;  // lanes of the warp, this one, behind the pairs
  uint64_t step[kOwn];
  int axis[kOwn];

  __device__ __forceinline__ explicit Lane(const RopeArgs& a) {
    const int lane = threadIdx.x & 31;
    l = lane % kLanes;
    r = lane / kLanes;
    // neighbours: 8 values in a row; halves: 4 of each half, behind the pairs 8 in a row
    const int with = a.pairs / 4;  // lanes with pairs
    some_stay = with < kLanes;
    stays = l >= with;
    e0 = kNext ? 8 * l : l < with ? 4 * l : 2 * a.pairs + 8 * (l - with);
    e1 = kNext || l >= with ? e0 + 4 : a.pairs + 4 * l;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int p = 4 * l + r * kOwn + i;
      step[i] = p < a.pairs ? turn_step(a.freqs[p]) : 0;
      axis[i] = p < a.pairs ? a.axis[p] : 0;
    }
  }
  // The members that turn into one another: none behind the pairs, where products with a
  // sine of 0 would be NaN beside an infinity (the zeros' signs keep those of the values).
  __device__ __forceinline__ void across(float2& u, float2& v, float u0) const {
    if (some_stay && stays) u = twice(u0), v = twice(-u0);
  }
  // cos and sin of the lane's four pairs for the token at pos
  __device__ __forceinline__ void angles(const int* pos, float2 (&c)[2], float2 (&s)[2]) const {
    float oc[kOwn], os[kOwn], ac[4], as[4];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) cos_sin(step[i], pos[axis[i]], oc[i], os[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int from = i / kOwn * kLanes + l;
      ac[i] = __shfl_sync(0xffffffffu, oc[i % kOwn], from);
      as[i] = __shfl_sync(0xffffffffu, os[i % kOwn], from);
    }
    c[0] = make_float2(ac[0], ac[1]), c[1] = make_float2(ac[2], ac[3]);
    s[0] = make_float2(as[0], as[1]), s[1] = make_float2(as[2], as[3]);
  }
  __device__ __forceinline__ void weights(const RopeArgs& a, const void* w, float2 (&u)[2], float2 (&v)[2]) const {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = element(j);
      x[j] = !w ? 1.f : a.w_f32 ? static_cast<const float*>(w)[e] : static_cast<float>(static_cast<const T*>(w)[e]);
    }
    apart<kNext>(x, u, v);
  }
  __device__ __forceinline__ int element(int j) const { return j < 4 ? e0 + j : e1 + j - 4; }
  // Brings the row about to 1 by a power of two: that of its largest value, or of sqrt(eps)
  // if that is larger. x r is the same then, and r as much less. Returns the power.
  static __device__ __forceinline__ float nearer(float2 (&u)[2], float2 (&v)[2], float eps) {
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) big = fmaxf(big, fmaxf(fmaxf(fabsf(u[i].x), fabsf(u[i].y)), fmaxf(fabsf(v[i].x), fabsf(v[i].y))));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    const uint32_t of_x = __float_as_uint(big) >> 23, of_eps = eps > 0.f ? ((__float_as_uint(eps) >> 23) + 127) / 2 : 0;
    const float by = __uint_as_float((254 - min(max(max(of_x, of_eps), 1u), 253u)) << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u[i] = mul2(u[i], twice(by));
      v[i] = mul2(v[i], twice(by));
    }
    return by;
  }
  static __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  }
};

// A CTA's part of every token: heads [first, last) of q or of k. Its warps take the
// tokens in turn.
struct Part {
  bool k;
  int first, last, token, stride;
  __device__ __forceinline__ Part(const RopeArgs& a, int rows) {
    const int group = blockIdx.x / a.parts, part = blockIdx.x - group * a.parts;
    k = part >= a.parts_q;
    const int heads = k ? a.Hkv : a.H, n = (heads + rows - 1) / rows;
    const int of = k ? a.parts - a.parts_q : a.parts_q, at = k ? part - a.parts_q : part;
    first = static_cast<int>(static_cast<int64_t>(at) * n / of) * rows;
    last = min(static_cast<int>(static_cast<int64_t>(at + 1) * n / of) * rows, heads);
    token = group * kRopeWarps + (threadIdx.x >> 5);
    stride = gridDim.x / a.parts * kRopeWarps;
  }
};

__device__ __forceinline__ int64_t row_at(const RopeRows& x, int b, int s, int head) {
  return b * x.sb + s * x.ss + head * x.sh;
}

// A warp's rows on their way through shared memory: batches of up to kBatch heads of a
// token (kB > 0: of two tensors), kStages - 1 of them under way while one is worked on,
// 2 KB (kB: 4 to 6 KB) each. As many loads in registers would halve the warps: 4608
// tokens of 24 + 24 heads of 128, bf16, with four rows in registers: forward 24.0 us where
// this took 21.7, backward 37.8 where it took 33.2 (32768 tokens forward: 134, 131). A
// warp with one batch in all gains nothing (700 tokens of 6 + 3 fp32 heads, backward:
// 7.7 us from registers, 8.5 here): not worth a second kernel beside some 20 us of calls.
template <int D, int kElemA, int kElemB>
struct Ring {
  // (backward of 4607 tokens with six steps 33.7 us, with four 34.8; forward of 4608 tokens
  // with three stages 22.2, with four 22.7, with two 22.8; of 32768 127.5, 128.0 and 126.4)
  static constexpr int kSteps = kElemA != 2 ? 2 : kElemB == 2 && D == 128 ? 6 : 4;
  static constexpr int kRows = 256 / D, kBatch = kRows * kSteps;
  static constexpr int kA = kBatch * D * kElemA, kB = kBatch * D * kElemB, kStage = kA + kB;
  static constexpr int kStages = kElemB ? 2 : 3;
  static constexpr int kSmem = kRopeWarps * kStages * kStage;
  static_assert(kBatch <= 16, "a lane a row and tensor");
  struct Shared {
    uint64_t full[kRopeWarps][kStages];
    uint32_t abort;
  };
  const RopeArgs& a;
  const Part& part;
  const RopeRows &x, &y;  // (y: the second tensor)
  Shared& sh;
  uint8_t* buf;
  uint32_t bars;
  int token, head, ask = 0, take = 0;  // of the next batch to ask for
  uint32_t phase = 0;

  __device__ __forceinline__ Ring(const RopeArgs& a_, const Part& p, const RopeRows& x_, const RopeRows& y_, uint8_t* smem, Shared& s)
      : a(a_), part(p), x(x_), y(y_), sh(s) {
    const int warp = threadIdx.x >> 5;
    buf = smem + warp * kStages * kStage;
    bars = smem_addr(&sh.full[warp][0]);
    token = p.token;
    head = p.first;
  }
  static __device__ __forceinline__ void set_up(const RopeArgs& a, Shared& sh) {
    if (threadIdx.x < kRopeWarps * kStages)
      mbar_init(smem_addr(&sh.full[0][0] + threadIdx.x), 1 + (a.stall >> threadIdx.x / kStages & 1u));
    if (threadIdx.x == 0) sh.abort = 0;
    fence_mbar_init();
    fence_async();
    __syncthreads();
  }
  __device__ __forceinline__ void next() {
    if (token >= a.tokens) return;
    const int lane = threadIdx.x & 31, n = min(kBatch, part.last - head), b = token / a.S, s = token - b * a.S;
    const uint32_t bar = bars + ask * 8, to = smem_addr(buf) + ask * kStage;
    const bool with_x = kB == 0 || a.norm;  // (without a norm the backward does not read x)
    if (lane == 0) mbar_arrive_expect_tx(bar, n * D * ((with_x ? kElemA : 0) + kElemB));
    __syncwarp();
    const bool second = kB > 0 && (lane & 16);
    const RopeRows& t = second ? y : x;
    const int elem = second ? kElemB : kElemA, i = kB > 0 ? lane & 15 : lane;
    if (second || with_x) {
      // heads side by side are one copy
      const int rows = t.sh == D ? (i == 0 ? n : 0) : (i < n ? 1 : 0);
      if (rows)
        bulk_g2s(to + (second ? kA : 0) + i * D * elem, static_cast<const uint8_t*>(t.p) + row_at(t, b, s, head + i) * elem,
                 rows * D * elem, bar);
    }
    if (++ask == kStages) ask = 0;
    if ((head += kBatch) >= part.last) {
      head = part.first;
      token += part.stride;
    }
    __syncwarp();
  }
  __device__ __forceinline__ void start() {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) next();
  }
  // The next batch, and the one that goes into the stage worked on before. nullptr: a wait ran out.
  __device__ __forceinline__ const uint8_t* batch() {
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(bars + take * 8, phase >> take & 1u, &sh.abort, a.err, a.timeout_ns)))
      return nullptr;
    next();
    return buf + take * kStage;
  }
  __device__ __forceinline__ void done() {
    phase ^= 1u << take;
    if (++take == kStages) take = 0;
    __syncwarp();
  }
  // After a wait that ran out: what is under way lands.
  __device__ __forceinline__ void drain() {
    for (; take != ask; done()) mbar_drain(bars + take * 8, phase >> take & 1u);
  }
};

// kTiny: a norm with an eps that does not hide what squares of small values lose in fp32, so
// that each row is brought about to 1 first (4608 tokens of 24 + 24 heads of 128, bf16: 25.5 us
// where others take 22.2; a look at every row and a second try took 23.2).
template <int D, typename T, bool kNext, bool kTiny>
__global__ void __launch_bounds__(kThreads, kFwdCtas) rope_fwd_kernel(const __grid_constant__ RopeArgs a) {
  using L = Lane<D, T, kNext>;
  using R = Ring<D, sizeof(T), 0>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ typename R::Shared shared;
  R::set_up(a, shared);
  grid_wait();  // (the launch may start while its predecessor in the stream ends)
  const Part part(a, L::kRows);
  const RopeRows &in = part.k ? a.k : a.q, &to = part.k ? a.ko : a.qo;
  R ring(a, part, in, in, smem, shared);
  ring.start();
  const L me(a);
  const int64_t to_step = L::kRows * to.sh;
  float2 wu[2], wv[2];
  me.weights(a, part.k ? a.wk : a.wq, wu, wv);
  for (int token = part.token; token < a.tokens; token += part.stride) {
    const int b = token / a.S, s = token - b * a.S;
    T* dest = static_cast<T*>(to.p) + row_at(to, b, s, part.first + me.r);
    // (u, v) -> n (u au - v bv, u bu + v av): weights and angles as one
    float2 au[2], av[2], bu[2], bv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      au[i] = wu[i];
      av[i] = wv[i];
      bu[i] = twice(0.f);
      bv[i] = twice(-0.f);
    }
    if (a.pairs) {
      float2 c[2], sn[2];
      me.angles(a.pos + b * a.pos_sb + static_cast<int64_t>(s) * a.axes, c, sn);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        au[i] = mul2(wu[i], c[i]);
        av[i] = mul2(wv[i], c[i]);
        bu[i] = mul2(wu[i], sn[i]);
        bv[i] = mul2(wv[i], make_float2(-sn[i].x, -sn[i].y));
      }
    }
    for (int head = part.first; head < part.last; head += R::kBatch) {
      const uint8_t* rows = ring.batch();
      if (!rows) return ring.drain();
#pragma unroll
      for (int i = 0; i < R::kSteps; ++i) {
        if (head + i * L::kRows >= part.last) break;
        const bool real = head + i * L::kRows + me.r < part.last;
        Raw<T> raw = {};
        if (real) raw.load(reinterpret_cast<const T*>(rows) + (i * L::kRows + me.r) * D, me.e0, me.e1, kNext);
        float2 u[2], v[2];
        raw.template get<kNext>(u, v);
        float n = 1.f;
        if (kTiny || a.norm) {
          const float by = kTiny ? L::nearer(u, v, a.eps) : 1.f;
          const float2 sq = fma2(v[1], v[1], fma2(v[0], v[0], fma2(u[1], u[1], mul2(u[0], u[0]))));
          n = rsqrtf(fmaf(L::row_sum(sq.x + sq.y), 1.f / D, kTiny ? a.eps * by * by : a.eps));
        }
        const float2 nn = twice(n);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float2 cu = u[j], cv = v[j];
          me.across(cu, cv, -0.f);
          u[j] = mul2(fma2(u[j], au[j], mul2(cv, bv[j])), nn);
          v[j] = mul2(fma2(v[j], av[j], mul2(cu, bu[j])), nn);
        }
        if (real) Raw<T>::template store<kNext>(dest, me.e0, me.e1, u, v);
        dest += to_step;
      }
      ring.done();
    }
  }
}

template <int D, typename T, typename G, bool kNext, bool kTiny>
__global__ void __launch_bounds__(kThreads, kBwdCtas) rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
  using L = Lane<D, T, kNext>;
  using R = Ring<D, sizeof(T), sizeof(G)>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ typename R::Shared shared;
  R::set_up(a, shared);
  grid_wait();  // (as the forward)
  const Part part(a, L::kRows);
  const RopeRows& to = part.k ? a.dk : a.dq;
  R ring(a, part, part.k ? a.k : a.q, part.k ? a.ko : a.qo, smem, shared);
  ring.start();
  const L me(a);
  const int64_t to_step = L::kRows * to.sh;
  float2 wu[2], wv[2], accu[2], accv[2];
  me.weights(a, part.k ? a.wk : a.wq, wu, wv);
#pragma unroll
  for (int i = 0; i < 2; ++i) accu[i] = accv[i] = make_float2(0.f, 0.f);
  bool ran_out = false;
  for (int token = part.token; token < a.tokens && !ran_out; token += part.stride) {
    const int b = token / a.S, s = token - b * a.S;
    T* dest = static_cast<T*>(to.p) + row_at(to, b, s, part.first + me.r);
    float2 c[2], sn[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[i] = make_float2(1.f, 1.f);
      sn[i] = make_float2(0.f, 0.f);
    }
    if (a.pairs) me.angles(a.pos + b * a.pos_sb + static_cast<int64_t>(s) * a.axes, c, sn);
    for (int head = part.first; head < part.last; head += R::kBatch) {
      const uint8_t* rows = ring.batch();
      if (!rows) {
        ran_out = true;
        break;
      }
#pragma unroll
      for (int i = 0; i < R::kSteps; ++i) {
        if (head + i * L::kRows >= part.last) break;
        const bool real = head + i * L::kRows + me.r < part.last;
        Raw<T> rx = {};
        Raw<G> rg = {};
        if (real) {
          rg.load(reinterpret_cast<const G*>(rows + R::kA) + (i * L::kRows + me.r) * D, me.e0, me.e1, kNext);
          if (a.norm) rx.load(reinterpret_cast<const T*>(rows) + (i * L::kRows + me.r) * D, me.e0, me.e1, kNext);
        }
        float2 u[2], v[2], gu[2], gv[2];
        rg.template get<kNext>(gu, gv);
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // back
          float2 cu = gu[j], cv = gv[j];
          me.across(cu, cv, 0.f);
          gu[j] = fma2(gu[j], c[j], mul2(cv, sn[j]));
          gv[j] = fma2(gv[j], c[j], mul2(cu, make_float2(-sn[j].x, -sn[j].y)));
        }
        if (kTiny || a.norm) {
          rx.template get<kNext>(u, v);
          const float by = kTiny ? L::nearer(u, v, a.eps) : 1.f;
          const float2 sq2 = fma2(v[1], v[1], fma2(v[0], v[0], fma2(u[1], u[1], mul2(u[0], u[0]))));
          float2 dot2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 2; ++j) dot2 = fma2(mul2(gv[j], wv[j]), v[j], fma2(mul2(gu[j], wu[j]), u[j], dot2));
          float sq = sq2.x + sq2.y, dot = dot2.x + dot2.y;
#pragma unroll
          for (int o = L::kLanes / 2; o > 0; o >>= 1) {
            sq += __shfl_xor_sync(0xffffffffu, sq, o);
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
          }
          const float n = real ? rsqrtf(fmaf(sq, 1.f / D, kTiny ? a.eps * by * by : a.eps)) : 0.f;  // (0 with eps = 0 adds nothing)
          const float back = -dot * n * n * (1.f / D);  // times x: - x r mean(g w x r)
          const float2 nn = twice(n), bb = twice(back);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            accu[j] = fma2(gu[j], mul2(u[j], nn), accu[j]);
            accv[j] = fma2(gv[j], mul2(v[j], nn), accv[j]);
            gu[j] = mul2(nn, fma2(gu[j], wu[j], mul2(u[j], bb)));
            gv[j] = mul2(nn, fma2(gv[j], wv[j], mul2(v[j], bb)));
            if constexpr (kTiny) {
              gu[j] = mul2(gu[j], twice(by));
              gv[j] = mul2(gv[j], twice(by));
            }
          }
        }
        if (real) Raw<T>::template store<kNext>(dest, me.e0, me.e1, gu, gv);
        dest += to_step;
      }
      ring.done();
    }
  }
  if (ran_out) ring.drain();
  if (!a.partial) return;
  // ---- this CTA's part of its weight's gradient, in a fixed order ----
  __shared__ float sums[kRopeWarps][D];
  float acc[8];
  together<kNext>(accu, accv, acc);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int o = L::kLanes; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    if (me.r == 0) sums[threadIdx.x >> 5][me.element(j)] = acc[j];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kRopeWarps; ++w) x += sums[w][threadIdx.x];
    a.partial[static_cast<int64_t>(blockIdx.x) * D + threadIdx.x] = x;
  }
}

// Sums the CTAs' parts of the weights' gradients (none: 0): 32 columns a CTA, 32 parts at a time.
__global__ void __launch_bounds__(1024) rope_weights_kernel(const float* partial, int groups, int parts, int parts_q, int D,
                                                            float* dwq, float* dwk) {
  __shared__ float sums[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, of_k = blockIdx.x * 32 >= D;
  const int col = blockIdx.x * 32 - of_k * D + x, first = of_k ? parts_q : 0, n = of_k ? parts - parts_q : parts_q;
  grid_wait();
  float sum = 0.f;
#pragma unroll 4
  for (int i = y; i < groups * n; i += 32) {
    const int group = i / n;
    sum += partial[static_cast<int64_t>(group * parts + first + i - group * n) * D + col];
  }
  sums[y][x] = sum;
  __syncthreads();
  sum = sums[x][y];  // a warp per column
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  float* to = of_k ? dwk : dwq;
  if (x == 0 && to) to[blockIdx.x * 32 - of_k * D + y] = sum;
}

// Parts of a token and CTAs of a launch. Many short parts fill the device when
// tokens are few; long ones share a token's angles. q's and k's parts should be of
// the same length, since the CTAs take equal numbers of tokens.
int plan(RopeArgs& a, int D, int sms, int per_sm) {
  const int rows = 256 / D, nq = (a.H + rows - 1) / rows, nk = (a.Hkv + rows - 1) / rows;
  const int64_t warps = static_cast<int64_t>(sms) * per_sm * kRopeWarps;
  const int64_t fill = (nq + nk) * static_cast<int64_t>(a.tokens) / warps;  // steps a warp if all are equal
  const int most = fill < 1 ? 1 : fill < kRopeSteps ? static_cast<int>(fill) : kRopeSteps;
  double least = 0;
  for (int per = most; per >= 1 && 2 * per >= most; --per) {
    int pq = (nq + per - 1) / per, pk = (nk + per - 1) / per;
    if (pq > kRopeCtas / 4) pq = kRopeCtas / 4;
    if (pk > kRopeCtas / 4) pk = kRopeCtas / 4;
    const int longest = std::max((nq + pq - 1) / pq, pk ? (nk + pk - 1) / pk : 0);
    const double cost = static_cast<double>(pq + pk) * (longest + 1.5);  // an angle costs some 1.5 steps
    if (per == most || cost < least) {
      least = cost;
      a.parts_q = pq;
      a.parts = pq + pk;
    }
  }
  const int needed = (a.tokens + kRopeWarps - 1) / kRopeWarps, room = std::max(1, std::min(kRopeCtas, sms * per_sm) / a.parts);
  return std::min(needed, room) * a.parts;
}

template <auto kKernel, int kSmem>
cudaError_t launch(const RopeArgs& a, int ctas, cudaStream_t s) {
  const cudaError_t e = allow_smem<kKernel>(kSmem);
  return e != cudaSuccess ? e : launch_clusters(kKernel, ctas, 1, 1, 1, kThreads, kSmem, true, s, a);
}

// Squares below 2^-126 lose what is below 2^-150: nothing beside an eps of 2^-110.
bool tiny(const RopeArgs& a) { return a.norm && a.eps < 0x1p-110f; }

template <int D, typename T>
cudaError_t fwd(RopeArgs& a, bool next, int sms, cudaStream_t s) {
  const int ctas = plan(a, D, sms, kFwdCtas);
  constexpr int kSmem = Ring<D, sizeof(T), 0>::kSmem;
  if (tiny(a))
    return next ? launch<rope_fwd_kernel<D, T, true, true>, kSmem>(a, ctas, s)
                : launch<rope_fwd_kernel<D, T, false, true>, kSmem>(a, ctas, s);
  return next ? launch<rope_fwd_kernel<D, T, true, false>, kSmem>(a, ctas, s)
              : launch<rope_fwd_kernel<D, T, false, false>, kSmem>(a, ctas, s);
}

template <int D, typename T, typename G>
cudaError_t bwd(RopeArgs& a, bool next, int sms, cudaStream_t s) {
  int ctas = 0;
  a.parts = 1;
  cudaError_t e = cudaSuccess;
  if (a.tokens > 0) {
    ctas = plan(a, D, sms, kBwdCtas);
    constexpr int kSmem = Ring<D, sizeof(T), sizeof(G)>::kSmem;
    if (tiny(a))
      e = next ? launch<rope_bwd_kernel<D, T, G, true, true>, kSmem>(a, ctas, s)
               : launch<rope_bwd_kernel<D, T, G, false, true>, kSmem>(a, ctas, s);
    else
      e = next ? launch<rope_bwd_kernel<D, T, G, true, false>, kSmem>(a, ctas, s)
               : launch<rope_bwd_kernel<D, T, G, false, false>, kSmem>(a, ctas, s);
  }
  if (e != cudaSuccess || !a.partial) return e;
  return launch_clusters(rope_weights_kernel, 2 * D / 32, 1, 1, 1, 1024, 0, true, s, static_cast<const float*>(a.partial),
                         ctas / a.parts, a.parts, a.parts_q, D, a.dwq, a.dwk);
}

}  // namespace

cudaError_t launch_rope_fwd(RopeArgs& a, int D, bool bf16, bool interleaved, int sms, cudaStream_t s) {
  if (D == 64) return bf16 ? fwd<64, __nv_bfloat16>(a, interleaved, sms, s) : fwd<64, float>(a, interleaved, sms, s);
  return bf16 ? fwd<128, __nv_bfloat16>(a, interleaved, sms, s) : fwd<128, float>(a, interleaved, sms, s);
}

cudaError_t launch_rope_bwd(RopeArgs& a, int D, bool bf16, bool g_f32, bool interleaved, int sms, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (!bf16) return D == 64 ? bwd<64, float, float>(a, interleaved, sms, s) : bwd<128, float, float>(a, interleaved, sms, s);
  if (g_f32) return D == 64 ? bwd<64, B, float>(a, interleaved, sms, s) : bwd<128, B, float>(a, interleaved, sms, s);
  return D == 64 ? bwd<64, B, B>(a, interleaved, sms, s) : bwd<128, B, B>(a, interleaved, sms, s);
}

}  // namespace cp
