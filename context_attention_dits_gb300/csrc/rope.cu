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
// Every value is read once and written once and costs some ten operations, so
// HBM bounds the long calls (2 or 3 streams) and the launch the short ones. A
// row lies in D / 8 lanes, 8 values each: its sums take 3 or 4 shuffles, and a
// lane holds both members of its four pairs, by one 16-byte piece where pairs
// are neighbours and two pieces of 8 where they are the row's halves. A warp
// walks the heads of one token, so an angle is formed once for all of them, each
// pair by one lane and handed round by shuffles.
//
// An angle of radians in fp32 is worth nothing far out (half a radian at position
// 2^23). It is kept in turns instead, as 64-bit fixed point: u = f 2^64 / 2 pi,
// whole turns dropped, and position u is exact but for what u itself is off,
// half of 2^-64 or so of a turn, times the position.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cp_ptx.cuh"
#include "cp_rope.h"

namespace cp {
namespace {

constexpr int kThreads = kRopeWarps * 32;

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

// Rows are touched once: past L1. (Not the read-only path: a row may be
// overwritten in place by the threads that have read it.)
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}

// A lane's 8 values of a row as they lie in memory: 4 from element e0, 4 from e1.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int e0, int e1, bool one) {
    if (one) {
      const uint4 v = ld16(row + e0);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 x = ld8(row + e0), y = ld8(row + e1);
      w[0] = x.x, w[1] = x.y, w[2] = y.x, w[3] = y.y;
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* row, int e0, int e1, bool one, const float (&x)[8]) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    if (one) {
      *reinterpret_cast<uint4*>(row + e0) = make_uint4(v[0], v[1], v[2], v[3]);
    } else {
      *reinterpret_cast<uint2*>(row + e0) = make_uint2(v[0], v[1]);
      *reinterpret_cast<uint2*>(row + e1) = make_uint2(v[2], v[3]);
    }
  }
};
template <>
struct Raw<float> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const float* row, int e0, int e1, bool) {
    const uint4 x = ld16(row + e0), y = ld16(row + e1);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
  static __device__ __forceinline__ void store(float* row, int e0, int e1, bool, const float (&x)[8]) {
    *reinterpret_cast<float4*>(row + e0) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(row + e1) = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// The four pairs of 8 values turned by (c, s): neighbours, or the two fours against each other.
template <bool kNext>
__device__ __forceinline__ void rotate(float (&x)[8], const float (&c)[4], const float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float &u = x[kNext ? 2 * i : i], &v = x[kNext ? 2 * i + 1 : 4 + i];
    const float y = fmaf(u, c[i], -v * s[i]);
    v = fmaf(u, s[i], v * c[i]);
    u = y;
  }
}

// What a lane is: its place in its row, its values, its weights and its own pairs' steps.
template <int D, typename T, bool kNext>
struct Lane {
  static constexpr int kLanes = D / 8;           // of a row
  static constexpr int kRows = 32 / kLanes;      // of a warp
  static constexpr int kOwn = 4 / kRows;         // pairs whose angle this lane forms
  int l, r, e0, e1;
  uint64_t step[kOwn];
  int axis[kOwn];

  __device__ __forceinline__ explicit Lane(const RopeArgs& a) {
    const int lane = threadIdx.x & 31;
    l = lane % kLanes;
    r = lane / kLanes;
    // neighbours: 8 values in a row; halves: 4 of each half, behind the pairs 8 in a row
    const int with = a.pairs / 4;  // lanes with pairs
    e0 = kNext ? 8 * l : l < with ? 4 * l : 2 * a.pairs + 8 * (l - with);
    e1 = kNext || l >= with ? e0 + 4 : a.pairs + 4 * l;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int p = 4 * l + r * kOwn + i;
      step[i] = p < a.pairs ? turn_step(a.freqs[p]) : 0;
      axis[i] = p < a.pairs ? a.axis[p] : 0;
    }
  }
  // cos and sin of the lane's four pairs for the token at pos
  __device__ __forceinline__ void angles(const int* pos, float (&c)[4], float (&s)[4]) const {
    float oc[kOwn], os[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) cos_sin(step[i], pos[axis[i]], oc[i], os[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int from = i / kOwn * kLanes + l;
      c[i] = __shfl_sync(0xffffffffu, oc[i % kOwn], from);
      s[i] = __shfl_sync(0xffffffffu, os[i % kOwn], from);
    }
  }
  __device__ __forceinline__ void weights(const RopeArgs& a, const void* w, float (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = j < 4 ? e0 + j : e1 + j - 4;
      x[j] = !w ? 1.f : a.w_f32 ? static_cast<const float*>(w)[e] : static_cast<float>(static_cast<const T*>(w)[e]);
    }
  }
  static __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  }
};

// The row steps of one unit: [q0, q1) of q, [k0, k1) of k, of token (b, s).
struct Unit {
  int b, s, q0, q1, k0, k1;
  __device__ __forceinline__ Unit(const RopeArgs& a, int unit, int rows) {
    const int token = unit / a.parts, part = unit - token * a.parts;
    const int nq = (a.H + rows - 1) / rows, n = nq + (a.Hkv + rows - 1) / rows;
    const int first = part * n / a.parts, last = (part + 1) * n / a.parts;
    b = token / a.S;
    s = token - b * a.S;
    q0 = first;
    q1 = min(last, nq);
    k0 = max(first - nq, 0);
    k1 = last - nq;
  }
};

template <typename T>
__device__ __forceinline__ T* row_of(const RopeRows& x, const Unit& u, int head) {
  return static_cast<T*>(x.p) + u.b * x.sb + u.s * x.ss + head * x.sh;
}

template <int D, typename T, bool kNext>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const __grid_constant__ RopeArgs a) {
  using L = Lane<D, T, kNext>;
  constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;  // rows whose loads are under way at once
  const L me(a);
  float wq[8], wk[8];
  me.weights(a, a.wq, wq);
  me.weights(a, a.wk, wk);
  const int units = a.tokens * a.parts, stride = gridDim.x * kRopeWarps;
  for (int unit = blockIdx.x * kRopeWarps + (threadIdx.x >> 5); unit < units; unit += stride) {
    const Unit u(a, unit, L::kRows);
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.pairs) me.angles(a.pos + u.b * a.pos_sb + static_cast<int64_t>(u.s) * a.axes, c, s);
    auto rows = [&](const RopeRows& in, const RopeRows& to, const float (&w)[8], int heads, int first, int last) {
      for (int at = first; at < last; at += kAhead) {
        Raw<T> raw[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int h = (at + i) * L::kRows + me.r;
          if (at + i < last && h < heads)
            raw[i].load(row_of<T>(in, u, h), me.e0, me.e1, kNext);
          else
            raw[i] = {};
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (at + i >= last) break;
          const int h = (at + i) * L::kRows + me.r;
          float x[8];
          raw[i].get(x);
          if (a.norm) {
            float sq = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = fmaf(x[j], x[j], sq);
            const float n = rsqrtf(fmaf(L::row_sum(sq), 1.f / D, a.eps));
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= n * w[j];
          }
          rotate<kNext>(x, c, s);
          if (h < heads) Raw<T>::store(row_of<T>(to, u, h), me.e0, me.e1, kNext, x);
        }
      }
    };
    rows(a.q, a.qo, wq, a.H, u.q0, u.q1);
    rows(a.k, a.ko, wk, a.Hkv, u.k0, u.k1);
  }
}

template <int D, typename T, typename G, bool kNext>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
  using L = Lane<D, T, kNext>;
  constexpr int kAhead = 2;
  const L me(a);
  float wq[8], wk[8], aq[8], ak[8];
  me.weights(a, a.wq, wq);
  me.weights(a, a.wk, wk);
#pragma unroll
  for (int j = 0; j < 8; ++j) aq[j] = ak[j] = 0.f;
  const int units = a.tokens * a.parts, stride = gridDim.x * kRopeWarps;
  for (int unit = blockIdx.x * kRopeWarps + (threadIdx.x >> 5); unit < units; unit += stride) {
    const Unit u(a, unit, L::kRows);
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.pairs) me.angles(a.pos + u.b * a.pos_sb + static_cast<int64_t>(u.s) * a.axes, c, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = -s[i];  // back
    auto rows = [&](const RopeRows& in, const RopeRows& grad, const RopeRows& to, const float (&w)[8], float (&acc)[8],
                    int heads, int first, int last) {
      for (int at = first; at < last; at += kAhead) {
        Raw<T> rx[kAhead];
        Raw<G> rg[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int h = (at + i) * L::kRows + me.r;
          rx[i] = {};
          rg[i] = {};
          if (at + i < last && h < heads) {
            rg[i].load(row_of<G>(grad, u, h), me.e0, me.e1, kNext);
            if (a.norm) rx[i].load(row_of<T>(in, u, h), me.e0, me.e1, kNext);
          }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (at + i >= last) break;
          const int h = (at + i) * L::kRows + me.r;
          float x[8], g[8];
          rg[i].get(g);
          rotate<kNext>(g, c, s);
          if (a.norm) {
            rx[i].get(x);
            float sq = 0.f, dot = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              sq = fmaf(x[j], x[j], sq);
              dot = fmaf(g[j] * w[j], x[j], dot);
            }
            sq = L::row_sum(sq);
            dot = L::row_sum(dot);
            const float n = h < heads ? rsqrtf(fmaf(sq, 1.f / D, a.eps)) : 0.f;  // (0 with eps = 0 adds nothing)
            const float back = dot * n * n * (1.f / D);  // times x: x r mean(g w x r)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              acc[j] = fmaf(g[j], x[j] * n, acc[j]);
              g[j] = n * fmaf(g[j], w[j], -x[j] * back);
            }
          }
          if (h < heads) Raw<T>::store(row_of<T>(to, u, h), me.e0, me.e1, kNext, g);
        }
      }
    };
    rows(a.q, a.qo, a.dq, wq, aq, a.H, u.q0, u.q1);
    rows(a.k, a.ko, a.dk, wk, ak, a.Hkv, u.k0, u.k1);
  }
  if (!a.partial) return;
  // ---- this CTA's part of the weights' gradients, in a fixed order ----
  __shared__ float sums[kRopeWarps][2][D];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int o = L::kLanes; o < 32; o <<= 1) {
      aq[j] += __shfl_xor_sync(0xffffffffu, aq[j], o);
      ak[j] += __shfl_xor_sync(0xffffffffu, ak[j], o);
    }
    const int e = j < 4 ? me.e0 + j : me.e1 + j - 4;
    if (me.r == 0) {
      sums[threadIdx.x >> 5][0][e] = aq[j];
      sums[threadIdx.x >> 5][1][e] = ak[j];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kRopeWarps; ++w) x += sums[w][i / D][i % D];
    a.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = x;
  }
}

// Sums the CTAs' parts of the weights' gradients (none: 0): 32 columns a CTA, 32 rows at a time.
__global__ void __launch_bounds__(1024) rope_weights_kernel(const float* partial, int ctas, int D, float* dwq, float* dwk) {
  __shared__ float sums[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + x;
  grid_wait();
  float sum = 0.f;
#pragma unroll 4
  for (int i = y; i < ctas; i += 32) sum += partial[static_cast<int64_t>(i) * 2 * D + col];
  sums[y][x] = sum;
  __syncthreads();
  sum = sums[x][y];  // a warp per column
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int of = blockIdx.x * 32 + y;
  float* to = of < D ? dwq : dwk;
  if (x == 0 && to) to[of % D] = sum;
}

// Parts of a token and CTAs of a launch. One unit is a warp's; many parts fill
// the device when tokens are few, few parts share a token's angles.
int plan(RopeArgs& a, int D, int sms, int per_sm) {
  const int steps = rope_steps(D, a.H, a.Hkv);
  const int64_t want = static_cast<int64_t>(sms) * per_sm * kRopeWarps * 2;
  const int64_t parts = (want + a.tokens - 1) / a.tokens;
  a.parts = static_cast<int>(parts < steps ? parts : steps);
  const int64_t ctas = (static_cast<int64_t>(a.tokens) * a.parts + kRopeWarps - 1) / kRopeWarps;
  const int most = sms * per_sm;
  return static_cast<int>(ctas < most ? ctas : most);
}

template <typename... P>
cudaError_t launch(void (*kernel)(P...), const RopeArgs& a, int ctas, cudaStream_t s) {
  kernel<<<ctas, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <int D, typename T>
cudaError_t fwd(RopeArgs& a, bool next, int sms, cudaStream_t s) {
  const int ctas = plan(a, D, sms, 4);
  return next ? launch(rope_fwd_kernel<D, T, true>, a, ctas, s) : launch(rope_fwd_kernel<D, T, false>, a, ctas, s);
}

template <int D, typename T, typename G>
cudaError_t bwd(RopeArgs& a, bool next, int sms, cudaStream_t s) {
  int ctas = 0;
  cudaError_t e = cudaSuccess;
  if (a.tokens > 0) {
    ctas = plan(a, D, sms < 152 ? sms : 152, 2);
    e = next ? launch(rope_bwd_kernel<D, T, G, true>, a, ctas, s) : launch(rope_bwd_kernel<D, T, G, false>, a, ctas, s);
  }
  if (e != cudaSuccess || !a.partial) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // prepared while the main kernel runs
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_weights_kernel, static_cast<const float*>(a.partial), ctas, D, a.dwq, a.dwk);
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
