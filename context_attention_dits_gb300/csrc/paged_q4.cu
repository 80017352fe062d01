// paged_q4.cu — the paged key/value cache in 4 bits: rows of new tokens written
// as codes, rows read back as values, and attention of one new token per sequence.
//
// A row (one token, one head, D values) is cut into groups of 64. A group is held
// as 64 codes c of 4 bits, a scale s and an offset z (bf16) and stands for z + s c:
//   z = the largest bf16 number not above the group's values
//   s = the smallest bf16 number not below (largest value - z) / 15 and 2^-100
//   c = min(15, floor((x - z) / s + 1/2))
// exactly, so that codes do not depend on how they are computed. A page holds the
// rows of one head after another, so that a warp's 32 keys are two contiguous
// pieces (codes, scales), or four in pages of 16 rows.
//
// The attention never forms z + s c. With x = q.k and p the weights,
//   x_j = sum over groups of s_j (q.c_j) + z_j (sum of q)
//   out = sum_j p_j s_j (c_j - 8) + sum_j p_j (z_j + 8 s_j)
// so that codes go to the matrix instructions as they are, 4-bit integers being
// exact in fp16, and scales meet only scores and weights, one number a key.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "cp_ptx.cuh"
#include "cp_score.h"
#include "paged_decode.cuh"

namespace cp {
namespace {

// The page of token pos of sequence b, or -1 (and the error word) if it is out of range.
__device__ __forceinline__ int page_of(const PagedArgs& a, int b, int pos) {
  const int id = a.table[static_cast<int64_t>(b) * a.max_pages + (pos >> a.page_shift)];
  if (id >= 0 && id < a.num_pages) return id;
  atomicOr(a.err, kDevErrPage);
  return -1;
}
// The row of head hk of the token that lies at `pos` in its sequence, counted in rows of one head.
__device__ __forceinline__ int64_t head_row(const PagedArgs& a, int page, int pos, int hk) {
  return ((static_cast<int64_t>(page) * a.Hkv + hk) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

// ----------------------------------------------------------------------------
// Append and read. A lane has 8 values of a row, 8 lanes a group: its least and
// largest value take three shuffles each.
// ----------------------------------------------------------------------------
constexpr int kRowThreads = 256;

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// a - b = h + l exactly.
__device__ __forceinline__ void exact_diff(float a, float b, float& h, float& l) {
  h = __fsub_rn(a, b);
  const float bb = __fsub_rn(h, a);
  l = __fsub_rn(__fsub_rn(a, __fsub_rn(h, bb)), __fadd_rn(b, bb));
}

// This lane's 8 codes (value i in bits 4 i) and its group's scale and offset (bf16,
// scale in the lower half), from the 8 lanes that share the group.
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint32_t& scale) {
  float least = x[0], most = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    least = min_nan(least, x[i]);
    most = max_nan(most, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    least = min_nan(least, __shfl_xor_sync(0xffffffffu, least, o));
    most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  const uint32_t lb = __float_as_uint(least), low = lb & 0xffffu;
  const float z = __uint_as_float(lb - low + (low && lb >> 31 ? 0x10000u : 0u));
  float h, l;
  exact_diff(most, z, h, l);
  if (!(fabsf(h) <= FLT_MAX)) {  // a value that is not finite, or a span that fp32 does not hold
    scale = 0x7fff7fffu;         // reads back as NaN
    return 0;
  }
  float s = __uint_as_float(__float_as_uint(__fdiv_rn(h, 15.f)) & 0xffff0000u);
  if (__fsub_rn(15.f * s, h) < l) s = __uint_as_float(__float_as_uint(s) + 0x10000u);  // both sides exact
  s = fmaxf(s, 0x1p-100f);
  scale = __float_as_uint(s) >> 16 | __float_as_uint(z);
  // The nearest integer, by a sum whose unit is 1: right unless the quotient, off by
  // 2^-19 at most, is next to a border.
  constexpr float kOne = 12582912.f;  // 1.5 2^23
  const float rs = __frcp_rn(s);
  uint32_t codes = 0;
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = __fsub_rn(x[i], z), g = fmaf(d, rs, kOne);
    far = fmaxf(far, fabsf(fmaf(d, rs, -__fsub_rn(g, kOne))));
    codes += __float_as_uint(g) << (4 * i);
  }
  codes -= 0x3f400000u;  // what the eight copies of kOne's bits, 0x4b400000, come to in 32 bits
  if (far > 0.5f - 0x1p-17f) {
    codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      exact_diff(x[i], z, h, l);
      int n = static_cast<int>(fminf(fmaf(h, rs, 0.5f), 15.f));
      if (n > 0 && __fadd_rn(__fsub_rn(h, (n - 0.5f) * s), l) < 0.f) --n;
      else if (n < 15 && __fadd_rn(__fsub_rn(h, (n + 0.5f) * s), l) >= 0.f) ++n;
      codes |= static_cast<uint32_t>(n) << (4 * i);
    }
  }
  return codes;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// Rows (token, head) of sequence blockIdx.y: a warp takes 256 / D of them.
template <int D, typename T>
__global__ void __launch_bounds__(kRowThreads) q4_append_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int kLanes = D / 8;
  const int b = blockIdx.y, l = threadIdx.x % kLanes;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kRowThreads / kLanes) + threadIdx.x / kLanes;
  const int64_t most = static_cast<int64_t>(a.T) * a.Hkv;
  const bool in = row < most;  // (lanes stay for the shuffles)
  const int t = static_cast<int>((in ? row : 0) / a.Hkv), hk = static_cast<int>((in ? row : 0) - static_cast<int64_t>(t) * a.Hkv);
  const int n = a.seq_lens[b];
  const bool live = in && !(a.new_lens && t >= a.new_lens[b]);
  float k[8] = {}, v[8] = {};
  if (live) {  // on their way before the row's place is looked up
    const int64_t at = (static_cast<int64_t>(b) * most + row) * D + l * 8;
    load8(static_cast<const T*>(a.k_new) + at, k);
    load8(static_cast<const T*>(a.v_new) + at, v);
  }
  const uint32_t pos = static_cast<uint32_t>(n) + static_cast<uint32_t>(t);  // (both below 2^31)
  int page = -1;
  if (live) {
    if (n < 0 || pos >= a.positions)
      atomicOr(a.err, kDevErrPage);
    else
      page = page_of(a, b, static_cast<int>(pos));
  }
  uint32_t ks, vs;
  const uint32_t kc = quantise(k, ks), vc = quantise(v, vs);
  if (page < 0) return;
  const int64_t dst = head_row(a, page, static_cast<int>(pos), hk);
  static_cast<uint32_t*>(a.k_cache)[dst * kLanes + l] = kc;
  static_cast<uint32_t*>(a.v_cache)[dst * kLanes + l] = vc;
  if (l % 8 == 0) {
    static_cast<uint32_t*>(a.k_scales)[dst * (D / kQ4Group) + l / 8] = ks;
    static_cast<uint32_t*>(a.v_scales)[dst * (D / kQ4Group) + l / 8] = vs;
  }
}

// Eight codes as values.
__device__ __forceinline__ void values8(uint32_t codes, uint32_t scale, float (&x)[8]) {
  const float s = __uint_as_float(scale << 16), z = __uint_as_float(scale & 0xffff0000u);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(s, static_cast<float>(codes >> (4 * i) & 15u), z);
}

// Rows (token, head) of sequence blockIdx.y: a warp takes kAhead times 256 / D, all
// of whose loads are under way at once (length, page, codes: one after the other).
template <int D, typename T>
__global__ void __launch_bounds__(kRowThreads) q4_read_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int kLanes = D / 8, kAhead = 4, kRows = kRowThreads / kLanes;
  const int b = blockIdx.y, l = threadIdx.x % kLanes;
  const int64_t most = static_cast<int64_t>(a.T) * a.Hkv;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kRows * kAhead) + threadIdx.x / kLanes;
  const int n = seq_len(a, b);
  uint32_t kc[kAhead], vc[kAhead], ks[kAhead], vs[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int64_t row = first + i * kRows;
    kc[i] = vc[i] = ks[i] = vs[i] = 0;
    if (row >= most) continue;
    const int t = static_cast<int>(row / a.Hkv), hk = static_cast<int>(row - static_cast<int64_t>(t) * a.Hkv);
    const int page = t < n ? page_of(a, b, t) : -1;
    if (page < 0) continue;
    const int64_t src = head_row(a, page, t, hk);
    kc[i] = static_cast<const uint32_t*>(a.k_cache)[src * kLanes + l];
    vc[i] = static_cast<const uint32_t*>(a.v_cache)[src * kLanes + l];
    ks[i] = static_cast<const uint32_t*>(a.k_scales)[src * (D / kQ4Group) + l / 8];
    vs[i] = static_cast<const uint32_t*>(a.v_scales)[src * (D / kQ4Group) + l / 8];
  }
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int64_t row = first + i * kRows;
    if (row >= most) break;
    const int64_t at = (static_cast<int64_t>(b) * most + row) * D + l * 8;
    float x[8];
    values8(kc[i], ks[i], x);
    store8(static_cast<T*>(a.k_out) + at, x);
    values8(vc[i], vs[i], x);
    store8(static_cast<T*>(a.v_out) + at, x);
  }
}

// ----------------------------------------------------------------------------
// Decode
// ----------------------------------------------------------------------------
constexpr int kChunk = 32;  // keys of a warp and step
static_assert(kChunk * kDecWarps == kQ4Block, "a block is a chunk of each warp");

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 tile of 16-bit numbers, two neighbours of a row in each lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t x) { return __half22float2(*reinterpret_cast<__half2*>(&x)); }
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Two codes (bits 0..3 of each half, or 4..7: kHigh) as fp16 numbers c - 8.
template <bool kHigh>
__device__ __forceinline__ uint32_t centred(uint32_t w) {
  uint32_t x;
  if (!kHigh) {  // 1024 + c
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(x) : "r"(w));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(0x64086408u));  // 1032
  } else {  // 1024 + 16 c
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(x) : "r"(w));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(x) : "r"(x), "r"(0x2c002c00u), "r"(0xd480d480u));  // / 16, - 72
  }
  return x;
}

// bf16 queries: one fp16 part of q and of the weights. fp32 ones: two of each, whose
// products leave 2^-22 out.
template <int D_, bool kF32, int kTiles>
struct Q4Unit {
  static constexpr int kD = D_, kRows = 8 * kTiles, kBlock = kQ4Block, kPerSm = q4_per_sm(!kF32, kRows);
  static constexpr int kGroups = D_ / kQ4Group, kParts = kF32 ? 2 : 1;
  static constexpr int kRowB = D_ / 2, kScaleB = kGroups * 4;  // a row's codes and scales
  static constexpr int kCodes = kChunk * kRowB, kScales = kChunk * kScaleB, kStage = 2 * (kCodes + kScales);
  static constexpr int kStages = 2;
  static constexpr int kState = kRows * (D_ + 2);
  static constexpr int kWarpB = (kStages * kStage > 2 * kState * 4 ? kStages * kStage : 2 * kState * 4) + 127 & ~127;
  static constexpr int kSmem = kDecWarps * kWarpB;
  struct Shared {
    uint64_t full[kDecWarps][kStages];
    uint32_t have[kDecWarps][kStages];  // the keys that a stage holds, a bit each
    uint32_t abort;
  };

  // stage and phase of the next chunk to ask for and to take
  int ask = 0, take = 0;
  uint32_t phase = 0;

  __device__ __forceinline__ Q4Unit(const PagedArgs& a, uint8_t*, Shared& sh) {
    if (threadIdx.x < kDecWarps * kStages)
      mbar_init(smem_addr(&sh.full[0][0] + threadIdx.x), a.page_shift >= 5 ? 4 : 8);
    if (threadIdx.x == 0) sh.abort = 0;
    fence_mbar_init();
    fence_async();
    __syncthreads();
  }

  __device__ __forceinline__ void run(const PagedArgs& a, int b, int n, int hk, int hg, int blk0, int blk1, uint8_t* smem,
                                      Shared& sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
    uint8_t* wbuf = smem + warp * kWarpB;
    const int h0 = hk * a.G + hg * kRows, nrow = min(kRows, a.G - hg * kRows);
    // this warp's chunks: keys (4 blk + warp) 32 on, the last below n
    const int last = min(blk1, n > warp * kChunk ? (n - warp * kChunk + kQ4Block - 1) / kQ4Block : 0);
    const int pieces = a.page_shift >= 5 ? 4 : 8;  // codes and scales of k and v, twice where pages are of 16 rows
    const int rows = a.page_shift >= 5 ? 32 : 16;

    // ---- loads: a lane a piece ----
    const int which = lane & 3, half = lane >> 2;  // k codes, k scales, v codes, v scales
    const uint8_t* base = static_cast<const uint8_t*>(which == 0   ? a.k_cache
                                                      : which == 1 ? a.k_scales
                                                      : which == 2 ? a.v_cache
                                                                   : a.v_scales);
    const int row_b = which & 1 ? kScaleB : kRowB;
    const uint32_t off = (which & 2 ? kCodes + kScales : 0) + (which & 1 ? kCodes : 0) + half * rows * row_b;
    auto find = [&](int blk) {
      const int pos = (blk * kDecWarps + warp) * kChunk + half * 16;
      const int page = lane < pieces && blk < last && pos < n ? page_of(a, b, pos) : -1;
      __syncwarp();
      return page;
    };
    auto load = [&](int blk, int page) {
      const int pos = (blk * kDecWarps + warp) * kChunk + half * 16;
      const uint32_t found = __ballot_sync(0xffffffffu, page >= 0);
      if (lane == 0) {
        uint32_t on = (found & 1u ? 0xffffu : 0u) | (found & (pieces == 8 ? 16u : 1u) ? 0xffff0000u : 0u);
        const int rest = n - pos;  // keys from here on
        if (rest < 32) on &= (1u << rest) - 1;
        sh.have[warp][ask] = on;
      }
      if (lane < pieces) {
        const uint32_t bar = smem_addr(&sh.full[warp][ask]), bytes = rows * row_b;
        mbar_arrive_expect_tx(bar, page >= 0 ? bytes : 0);
        if (page >= 0)
          bulk_g2s(smem_addr(wbuf) + ask * kStage + off, base + head_row(a, page, pos, hk) * row_b, bytes, bar);
      }
      if (++ask == kStages) ask = 0;
      __syncwarp();
    };
    fence_async();  // (what was read and written here before, by this and by other warps ahead of the barrier)
    int next = find(blk0), asked = blk0;
    if (!aborted(sh)) {
#pragma unroll
      for (int st = 0; st < kStages - 1; ++st) {
        if (asked < last) load(asked++, next);
        next = find(asked);
      }
    }

    // ---- q: each head's column in fp16, scaled by a power of two so that its largest
    // value lies in [2^14, 2^15); what is below 2^-39 of that is lost ----
    uint32_t qf[kTiles][kGroups][4][kParts][2];  // per step of 16 values
    float undo[kTiles][2], qsum[kTiles][kGroups][2], slope[kTiles][2];
#pragma unroll
    for (int x = 0; x < kTiles; ++x) {
      const int h = x * 8 + g;
      float v[kGroups][16], big = 0.f, sum[kGroups];
#pragma unroll
      for (int y = 0; y < kGroups; ++y) {
        float lo[8] = {}, hi[8] = {};
        if (h < nrow) {
          using T = std::conditional_t<kF32, float, __nv_bfloat16>;
          const T* q = static_cast<const T*>(a.q) + (static_cast<int64_t>(b) * a.H + h0 + h) * kD + y * kQ4Group + tq * 16;
          load8(q, lo);
          load8(q + 8, hi);
        }
        sum[y] = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          v[y][i] = i < 8 ? lo[i & 7] : hi[i & 7];
          big = fmaxf(big, fabsf(v[y][i]));
          sum[y] += v[y][i];
        }
        sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 1);
        sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 2);
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      const int e = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -100), 100);
#pragma unroll
      for (int y = 0; y < kGroups; ++y)
#pragma unroll
        for (int st = 0; st < 4; ++st)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            // codes i and i + 4 of a word of 8; those of odd i come times 16
            const int i = (st >> 1) * 8 + (st & 1) * 2 + r;
            const float up = power_of_2(r ? 10 - e : 14 - e), lo = v[y][i] * up, hi = v[y][i + 4] * up;
            qf[x][y][st][0][r] = pack_f16x2(lo, hi);
            if constexpr (kF32) {
              const float2 have = unpack_f16x2(qf[x][y][st][0][r]);
              qf[x][y][st][1][r] = pack_f16x2(lo - have.x, hi - have.y);
            }
          }
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // the columns of this lane's scores: heads 2 tq, 2 tq + 1
        const int from = (2 * tq + c) * 4, hc = x * 8 + 2 * tq + c;
        undo[x][c] = power_of_2(__shfl_sync(0xffffffffu, e, from) + 10);  // of 2^(14 - e), and 2^-24 of the codes
#pragma unroll
        for (int y = 0; y < kGroups; ++y) qsum[x][y][c] = __shfl_sync(0xffffffffu, sum[y], from);
        slope[x][c] = a.slopes && hc < nrow ? a.slopes[h0 + hc] * kL2e : 0.f;
      }
    }

    DecScore score;
    score.scale = a.scale;
    score.cap = a.cap;
    score.inv_cap = a.cap > 0.f ? 1.f / a.cap : 0.f;
    float m[kTiles][2], l[kTiles][2], zs[kTiles][kGroups][2], o[kTiles][kGroups][4][4];
#pragma unroll
    for (int x = 0; x < kTiles; ++x)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[x][c] = -INFINITY;
        l[x][c] = 0.f;
#pragma unroll
        for (int y = 0; y < kGroups; ++y) {
          zs[x][y][c] = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) o[x][y][j][2 * c] = o[x][y][j][2 * c + 1] = 0.f;
        }
      }
    int top = 27;  // exponent (biased) of the largest value scale so far: o is in units of 2^(top - 141)
    // Row r of a 16-key tile is key turn(r): neighbours change places in every other
    // pair, so that the lanes of a quarter that read v's rows differ in parity
    auto turn = [](int r) { return r ^ (r >> 1 & 1); };
    const int kr = turn(g), va = turn(2 * tq), vb = turn(2 * tq + 1);

    for (int blk = blk0; blk < last; ++blk) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&sh.full[warp][take]), phase >> take & 1u, &sh.abort, a.err,
                                                     a.timeout_ns)))
        break;
      if (asked < last) load(asked++, next);  // into the stage that the last step read
      next = find(asked);
      const uint8_t* kt = wbuf + take * kStage;
      const uint8_t *kz = kt + kCodes, *vt = kz + kScales, *vz = vt + kCodes;
      const uint32_t on = sh.have[warp][take];

      // ---- scores, keys as rows: two tiles of 16 ----
      float s[2][kTiles][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float dot[kTiles][kGroups][4];
#pragma unroll
        for (int y = 0; y < kGroups; ++y) {
          const uint2 wa = *reinterpret_cast<const uint2*>(kt + (16 * t + kr) * kRowB + y * 32 + tq * 8);
          const uint2 wb = *reinterpret_cast<const uint2*>(kt + (16 * t + kr + 8) * kRowB + y * 32 + tq * 8);
#pragma unroll
          for (int x = 0; x < kTiles; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) dot[x][y][e] = 0.f;
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            const uint32_t ua = (st >> 1 ? wa.y : wa.x) >> (st & 1 ? 8 : 0), ub = (st >> 1 ? wb.y : wb.x) >> (st & 1 ? 8 : 0);
            // codes as they are: subnormal fp16 numbers, c 2^-24, and 16 c 2^-24
            const uint32_t a0 = ua & 0x000f000fu, a1 = ub & 0x000f000fu, a2 = ua & 0x00f000f0u, a3 = ub & 0x00f000f0u;
#pragma unroll
            for (int x = 0; x < kTiles; ++x)
#pragma unroll
              for (int p = kParts - 1; p >= 0; --p)
                mma_f16(dot[x][y], a0, a1, a2, a3, qf[x][y][st][p][0], qf[x][y][st][p][1]);
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int key = 16 * t + kr + 8 * r;
          const bool there = on >> key & 1u;
          const float dist = static_cast<float>(n - 1 - ((blk * kDecWarps + warp) * kChunk + key));
          float ks[kGroups], kzz[kGroups];
#pragma unroll
          for (int y = 0; y < kGroups; ++y) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(kz + key * kScaleB + y * 4);
            ks[y] = __uint_as_float(w << 16);
            kzz[y] = __uint_as_float(w & 0xffff0000u);
          }
#pragma unroll
          for (int x = 0; x < kTiles; ++x)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float d = ks[0] * dot[x][0][2 * r + c], zq = kzz[0] * qsum[x][0][c];
#pragma unroll
              for (int y = 1; y < kGroups; ++y) {
                d = fmaf(ks[y], dot[x][y][2 * r + c], d);
                zq = fmaf(kzz[y], qsum[x][y][c], zq);
              }
              s[t][x][2 * r + c] = there ? score(fmaf(d, undo[x][c], zq), slope[x][c], dist) : -INFINITY;
            }
        }
      }

      // ---- weights ----
      float f[kTiles][2];
#pragma unroll
      for (int x = 0; x < kTiles; ++x)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(fmaxf(s[0][x][c], s[0][x][2 + c]), fmaxf(s[1][x][c], s[1][x][2 + c]));
#pragma unroll
          for (int of = 4; of < 32; of <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, of));
          const float mn = fmaxf(m[x][c], mx), ref = mn == -INFINITY ? 0.f : mn;
          f[x][c] = kF32 ? exp2f(m[x][c] - ref) : ex2_approx(m[x][c] - ref);
          m[x][c] = mn;
          float sum = 0.f;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float& p = s[t][x][2 * r + c];
              p = kF32 ? exp2f(p - ref) : ex2_approx(p - ref);
              sum += p;
            }
          l[x][c] = fmaf(l[x][c], f[x][c], sum);
        }

      // ---- the values' scales meet the weights: p s in fp16, scaled so that it stays
      // below 2^15; p (z + 8 s) summed as it is ----
      float vs[2][2][kGroups];  // [tile][row]
      uint32_t largest = 0;
#pragma unroll
      for (int x = 0; x < kTiles; ++x)
#pragma unroll
        for (int y = 0; y < kGroups; ++y)
#pragma unroll
          for (int c = 0; c < 2; ++c) zs[x][y][c] *= f[x][c];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int key = 16 * t + kr + 8 * r;
          const bool there = on >> key & 1u;
#pragma unroll
          for (int y = 0; y < kGroups; ++y) {
            uint32_t w = *reinterpret_cast<const uint32_t*>(vz + key * kScaleB + y * 4);
            w = there ? w : 0u;  // (a row that holds no key may hold anything)
            const float sv = __uint_as_float(w << 16), zz = fmaf(8.f, sv, __uint_as_float(w & 0xffff0000u));
            vs[t][r][y] = sv;
            largest = max(largest, w & 0x7fffu);
#pragma unroll
            for (int x = 0; x < kTiles; ++x)
#pragma unroll
              for (int c = 0; c < 2; ++c) zs[x][y][c] = fmaf(s[t][x][2 * r + c], zz, zs[x][y][c]);
          }
        }
      const int now = max(top, static_cast<int>(__reduce_max_sync(0xffffffffu, largest) >> 7));
      if (now != top) {
        const float down = now - top > 126 ? 0.f : power_of_2(top - now);
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
#pragma unroll
          for (int c = 0; c < 2; ++c) f[x][c] *= down;
        top = now;
      }
      const float fit = power_of_2(141 - top);
      uint32_t pf[kTiles][kGroups][2][kParts][2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int y = 0; y < kGroups; ++y) {
            const float sv = vs[t][r][y] * fit;
#pragma unroll
            for (int x = 0; x < kTiles; ++x) {
              const float u = s[t][x][2 * r] * sv, v = s[t][x][2 * r + 1] * sv;
              const uint32_t w = pack_f16x2(u, v);
              pf[x][y][t][0][r] = transpose8(w);
              if constexpr (kF32) {
                const float2 have = unpack_f16x2(w);
                pf[x][y][t][1][r] = transpose8(pack_f16x2(u - have.x, v - have.y));
              }
            }
          }

      // ---- O^T += V^T P^T, summed over the chunk apart (the instruction's own sums
      // truncate, which would add up along a long sequence) ----
#pragma unroll
      for (int y = 0; y < kGroups; ++y) {
        float add[kTiles][4][4];
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) add[x][j][e] = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          auto word = [&](int r) {
            return *reinterpret_cast<const uint32_t*>(vt + (16 * t + r) * kRowB + y * 32 + g * 4);
          };
          const uint32_t w0 = word(va), w1 = word(vb), w2 = word(va + 8), w3 = word(vb + 8);
          // two keys' codes side by side: 0 .. 3 of the word, and 4 .. 7
          uint32_t a01 = __byte_perm(w0, w1, 0x5410), b01 = __byte_perm(w0, w1, 0x7632);
          uint32_t a23 = __byte_perm(w2, w3, 0x5410), b23 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j == 2) a01 >>= 8, b01 >>= 8, a23 >>= 8, b23 >>= 8;
            const uint32_t a0 = j & 1 ? centred<true>(a01) : centred<false>(a01);
            const uint32_t a1 = j & 1 ? centred<true>(b01) : centred<false>(b01);
            const uint32_t a2 = j & 1 ? centred<true>(a23) : centred<false>(a23);
            const uint32_t a3 = j & 1 ? centred<true>(b23) : centred<false>(b23);
#pragma unroll
            for (int x = 0; x < kTiles; ++x)
#pragma unroll
              for (int p = kParts - 1; p >= 0; --p) mma_f16(add[x][j], a0, a1, a2, a3, pf[x][y][t][p][0], pf[x][y][t][p][1]);
          }
        }
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[x][y][j][e] = fmaf(o[x][y][j][e], f[x][e & 1], add[x][j][e]);
      }
      phase ^= 1u << take;
      if (++take == kStages) take = 0;
      __syncwarp();
    }
    if (aborted(sh)) {  // copies under way land before the buffers change hands; nothing is asked for any more
      while (take != ask) {
        mbar_drain(smem_addr(&sh.full[warp][take]), phase >> take & 1u, a.timeout_ns);
        phase ^= 1u << take;
        if (++take == kStages) take = 0;
      }
      __syncwarp();
    }

    // ---- this warp's state into its buffers ----
    float* w = reinterpret_cast<float*>(wbuf);
    const float unit = power_of_2(top - 141);
#pragma unroll
    for (int x = 0; x < kTiles; ++x)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = x * 8 + 2 * tq + c;
#pragma unroll
        for (int of = 4; of < 32; of <<= 1) l[x][c] += __shfl_xor_sync(0xffffffffu, l[x][c], of);
#pragma unroll
        for (int y = 0; y < kGroups; ++y) {
#pragma unroll
          for (int of = 4; of < 32; of <<= 1) zs[x][y][c] += __shfl_xor_sync(0xffffffffu, zs[x][y][c], of);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[r * kD + y * kQ4Group + g * 8 + j] = fmaf(o[x][y][j][c], unit, zs[x][y][c]);
            w[r * kD + y * kQ4Group + g * 8 + j + 4] = fmaf(o[x][y][j][2 + c], unit, zs[x][y][c]);
          }
        }
        if (g == 0) {
          w[kRows * kD + 2 * r] = m[x][c];
          w[kRows * kD + 2 * r + 1] = l[x][c];
        }
      }
    fence_async();
  }

  // The same answer for the whole warp.
  static __device__ __forceinline__ bool aborted(Shared& sh) {
    return __any_sync(0xffffffffu, *static_cast<volatile uint32_t*>(&sh.abort));
  }
  // A wait for a copy that is under way after something else has given up.
  static __device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < timeout_ns) {
    }
  }
};

template <int D, bool kF32, int kTiles>
cudaError_t decode_q4(const PagedArgs& a, cudaStream_t s) {
  using U = Q4Unit<D, kF32, kTiles>;
  return launch_decode<U>(a, q4_cluster(!kF32, a.B, a.Hkv, a.G, a.max_pages, a.page_shift),
                          q4_ctas(!kF32, U::kRows, a.sms), s);
}

template <typename... P>
cudaError_t launch_rows(void (*kernel)(P...), const PagedArgs& a, int rows_per_cta, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.T) * a.Hkv;
  const int64_t ctas = (rows + rows_per_cta - 1) / rows_per_cta;
  if (ctas > INT_MAX) return cudaErrorInvalidValue;
  kernel<<<dim3(static_cast<unsigned>(ctas), a.B), kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q4_append(const PagedArgs& a, bool bf16, cudaStream_t s) {
  const int rows = kRowThreads / (a.D / 8);
  if (a.D == 64)
    return bf16 ? launch_rows(q4_append_kernel<64, __nv_bfloat16>, a, rows, s) : launch_rows(q4_append_kernel<64, float>, a, rows, s);
  return bf16 ? launch_rows(q4_append_kernel<128, __nv_bfloat16>, a, rows, s) : launch_rows(q4_append_kernel<128, float>, a, rows, s);
}

cudaError_t launch_q4_read(const PagedArgs& a, bool bf16, cudaStream_t s) {
  const int rows = kRowThreads / (a.D / 8) * 4;
  if (a.D == 64)
    return bf16 ? launch_rows(q4_read_kernel<64, __nv_bfloat16>, a, rows, s) : launch_rows(q4_read_kernel<64, float>, a, rows, s);
  return bf16 ? launch_rows(q4_read_kernel<128, __nv_bfloat16>, a, rows, s) : launch_rows(q4_read_kernel<128, float>, a, rows, s);
}

cudaError_t launch_q4_decode(const PagedArgs& a, bool bf16, cudaStream_t s) {
  const int rows = q4_rows(bf16, a.G);
  if (a.D == 64) return !bf16 ? decode_q4<64, true, 1>(a, s) : rows == 8 ? decode_q4<64, false, 1>(a, s) : decode_q4<64, false, 2>(a, s);
  return !bf16 ? decode_q4<128, true, 1>(a, s) : rows == 8 ? decode_q4<128, false, 1>(a, s) : decode_q4<128, false, 2>(a, s);
}

}  // namespace cp
