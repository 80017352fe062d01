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
//   x_j = sum over groups of s_j (q.(c_j - 8)) + (z_j + 8 s_j) (sum of q)
//   out = sum_j p_j s_j (c_j - 8) + sum_j p_j (z_j + 8 s_j)
// so that codes go to the matrix instructions alone, as c - 8, which is exact in fp16,
// and scales meet only scores and weights, one number a key.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "cp_ptx.cuh"
#include "cp_score.h"
#include "packed.cuh"
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
// Append and read
// ----------------------------------------------------------------------------
constexpr int kRowThreads = 128;

__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float y;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float y;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// 1 where a >= b, else 0.
__device__ __forceinline__ float at_least(float a, float b) {
  float y;
  asm("set.ge.f32.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// a - b = h + l exactly (the two-sum of Knuth, of a and -b).
__device__ __forceinline__ void exact_diff(float a, float b, float& h, float& l) {
  h = __fsub_rn(a, b);
  const float bb = __fsub_rn(h, a);
  l = __fsub_rn(__fsub_rn(a, __fsub_rn(h, bb)), __fadd_rn(b, bb));
}

// This lane's 16 codes (value i of 8 in bits 4 i of a word) and its group's scale and
// offset (bf16, scale in the lower half), from the 4 lanes that share the group. kB16:
// the values are bf16 numbers. Everything is decided exactly, by candidates from
// approximate quotients that are never too large and a comparison that raises them.
template <bool kB16>
__device__ __forceinline__ uint2 quantise(const float (&x)[16], uint32_t& scale) {
  float least = x[0], most = x[0];
#pragma unroll
  for (int i = 1; i < 16; i += 2) {
    least = min_nan(least, x[i], x[(i + 1) & 15]);  // (the last with x[0] again)
    most = max_nan(most, x[i], x[(i + 1) & 15]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const float a = __shfl_xor_sync(0xffffffffu, least, o), b = __shfl_xor_sync(0xffffffffu, most, o);
    least = min_nan(least, a, a);
    most = max_nan(most, b, b);
  }
  float z = least;
  if constexpr (!kB16) {
    const uint32_t lb = __float_as_uint(least), low = lb & 0xffffu;
    z = __uint_as_float(lb - low + (low && lb >> 31 ? 0x10000u : 0u));
  }
  float h, l;
  exact_diff(most, z, h, l);
  // a value that is not finite, or a span that fp32 does not hold: reads back as NaN, whatever is formed meanwhile
  const bool bad = !(fabsf(h) <= FLT_MAX);
  // s: upper bits of a quotient that is at most 2^-19 of itself too small, so two steps up at most
  uint32_t sb = __float_as_uint(h * (1.f / 15 * (1 - 0x1p-20f))) & 0xffff0000u;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (__fsub_rn(15.f * __uint_as_float(sb), h) < l) sb += 0x10000u;  // both sides exact
  const float s = fmaxf(__uint_as_float(sb), 0x1p-100f);
  scale = bad ? 0x7fff7fffu : __float_as_uint(s) >> 16 | __float_as_uint(z);
  // c: the integer nearest to a quotient that is at most 15 2^-18 too small (by a sum
  // whose unit is 1), raised where the value lies half a step above it or more
  constexpr float kOne = 12582912.f;  // 1.5 2^23
  const float2 rs = twice(rcp_approx(s) * (1 - 0x1p-20f)), down = twice(-s), zz = twice(-z);
  const float half = 0.5f * s;
  bool exact = kB16;
  if constexpr (kB16) {
    // Differences of 8-bit numbers are exact while none is 2^15 times another (or an
    // offset 0); seldom otherwise, and zeros then count as otherwise too.
    float small = fabsf(z);
#pragma unroll
    for (int i = 0; i < 16; i += 2) small = fmin3(small, fabsf(x[i]), fabsf(x[i + 1]));
    exact = z == 0.f || small >= fmaxf(fabsf(least), fabsf(most)) * 0x1p-14f;
  }
  float2 c[8];  // codes i and i + 8
  if (kB16 && __all_sync(0xffffffffu, exact)) {
    // r - s / 2 is 0 or 2^-19.1 s at least (the values' unit, and that of s, of which all
    // are multiples), so r times a little more than 1 / s rounds to 1 just where r is half
    // a step or more; and r > - s / 2, since the first quotient was too small
    const float2 more = twice(rcp_approx(s) * (1 + 0x1p-21f));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 d = add2(make_float2(x[i], x[i + 8]), zz);
      const float2 g = fma2(d, rs, twice(kOne));
      const float2 r = fma2(add2(g, twice(-kOne)), down, d);  // exact: d - c s, within a step
      c[i] = add2(fma2(r, more, g), twice(-kOne));
    }
  } else {  // what the difference has lost decides where the rest is half a step
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = make_float2(x[i], x[i + 8]), minus = twice(-1.f);
      const float2 d = add2(v, zz);
      const float2 back = fma2(v, minus, d);
      const float2 lost = fma2(add2(twice(z), back), minus, fma2(fma2(back, minus, d), minus, v));
      const float2 g = add2(fma2(d, rs, twice(kOne)), twice(-kOne));
      const float2 r = add2(add2(fma2(g, down, d), twice(-half)), lost);
      c[i] = add2(g, make_float2(at_least(r.x, 0.f), at_least(r.y, 0.f)));
    }
  }
  // four codes at a time are a number below 2^16, exact in fp32
  uint2 codes;
  const float2 c03 = fma2(fma2(c[3], twice(16.f), c[2]), twice(256.f), fma2(c[1], twice(16.f), c[0]));
  const float2 c47 = fma2(fma2(c[7], twice(16.f), c[6]), twice(256.f), fma2(c[5], twice(16.f), c[4]));
  const float2 lo = add2(c03, twice(0x1p23f)), hi = add2(c47, twice(0x1p23f));
  codes.x = __byte_perm(__float_as_uint(lo.x), __float_as_uint(hi.x), 0x5410);
  codes.y = __byte_perm(__float_as_uint(lo.y), __float_as_uint(hi.y), 0x5410);
  return bad ? make_uint2(0, 0) : codes;
}

// Token and head of a row (row < 2^31).
__device__ __forceinline__ void token_head(const PagedArgs& a, int row, int& t, int& hk) {
  const uint64_t wide = static_cast<uint64_t>(static_cast<uint32_t>(row)) * a.hkv_mul;
  t = static_cast<int>(wide >> (32 + a.hkv_shift));
  hk = row - t * a.Hkv;
}

// Rows (token, head) of sequence blockIdx.y: a warp takes 512 / D of them, 16 values a
// lane. Bound by instructions, so the work that a group takes once is spread over few
// lanes (8 values a lane: 31.6 us where 16 took 26.3), and keys and values share the
// look-up of their place (a CTA of either alone: 26.3 us where both took 22.9; now 22.2: some
// 17000 new tokens of 6 sequences, 8 heads of 128, bf16, 4.0 TB/s of rows and codes).
template <int D, typename T>
__global__ void __launch_bounds__(kRowThreads) q4_append_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int kLanes = D / 16;
  grid_wait();  // (the launch may start while its predecessor in the stream ends)
  const int b = blockIdx.y, l = threadIdx.x % kLanes;
  const int row = blockIdx.x * (kRowThreads / kLanes) + threadIdx.x / kLanes, most = a.T * a.Hkv;
  const bool in = row < most;  // (lanes stay for the shuffles)
  int t, hk;
  token_head(a, in ? row : 0, t, hk);
  const int n = a.seq_lens[b];
  const bool live = in && !(a.new_lens && t >= a.new_lens[b]);
  if (!__any_sync(0xffffffffu, live)) return;  // padding
  float k[16] = {}, v[16] = {};
  auto load16 = [&](const void* from, float (&x)[16]) {
    const T* p = static_cast<const T*>(from) + (static_cast<int64_t>(b) * most + row) * D + l * 16;
    float lo[8], hi[8];
    load8(p, lo);
    load8(p + 8, hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = lo[i];
      x[8 + i] = hi[i];
    }
  };
  if (live) {  // on their way before the row's place is looked up
    load16(a.k_new, k);
    load16(a.v_new, v);
  }
  const uint32_t pos = static_cast<uint32_t>(n) + static_cast<uint32_t>(t);  // (both below 2^31)
  int page = -1;
  if (live) {
    if (n < 0 || pos >= a.positions)
      atomicOr(a.err, kDevErrPage);
    else
      page = page_of(a, b, static_cast<int>(pos));
  }
  constexpr bool kB16 = sizeof(T) == 2;
  uint32_t ks, vs;
  const uint2 kc = quantise<kB16>(k, ks), vc = quantise<kB16>(v, vs);
  if (page < 0) return;
  const int64_t dst = head_row(a, page, static_cast<int>(pos), hk);
  static_cast<uint2*>(a.k_cache)[dst * kLanes + l] = kc;
  static_cast<uint2*>(a.v_cache)[dst * kLanes + l] = vc;
  if (l % 4 == 0) {
    static_cast<uint32_t*>(a.k_scales)[dst * (D / kQ4Group) + l / 4] = ks;
    static_cast<uint32_t*>(a.v_scales)[dst * (D / kQ4Group) + l / 4] = vs;
  }
}

// Eight codes as values: code i of a half word, in its place within the mantissa of
// 2^23, is 16^i times itself.
__device__ __forceinline__ void values8(uint32_t codes, uint32_t scale, float (&x)[8]) {
  const float s = __uint_as_float(scale << 16);
  const float2 z = twice(__uint_as_float(scale & 0xffff0000u)), one = twice(-0x1p23f);
  const float2 s01 = make_float2(s, s * 0x1p-4f), s23 = make_float2(s * 0x1p-8f, s * 0x1p-12f);
#pragma unroll
  for (int i = 0; i < 2; ++i, codes >>= 16) {
    auto at = [&](uint32_t mask) { return __uint_as_float((codes & mask) | 0x4b000000u); };
    const float2 a = fma2(s01, add2(make_float2(at(0xfu), at(0xf0u)), one), z);
    const float2 b = fma2(s23, add2(make_float2(at(0xf00u), at(0xf000u)), one), z);
    x[4 * i] = a.x, x[4 * i + 1] = a.y, x[4 * i + 2] = b.x, x[4 * i + 3] = b.y;
  }
}

// Rows (token, head) of sequence blockIdx.y: a warp takes kAhead times 256 / D, all
// of whose loads are under way at once (length, page, codes: one after the other).
// Bound by HBM, most of it the values written: 24.0 us for 6 sequences of up to 5119
// tokens, 8 heads of 128, 6.0 TB/s (four times 256 / D: 24.6).
template <int D, typename T>
__global__ void __launch_bounds__(kRowThreads) q4_read_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int kLanes = D / 8, kAhead = 2, kRows = kRowThreads / kLanes;
  grid_wait();
  const int b = blockIdx.y, l = threadIdx.x % kLanes;
  const int most = a.T * a.Hkv, first = blockIdx.x * (kRows * kAhead) + threadIdx.x / kLanes;
  const int n = seq_len(a, b);
  uint32_t kc[kAhead], vc[kAhead], ks[kAhead], vs[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int row = first + i * kRows;
    kc[i] = vc[i] = ks[i] = vs[i] = 0;
    if (row >= most) continue;
    int t, hk;
    token_head(a, row, t, hk);
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
    const int row = first + i * kRows;
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
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
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
// Four such tiles from shared memory, of rows that the lanes name, eight each, transposed.
__device__ __forceinline__ void load_transposed(uint32_t at, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t x) { return __half22float2(*reinterpret_cast<__half2*>(&x)); }
// The nearest multiple of 16, of |x| < 2^25.
__device__ __forceinline__ float multiple(float x) { return __fadd_rn(__fadd_rn(x, 0x1.8p27f), -0x1.8p27f); }
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// x plus the offset of a scale word, its upper bf16 number.
__device__ __forceinline__ float plus_offset(float x, uint32_t w) {
  float y;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.rn.f32.bf16 %0, hi, %1;\n\t}" : "=f"(y) : "f"(x), "r"(w));
  return y;
}

// Codes i and i + 4 of a word of 8 (i known when compiled) as fp16 numbers c - 8: a code
// put into the mantissa of 1024 is 1024 + c (or 1024 + 16 c), and the rest is taken off.
// (The usual way from short integers to floating point: the bits of a fixed exponent.)
__device__ __forceinline__ uint32_t codes(uint32_t w, int i) {
  uint32_t x;
  if (i & 2) w >>= 8;
  if (!(i & 1)) {
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(x) : "r"(w));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(0x64086408u));  // 1032
  } else {
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(x) : "r"(w));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(x) : "r"(x), "r"(0x2c002c00u), "r"(0xd480d480u));  // / 16, - 72
  }
  return x;
}

// cap tanh(y) for y = x / cap within 1: the polynomial of score_math.cuh (relative
// error 5.0e-8), as a factor of y.
__device__ __forceinline__ float2 tanh_poly(float2 u) {
  constexpr float c[7] = {0.9999999502f,  -0.3333283915f,  0.1332520408f, -0.05345702957f,
                          0.02028998042f, -0.006203379104f, 0.001041022634f};
  float2 p = twice(c[6]);
#pragma unroll
  for (int i = 5; i >= 0; --i) p = fma2(p, u, twice(c[i]));
  return p;
}

// A warp's part of a unit: chunks first, first + step, ... below last, of sequence b's n
// keys, for group hg of key/value head hk's query heads.
struct Part {
  int b, n, hk, hg, first, last, step;
};

// Codes come as c - 8: the instruction aligns products by the exponents that its operands
// name and truncates, so that sums of numbers above zero lean, and those of subnormal
// operands, which name one too large, the more. (The bits of c as they lie are the fp16
// number c 2^-24 and take one instruction less a pair: 2 x 262144 keys 69 us where this
// takes 75.6. But answers of so many keys leaned by 4e-4 of themselves, where the weights'
// rounding costs 7e-5, and scores were 4e-7 off, here 8e-8.)
// bf16 queries: one fp16 part of q and of the weights. fp32 queries: two parts of each,
// whose products leave 2^-22 out; the upper part of q is cut to multiples of 16 of at
// most 2^15, so that its products with codes and their sums over a group are whole
// numbers of 20 bits, which nothing truncates (with parts of 11 bits each wherever they
// lie, scores were ten times as far off as fp32's).
template <int D_, bool kF32, int kTiles, int kChunk>
struct Q4Unit {
  static constexpr int kT = kChunk / 16;  // tiles of a warp's keys in a step
  static constexpr int kD = D_, kRows = 8 * kTiles, kBlock = kChunk, kPerSm = q4_per_sm(!kF32, kRows, kChunk);
  static constexpr int kGroups = D_ / kQ4Group, kParts = kF32 ? 2 : 1;
  static constexpr int kRowB = D_ / 2, kScaleB = kGroups * 4;  // a row's codes and scales
  static constexpr int kCodes = kChunk * kRowB, kScales = kChunk * kScaleB, kStage = 2 * (kCodes + kScales);
  static constexpr int kStages = 2;
  static constexpr int kState = kRows * (D_ + 2);
  static constexpr int kWarpB = ((kStages * kStage > 2 * kState * 4 ? kStages * kStage : 2 * kState * 4) + 127) & ~127;
  static constexpr int kSmem = kDecWarps * kWarpB;
  using Keys = std::conditional_t<kChunk == 64, uint64_t, uint32_t>;  // a bit a key of a chunk
  static constexpr bool kEarly = true;
  // the next part's first loads go ahead of this one's end where a stage has room for the state
  static constexpr bool kAhead = kStages == 2 && kStage >= kState * 4;
  struct Shared {
    uint64_t full[kDecWarps][kStages];
    uint32_t abort;
  };

  // stage of the next chunk to ask for and to take, and the stages' phases
  int ask = 0, take = 0;
  uint32_t phase = 0;
  // the loads of a part, a lane a piece (codes and scales of k and v, each as often as a chunk meets pages)
  int pos, page = 0, asked, last, step;  // of the lane's piece of chunk `asked`
  const uint8_t* base;
  const int* table;
  Keys coming[kStages - 1];  // the keys of the chunks under way

  __device__ __forceinline__ Q4Unit(const PagedArgs& a, uint8_t*, Shared& sh) {
    if (threadIdx.x < kDecWarps * kStages)
      mbar_init(smem_addr(&sh.full[0][0] + threadIdx.x), 4 * runs(a) + (a.stall >> threadIdx.x / kStages & 1u));
    if (threadIdx.x == 0) sh.abort = 0;
    fence_mbar_init();
    fence_async();
    __syncthreads();
  }

  static __device__ __forceinline__ int row_bytes() { return threadIdx.x & 1 ? kScaleB : kRowB; }
  // (the page is looked at when its chunk is asked for: an instruction that needs it earlier would wait for the table)
  __device__ __forceinline__ bool wanted(const PagedArgs& a, int n) const {
    return static_cast<int>(threadIdx.x & 31) < 4 * runs(a) && asked < last && pos < n;
  }
  __device__ __forceinline__ void find(const PagedArgs& a, int n) {
    if (wanted(a, n)) page = table[pos >> a.page_shift];
  }
  // Asks for chunk `asked` of n keys and looks the warp's next one's page up: which keys there are, a bit each.
  __device__ __forceinline__ Keys load(const PagedArgs& a, int n, uint8_t* smem, Shared& sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pieces = 4 * runs(a), rows = kChunk / runs(a);
    bool ok = wanted(a, n);
    if (ok && (page < 0 || page >= a.num_pages)) {
      atomicOr(a.err, kDevErrPage);
      ok = false;
    }
    uint32_t found = __ballot_sync(0xffffffffu, ok) & 0x11111111u;  // a bit a run
    Keys on = 0;
    if (found == (0x11111111u >> (32 - pieces))) {
      on = ~Keys{0};
    } else {
      const Keys one = rows == 64 ? ~Keys{0} : (Keys{1} << (rows & 63)) - 1;
      for (int at = 0; found; at += rows, found >>= 4)
        if (found & 1u) on |= one << at;
    }
    const int rest = n - asked * kChunk;
    if (rest < kChunk) on &= (Keys{1} << rest) - 1;
    if (lane < pieces) {
      const int row_b = row_bytes(), which = lane & 3;  // k codes, k scales, v codes, v scales
      const uint32_t bar = smem_addr(&sh.full[warp][ask]), bytes = rows * row_b;
      const uint32_t dst = smem_addr(smem + warp * kWarpB) + ask * kStage + (which & 2 ? kCodes + kScales : 0) +
                           (which & 1 ? kCodes : 0) + (lane >> 2) * bytes;
      const int64_t page_b = (static_cast<int64_t>(row_b) << a.page_shift) * a.Hkv;
      mbar_arrive_expect_tx(bar, ok ? bytes : 0);
      if (ok) bulk_g2s(dst, base + page * page_b + (pos & ((1 << a.page_shift) - 1)) * row_b, bytes, bar);
    }
    if (++ask == kStages) ask = 0;
    asked += step;
    pos += step * kChunk;
    find(a, n);
    return on;
  }

  // The loads of a part's first chunks.
  __device__ __forceinline__ void start(const PagedArgs& a, const Part& p, uint8_t* smem, Shared& sh) {
    const int which = threadIdx.x & 3, run = (threadIdx.x & 31) >> 2;
    base = static_cast<const uint8_t*>(which == 0   ? a.k_cache
                                       : which == 1 ? a.k_scales
                                       : which == 2 ? a.v_cache
                                                    : a.v_scales) +
           p.hk * (static_cast<int64_t>(row_bytes()) << a.page_shift);
    table = a.table + static_cast<int64_t>(p.b) * a.max_pages;
    asked = p.first;
    step = p.step;
    last = p.last;
    pos = asked * kChunk + run * (kChunk / runs(a));
    fence_async();  // (what was read and written here before)
    find(a, p.n);
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st)
      if (asked < last && !aborted(sh)) coming[st] = load(a, p.n, smem, sh);
  }

  // For a cluster: a warp's chunks of blocks [blk0, blk1); its state at the start of its buffers.
  __device__ __forceinline__ void run(const PagedArgs& a, int b, int n, int hk, int hg, int blk0, int blk1, uint8_t* smem,
                                      Shared& sh) {
    const Part p{b, n, hk, hg, blk0 + static_cast<int>(threadIdx.x >> 5), blk1, kDecWarps};
    start(a, p, smem, sh);
    take_part(a, p, nullptr, smem, sh);
  }

  // A part whose first loads are under way, and those of the following one ahead of its
  // end. Returns the warp's state: O [kRows][kD], then m and l.
  __device__ __forceinline__ float* take_part(const PagedArgs& a, const Part& part, const Part* following, uint8_t* smem,
                                              Shared& sh) {
    const int b = part.b, n = part.n, hk = part.hk, hg = part.hg;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
    uint8_t* wbuf = smem + warp * kWarpB;
    const uint32_t bars = smem_addr(&sh.full[warp][0]);
    const int h0 = hk * a.G + hg * kRows, nrow = min(kRows, a.G - hg * kRows);

    // ---- q: each head's column in fp16, scaled by a power of two so that its largest
    // value lies in [2^14, 2^15); what is below 2^-39 of that is lost ----
    // Scores leave the products as x / cap, or in units of log2 where there is no cap.
    const float unit_x = a.cap > 0.f ? a.scale / a.cap : a.scale * kL2e, cap2 = a.cap * kL2e;
    uint32_t qf[kTiles][kGroups][4][kParts][2];  // per step of 16 values
    float2 undo[kTiles], qsum[kTiles][kGroups], slope[kTiles];  // of this lane's columns, heads 2 tq and 2 tq + 1
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
            // codes i and i + 4 of a word of 8
            const int i = (st >> 1) * 8 + (st & 1) * 2 + r;
            const float up = power_of_2(14 - e), lo = v[y][i] * up, hi = v[y][i + 4] * up;
            if constexpr (!kF32) {
              qf[x][y][st][0][r] = pack_f16x2(lo, hi);
            } else {
              qf[x][y][st][0][r] = pack_f16x2(multiple(lo), multiple(hi));
              const float2 have = unpack_f16x2(qf[x][y][st][0][r]);
              qf[x][y][st][1][r] = pack_f16x2(lo - have.x, hi - have.y);
            }
          }
      auto column = [&](float z) {  // of heads 2 tq and 2 tq + 1, from the lanes that hold heads g
        return make_float2(__shfl_sync(0xffffffffu, z, 8 * tq), __shfl_sync(0xffffffffu, z, 8 * tq + 4));
      };
      undo[x] = column(power_of_2(e - 14) * unit_x);
#pragma unroll
      for (int y = 0; y < kGroups; ++y) qsum[x][y] = column(sum[y] * unit_x);
      const int hc = x * 8 + 2 * tq;
      slope[x] = make_float2(a.slopes && hc < nrow ? a.slopes[h0 + hc] * kL2e : 0.f,
                             a.slopes && hc + 1 < nrow ? a.slopes[h0 + hc + 1] * kL2e : 0.f);
    }

    float2 m[kTiles], l[kTiles], zs[kTiles][kGroups], o[kTiles][kGroups][4][2];
#pragma unroll
    for (int x = 0; x < kTiles; ++x) {
      m[x] = twice(-INFINITY);
      l[x] = twice(0.f);
#pragma unroll
      for (int y = 0; y < kGroups; ++y) {
        zs[x][y] = twice(0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[x][y][j][0] = o[x][y][j][1] = twice(0.f);
      }
    }
    // exponent (biased) of the largest value scale so far, and what brings it below 2^15: o is in units of 2^(top - 141)
    int top = 27;
    float fit = power_of_2(141 - 27);
    const uint8_t* krow = wbuf + g * kRowB + tq * 8;
    const uint8_t* zrow = wbuf + kCodes + g * kScaleB;
    const uint32_t vrows = smem_addr(wbuf) + kCodes + kScales + ((lane & 7) + (lane >> 4) * 8) * kRowB + (lane & 8) * 2;
    auto scales = [](const uint8_t* p, uint32_t (&w)[kGroups]) {
      if constexpr (kGroups == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      }
    };

    for (int chunk = part.first; chunk < part.last; chunk += part.step) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bars + take * 8, phase >> take & 1u, &sh.abort, a.err, a.timeout_ns)))
        break;
      const Keys on = coming[0];
#pragma unroll
      for (int st = 1; st < kStages - 1; ++st) coming[st - 1] = coming[st];
      if (asked < last) coming[kStages - 2] = load(a, n, smem, sh);  // into the stage that the last step read
      const int stage = take * kStage;
      const bool part = on != ~Keys{0};
      if (part) {  // rows that hold no key may hold anything: their scales become 0, and no result depends on them
#pragma unroll
        for (int i = lane; i < kChunk; i += 32)
          if (!(on >> i & 1u))
#pragma unroll
            for (int y = 0; y < 2 * kGroups; ++y)
              *reinterpret_cast<uint32_t*>(wbuf + stage + kCodes + (y & 1 ? kCodes + kScales : 0) + i * kScaleB + (y >> 1) * 4) = 0;
        fence_async();  // (before copies come here again)
        __syncwarp();
      }

      // ---- scores, keys as rows: tiles of 16; [tile][row] over the lane's two heads ----
      float2 s[kT][kTiles][2];
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        float dot[kTiles][kGroups][4];
#pragma unroll
        for (int y = 0; y < kGroups; ++y) {
          const uint2 wa = *reinterpret_cast<const uint2*>(krow + stage + 16 * t * kRowB + y * 32);
          const uint2 wb = *reinterpret_cast<const uint2*>(krow + stage + (16 * t + 8) * kRowB + y * 32);
          float low[kTiles][4];
#pragma unroll
          for (int x = 0; x < kTiles; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) dot[x][y][e] = low[x][e] = 0.f;
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            const uint32_t ua = st >> 1 ? wa.y : wa.x, ub = st >> 1 ? wb.y : wb.x;
            const uint32_t a0 = codes(ua, 2 * (st & 1)), a1 = codes(ub, 2 * (st & 1));
            const uint32_t a2 = codes(ua, 2 * (st & 1) + 1), a3 = codes(ub, 2 * (st & 1) + 1);
#pragma unroll
            for (int x = 0; x < kTiles; ++x) {
              if constexpr (kF32) mma_f16(low[x], a0, a1, a2, a3, qf[x][y][st][1][0], qf[x][y][st][1][1]);
              mma_f16(dot[x][y], a0, a1, a2, a3, qf[x][y][st][0][0], qf[x][y][st][0][1]);
            }
          }
          if constexpr (kF32)
#pragma unroll
            for (int x = 0; x < kTiles; ++x)
#pragma unroll
              for (int e = 0; e < 4; ++e) dot[x][y][e] += low[x][e];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t w[kGroups];
          scales(zrow + stage + (16 * t + 8 * r) * kScaleB, w);
#pragma unroll
          for (int x = 0; x < kTiles; ++x) {
            float2 d, zq;
#pragma unroll
            for (int y = 0; y < kGroups; ++y) {
              const float ks = __uint_as_float(w[y] << 16), kz = plus_offset(8.f * ks, w[y]);
              const float d0 = dot[x][y][2 * r], d1 = dot[x][y][2 * r + 1];
              d.x = y ? fmaf(ks, d0, d.x) : ks * d0;
              d.y = y ? fmaf(ks, d1, d.y) : ks * d1;
              zq.x = y ? fmaf(kz, qsum[x][y].x, zq.x) : kz * qsum[x][y].x;
              zq.y = y ? fmaf(kz, qsum[x][y].y, zq.y) : kz * qsum[x][y].y;
            }
            s[t][x][r] = fma2(d, undo[x], zq);
          }
        }
      }
      if (a.cap > 0.f) {
        float far = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * kT * kTiles; ++i) {
          float2& y = s[i / 2 % kT][i / (2 * kT)][i & 1];
          far = fmax3(far, fabsf(y.x), fabsf(y.y));
        }
        if (__all_sync(0xffffffffu, far <= 1.f)) {
#pragma unroll
          for (int i = 0; i < 2 * kT * kTiles; ++i) {
            float2& y = s[i / 2 % kT][i / (2 * kT)][i & 1];
            y = mul2(mul2(y, twice(cap2)), tanh_poly(mul2(y, y)));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2 * kT * kTiles; ++i) {
            float2& y = s[i / 2 % kT][i / (2 * kT)][i & 1];
            y = make_float2(cap2 * tanhf(y.x), cap2 * tanhf(y.y));
          }
        }
      }
      if (a.slopes) {
        const float dist = static_cast<float>(n - 1 - chunk * kChunk - g);
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int x = 0; x < kTiles; ++x) s[t][x][r] = fma2(twice(16 * t + 8 * r - dist), slope[x], s[t][x][r]);
      }
      if (part)
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int x = 0; x < kTiles; ++x)
              if (!(on >> (g + 16 * t + 8 * r) & 1u)) s[t][x][r] = twice(-INFINITY);

      // ---- weights ----
      float2 f[kTiles];
#pragma unroll
      for (int x = 0; x < kTiles; ++x) {
        auto weigh = [&](float& mm, float& ll, float& ff, auto p) {
          float mx = p(0, 0), sum = 0.f;
#pragma unroll
          for (int i = 1; i < 2 * kT; ++i) mx = fmaxf(mx, p(i >> 1, i & 1));
#pragma unroll
          for (int of = 4; of < 32; of <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, of));
          const float mn = fmaxf(mm, mx), ref = mn == -INFINITY ? 0.f : mn;
          auto ex2 = [](float z) { return kF32 ? exp2f(z) : ex2_approx(z); };
          ff = ex2(mm - ref);
          mm = mn;
#pragma unroll
          for (int i = 0; i < 2 * kT; ++i) {
            float& y = p(i >> 1, i & 1);
            y = ex2(y - ref);
            sum += y;
          }
          ll = fmaf(ll, ff, sum);
        };
        weigh(m[x].x, l[x].x, f[x].x, [&](int t, int r) -> float& { return s[t][x][r].x; });
        weigh(m[x].y, l[x].y, f[x].y, [&](int t, int r) -> float& { return s[t][x][r].y; });
      }

      // ---- the values' scales meet the weights: p s in fp16, scaled so that it stays
      // below 2^15; p (z + 8 s) summed as it is ----
      float largest = 0.f;  // (a lane a key here)
#pragma unroll
      for (int i = 0; i < kChunk; i += 32) {
        uint32_t w[kGroups];
        scales(wbuf + stage + 2 * kCodes + kScales + (lane + i) * kScaleB, w);
#pragma unroll
        for (int y = 0; y < kGroups; ++y) {
          largest = fmaxf(largest, fabsf(__uint_as_float(w[y] << 16)));
        }
      }
      float2 fz[kTiles];
#pragma unroll
      for (int x = 0; x < kTiles; ++x) fz[x] = f[x];
      if (__any_sync(0xffffffffu, largest * fit >= 32768.f)) {  // seldom: a larger scale than any before
        const int now = max(top, static_cast<int>(__reduce_max_sync(0xffffffffu, __float_as_uint(largest)) >> 23));
        const float2 down = twice(now - top > 126 ? 0.f : power_of_2(top - now));
#pragma unroll
        for (int x = 0; x < kTiles; ++x) f[x] = mul2(f[x], down);
        top = now;
        fit = power_of_2(141 - top);
      }

      // ---- O^T += V^T P^T, summed over the chunk apart (the instruction's own sums
      // truncate, which would add up along a long sequence) ----
#pragma unroll
      for (int y = 0; y < kGroups; ++y) {
        uint32_t pf[kTiles][kT][kParts][2];
#pragma unroll
        for (int x = 0; x < kTiles; ++x) zs[x][y] = mul2(zs[x][y], fz[x]);
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(zrow + stage + kCodes + kScales + (16 * t + 8 * r) * kScaleB + 4 * y);
            const float sv = __uint_as_float(w << 16), zz = plus_offset(8.f * sv, w), fs = sv * fit;
#pragma unroll
            for (int x = 0; x < kTiles; ++x) {
              const float2 p = s[t][x][r];
              zs[x][y].x = fmaf(p.x, zz, zs[x][y].x);
              zs[x][y].y = fmaf(p.y, zz, zs[x][y].y);
              const float2 ps = make_float2(p.x * fs, p.y * fs);
              const uint32_t u = pack_f16x2(ps.x, ps.y);
              pf[x][t][0][r] = transpose8(u);
              if constexpr (kF32) {
                const float2 have = unpack_f16x2(u);
                pf[x][t][1][r] = transpose8(pack_f16x2(ps.x - have.x, ps.y - have.y));
              }
            }
          }
        // (fp32: the lower parts' products apart, or the instruction drops them beside the upper ones':
        // 50000 keys were then 1.2e-6 of the result off, now 3e-7)
        float add[kTiles][4][4], low[kTiles][4][4];
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) add[x][j][e] = low[x][j][e] = 0.f;
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          const int at = stage + 16 * t * kRowB + y * 32;
          // two keys' codes side by side: values 4 g to 4 g + 3, and those 32 behind them (rows
          // 64 bytes apart meet four to a bank here, which costs less than eight instructions a tile)
          uint32_t a01, b01, a23, b23;
          load_transposed(vrows + at, a01, b01, a23, b23);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = codes(a01, j), a1 = codes(b01, j), a2 = codes(a23, j), a3 = codes(b23, j);
#pragma unroll
            for (int x = 0; x < kTiles; ++x) {
              mma_f16(add[x][j], a0, a1, a2, a3, pf[x][t][0][0], pf[x][t][0][1]);
              if constexpr (kF32) mma_f16(low[x][j], a0, a1, a2, a3, pf[x][t][1][0], pf[x][t][1][1]);
            }
          }
        }
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float2& to = o[x][y][j][e];
              to = fma2(to, f[x], make_float2(add[x][j][2 * e], add[x][j][2 * e + 1]));
              if constexpr (kF32) to = add2(to, make_float2(low[x][j][2 * e], low[x][j][2 * e + 1]));
            }
      }
      phase ^= 1u << take;
      if (++take == kStages) take = 0;
      __syncwarp();
    }
    if constexpr (kAhead)
      if (following) start(a, *following, smem, sh);
    if (aborted(sh)) {  // copies under way land before the buffers change hands; nothing is asked for any more
      while (take != ask) {
        mbar_drain(bars + take * 8, phase >> take & 1u);
        phase ^= 1u << take;
        if (++take == kStages) take = 0;
      }
      __syncwarp();
    }

    // ---- this warp's state into its buffers ----
    // (not where the next copies go)
    float* const w = reinterpret_cast<float*>(wbuf + (kAhead && following && take == 0 ? kStage : 0));
    const float unit = power_of_2(top - 141);
#pragma unroll
    for (int x = 0; x < kTiles; ++x) {
      auto keep = [&](int r, float mm, float ll, const float (&zz)[kGroups], auto column) {
#pragma unroll
        for (int of = 4; of < 32; of <<= 1) ll += __shfl_xor_sync(0xffffffffu, ll, of);
#pragma unroll
        for (int y = 0; y < kGroups; ++y) {
          float z = zz[y];
#pragma unroll
          for (int of = 4; of < 32; of <<= 1) z += __shfl_xor_sync(0xffffffffu, z, of);
          float out[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            out[j] = fmaf(column(o[x][y][j][0]), unit, z);
            out[j + 4] = fmaf(column(o[x][y][j][1]), unit, z);
          }
          float4* const to = reinterpret_cast<float4*>(w + r * kD + y * kQ4Group + g * 4);
          to[0] = make_float4(out[0], out[1], out[2], out[3]);
          to[8] = make_float4(out[4], out[5], out[6], out[7]);
        }
        if (g == 0) {
          w[kRows * kD + 2 * r] = mm;
          w[kRows * kD + 2 * r + 1] = ll;
        }
      };
      float zx[kGroups], zy[kGroups];
#pragma unroll
      for (int y = 0; y < kGroups; ++y) {
        zx[y] = zs[x][y].x;
        zy[y] = zs[x][y].y;
      }
      keep(x * 8 + 2 * tq, m[x].x, l[x].x, zx, [](float2 v) { return v.x; });
      keep(x * 8 + 2 * tq + 1, m[x].y, l[x].y, zy, [](float2 v) { return v.y; });
    }
    fence_async();
    return w;
  }

  // Pages that a chunk meets.
  static __device__ __forceinline__ int runs(const PagedArgs& a) {
    return (1 << a.page_shift) >= kChunk ? 1 : kChunk >> a.page_shift;
  }
  // The same answer for the whole warp.
  static __device__ __forceinline__ bool aborted(Shared& sh) {
    return __any_sync(0xffffffffu, *static_cast<volatile uint32_t*>(&sh.abort));
  }
};

// The list: all units' chunks, cut into equal contiguous ranges, one per warp. A warp
// waits for no other: units within its range it writes out, the one that began before
// and the one that goes on it leaves as partials, for the join.
// 2 x 262144 keys, 32 heads on 4 of 128, bf16, capped: 75.5 us with the join, 4.0 TB/s of
// the cache; the copies alone, with nothing formed of them, take 54. Waiting bounds it: a
// scheduler has two warps, each of which waits for its own last result half of the time,
// so that half of the issue slots go by (a warp takes some 20 instructions for a key and
// head, 128 codes of k and of v for 8 query heads). More warps have shorter steps, with
// more overhead a key, or spill: three CTAs 74.0 us, but a ragged batch 49.8 where this
// takes 49.1; of 32 keys a step three take 80.4 (48.7), four 87.7 (52.7).
template <class U>
__global__ void __launch_bounds__(kDecThreads, U::kPerSm) q4_decode_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int D = U::kD;
  extern __shared__ __align__(128) uint8_t smem[];
  int* cum = reinterpret_cast<int*>(smem + U::kSmem);  // [B + 1]: chunks before sequence b
  __shared__ int wsum[kDecWarps];
  __shared__ typename U::Shared shared;
  U unit(a, smem, shared);
  grid_wait();
  const int groups = (a.G + U::kRows - 1) / U::kRows, HG = a.Hkv * groups;
  const int total = work_list<U::kBlock>(a, HG, cum, wsum);
  grid_release();  // the join's CTAs take their places as these leave
  no_tokens<D>(a, cum);
  // (each warp that takes part has a chunk at least, so that a unit's partials lie with neighbours)
  const int worker = blockIdx.x * kDecWarps + (threadIdx.x >> 5), workers = min(static_cast<int>(gridDim.x) * kDecWarps, total);
  const int lane = threadIdx.x & 31;
  if (worker >= workers) return;
  const int begin = static_cast<int>(static_cast<int64_t>(total) * worker / workers);
  const int end = static_cast<int>(static_cast<int64_t>(total) * (worker + 1) / workers);
  int b = sequence_of(a, cum, begin), u = 0, nblk = 0;  // the unit within its sequence, and its chunks
  auto place = [&](int at) {
    while (cum[b + 1] <= at) ++b;
    const int n = min(max(a.seq_lens[b], 0), table_len(a));
    nblk = (n + U::kBlock - 1) / U::kBlock;
    u = (at - cum[b]) / nblk;
    const int first = (at - cum[b]) - u * nblk, hk = u / groups;
    return Part{b, n, hk, u - hk * groups, first, min(nblk, first + end - at), 1};
  };
  const int width = min(U::kRows, a.G);  // heads of a partial: O, then m and l
  Part p = place(begin);
  unit.start(a, p, smem, shared);
  for (int at = begin; at < end;) {
    const int64_t info = static_cast<int64_t>(p.b) * HG + u;
    const int h0 = p.hk * a.G + p.hg * U::kRows, nrow = min(U::kRows, a.G - p.hg * U::kRows);
    const int unit0 = at - p.first, unit1 = unit0 + nblk;  // the unit's chunks in the list
    const bool whole = at == unit0 && at + p.last - p.first == unit1;
    const int next = at + p.last - p.first, slot = at == begin ? 0 : 1;
    Part q = p;
    if (next < end) q = place(next);
    const float* w = unit.take_part(a, p, next < end ? &q : nullptr, smem, shared);
    __syncwarp();
    if (whole) {
      const int64_t row0 = static_cast<int64_t>(p.b) * a.H + h0;
      for (int i = lane; i < nrow * D; i += 32) {
        const float sum = w[U::kRows * D + 2 * (i / D) + 1];
        put_out(a, row0 * D + i, sum != 0.f ? w[i] / sum : 0.f);
      }
      if (lane < nrow) a.lse[row0 + lane] = natural_lse(w[U::kRows * D + 2 * lane], w[U::kRows * D + 2 * lane + 1]);
    } else {
      float* part = a.partial + (static_cast<int64_t>(worker) * 2 + slot) * width * (D + 2);
      for (int i = 2 * lane; i < nrow * D; i += 64)  // (D + 2 floats a head: 8-byte alignment)
        *reinterpret_cast<float2*>(part + i) = *reinterpret_cast<const float2*>(w + i);
      for (int i = lane; i < 2 * nrow; i += 32) part[width * D + i] = w[U::kRows * D + i];
    }
    // the warp that begins a unit says which partials make it up; a chunk x lies with warp ((x + 1) workers - 1) / total
    if (lane == 0 && at == unit0)
      a.info[info] = whole ? make_int2(0, -1)
                           : make_int2(worker * 2 + slot, static_cast<int>((static_cast<int64_t>(unit1) * workers - 1) / total));
    __syncwarp();
    if constexpr (!U::kAhead)
      if (next < end) unit.start(a, q, smem, shared);
    p = q;
    at = next;
  }
}

// Joins the partials of a unit that lay with more than one warp: the first in the slot
// that info names, the others in slot 0 of the warps up to info.y. kSplit warps a query
// head take its partials in turn, with a running maximum each, eight under way at once,
// and meet at the end: three loads one after the other in all. Many warps a head where a
// unit has many partials, one where it has few (48 ragged sequences of 24 heads, three
// partials a unit on average: the call 49.1 us with one, 49.4 with four).
template <int D, int kSplit>
__global__ void __launch_bounds__(kSplit == 1 ? 128 : kSplit * 32) q4_join_kernel(const __grid_constant__ PagedArgs a, int rows) {
  constexpr int kLane = D / 32, kFlight = 8;
  __shared__ float acc[kSplit][D], stat[kSplit][2];
  const int warp = kSplit == 1 ? 0 : threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = kSplit == 1 ? blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x, b = blockIdx.y;
  if (h >= a.H) return;  // (a warp a head: whole warps)
  const int groups = (a.G + rows - 1) / rows, width = min(rows, a.G), slot_floats = width * (D + 2);
  const int hk = h / a.G, r = (h - hk * a.G) % rows, hg = (h - hk * a.G) / rows;
  grid_wait();
  const int tokens = a.seq_lens[b];
  const int2 w = a.info[(static_cast<int64_t>(b) * a.Hkv + hk) * groups + hg];  // (of no use where there are no tokens)
  if (min(tokens, table_len(a)) <= 0 || w.y < 0) return;
  const int c0 = w.x >> 1, n = w.y - c0 + 1;
  float m = -INFINITY, l = 0.f, o[kLane] = {};
  for (int i = warp; i < n; i += kSplit * kFlight) {
    float2 ml[kFlight];
    float x[kFlight][kLane];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int at = i + u * kSplit;
      ml[u] = make_float2(-INFINITY, 0.f);
      if (at < n) {
        const float* p = a.partial + (static_cast<int64_t>(c0 + at) * 2 + (at == 0 ? w.x & 1 : 0)) * slot_floats;
        ml[u] = *reinterpret_cast<const float2*>(p + width * D + 2 * r);
#pragma unroll
        for (int c = 0; c < kLane; c += 2)
          *reinterpret_cast<float2*>(&x[u][c]) = *reinterpret_cast<const float2*>(p + r * D + lane * kLane + c);
      }
    }
    float now = m;
#pragma unroll
    for (int u = 0; u < kFlight; ++u) now = fmaxf(now, ml[u].x);
    const float base = now == -INFINITY ? 0.f : now, f = exp2f(m - base);
    m = now;
    l *= f;
#pragma unroll
    for (int c = 0; c < kLane; ++c) o[c] *= f;
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (i + u * kSplit >= n) break;
      const float g = exp2f(ml[u].x - base);
      l = fmaf(ml[u].y, g, l);
#pragma unroll
      for (int c = 0; c < kLane; ++c) o[c] = fmaf(x[u][c], g, o[c]);
    }
  }
  const int64_t row = static_cast<int64_t>(b) * a.H + h;
  if constexpr (kSplit == 1) {
#pragma unroll
    for (int c = 0; c < kLane; ++c) put_out(a, row * D + lane * kLane + c, l != 0.f ? o[c] / l : 0.f);
    if (lane == 0) a.lse[row] = natural_lse(m, l);
    return;
  }
#pragma unroll
  for (int c = 0; c < kLane; ++c) acc[warp][lane * kLane + c] = o[c];
  if (lane == 0) {
    stat[warp][0] = m;
    stat[warp][1] = l;
  }
  __syncthreads();
  if (threadIdx.x >= D) return;
  float mx = -INFINITY, sum = 0.f, x = 0.f;
#pragma unroll
  for (int i = 0; i < kSplit; ++i) mx = fmaxf(mx, stat[i][0]);
  const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
  for (int i = 0; i < kSplit; ++i) {
    const float g = exp2f(stat[i][0] - base);
    sum = fmaf(stat[i][1], g, sum);
    x = fmaf(acc[i][threadIdx.x], g, x);
  }
  put_out(a, row * D + threadIdx.x, sum != 0.f ? x / sum : 0.f);
  if (threadIdx.x == 0) a.lse[row] = natural_lse(mx, sum);
}

template <int D, bool kF32, int kTiles>
cudaError_t decode_q4(const PagedArgs& a, cudaStream_t s) {
  using Few = Q4Unit<D, kF32, kTiles, kQ4FewKeys>;
  const int cs = q4_cluster(!kF32, a.B, a.Hkv, a.G, a.max_pages, a.page_shift);
  if (cs > 0) return launch_clustered<Few>(a, cs, s);
  using U = Q4Unit<D, kF32, kTiles, q4_chunk(!kF32, 8 * kTiles)>;
  const int smem = U::kSmem + (a.B + 1) * 4;
  static_assert(U::kSmem + (kPagedMaxBatch + 8) * 4 <= 227 * 1024, "shared memory budget");
  cudaError_t e;
  if ((e = allow_smem<q4_decode_kernel<U>>(U::kSmem + (kPagedMaxBatch + 1) * 4)) != cudaSuccess) return e;
  const int ctas = q4_ctas(!kF32, U::kRows, smem, a.sms), rows = U::kRows;
  e = launch_clusters(q4_decode_kernel<U>, ctas, 1, 1, 1, kDecThreads, smem, true, s, a);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.B) * a.Hkv * ((a.G + rows - 1) / rows), partials = ctas * kDecWarps / units;
  if (partials <= 8) return launch_clusters(q4_join_kernel<D, 1>, (a.H + 3) / 4, a.B, 1, 1, 128, 0, true, s, a, rows);
  if (partials <= 32) return launch_clusters(q4_join_kernel<D, 4>, a.H, a.B, 1, 1, 128, 0, true, s, a, rows);
  return launch_clusters(q4_join_kernel<D, 16>, a.H, a.B, 1, 1, 512, 0, true, s, a, rows);
}

template <typename... P>
cudaError_t launch_rows(void (*kernel)(P...), const PagedArgs& a, int rows_per_cta, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.T) * a.Hkv;  // below 2^31
  return launch_clusters(kernel, (rows + rows_per_cta - 1) / rows_per_cta, a.B, 1, 1, kRowThreads, 0, true, s, a);
}

}  // namespace

cudaError_t launch_q4_append(const PagedArgs& a, bool bf16, cudaStream_t s) {
  const int rows = kRowThreads / (a.D / 16);
  if (a.D == 64)
    return bf16 ? launch_rows(q4_append_kernel<64, __nv_bfloat16>, a, rows, s) : launch_rows(q4_append_kernel<64, float>, a, rows, s);
  return bf16 ? launch_rows(q4_append_kernel<128, __nv_bfloat16>, a, rows, s) : launch_rows(q4_append_kernel<128, float>, a, rows, s);
}

cudaError_t launch_q4_read(const PagedArgs& a, bool bf16, cudaStream_t s) {
  const int rows = kRowThreads / (a.D / 8) * 2;
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
