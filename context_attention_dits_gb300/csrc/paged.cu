// paged.cu — the paged key/value cache: rows of new tokens written into pages,
// and attention of one new token per sequence over the pages.
//
// A cache is [num_pages, page, Hkv, D]; key j of sequence b is row j mod page
// of page table[b][j / page]. With n = seq_lens[b] and q the sequence's new
// token (position n - 1):
//   x_j = scale q.k_j, capped to cap tanh(x / cap), less slope_h (n - 1 - j)
//   out = sum_j softmax_j(x_j) v_j,  lse = ln sum_j exp(x_j),  j < n
//
// Decode reads every cached row once and computes 4 G D flop per row pair of
// 4 D bytes (bf16): it is bound by HBM. What the split has to give is enough
// bytes in flight on every multiprocessor whatever the batch: all work is laid
// out as one list of 64-key blocks (sequence, key/value head, group of query
// heads, block), cut into equal contiguous ranges, one per CTA. A CTA's range
// holds at most one unit (sequence, head) that began in an earlier CTA and one
// that goes on in the next; those leave a partial (O, m, l) each, which a
// second launch joins. Units that lie within one CTA are written directly.
// Where the tables are short and the units few (paged_cluster), a unit is taken
// by a cluster of CTAs instead, which joins its parts itself: one launch.
// Each warp streams its own 16 keys of every block through kStages buffers of
// its own with 16-byte asynchronous copies (one row of one head is 128 to 512
// contiguous bytes), so no barrier of the CTA stands in the loop; the warps'
// states are joined at the end of a unit.
// bf16: Q K^T and P V on m16n8k16 matrix instructions (16 query heads, 16
// keys); the tile is far too small for a 128-row tensor-memory MMA, and the
// instruction's rate is not what bounds it. fp32: the same in three passes of
// tf32, 8 query heads.
// Measured, device time: 2 x 262144 keys, 32 heads on 4, D = 128, bf16 170 us
// (6.3 TB/s), 48 x 4096 keys, 24 on 8 125 us (6.4), 48 ragged ones, log-uniform
// from 512 to 8192, 90 us for one draw of 131167 keys (6.0; 5.2 to 6.0 by the
// draw: units end inside the ranges, and a pipeline starts anew with each); fp32
// 8 x 16384 keys 183 us (5.9); 1 x 1000 keys 5.9 us under a table for 1000, 9.1
// under one for 65536 tokens (the path goes by the table's width, all that the
// host knows). More than 16 query heads on one (8 in fp32) read its rows once for
// each 16: 32 on one 3.0 TB/s of the cache's bytes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "cp_internal.h"
#include "cp_ptx.cuh"
#include "cp_score.h"
#include "tf32.cuh"

namespace cp {
namespace {

constexpr float kL2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

// Row (page * page_size + row in page) of token pos of sequence b, or -1 (and
// the error word) if its page is out of range.
__device__ __forceinline__ int cache_row(const PagedArgs& a, int b, int pos) {
  const int pg = pos >> a.page_shift;
  const int id = a.table[static_cast<int64_t>(b) * a.max_pages + pg];
  if (id < 0 || id >= a.num_pages) {
    atomicOr(a.err, kDevErrPage);
    return -1;
  }
  return (id << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

// ----------------------------------------------------------------------------
// Append. A row of a token is Hkv * D elements, contiguous on both sides; TPR
// threads share a row, each moving 16 bytes of k and of v at a time. Bound by
// HBM where there are many rows, by the launch where there are few. The first
// pieces are on their way before the row's place is looked up (a length, then a
// page), whose latency is as long as theirs. 6 sequences with up to 4607 new
// tokens of 8 heads of 128, bf16, 113 MB read and written in all: 21.2 us; one
// token of 64 sequences 1.7 us.
// ----------------------------------------------------------------------------
template <int TPR>
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ PagedArgs a, int pieces) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / TPR) + threadIdx.x / TPR;
  if (row >= static_cast<int64_t>(a.B) * a.T) return;
  const int b = static_cast<int>(row) / a.T, t = static_cast<int>(row) - b * a.T;  // B * T < 2^31
  const int n = a.seq_lens[b];
  if (a.new_lens && t >= a.new_lens[b]) return;
  const uint4* ks = static_cast<const uint4*>(a.k_new) + row * pieces;
  const uint4* vs = static_cast<const uint4*>(a.v_new) + row * pieces;
  int p = threadIdx.x % TPR;
  uint4 x, y;
  if (p < pieces) {
    x = ks[p];
    y = vs[p];
  }
  const uint32_t pos = static_cast<uint32_t>(n) + static_cast<uint32_t>(t);  // (both below 2^31)
  if (n < 0 || pos >= a.positions) {
    atomicOr(a.err, kDevErrPage);
    return;
  }
  const int dst = cache_row(a, b, static_cast<int>(pos));
  if (dst < 0) return;
  uint4* kd = static_cast<uint4*>(a.k_cache) + static_cast<int64_t>(dst) * pieces;
  uint4* vd = static_cast<uint4*>(a.v_cache) + static_cast<int64_t>(dst) * pieces;
  while (p < pieces) {
    kd[p] = x;
    vd[p] = y;
    if ((p += TPR) < pieces) {
      x = ks[p];
      y = vs[p];
    }
  }
}

// ----------------------------------------------------------------------------
// Decode
// ----------------------------------------------------------------------------
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kDecThreads = 128;
constexpr int kDecWarps = 4;
constexpr int kChunk = 16;  // keys of a warp and step
static_assert(kChunk * kDecWarps == kPagedBlock, "a block is a chunk of each warp");

template <int D, typename T>
struct DecCfg {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int kRows = kBf16 ? 16 : 8;          // query heads of a unit
  static constexpr int kRowB = D * sizeof(T);           // bytes of a cached row
  static constexpr int kPieces = kRowB / 16;            // 16-byte pieces of it
  static constexpr int kTile = kChunk * kRowB;          // a chunk's k (or v)
  static constexpr int kStages = kBf16 && D == 64 ? 4 : 3;
  static constexpr int kWarpB = kStages * 2 * kTile;    // a warp's buffers
  static constexpr int kState = kRows * (D + 2);        // floats of a warp's state: O, then m and l
  static_assert(kStages <= 4, "have");
  static_assert(kWarpB >= 2 * kState * 4, "a warp's buffers hold its state at the end of a unit, the first's the CTA's too");
  static constexpr int kSmem = kDecWarps * kWarpB;
  static constexpr int kCtas = paged_ctas(D, kBf16);
  static_assert(kCtas == 152 || 2 * (kSmem + kPagedMaxBatch * 4 + 2048) <= 228 * 1024, "two CTAs on a multiprocessor");
};

// A score in units of log2, dist keys back.
struct DecScore {
  float scale, cap, inv_cap;
  __device__ __forceinline__ float operator()(float dot, float slope2, float dist) const {
    float x = dot * scale;
    if (cap > 0.f) x = cap * tanhf(x * inv_cap);
    return fmaf(x, kL2e, -slope2 * dist);
  }
};

// The length of sequence b, held within what its row of the table can address.
__device__ __forceinline__ int table_len(const PagedArgs& a) {
  return static_cast<int>(min(static_cast<int64_t>(a.max_pages) << a.page_shift, int64_t{INT_MAX - 64}));
}
__device__ __forceinline__ int seq_len(const PagedArgs& a, int b) {
  const int n = a.seq_lens[b], most = table_len(a);
  if (n < 0 || n > most) {
    atomicOr(a.err, kDevErrPage);
    return n < 0 ? 0 : most;
  }
  return n;
}

__device__ __forceinline__ void put_out(const PagedArgs& a, int64_t at, float x) {
  if (a.out_bf16)
    static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16(x);
  else
    static_cast<float*>(a.out)[at] = x;
}
__device__ __forceinline__ float natural_lse(float mx, float sum) {
  return sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

// Blocks [blk0, blk1) of group hg of key/value head hk's query heads, sequence b
// of n tokens: each warp's state into its buffers, O [kRows][D], then m and l.
template <int D, typename T>
__device__ __forceinline__ void decode_unit(const PagedArgs& a, int b, int n, int hk, int hg, int blk0, int blk1,
                                            uint8_t* smem, uint32_t (*have)[4]) {
  using C = DecCfg<D, T>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* wbuf = smem + warp * C::kWarpB;
  const uint32_t wb = smem_addr(wbuf);
  const int64_t tok_b = static_cast<int64_t>(a.Hkv) * C::kRowB;  // bytes of a token's row of all heads
  DecScore score;
  score.scale = a.scale;
  score.cap = a.cap;
  score.inv_cap = a.cap > 0.f ? 1.f / a.cap : 0.f;
  const int h0 = hk * a.G + hg * C::kRows, nrow = min(C::kRows, a.G - hg * C::kRows);
  const uint8_t* kc = static_cast<const uint8_t*>(a.k_cache) + static_cast<int64_t>(hk) * C::kRowB;
  const uint8_t* vc = static_cast<const uint8_t*>(a.v_cache) + static_cast<int64_t>(hk) * C::kRowB;

  // a chunk's rows: lane r < 16 finds row r (-1 past the end)
  auto find = [&](int blk) {
    const int j = blk * kPagedBlock + warp * kChunk + lane;
    const int row = lane < kChunk && blk < blk1 && j < n ? cache_row(a, b, j) : -1;
    __syncwarp();  // the matrix loads and products that follow want the warp converged
    return row;
  };
  auto load = [&](int rows, int stage) {
    const uint32_t base = wb + stage * 2 * C::kTile;
    const uint32_t found = __ballot_sync(0xffffffffu, rows >= 0);
    if (lane == 0) have[warp][stage] = found;
#pragma unroll
    for (int i = lane; i < kChunk * C::kPieces; i += 32) {
      const int r = i / C::kPieces, p = i % C::kPieces;
      const int row = __shfl_sync(0xffffffffu, rows, r);
      const int64_t off = static_cast<int64_t>(max(row, 0)) * tok_b + p * 16;
      const uint32_t d = base + r * C::kRowB + ((p ^ (r & 7)) * 16);
      cp_async16(d, kc + off, row >= 0);
      cp_async16(d + C::kTile, vc + off, row >= 0);
    }
  };

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int rows_next = find(blk0);
#pragma unroll
  for (int st = 0; st < C::kStages - 1; ++st) {
    if (blk0 + st < blk1) load(rows_next, st);
    rows_next = find(blk0 + st + 1);
    cp_async_commit();
  }

  if constexpr (C::kBf16) {
    const int g = lane >> 2, tq = lane & 3;
    uint32_t qf[D / 16][4];
    {
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(b) * a.H + h0) * D;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = g + (e & 1) * 8, d = kk * 16 + tq * 2 + (e >> 1) * 8;
          qf[kk][e] = r < nrow ? *reinterpret_cast<const uint32_t*>(q + r * D + d) : 0u;
        }
    }
    float slope[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) slope[e] = a.slopes && g + 8 * e < nrow ? a.slopes[h0 + g + 8 * e] * kL2e : 0.f;
    float o[D / 8][4];
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[x][e] = 0.f;
    const int lm = lane >> 3, lr = lane & 7;
    const bool two = nrow > 8;
    int stage = 0;
    for (int blk = blk0; blk < blk1; ++blk) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();
      {  // the stage that the last step read is free again
        int st = stage + C::kStages - 1;
        if (st >= C::kStages) st -= C::kStages;
        if (blk + C::kStages - 1 < blk1) load(rows_next, st);
        rows_next = find(blk + C::kStages);
        cp_async_commit();
      }
      const uint32_t kb = wb + stage * 2 * C::kTile, vb = kb + C::kTile;
      const uint32_t on = have[warp][stage];
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const int krow = (lm >> 1) * 8 + lr;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t f[4];
        ldsm4(f, kb + krow * C::kRowB + (((2 * kk + (lm & 1)) ^ (krow & 7)) * 16));
        mma16816(s[0], qf[kk], f[0], f[1]);
        mma16816(s[1], qf[kk], f[2], f[3]);
      }
      const int j0 = blk * kPagedBlock + warp * kChunk + tq * 2;
      uint32_t pf[4];
      float fsc[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // rows g and g + 8
        if (e == 1 && !two) {
          pf[1] = pf[3] = 0u;
          fsc[1] = 1.f;
          break;
        }
        float x[4], mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int j = j0 + (c >> 1) * 8 + (c & 1);
          x[c] = (on >> (tq * 2 + (c >> 1) * 8 + (c & 1))) & 1u ? score(s[c >> 1][2 * e + (c & 1)], slope[e], static_cast<float>(n - 1 - j)) : -INFINITY;
          mx = fmaxf(mx, x[c]);
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[e], mx), base = mn == -INFINITY ? 0.f : mn;
        fsc[e] = ex2_approx(m[e] - base);
        m[e] = mn;
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[c] = ex2_approx(x[c] - base);
          sum += x[c];
        }
        l[e] = l[e] * fsc[e] + sum;
        // P rounded to bf16 for the matrix product; l sums it unrounded
        pf[e] = pack_bf16x2(x[0], x[1]);
        pf[2 + e] = pack_bf16x2(x[2], x[3]);
      }
      if (__any_sync(0xffffffffu, fsc[0] != 1.f || fsc[1] != 1.f)) {
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
          o[x][0] *= fsc[0];
          o[x][1] *= fsc[0];
          o[x][2] *= fsc[1];
          o[x][3] *= fsc[1];
        }
      }
      const int vrow = (lm & 1) * 8 + lr;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        uint32_t f[4];
        ldsm4t(f, vb + vrow * C::kRowB + (((2 * x + (lm >> 1)) ^ (vrow & 7)) * 16));
        mma16816(o[2 * x], pf, f[0], f[1]);
        mma16816(o[2 * x + 1], pf, f[2], f[3]);
      }
      __syncwarp();
      if (++stage == C::kStages) stage = 0;
    }
    // ---- this warp's state into its buffers: O [kRows][D], then m, l ----
    cp_async_wait<0>();
    __syncwarp();
    float* w = reinterpret_cast<float*>(wbuf);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      const int r = g + 8 * e;
#pragma unroll
      for (int x = 0; x < D / 8; ++x)
        *reinterpret_cast<float2*>(w + r * D + x * 8 + tq * 2) = make_float2(o[x][2 * e], o[x][2 * e + 1]);
      if (tq == 0) {
        w[C::kRows * D + 2 * r] = m[e];
        w[C::kRows * D + 2 * r + 1] = l[e];
      }
    }
  } else {
    // fp32 in three passes of tf32 (tf32.cuh), keys as the rows: S^T = K Q^T
    // (16 keys x 8 heads), then O^T = V^T P^T (D x 8 heads, 16 keys); a lane
    // holds the statistics of heads 2 tq and 2 tq + 1
    const int g = lane >> 2, tq = lane & 3;
    const float* q = static_cast<const float*>(a.q) + (static_cast<int64_t>(b) * a.H + h0 + g) * D;
    uint32_t qh[D / 8][2], ql[D / 8][2];
#pragma unroll
    for (int kk = 0; kk < D / 8; ++kk)
#pragma unroll
      for (int e = 0; e < 2; ++e) split_tf32(g < nrow ? q[8 * kk + tq + 4 * e] : 0.f, qh[kk][e], ql[kk][e]);
    float slope[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) slope[e] = a.slopes && 2 * tq + e < nrow ? a.slopes[h0 + 2 * tq + e] * kL2e : 0.f;
    float o[D / 16][4];
#pragma unroll
    for (int x = 0; x < D / 16; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[x][e] = 0.f;
    int stage = 0;
    for (int blk = blk0; blk < blk1; ++blk) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();
      {
        int st = stage + C::kStages - 1;
        if (st >= C::kStages) st -= C::kStages;
        if (blk + C::kStages - 1 < blk1) load(rows_next, st);
        rows_next = find(blk + C::kStages);
        cp_async_commit();
      }
      const uint8_t* kb = wbuf + stage * 2 * C::kTile;
      const uint8_t* vb = kb + C::kTile;
      const uint32_t on = have[warp][stage];
      // element d of row r of a tile
      auto at = [&](const uint8_t* tile, int r, int d) {
        return *reinterpret_cast<const float*>(tile + r * C::kRowB + (((d >> 2) ^ (r & 7)) * 16) + (d & 3) * 4);
      };
      float s[4] = {0.f, 0.f, 0.f, 0.f}, small[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k0 = 0; k0 < D / 8; k0 += 4) {
        float big[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = k0; kk < k0 + 4; ++kk) {
          uint32_t ah[4], al[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split_tf32(at(kb, g + (e & 1) * 8, 8 * kk + tq + (e >> 1) * 4), ah[e], al[e]);
          mma3_tf32(big, small, ah, al, qh[kk], ql[kk]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += big[e];
      }
      // rows (keys) g and g + 8: elements 0, 1 and 2, 3; columns (heads) 2 tq, 2 tq + 1
      const int j0 = blk * kPagedBlock + warp * kChunk + g;
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x[2], mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          x[u] = -INFINITY;
          if ((on >> (g + 8 * u)) & 1u) {
            x[u] = score(s[2 * u + e] + small[2 * u + e], slope[e], static_cast<float>(n - 1 - j0 - 8 * u));
          }
          mx = fmaxf(mx, x[u]);
        }
#pragma unroll
        for (int of = 16; of > 2; of >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, of));
        const float mn = fmaxf(m[e], mx), base = mn == -INFINITY ? 0.f : mn;
        f[e] = exp2f(m[e] - base);
        m[e] = mn;
        s[e] = exp2f(x[0] - base);
        s[2 + e] = exp2f(x[1] - base);
        l[e] = l[e] * f[e] + s[e] + s[2 + e];
      }
      // P^T as the B operand: key tq (+ 4, 8, 12), head g, from lane 4 key + head / 2
      uint32_t ph[2][2], pl[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int src = (tq + 4 * e) * 4 + (g >> 1);
          const float y0 = __shfl_sync(0xffffffffu, s[2 * u], src), y1 = __shfl_sync(0xffffffffu, s[2 * u + 1], src);
          split_tf32(g & 1 ? y1 : y0, ph[u][e], pl[u][e]);
        }
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        float big[4] = {0.f, 0.f, 0.f, 0.f}, sm[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t ah[4], al[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            split_tf32(at(vb, 8 * u + tq + (e >> 1) * 4, 16 * x + g + (e & 1) * 8), ah[e], al[e]);
          mma3_tf32(big, sm, ah, al, ph[u], pl[u]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x][e] = fmaf(o[x][e], f[e & 1], big[e] + sm[e]);
      }
      __syncwarp();
      if (++stage == C::kStages) stage = 0;
    }
    cp_async_wait<0>();
    __syncwarp();
    float* w = reinterpret_cast<float*>(wbuf);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int of = 16; of > 2; of >>= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], of);
      const int r = 2 * tq + e;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        w[r * D + 16 * x + g] = o[x][e];
        w[r * D + 16 * x + g + 8] = o[x][2 + e];
      }
      if (g == 0) {
        w[C::kRows * D + 2 * r] = m[e];
        w[C::kRows * D + 2 * r + 1] = l[e];
      }
    }
  }
}

// Element i of a unit's O over the CTA's four warps, relative to the largest
// maximum mx of its head; sum: the weights'.
template <int D, typename T>
__device__ __forceinline__ float join_warps(const uint8_t* smem, int i, float& mx, float& sum) {
  using C = DecCfg<D, T>;
  const int r = i / D;
  float mw[kDecWarps], acc = 0.f;
  mx = -INFINITY;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    mw[w] = reinterpret_cast<const float*>(smem + w * C::kWarpB)[C::kRows * D + 2 * r];
    mx = fmaxf(mx, mw[w]);
  }
  const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    const float* st = reinterpret_cast<const float*>(smem + w * C::kWarpB);
    const float f = exp2f(mw[w] - base);
    sum = fmaf(st[C::kRows * D + 2 * r + 1], f, sum);
    acc = fmaf(st[i], f, acc);
  }
  return acc;
}

template <int D, typename T>
__global__ void __launch_bounds__(kDecThreads) paged_decode_kernel(const __grid_constant__ PagedArgs a) {
  using C = DecCfg<D, T>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int cum[kPagedMaxBatch + 1];  // blocks before sequence b
  __shared__ int wsum[kDecWarps];
  __shared__ uint32_t have[kDecWarps][4];  // the rows that a stage holds, a bit each
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (a.G + C::kRows - 1) / C::kRows;
  const int HG = a.Hkv * groups;
  // ---- the work list: an exclusive sum of the sequences' blocks ----
  int carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += kDecThreads) {
    const int b = b0 + threadIdx.x;
    const int x = b < a.B ? (seq_len(a, b) + kPagedBlock - 1) / kPagedBlock * HG : 0;
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    if (lane == 31) wsum[warp] = s;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < kDecWarps; ++w) {
      if (w < warp) before += wsum[w];
      carry += wsum[w];
    }
    if (b < a.B) cum[b] = before + s - x;
    __syncthreads();
  }
  if (threadIdx.x == 0) cum[a.B] = carry;
  __syncthreads();
  const int total = carry;
  // sequences without a token: out 0, lse -inf
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (cum[b + 1] != cum[b]) continue;
    for (int i = threadIdx.x; i < a.H * D; i += kDecThreads) put_out(a, static_cast<int64_t>(b) * a.H * D + i, 0.f);
    for (int i = threadIdx.x; i < a.H; i += kDecThreads) a.lse[static_cast<int64_t>(b) * a.H + i] = -INFINITY;
  }
  const int share = (total + gridDim.x - 1) / gridDim.x;
  const int begin = min(total, static_cast<int>(blockIdx.x) * share), end = min(total, begin + share);
  if (begin >= end) return;

  int b = 0;
  {  // the sequence of the first block
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (cum[mid] <= begin) lo = mid; else hi = mid - 1;
    }
    b = lo;
  }
  for (int at = begin; at < end;) {
    while (cum[b + 1] <= at) ++b;
    const int n = min(max(a.seq_lens[b], 0), table_len(a));
    const int nblk = (n + kPagedBlock - 1) / kPagedBlock;
    const int u = (at - cum[b]) / nblk, blk0 = (at - cum[b]) - u * nblk;
    const int blk1 = min(nblk, blk0 + end - at);
    const int unit0 = at - blk0;  // the unit's first block in the list
    const int hk = u / groups, hg = u - hk * groups;
    const int h0 = hk * a.G + hg * C::kRows, nrow = min(C::kRows, a.G - hg * C::kRows);
    decode_unit<D, T>(a, b, n, hk, hg, blk0, blk1, smem, have);
    // ---- the warps' states joined: written out, or left as a partial ----
    __syncthreads();
    const bool whole = blk0 == 0 && blk1 == nblk;
    const int slot = at == begin ? 0 : 1;
    const int width = min(C::kRows, a.G);  // heads of a partial: O, then m and l
    float* part = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * width * (D + 2);
    for (int i = threadIdx.x; i < nrow * D; i += kDecThreads) {
      const int r = i / D;
      float mx, sum;
      const float acc = join_warps<D, T>(smem, i, mx, sum);
      if (whole) {
        const int64_t row = static_cast<int64_t>(b) * a.H + h0 + r;
        put_out(a, row * D + i % D, sum != 0.f ? acc / sum : 0.f);
        if (i % D == 0) a.lse[row] = natural_lse(mx, sum);
      } else {
        part[i] = acc;
        if (i % D == 0) {
          part[width * D + 2 * r] = mx;
          part[width * D + 2 * r + 1] = sum;
        }
      }
    }
    if (threadIdx.x == 0 && blk0 == 0)  // the CTA that begins a unit says which partials make it up
      a.info[static_cast<int64_t>(b) * HG + u] =
          whole ? make_int2(0, -1) : make_int2(blockIdx.x * 2 + slot, (unit0 + nblk - 1) / share);
    __syncthreads();  // the buffers are free for the next unit's copies
    at += blk1 - blk0;
  }
}

// Joins the partials of a unit that lay in more than one CTA: the first in the
// slot that info names, the others in slot 0 of the CTAs up to info.y. A thread
// per column; the partials' weights first, a thread each, then the columns with
// eight loads under way (a dependent walk over 32 partials took 10 us).
template <int D>
__global__ void __launch_bounds__(D) paged_join_kernel(const __grid_constant__ PagedArgs a, int rows) {
  __shared__ float weight[kPagedCtas];
  __shared__ float red[2][D / 32];
  const int h = blockIdx.x, b = blockIdx.y, d = threadIdx.x, warp = d >> 5;
  grid_wait();
  if (a.seq_lens[b] <= 0) return;
  const int groups = (a.G + rows - 1) / rows;
  const int hk = h / a.G, r = (h - hk * a.G) % rows, hg = (h - hk * a.G) / rows;
  const int2 w = a.info[(static_cast<int64_t>(b) * a.Hkv + hk) * groups + hg];
  if (w.y < 0) return;
  const int c0 = w.x >> 1, n = w.y - c0 + 1, width = min(rows, a.G), slot_floats = width * (D + 2);
  auto part = [&](int i) {
    return a.partial + (static_cast<int64_t>(c0 + i) * 2 + (i == 0 ? w.x & 1 : 0)) * slot_floats;
  };
  float mx = -INFINITY, sum = 0.f, acc = 0.f;
  auto store = [&]() {
    const int64_t row = static_cast<int64_t>(b) * a.H + h;
    put_out(a, row * D + d, sum != 0.f ? acc / sum : 0.f);
    if (d == 0) a.lse[row] = natural_lse(mx, sum);
  };
  if (n <= 4) {  // every load at once
    float pm[4], pl[4], po[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      pm[i] = -INFINITY;
      pl[i] = po[i] = 0.f;
      if (i < n) {
        const float2 ml = *reinterpret_cast<const float2*>(part(i) + width * D + 2 * r);
        pm[i] = ml.x;
        pl[i] = ml.y;
        po[i] = part(i)[r * D + d];
      }
      mx = fmaxf(mx, pm[i]);
    }
    const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = exp2f(pm[i] - base);
      sum = fmaf(pl[i], f, sum);
      acc = fmaf(po[i], f, acc);
    }
    store();
    return;
  }
  for (int i = d; i < n; i += D) {
    weight[i] = part(i)[width * D + 2 * r];
    mx = fmaxf(mx, weight[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if ((d & 31) == 0) red[0][warp] = mx;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < D / 32; ++i) mx = fmaxf(mx, red[0][i]);
  const float base = mx == -INFINITY ? 0.f : mx;
  for (int i = d; i < n; i += D) {
    weight[i] = exp2f(weight[i] - base);
    sum = fmaf(part(i)[width * D + 2 * r + 1], weight[i], sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((d & 31) == 0) red[1][warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) sum += red[1][i];
  int i = 0;
  for (; i + 8 <= n; i += 8) {
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = part(i + u)[r * D + d];
#pragma unroll
    for (int u = 0; u < 8; ++u) acc = fmaf(x[u], weight[i + u], acc);
  }
  for (; i < n; ++i) acc = fmaf(part(i)[r * D + d], weight[i], acc);
  store();
}

// A unit by a cluster of CTAs, each with an equal part of its blocks; the parts
// are joined through distributed shared memory. One launch and no workspace, for
// short tables (paged_cluster).
template <int D, typename T>
__global__ void __launch_bounds__(kDecThreads) paged_decode_cluster_kernel(const __grid_constant__ PagedArgs a) {
  using C = DecCfg<D, T>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t have[kDecWarps][4];
  const int cs = cluster_size(), rank = cluster_rank();
  const int groups = (a.G + C::kRows - 1) / C::kRows;
  const int u = blockIdx.x / cs, b = blockIdx.y, hk = u / groups, hg = u - hk * groups;
  const int h0 = hk * a.G + hg * C::kRows, nrow = min(C::kRows, a.G - hg * C::kRows);
  const int64_t row0 = static_cast<int64_t>(b) * a.H + h0;
  const int n = seq_len(a, b);
  if (n == 0) {  // the whole cluster leaves
    for (int i = threadIdx.x; rank == 0 && i < nrow * D; i += kDecThreads) put_out(a, row0 * D + i, 0.f);
    for (int r = threadIdx.x; rank == 0 && r < nrow; r += kDecThreads) a.lse[row0 + r] = -INFINITY;
    return;
  }
  const int nblk = (n + kPagedBlock - 1) / kPagedBlock;
  decode_unit<D, T>(a, b, n, hk, hg, cluster_part(nblk, rank, cs), cluster_part(nblk, rank + 1, cs), smem, have);
  __syncthreads();
  // this CTA's state, behind the first warp's
  float* part = reinterpret_cast<float*>(smem) + C::kState;
  for (int i = threadIdx.x; i < nrow * D; i += kDecThreads) {
    float mx, sum;
    const float acc = join_warps<D, T>(smem, i, mx, sum);
    if (cs == 1) {
      put_out(a, row0 * D + i, sum != 0.f ? acc / sum : 0.f);
      if (i % D == 0) a.lse[row0 + i / D] = natural_lse(mx, sum);
    } else {
      part[i] = acc;
      if (i % D == 0) {
        part[C::kRows * D + 2 * (i / D)] = mx;
        part[C::kRows * D + 2 * (i / D) + 1] = sum;
      }
    }
  }
  if (cs == 1) return;
  cluster_sync();
  const uint32_t mine = smem_addr(part);
  auto join = [&](auto most_c) {
    constexpr int kMost = decltype(most_c)::value;
    const int end = 2 * cluster_part(nrow * D / 2, rank + 1, cs);
    for (int i = 2 * (cluster_part(nrow * D / 2, rank, cs) + threadIdx.x); i < end; i += 2 * kDecThreads) {
      const int r = i / D;
      float2 ml[kMost], o[kMost];
#pragma unroll
      for (int c = 0; c < kMost; ++c) {
        ml[c] = make_float2(-INFINITY, 0.f);
        o[c] = make_float2(0.f, 0.f);
        if (c < cs) {  // every load under way at once
          const uint32_t at = cluster_peer(mine, c);
          ml[c] = ld_peer2(at + (C::kRows * D + 2 * r) * 4);
          o[c] = ld_peer2(at + i * 4);
        }
      }
      float mx = -INFINITY, sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int c = 0; c < kMost; ++c) mx = fmaxf(mx, ml[c].x);
      const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int c = 0; c < kMost; ++c) {
        const float f = exp2f(ml[c].x - base);
        sum = fmaf(ml[c].y, f, sum);
        x = fmaf(o[c].x, f, x);
        y = fmaf(o[c].y, f, y);
      }
      put_out(a, row0 * D + i, sum != 0.f ? x / sum : 0.f);
      put_out(a, row0 * D + i + 1, sum != 0.f ? y / sum : 0.f);
      if (i % D == 0) a.lse[row0 + r] = natural_lse(mx, sum);
    }
  };
  if (cs <= 8)
    join(std::integral_constant<int, 8>{});
  else
    join(std::integral_constant<int, kPagedCluster>{});
  cluster_sync();  // a CTA's shared memory stays until its peers have read it
}

template <int D, typename T>
cudaError_t decode_d(const PagedArgs& a, cudaStream_t s) {
  using C = DecCfg<D, T>;
  static_assert(C::kSmem + (kPagedMaxBatch + 8) * 4 <= 227 * 1024, "shared memory budget");
  cudaError_t e;
  const int cs = paged_cluster(D, C::kBf16, a.B, a.Hkv, a.G, a.max_pages, a.page_shift);
  if (cs > 0) {
    if ((e = allow_smem<paged_decode_cluster_kernel<D, T>, true>(C::kSmem)) != cudaSuccess) return e;
    const int units = a.Hkv * ((a.G + C::kRows - 1) / C::kRows);
    return launch_clusters(paged_decode_cluster_kernel<D, T>, units, a.B, 1, cs, kDecThreads, C::kSmem, false, s, a);
  }
  if ((e = allow_smem<paged_decode_kernel<D, T>>(C::kSmem)) != cudaSuccess) return e;
  // blocks of the list if every table were full; a unit of one block is never split
  const int groups = (a.G + C::kRows - 1) / C::kRows;
  const int64_t per_unit = ((static_cast<int64_t>(a.max_pages) << a.page_shift) + kPagedBlock - 1) / kPagedBlock;
  const int64_t bound = per_unit * a.Hkv * groups * a.B;
  paged_decode_kernel<D, T><<<paged_grid(D, C::kBf16, bound, a.sms), kDecThreads, C::kSmem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || per_unit <= 1) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.H, a.B);
  cfg.blockDim = dim3(D);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  // prepared while the decode kernel runs, which does not release it early: the
  // join's CTAs start when the last of decode's have left
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, a, static_cast<int>(C::kRows));
}

}  // namespace

cudaError_t launch_paged_append(const PagedArgs& a, int elem_bytes, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.T;
  if (rows == 0) return cudaSuccess;
  const int pieces = a.Hkv * a.D * elem_bytes / 16;
  // threads a row: enough for one piece each, where a row has as many
  if (pieces <= 32)
    paged_append_kernel<32><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, s>>>(a, pieces);
  else if (pieces <= 64)
    paged_append_kernel<64><<<static_cast<unsigned>((rows + 3) / 4), 256, 0, s>>>(a, pieces);
  else
    paged_append_kernel<128><<<static_cast<unsigned>((rows + 1) / 2), 256, 0, s>>>(a, pieces);
  return cudaGetLastError();
}

cudaError_t launch_paged_decode(const PagedArgs& a, bool bf16, cudaStream_t s) {
  if (a.D == 64) return bf16 ? decode_d<64, __nv_bfloat16>(a, s) : decode_d<64, float>(a, s);
  return bf16 ? decode_d<128, __nv_bfloat16>(a, s) : decode_d<128, float>(a, s);
}

}  // namespace cp
