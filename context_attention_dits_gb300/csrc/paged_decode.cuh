// paged_decode.cuh — one-token attention over a paged cache. The clusters, the work
// list's sums and the writing of results serve both caches; the kernel over the list and
// its join serve paged.cu alone (paged_q4.cu cuts the list among warps and has its own).
// A kernel's class C says what a cached row is:
//   kD, kRows      head width, query heads of a unit (a sequence's key/value head and
//                  a group of the query heads that share it)
//   kBlock         keys of a work block, of which each of the CTA's warps has a part
//   kWarpB, kState bytes between the warps' buffers, and the floats of a warp's state:
//                  O [kRows][kD], then m (units of log2) and l of each head
//   kPerSm         CTAs on a multiprocessor that its registers leave room for (0: whatever comes)
//   kEarly         clusters may start while their predecessor in the stream ends
//   Shared, C(a, smem, shared), run(a, b, n, hk, hg, blk0, blk1, smem, shared)
//                  what a CTA shares and keeps, and a unit's blocks [blk0, blk1) of n
//                  keys: leaves each warp's state at the start of its buffers
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "cp_ptx.cuh"
#include "cp_score.h"

namespace cp {
namespace {

constexpr float kL2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

constexpr int kDecThreads = 128;
constexpr int kDecWarps = 4;

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

// Element i of a unit's O over the CTA's four warps, relative to the largest
// maximum mx of its head; sum: the weights'.
template <class C>
__device__ __forceinline__ float join_warps(const uint8_t* smem, int i, float& mx, float& sum) {
  constexpr int D = C::kD;
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

// The work list: cum[b], b = 0 .. B, becomes the blocks of kBlock keys before sequence
// b, counting each block HG times. The CTA's threads all come here.
template <int kBlock>
__device__ __forceinline__ int work_list(const PagedArgs& a, int HG, int* cum, int* wsum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += kDecThreads) {
    const int b = b0 + threadIdx.x;
    const int x = b < a.B ? (seq_len(a, b) + kBlock - 1) / kBlock * HG : 0;
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
  return carry;
}
// Sequences without a token: out 0, lse -inf.
template <int D>
__device__ __forceinline__ void no_tokens(const PagedArgs& a, const int* cum) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (cum[b + 1] != cum[b]) continue;
    for (int i = threadIdx.x; i < a.H * D; i += kDecThreads) put_out(a, static_cast<int64_t>(b) * a.H * D + i, 0.f);
    for (int i = threadIdx.x; i < a.H; i += kDecThreads) a.lse[static_cast<int64_t>(b) * a.H + i] = -INFINITY;
  }
}
// The sequence of the list's block `at`.
__device__ __forceinline__ int sequence_of(const PagedArgs& a, const int* cum, int at) {
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (cum[mid] <= at) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The list: all units' blocks of C::kBlock keys, cut into equal contiguous ranges,
// one per CTA.
template <class C>
__global__ void __launch_bounds__(kDecThreads, C::kPerSm) paged_decode_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int D = C::kD;
  extern __shared__ __align__(128) uint8_t smem[];
  int* cum = reinterpret_cast<int*>(smem + C::kSmem);  // [B + 1]: blocks before sequence b
  __shared__ int wsum[kDecWarps];
  __shared__ typename C::Shared shared;
  C unit(a, smem, shared);
  const int groups = (a.G + C::kRows - 1) / C::kRows;
  const int HG = a.Hkv * groups;
  const int total = work_list<C::kBlock>(a, HG, cum, wsum);
  no_tokens<D>(a, cum);
  const int share = (total + gridDim.x - 1) / gridDim.x;
  const int begin = min(total, static_cast<int>(blockIdx.x) * share), end = min(total, begin + share);
  if (begin >= end) return;

  int b = sequence_of(a, cum, begin);
  for (int at = begin; at < end;) {
    while (cum[b + 1] <= at) ++b;
    const int n = min(max(a.seq_lens[b], 0), table_len(a));
    const int nblk = (n + C::kBlock - 1) / C::kBlock;
    const int u = (at - cum[b]) / nblk, blk0 = (at - cum[b]) - u * nblk;
    const int blk1 = min(nblk, blk0 + end - at);
    const int unit0 = at - blk0;  // the unit's first block in the list
    const int hk = u / groups, hg = u - hk * groups;
    const int h0 = hk * a.G + hg * C::kRows, nrow = min(C::kRows, a.G - hg * C::kRows);
    unit.run(a, b, n, hk, hg, blk0, blk1, smem, shared);
    // ---- the warps' states joined: written out, or left as a partial ----
    __syncthreads();
    const bool whole = blk0 == 0 && blk1 == nblk;
    const int slot = at == begin ? 0 : 1;
    const int width = min(C::kRows, a.G);  // heads of a partial: O, then m and l
    float* part = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * width * (D + 2);
    for (int i = threadIdx.x; i < nrow * D; i += kDecThreads) {
      const int r = i / D;
      float mx, sum;
      const float acc = join_warps<C>(smem, i, mx, sum);
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
// 32 loads under way (a dependent walk over 32 partials took 10 us).
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
  for (int i = 0; i < n; i += 32) {
    float x[32];
#pragma unroll
    for (int u = 0; u < 32; ++u)
      if (i + u < n) x[u] = part(i + u)[r * D + d];
#pragma unroll
    for (int u = 0; u < 32; ++u)
      if (i + u < n) acc = fmaf(x[u], weight[i + u], acc);
  }
  store();
}

// A unit by a cluster of CTAs, each with an equal part of its blocks; the parts
// are joined through distributed shared memory. One launch and no workspace, for
// short tables (paged_cluster).
template <class C>
__global__ void __launch_bounds__(kDecThreads, C::kPerSm) paged_decode_cluster_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int D = C::kD;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ typename C::Shared shared;
  C unit(a, smem, shared);
  if (C::kEarly) grid_wait();
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
  const int nblk = (n + C::kBlock - 1) / C::kBlock;
  unit.run(a, b, n, hk, hg, cluster_part(nblk, rank, cs), cluster_part(nblk, rank + 1, cs), smem, shared);
  __syncthreads();
  // this CTA's state, behind the first warp's
  float* part = reinterpret_cast<float*>(smem) + C::kState;
  for (int i = threadIdx.x; i < nrow * D; i += kDecThreads) {
    float mx, sum;
    const float acc = join_warps<C>(smem, i, mx, sum);
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

// One launch by clusters of cs CTAs.
template <class C>
cudaError_t launch_clustered(const PagedArgs& a, int cs, cudaStream_t s) {
  cudaError_t e;
  if ((e = allow_smem<paged_decode_cluster_kernel<C>, true>(C::kSmem)) != cudaSuccess) return e;
  const int units = a.Hkv * ((a.G + C::kRows - 1) / C::kRows);
  return launch_clusters(paged_decode_cluster_kernel<C>, units, a.B, 1, cs, kDecThreads, C::kSmem, C::kEarly, s, a);
}

// At most `ctas` (kPagedCtas or fewer) CTAs over the list, and the join of what they leave.
template <class C>
cudaError_t launch_listed(const PagedArgs& a, int ctas, cudaStream_t s) {
  constexpr int D = C::kD;
  static_assert(C::kSmem + (kPagedMaxBatch + 8) * 4 <= 227 * 1024, "shared memory budget");
  if (ctas > kPagedCtas) return cudaErrorInvalidValue;  // (what the workspace and the join hold)
  cudaError_t e;
  if ((e = allow_smem<paged_decode_kernel<C>>(C::kSmem + (kPagedMaxBatch + 1) * 4)) != cudaSuccess) return e;
  // blocks of the list if every table were full; a unit of one block is never split
  const int groups = (a.G + C::kRows - 1) / C::kRows;
  const int64_t per_unit = ((static_cast<int64_t>(a.max_pages) << a.page_shift) + C::kBlock - 1) / C::kBlock;
  const int64_t bound = per_unit * a.Hkv * groups * a.B;
  const int grid = bound < 1 ? 1 : bound < ctas ? static_cast<int>(bound) : ctas;
  paged_decode_kernel<C><<<grid, kDecThreads, C::kSmem + (a.B + 1) * 4, s>>>(a);
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
}  // namespace cp
