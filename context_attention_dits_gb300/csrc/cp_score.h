// cp_score.h — launch parameters of the score-rule attention (forward,
// backward) and of the paged cache, shared by their kernels and entry points.
// Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>

namespace cp {

// One 64-row block of a document-id row: the smallest and largest id >= 0 in
// it (INT_MAX, -1 if none) and whether it holds a negative id.
struct DocRange {
  int lo, hi, neg, pad;
};
constexpr int kDocBlock = 64;
constexpr int kScoreMaxTokens = 1 << 21;  // query rows or keys of a call

// A scored attention launch. Tensors are dense: q, out, dout, dq [B, Sq, H, D];
// k, v, dk, dv [B, Skv, Hkv, D]; lse, delta [B, H, Sq].
struct ScoreArgs {
  int B, H, Hkv, G, Sq, Skv;  // G = H / Hkv query heads share a key/value head
  float scale;
  float cap;              // 0: none
  const float* slopes;    // [H], or nullptr
  int causal;
  int rel;                // position of query row 0 minus position of key row 0
  const int* prefix;      // [B] positions, or nullptr
  int kv_pos0;            // position of key row 0 (prefix is in positions)
  const int* qdoc;        // [B, Sq], or nullptr
  const int* kdoc;        // [B, Skv]
  const DocRange* qrange;  // [B, ceil(Sq / 64)], set with qdoc
  const DocRange* krange;  // [B, ceil(Skv / 64)]
  const void *q, *k, *v;
  const void *o, *dout;  // backward: the forward's out, and its gradient
  void* out;             // forward
  float* lse;            // forward: written; backward: read
  float* delta;          // backward, fp32 inputs: [B, H, Sq]
  float* lse2p;          // backward, bf16: -lse log2e and delta, each (batch entry, head) padded to 64 rows
  float* dltp;
  void *dq, *dk, *dv;
  int out_bf16;   // type of out
  int grad_bf16;  // type of dq, dk, dv
  int sms;        // multiprocessors of the device
  uint32_t* err;  // tensor-core kernels: device error word and the bound on each wait
  uint64_t timeout_ns;
};

// Keys j < key_limit(i) satisfy the causal rule for query row i of batch entry
// b: position(j) <= position(i), or position(j) < prefix.
__device__ __forceinline__ int prefix_limit(const ScoreArgs& a, int b) {
  return a.prefix ? max(a.prefix[b], 0) - a.kv_pos0 : INT_MIN;
}
__device__ __forceinline__ int key_limit(const ScoreArgs& a, int plim, int i) {
  return a.causal ? max(a.rel + i + 1, plim) : INT_MAX;
}

// Whether any pair of two blocks can share a document.
__device__ __forceinline__ bool docs_meet(const DocRange& q, const DocRange& k) {
  return q.lo <= k.hi && k.lo <= q.hi;  // an empty block has lo = INT_MAX, hi = -1
}
__device__ __forceinline__ DocRange docs_join(const DocRange& x, const DocRange& y) {
  return DocRange{min(x.lo, y.lo), max(x.hi, y.hi), x.neg | y.neg, 0};
}
// Whether every pair of the two blocks is of one document.
__device__ __forceinline__ bool docs_same(const DocRange& q, const DocRange& k) {
  return q.lo == q.hi && k.lo == k.hi && q.lo == k.lo && !q.neg && !k.neg;
}

// Fills qrange and krange from qdoc and kdoc.
cudaError_t launch_doc_ranges(const ScoreArgs& a, cudaStream_t s);
// bf16 on the tensor cores.
cudaError_t launch_score_fwd_tc(const ScoreArgs& a, int D, cudaStream_t s);
cudaError_t launch_score_bwd_tc(const ScoreArgs& a, int D, cudaStream_t s);
// fp32, its products in three passes of tf32.
cudaError_t launch_score_fwd_f32(const ScoreArgs& a, int D, cudaStream_t s);
cudaError_t launch_score_bwd_f32(const ScoreArgs& a, int D, cudaStream_t s);

// The paged cache.
constexpr int kPagedCtas = 304;     // CTAs over the list of blocks at most: two on each of 152 multiprocessors
constexpr int kPagedBlock = 64;     // keys of one work block
constexpr int kPagedMaxBatch = 4096;
struct PagedArgs {
  int B, T, H, Hkv, G, D;
  int num_pages, page_shift, max_pages;
  uint32_t positions;  // append: what the tables hold a place for, 2^31 at most (a 64-bit test took 7% more)
  const int* table;     // [B, max_pages]
  const int* seq_lens;  // [B]
  const int* new_lens;  // append: [B], or nullptr (all T)
  const void *k_new, *v_new;  // append: [B, T, Hkv, D]
  void *k_cache, *v_cache;    // [num_pages, page, Hkv, D]; in 4 bits: codes [num_pages, Hkv, page, D / 2]
  void *k_scales, *v_scales;  // in 4 bits: [num_pages, Hkv, page, D / 64, 2], scale and offset
  void *k_out, *v_out;        // read: [B, T, Hkv, D]
  const void* q;  // decode: [B, H, D]
  void* out;
  float* lse;  // [B, H]
  int out_bf16;
  float scale, cap;
  const float* slopes;
  float* partial;  // workspace: [CTAs over the list; in 4 bits their warps][2] partial results
  int2* info;      // workspace: [B * Hkv * groups] which partials make up a unit
  int sms;         // multiprocessors of the device
  uint32_t* err;
  // in 4 bits
  uint64_t timeout_ns;  // bound on each wait
  uint32_t stall;       // 0; in tests, warps of each decode CTA (a bit each) whose copies never count as done
  uint32_t hkv_mul;     // x / Hkv is the upper word of x hkv_mul, hkv_shift bits less, for x < 2^31
  int hkv_shift;
};
// Query heads that share a key/value head are taken this many at a time.
constexpr int paged_rows(bool bf16) { return bf16 ? 16 : 8; }
// CTAs that run at once on 152 multiprocessors: two on each where their buffers fit.
constexpr int paged_ctas(int D, bool bf16) { return D * (bf16 ? 2 : 4) <= 256 ? kPagedCtas : kPagedCtas / 2; }
// CTAs that share a list of `blocks` blocks: as many as run at once, so that no
// second wave of equal ranges follows, on a device with fewer multiprocessors too.
inline int paged_grid(int D, bool bf16, int64_t blocks, int sms) {
  const int most = paged_ctas(D, bf16), at_once = most / 152 * sms, ctas = at_once < most ? at_once : most;
  return blocks < 1 ? 1 : blocks < ctas ? static_cast<int>(blocks) : ctas;
}
// Decode in one launch: the CTAs (1 to 16, a cluster) that share a unit (a
// sequence's key/value head and group of query heads), or 0 where the list of all
// blocks is cut among the CTAs instead. Clusters save the second launch and the
// workspace, but a unit has 8 or 16 CTAs at most and idle ones take no other's work. So:
// two blocks a CTA where all units' CTAs run at once (on 152 multiprocessors: the
// workspace's size, which hangs on this, is asked for without a device), more
// where they would not, up to 8 (bf16) or 4 (fp32, whose blocks are twice the
// bytes). Clusters against the list, 24 heads on 8, D = 128, device us: bf16 1 x 1000 keys 5.6 / 8.4,
// 1 x 4096 10.0 / 11.7, 8 x 1000 8.7 / 10.4, 4 x 4096 11.7 / 15.9, 1 x 8000
// (16 blocks a CTA) 15.9 / 15.1; fp32 1 x 1000 8.2 / 9.9, 1 x 4096 (8) 18.1 / 15.0.
// Clusters of 16 find room beside each other for some 8 units, and only where two
// CTAs fit a multiprocessor: against clusters of 8, bf16 1 x 4096 8.7 / 10.0,
// 1 x 8192 12.1 / 13.7, 1 x 2000 6.7 / 6.9, 1 x 1500 6.8 / 6.2, but 2 x 2000 (16
// units) 12.5 / 7.9, fp32 1 x 2000 16.1 / 11.3.
constexpr int kPagedCluster = 16;
inline int paged_cluster(int D, bool bf16, int B, int Hkv, int G, int max_pages, int page_shift) {
  const int64_t blocks = ((static_cast<int64_t>(max_pages) << page_shift) + kPagedBlock - 1) / kPagedBlock;
  const int64_t units = static_cast<int64_t>(B) * Hkv * ((G + paged_rows(bf16) - 1) / paged_rows(bf16));
  const int ctas = paged_ctas(D, bf16);
  int cs = 1;
  const int most = units <= 8 && ctas == kPagedCtas ? kPagedCluster : kPagedCluster / 2;
  while (cs < most && blocks > (cs < 8 ? 2 : 4) * cs && units * cs * 2 <= ctas) cs *= 2;
  return units <= ctas && blocks <= cs * (bf16 ? 8 : 4) ? cs : 0;
}
cudaError_t launch_paged_append(const PagedArgs& a, int elem_bytes, cudaStream_t s);
cudaError_t launch_paged_decode(const PagedArgs& a, bool bf16, cudaStream_t s);

// The cache in 4 bits.
constexpr int kQ4Group = 64;   // values that share a scale and an offset
constexpr int kQ4MinPage = 16;
// Query heads of a unit: as many columns of the matrix instruction, or twice.
constexpr int q4_rows(bool bf16, int G) { return bf16 && G > 8 ? 16 : 8; }
// Keys of a warp's step. Longer steps have more products under way and fewer
// overheads a key, shorter ones share few keys among more CTAs (clusters).
constexpr int kQ4FewKeys = 32;
constexpr int q4_chunk(bool bf16, int rows) { return bf16 && rows == 8 ? 64 : 32; }
// CTAs on a multiprocessor, as far as their registers go.
constexpr int q4_per_sm(bool bf16, int rows, int chunk) { return bf16 && rows == 8 ? (chunk == 64 ? 2 : 4) : 2; }
// CTAs over the list: as many as run at once on 152 multiprocessors at most, with
// `smem` bytes of shared memory each (the list's own share grows with the batch).
inline int q4_ctas(bool bf16, int rows, int smem, int sms) {
  const int by_smem = 228 * 1024 / (smem + 1536), by_regs = q4_per_sm(bf16, rows, q4_chunk(bf16, rows));
  return (by_smem < by_regs ? by_smem : by_regs) * (sms < 152 ? sms : 152);
}
// CTAs of a cluster that share a unit, or 0 for the list, as paged_cluster.
inline int q4_cluster(bool bf16, int B, int Hkv, int G, int max_pages, int page_shift) {
  const int rows = q4_rows(bf16, G);
  const int64_t blocks = ((static_cast<int64_t>(max_pages) << page_shift) + 4 * kQ4FewKeys - 1) / (4 * kQ4FewKeys);
  const int64_t units = static_cast<int64_t>(B) * Hkv * ((G + rows - 1) / rows);
  const int ctas = q4_per_sm(bf16, rows, kQ4FewKeys) * 152;
  const int most = units <= 8 ? kPagedCluster : kPagedCluster / 2;
  int cs = 1;
  while (cs < most && blocks > cs && units * cs * 2 <= ctas) cs *= 2;
  return units <= ctas && blocks <= cs * 4 ? cs : 0;
}
// Division by d (1 .. 65535) of numbers below 2^31 by a multiplication (that by an invariant
// integer of Granlund and Montgomery): with 2^s >= d > 2^(s - 1), mul is
// 2^(31 + s) / d rounded up, off by less than 1, which n < 2^31 makes less than 1 / d.
inline void divide_by(int d, uint32_t* mul, int* shift) {
  int s = 0;
  while ((1 << s) < d) ++s;
  *mul = static_cast<uint32_t>((uint64_t{1} << (31 + s)) / d + (d & (d - 1) ? 1 : 0));
  *shift = s - 1;  // (d = 1: -1, and mul 2^31)
}
cudaError_t launch_q4_append(const PagedArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_q4_read(const PagedArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_q4_decode(const PagedArgs& a, bool bf16, cudaStream_t s);

// Lets a kernel use `bytes` of dynamic shared memory, once per device (the call
// costs as much host time as a launch).
template <auto kKernel, bool kClusters16 = false>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (kClusters16 && e == cudaSuccess) e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t{1} << dev, std::memory_order_release);
  return e;
}

// CTAs that share an item, 1 to 8: the size with the least estimated time. Items
// of kind a (taken by clusters) and b (by clusters too if b_clusters, else by
// single CTAs) have up to tiles_a and tiles_b steps, `over` steps of their own
// for start and join, and a part `fill` of the steps on average; the estimate is
// the longest item's time or all items' over the multiprocessors. Where items
// fill a wave of their own a cluster only adds starts and joins (fp32, 104 items
// of 7 tiles: 22 us alone, 29 in clusters of 2); it pays where a few are long
// (fp32, 32 query heads on one: backward 2544 us alone, 1288 in clusters of 2).
inline int cluster_for(double over, int64_t items_a, int64_t tiles_a, int64_t items_b, int64_t tiles_b, double fill,
                       bool b_clusters, int sms) {
  int best = 1;
  double least = 0;
  for (int cs = 1; cs <= 8; cs *= 2) {
    const int cb = b_clusters ? cs : 1;
    const double ta = static_cast<double>((tiles_a + cs - 1) / cs), tb = static_cast<double>((tiles_b + cb - 1) / cb);
    const double all = (items_a * cs * (fill * ta + over) + items_b * cb * (fill * tb + over)) / sms;
    double t = all;
    if (items_a > 0 && ta + over > t) t = ta + over;
    if (items_b > 0 && tb + over > t) t = tb + over;
    if (cs == 1 || t < 0.9 * least) {
      best = cs;
      least = t;
    }
  }
  return best;
}

// Launches items x y x z clusters of `cluster` CTAs each; `after`: the launch may
// start while its predecessor in the stream ends (the kernel calls grid_wait).
template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), int64_t items, unsigned y, unsigned z, int cluster, int threads,
                            int smem, bool after, cudaStream_t s, const A&... args) {
  if (items * cluster > 0x7fffffff || y > 65535 || z > 65535) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(items * cluster), y, z);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2]{};
  cfg.attrs = at;
  if (cluster > 1) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = cluster;
    at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (after) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// From cp_api.cu: the checks and tensor maps that the entry points share.
// 0, or the cp_status of the current device's check.
int host_device(uint32_t** err, int* sms);
// bf16 [Bn, S, H, D] with 64-column x box_rows boxes of one head, 128-byte swizzle.
bool host_tmap_bf16(CUtensorMap* m, const void* base, int D, int H, int S, int Bn, int box_rows);

}  // namespace cp
