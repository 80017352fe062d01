// score_fwd_tc.cu — forward of attention with a score rule on the
// 5th-generation tensor cores (tcgen05 + TMEM + TMA), bf16 q, k, v.
//
// With s = q.k: x = scale s, capped to cap tanh(x / cap), less slope |i - j|;
// out = softmax(x) v and lse = ln sum exp x over the pairs that take part.
// An item is two 128-row query tiles of one (batch entry, query head); a CTA walks
// the 128-key tiles that any of their rows reach, with the reference m, sum l and
// unnormalised O of the online softmax; S and O live in tensor memory, P =
// 2^(x log2e - m) is rounded to bf16 over S for the second product (l sums P
// before the rounding, so lse has fp32's accuracy and the rounding errors of out
// average out over the keys).
//
// TMEM layout and the MMA issue order are those of the plain forward kernel. Warp
// roles (352 threads): TMA producer, MMA issuer, two groups of four softmax warps
// (one thread per query row), and one warp that finds the items. What the rule
// adds sits in the softmax warps and in the choice of tiles:
//   * masks: causal with an open prefix is a limit per row (keys below
//     max(position + 1, prefix)), applied only in the tiles it cuts; documents
//     compare ids only in tiles that hold more than one. Tiles that no row
//     reaches are not loaded: past the last row's limit, and, with documents,
//     those whose id range misses the rows' (a bitmap in shared memory, built
//     from the ranges of 64-row blocks that a small launch has put down);
//   * cap: an odd polynomial in s while every |x / cap| of a warp's tile stays
//     below 1/2 (or 1), checked after the fact by the largest s^2; see
//     score_math.cuh;
//   * bias: one more FMA a score in tiles on one side of the diagonal.
// P is formed with whatever reference the row has, 0 at first (the maximum in
// rows of few keys), in place of the running maximum, and checked afterwards by
// the row's sum over the tile (2^-20 to 2^20) and up to it (at most 2^26, which
// leaves v up to 2^96 in rows of any length, and down to 2^-96), and the largest
// s^2; a warp that fails reloads S and takes the exact path (maximum first).
//
// What bounds it: a query tile's step is a chain of S (512 cycles of the tensor
// pipe at D = 128), the softmax (some 1050: 128 exponentials a thread), P V (512)
// and their hand-overs, and two tiles are what tensor memory holds, so that the
// pipe stands still a fifth of the 2650 cycles. Short items are bound by their
// ends: the first loads and S (5000 cycles after a cold start) and the stores of
// out, which come from all multiprocessors at once. A CTA therefore goes on to
// the item of a block that has not started, and the loads and S of its first tile
// go by under the stores of the last (900 cycles from item to item); those with
// the most causal keys first. Measured, 4608 tokens, 24 heads on 8, bf16, D =
// 128: plain 161 us (1618 TFLOP/s; the plain kernel 165), causal 94, cap 50 219,
// causal with it 130, slopes 171, causal with them 99, causal with both 145;
// documents of 512 32 (24 heads on 24: 35). D = 64: 123, 76, 194, 121, 149, 87,
// 145. The eleven warps leave 168 registers a thread; every form spills 28 to 98
// bytes.
// Every wait is bounded (cp_ptx.cuh); on expiry the CTA drains its copies and
// MMAs, frees TMEM and returns.
// A few rows against many keys (a chunk of a long prompt) are too few items for
// the multiprocessors: then the CTAs of a cluster take equal ranges of an item's
// key tiles, leave their (m, l, O) in shared memory, and each joins and stores
// the rows of its share.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "cp_internal.h"
#include "cp_ptx.cuh"
#include "cp_score.h"
#include "score_math.cuh"

namespace cp {
namespace {

constexpr int kThreads = 352;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: rescale only when the max grows by > 2^8
constexpr float kSumMost = 1048576.f;      // of a row's P over a tile
constexpr float kTotalMost = 67108864.f;   // 2^26, over its tiles: beyond, the reference moves up as far
constexpr int kFewKeys = 32;
constexpr uint32_t kTmemCols = 512;
// Words of a bitmap of key tiles: a bit for a tile up to 262144 keys, for 2, 4
// or 8 neighbours beyond.
constexpr int kMapWords = 64;
static_assert(kScoreMaxTokens / kTileN <= kMapWords * 32 * 8, "groups of 8 at most");

template <int D>
struct Smem {
  static constexpr int kQTile = kTileM * D * 2;   // bytes of one bf16 Q tile
  static constexpr int kKVTile = kTileN * D * 2;  // bytes of one bf16 K or V tile
  static constexpr int kHalf = kTileM * 128;      // one 64-column (128-byte) box of a 128-row tile
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + 2 * kQTile;
  static constexpr int kOffV = kOffK + 2 * kKVTile;
  static constexpr int kOffStage = kOffV + 2 * kKVTile;  // a softmax warp's 32 rows x 128 bytes of out on their way
  static constexpr int kOffStat = kOffStage;             // (clusters) [256] rows' m, l
  static constexpr int kOffBar = kOffStage + 8 * 4096;
  static constexpr int kNumBars = 25;
  static constexpr int kOffNext = (kOffBar + kNumBars * 8 + 15) / 16 * 16;  // the next block's index
  static constexpr int kOffItem = kOffNext + 16;                          // [2] Item
  static constexpr int kOffMisc = kOffItem + 2 * 32;
  static constexpr int kOffMap = kOffMisc + 16;  // [2] act, then which tiles are mixed for query tile 0, 1
  static constexpr int kBytes = kOffMap + 2 * 3 * kMapWords * 4;
  // slack to align the base to 1024 bytes; at least 116 KB so that two CTAs
  // never share an SM (each allocates all 512 TMEM columns)
  static constexpr int kAlloc = (kBytes + 1024) > 116 * 1024 ? (kBytes + 1024) : 116 * 1024;
};

// A work item: a pair of query tiles (the last may be single) of one head, and
// this CTA's part of the walk over its key tiles.
struct Item {
  int valid;  // 0: there are no more
  int h, b, row0;
  int plim, ntile;  // prefix_limit; key tiles that the last row reaches
  int n0, NT;       // this CTA's tiles: NT of those that take part, from the n0-th on
};
static_assert(sizeof(Item) == 32, "kOffMisc");

// barrier indices
enum : int {
  kBarQFull = 0,      // +tile
  kBarQEmpty = 2,     // +tile: the item's last S has read Q
  kBarKFull = 4,      // +stage
  kBarKEmpty = 6,     // +stage
  kBarVFull = 8,      // +stage
  kBarVEmpty = 10,    // +stage
  kBarSFull = 12,     // +tile
  kBarPFull = 14,     // +tile
  kBarOFull = 16,     // +tile
  kBarItemFull = 18,  // +slot: an Item and its bitmaps are set
  kBarItemEmpty = 20, // +slot: producer, issuer and the softmax warps have read them
  kBarNear = 22,      // the item's last tiles are being loaded
  kBarNext = 23,      // the next block's index is there
  kBarDrain = 24,
};

template <int D, bool kCap, bool kBias>
__global__ void __launch_bounds__(kThreads, 1)
    score_fwd_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to, const __grid_constant__ ScoreArgs a,
                        const __grid_constant__ CapCoef cc) {
  using L = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);  // [0] TMEM base, [1] abort flag, [2] tiles
  volatile uint32_t* abort_flag = misc + 1;
  auto bar = [&](int i) -> uint32_t { return sb + L::kOffBar + 8 * i; };
  auto item_at = [&](int slot) { return reinterpret_cast<Item*>(smem + L::kOffItem) + slot; };
  auto map_at = [&](int slot) { return reinterpret_cast<uint32_t*>(smem + L::kOffMap) + slot * 3 * kMapWords; };
  const int cs = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  int shift = 0;  // a bit of the bitmaps is for 2^shift key tiles
  while (((a.Skv + kTileN - 1) / kTileN) >> shift > kMapWords * 32) ++shift;
  // with a bias the nearest keys weigh most: from the rows' own position
  // outwards, so that the running maximum is found first and keeps
  auto walk_start = [&](const Item& t) {
    return kBias ? min(t.ntile - 1, max(-1, (a.rel + min(t.row0 + 2 * kTileM, a.Sq) - 1) / kTileN)) : -1;
  };

  // No copy, product or wait meets a barrier before this: initialised, the
  // initialisation fenced for the cluster and for the async proxy (the copies' and
  // the commits' arrivals), then the CTA's barrier. No peer's shared memory is
  // touched before the first cluster_sync.
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i)
      mbar_init(bar(i), (i == kBarPFull || i == kBarPFull + 1) ? 4 : (i == kBarItemEmpty || i == kBarItemEmpty + 1) ? 10 : 1);
    misc[1] = 0;
    fence_mbar_init();
    fence_async();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(misc), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const uint64_t tmo = a.timeout_ns;

  if (warp == kThreads / 32 - 1) {
    // ===================== items =====================
    // The first is this block's own; then, once the last tiles of an item are
    // being loaded, a block that has not started gives up its own: setting up
    // and the first loads of an item then go by under the last products and the
    // stores of the one before. In a cluster there is the one item.
    if (a.qdoc) grid_wait();  // the document ranges
    // (head and rank in x, batch entry in y, pair in z, the pairs with the most
    // causal keys first, heads fastest: no index needs a division)
    int x = static_cast<int>(blockIdx.x) >> (__ffs(cs) - 1), y = blockIdx.y, z = blockIdx.z;
    bool more = true;
    for (int n = 0;; ++n) {
      const int slot = n & 1;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarItemEmpty + slot), ((n >> 1) & 1) ^ 1, abort_flag, a.err, tmo)))
        break;
      Item t{};
      if (more) {
        t.valid = 1;
        t.h = x;
        t.b = y;
        t.row0 = (static_cast<int>(gridDim.z) - 1 - z) * 2 * kTileM;
        t.plim = prefix_limit(a, t.b);
        // key tiles that the last row (the largest limit) reaches
        t.ntile = (max(0, min(a.Skv, key_limit(a, t.plim, min(t.row0 + 2 * kTileM, a.Sq) - 1))) + kTileN - 1) / kTileN;
        int tiles = t.ntile;
        if (a.qdoc) {
          uint32_t* act = map_at(slot);
          const int nqb = (a.Sq + kDocBlock - 1) / kDocBlock, nkb = (a.Skv + kDocBlock - 1) / kDocBlock;
          const DocRange* qr = a.qrange + static_cast<int64_t>(t.b) * nqb;
          const DocRange* kr = a.krange + static_cast<int64_t>(t.b) * nkb;
          const DocRange q0 = doc_span(qr, nqb, t.row0 / kDocBlock, 2), q1 = doc_span(qr, nqb, t.row0 / kDocBlock + 2, 2);
          tiles = 0;
          const int groups = (t.ntile + (1 << shift) - 1) >> shift;
#pragma unroll 4
          for (int g0 = 0; g0 < groups; g0 += 32) {
            const int gr = g0 + lane;
            const DocRange k = doc_span(kr, nkb, (2 * gr) << shift, 2 << shift);
            const bool on = gr < groups && (docs_meet(q0, k) || docs_meet(q1, k));
            const uint32_t w = __ballot_sync(0xffffffffu, on);
            const uint32_t m0 = __ballot_sync(0xffffffffu, !docs_same(q0, k)), m1 = __ballot_sync(0xffffffffu, !docs_same(q1, k));
            if (lane == 0) {
              act[g0 >> 5] = w;
              act[kMapWords + (g0 >> 5)] = m0;
              act[2 * kMapWords + (g0 >> 5)] = m1;
            }
            tiles += on ? min(1 << shift, t.ntile - (gr << shift)) : 0;
          }
          tiles = __reduce_add_sync(0xffffffffu, tiles);
        }
        // this CTA's part of the walk
        t.n0 = cluster_part(tiles, rank, cs);
        t.NT = cluster_part(tiles, rank + 1, cs) - t.n0;
      }
      if (lane == 0) {
        *item_at(slot) = t;
        mbar_arrive(bar(kBarItemFull + slot));
      }
      if (!more) break;
      more = false;
      if (cs > 1) continue;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarNear), n & 1, abort_flag, a.err, tmo))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(kBarNext), 16);
        next_block_ask(sb + L::kOffNext, bar(kBarNext));
      }
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarNext), n & 1, abort_flag, a.err, tmo))) {
        drain_wait(bar(kBarNext), n & 1, tmo);
        break;
      }
      more = next_block(sb + L::kOffNext, x, y, z);
      __syncwarp();  // every lane has read the answer
    }
  } else if (warp == 0) {
    // ===================== TMA producer =====================
    const bool leader = elect_one();
    if (leader) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
      tma_prefetch_desc(&to);
    }
    int k_issued[2] = {0, 0}, v_issued[2] = {0, 0}, q_issued[2] = {0, 0};
    int g = 0;  // key tiles so far, of all items
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int slot = n & 1;
      if (!mbar_wait_bounded(bar(kBarItemFull + slot), (n >> 1) & 1, abort_flag, a.err, tmo)) break;
      const Item t = *item_at(slot);
      if (!t.valid) break;
      const int hk = t.h / a.G;
      auto load_q = [&](int i) -> bool {
        const uint32_t qb = bar(kBarQFull + i);
        if (!mbar_wait_bounded(bar(kBarQEmpty + i), (q_issued[i] & 1) ^ 1, abort_flag, a.err, tmo)) return false;
        if (leader) {
          mbar_arrive_expect_tx(qb, L::kQTile);
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sb + L::kOffQ + i * L::kQTile + c * L::kHalf, &tq, qb, c * 64, t.h, t.row0 + i * kTileM, t.b);
        }
        ++q_issued[i];
        return true;
      };
      const int near = max(0, t.NT - 3);
      if (t.NT == 0 && leader) mbar_arrive(bar(kBarNear));
      if (t.NT > 0) ok = load_q(0);
      TileWalk<true> cur(a.qdoc ? map_at(slot) : nullptr, 0, t.ntile, walk_start(t), shift);
      for (int k = 0; k < t.n0; ++k) cur.next();
      for (int it = 0; ok && it < t.NT; ++it, ++g) {
        const int s = g & 1;
        const uint32_t ph = (g >> 1) & 1;
        if (it == near && leader) mbar_arrive(bar(kBarNear));
        if (!(ok = mbar_wait_bounded(bar(kBarKEmpty + s), ph ^ 1, abort_flag, a.err, tmo))) break;
        if (leader) {
          mbar_arrive_expect_tx(bar(kBarKFull + s), L::kKVTile);
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sb + L::kOffK + s * L::kKVTile + c * L::kHalf, &tk, bar(kBarKFull + s), c * 64, hk,
                        cur.t * kTileN, t.b);
        }
        ++k_issued[s];
        if (it == 0 && t.row0 + kTileM < a.Sq && !(ok = load_q(1))) break;
        if (!(ok = mbar_wait_bounded(bar(kBarVEmpty + s), ph ^ 1, abort_flag, a.err, tmo))) break;
        if (leader) {
          mbar_arrive_expect_tx(bar(kBarVFull + s), L::kKVTile);
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sb + L::kOffV + s * L::kKVTile + c * L::kHalf, &tv, bar(kBarVFull + s), c * 64, hk,
                        cur.t * kTileN, t.b);
        }
        ++v_issued[s];
        cur.next();
      }
      __syncwarp();
      if (leader) mbar_arrive(bar(kBarItemEmpty + slot));
    }
    if (*abort_flag) {
      // let every issued copy land before the CTA's shared memory goes away
      for (int s = 0; s < 2; ++s) {
        if (q_issued[s]) drain_wait(bar(kBarQFull + s), (q_issued[s] - 1) & 1, tmo);
        if (k_issued[s]) drain_wait(bar(kBarKFull + s), (k_issued[s] - 1) & 1, tmo);
        if (v_issued[s]) drain_wait(bar(kBarVFull + s), (v_issued[s] - 1) & 1, tmo);
      }
    }
  } else if (warp == 1) {
    // ===================== MMA issuer =====================
    // The whole warp runs the loop (every operand is warp-uniform); one
    // elected lane issues the MMAs and commits.
    const bool leader = elect_one();
    constexpr uint32_t idesc_s = idesc_bf16_f32(kTileM, kTileN, false, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(kTileM, D, false, true);
    // Descriptor halves of every operand buffer, built once (see
    // mma_ss_lohi: nothing but an add may sit between two MMAs).
    const uint64_t dq = smem_desc_sw128(sb + L::kOffQ, 16, 1024);
    const uint64_t dk = smem_desc_sw128(sb + L::kOffK, 16, 1024);
    const uint64_t dv = smem_desc_sw128(sb + L::kOffV, L::kHalf, 1024);
    const uint32_t qk_hi = static_cast<uint32_t>(dq >> 32);  // same for Q and K (SBO 1024, 128B swizzle)
    const uint32_t v_hi = static_cast<uint32_t>(dv >> 32);
    const uint32_t q_lo = static_cast<uint32_t>(dq), k_lo = static_cast<uint32_t>(dk);
    const uint32_t v_lo = static_cast<uint32_t>(dv);
    auto commit = [&](uint32_t bar_addr) {
      if (leader) mma_commit(bar_addr);
    };
    auto issue_s = [&](int i, int stage) {
      const uint32_t a0 = q_lo + ((i * L::kQTile) >> 4);
      const uint32_t b0 = k_lo + ((stage * L::kKVTile) >> 4);
      const uint32_t d_tmem = tmem + i * kTileN;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * L::kHalf + (kk & 3) * 32) >> 4;
        if (leader) mma_ss_lohi(d_tmem, a0 + off, qk_hi, b0 + off, qk_hi, idesc_s, kk > 0 ? 1u : 0u);
      }
    };
    auto issue_pv = [&](int i, int stage, bool acc) {
      const uint32_t b0 = v_lo + ((stage * L::kKVTile) >> 4);
      const uint32_t d_tmem = tmem + 256 + i * D;
      const uint32_t a_tmem = tmem + i * kTileN;
      const uint32_t acc0 = acc ? 1u : 0u;
#pragma unroll
      for (int kk = 0; kk < kTileN / 16; ++kk)
        if (leader) mma_ts_lohi(d_tmem, a_tmem + kk * 8, b0 + ((kk * 2048) >> 4), v_hi, idesc_o, kk > 0 ? 1u : acc0);
    };
    int g = 0;              // key tiles so far, of all items
    int pc[2] = {0, 0};     // and those of each query tile
    int qc[2] = {0, 0};     // items of each query tile
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!(ok = mbar_wait_bounded(bar(kBarItemFull + (n & 1)), (n >> 1) & 1, abort_flag, a.err, tmo))) break;
      const Item* t = item_at(n & 1);
      const int valid = t->valid, NT = t->NT, nq = t->row0 + kTileM < a.Sq ? 2 : 1;
      __syncwarp();
      if (leader) mbar_arrive(bar(kBarItemEmpty + (n & 1)));
      if (!valid) break;
      if (NT == 0) continue;
      // S of the first tile: behind the last products of the item before, whose P
      // it writes over
      ok = mbar_wait_bounded(bar(kBarQFull), qc[0] & 1, abort_flag, a.err, tmo) &&
           mbar_wait_bounded(bar(kBarKFull + (g & 1)), (g >> 1) & 1, abort_flag, a.err, tmo);
      for (int i = 0; i < nq && ok; ++i) {
        if (i == 1 && !mbar_wait_bounded(bar(kBarQFull + 1), qc[1] & 1, abort_flag, a.err, tmo)) {
          ok = false;
          break;
        }
        tc_fence_after();
        issue_s(i, g & 1);
        commit(bar(kBarSFull + i));
        if (NT == 1) commit(bar(kBarQEmpty + i));
      }
      if (ok) commit(bar(kBarKEmpty + (g & 1)));
      // The tensor pipe queues about one MMA: whatever this thread does
      // between two MMA groups leaves the pipe idle. Each step therefore
      // waits at two points only: V(it), K(it+1) and P_0(it) before
      // PV_0(it) + S_0(it+1); P_1(it) before PV_1(it) + S_1(it+1). The step
      // is instantiated per tile count and ring stage so that every MMA
      // operand is a compile-time offset from one base: a run-time tile or
      // stage index in the issue sequence measurably stalls the pipe. P of an
      // item's first tile comes after its softmax warps have read the O before.
      auto step = [&](auto nq_c, auto stage_c, int it) -> bool {
        constexpr int kNq = decltype(nq_c)::value;
        constexpr int s = decltype(stage_c)::value;
        constexpr int s2 = s ^ 1;
        const bool more = it + 1 < NT;
        if (!mbar_wait_bounded(bar(kBarVFull + s), ((g + it) >> 1) & 1, abort_flag, a.err, tmo) ||
            (more && !mbar_wait_bounded(bar(kBarKFull + s2), ((g + it + 1) >> 1) & 1, abort_flag, a.err, tmo)))
          return false;
#pragma unroll
        for (int i = 0; i < kNq; ++i) {
          if (!mbar_wait_bounded(bar(kBarPFull + i), (pc[i] + it) & 1, abort_flag, a.err, tmo)) return false;
          tc_fence_after();
          issue_pv(i, s, it > 0);
          if (more) {
            issue_s(i, s2);
            commit(bar(kBarSFull + i));
            if (it + 2 == NT) commit(bar(kBarQEmpty + i));
          } else {
            commit(bar(kBarOFull + i));
          }
          if (i == kNq - 1) {
            commit(bar(kBarVEmpty + s));
            if (more) commit(bar(kBarKEmpty + s2));
          }
        }
        return true;
      };
      auto run_steps = [&](auto nq_c) {
        int it = 0;
        if (ok && (g & 1)) ok = step(nq_c, std::integral_constant<int, 1>{}, it++);
        for (; ok && it < NT; it += 2) {
          ok = step(nq_c, std::integral_constant<int, 0>{}, it);
          if (ok && it + 1 < NT) ok = step(nq_c, std::integral_constant<int, 1>{}, it + 1);
        }
      };
      if (nq == 2)
        run_steps(std::integral_constant<int, 2>{});
      else
        run_steps(std::integral_constant<int, 1>{});
      g += NT;
      for (int i = 0; i < nq; ++i) {
        pc[i] += NT;
        ++qc[i];
      }
    }
    if (!ok) {
      commit(bar(kBarDrain));
      drain_wait(bar(kBarDrain), 0, tmo);
    }
  } else {
    // ===================== softmax + epilogue =====================
    const int i = (warp - 2) >> 2;  // query tile of this warpgroup
    const int wq = warp & 3;        // TMEM lane quadrant of this warp (warp id mod 4)
    const int row = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t t_s = tmem + lane_off + i * kTileN;
    const uint32_t t_o = tmem + lane_off + 256 + i * D;
    const float sl2 = a.scale * kLog2e;
    int pc = 0, oc = 0;  // key tiles and items with any so far
    bool ok = true;
    for (int n = 0; ok; ++n) {
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarItemFull + (n & 1)), (n >> 1) & 1, abort_flag, a.err, tmo));
      if (!ok) break;
      const Item* item = item_at(n & 1);
      if (!item->valid) break;
      if (item->row0 + i * kTileM >= a.Sq) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarItemEmpty + (n & 1)));
        continue;
      }
      const int NT = item->NT;
      const int at = item->row0 + i * kTileM + row;  // this thread's query row
      const int lim = min(a.Skv, key_limit(a, item->plim, at));
      const int qd = a.qdoc && at < a.Sq ? a.qdoc[static_cast<int64_t>(item->b) * a.Sq + at] : -1;
      const float slope2 = kBias ? a.slopes[item->h] * kLog2e : 0.f;
      float m_used = -INFINITY, l = 0.f;
      // 0: as below; with a cap, of whose polynomial these are the 3 terms' range, 1: the
      // 6 terms' range; 2: the next tile exactly. Each item's own: which CTA takes it,
      // and after which, must not show in its bits. With the reference 0 the heaviest
      // key's P is rounded, with the maximum it is 1: rows of few keys, whose result
      // hangs on that one, begin exactly (their error would be up to twice that of out's
      // own rounding; so it is below 1.4 of it)
      int level = __any_sync(0xffffffffu, lim < kFewKeys) ? 2 : 0;
      TileWalk<true> cur(a.qdoc ? map_at(n & 1) : nullptr, 0, item->ntile, walk_start(*item), shift);
      for (int k = item->n0; k > 0; --k) cur.next();
      for (int it = 0; it < NT; ++it) {
        const int kv0 = cur.t * kTileN;
        const bool mix = a.qdoc && cur.in(map_at(n & 1) + (1 + i) * kMapWords);
        const int nv = lim - kv0;                  // this row's keys of the tile: those below nv
        const int dq = a.rel + at - kv0;   // position of the row less that of the tile's first key
        const bool cut = __any_sync(0xffffffffu, nv < kTileN);
        // where every pair that takes part has the same order, the bias is linear in the key
        const bool below = __all_sync(0xffffffffu, dq >= kTileN - 1 || nv <= dq + 1);
        const bool above = __all_sync(0xffffffffu, dq <= 0);
        // the places that take part, a bit each (found before the wait, which hides it)
        const bool masked = cut || mix;
        uint32_t on[4] = {~0u, ~0u, ~0u, ~0u};
        if (masked) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int n = nv - 32 * w;
            on[w] = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
          }
        }
        if (mix) {
          const int* kd = a.kdoc + static_cast<int64_t>(item->b) * a.Skv;
          int ids[4];
          uint32_t same[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int j = kv0 + 32 * w + lane;
            ids[w] = j < a.Skv ? __ldg(kd + j) : -1;
          }
          same_docs<4>(qd, ids, same);
#pragma unroll
          for (int w = 0; w < 4; ++w) on[w] &= same[w];
        }
        if (masked && a.qdoc) {
          const int keys = __popc(on[0]) + __popc(on[1]) + __popc(on[2]) + __popc(on[3]);
          if (__any_sync(0xffffffffu, m_used == -INFINITY && keys > 0 && keys < kFewKeys)) level = 2;
        }
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarSFull + i), (pc + it) & 1, abort_flag, a.err, tmo));
        if (!ok) break;
        tc_fence_after();
        uint32_t pk[kTileN / 2];
        // P = 2^(x - m) in pairs, rounded to bf16 into pk, 16 columns at a time
        // (the next columns' load is under way meanwhile); returns the row sum
        // before the rounding. kMode 1: no cap; 3, 6: the polynomial of that
        // degree, umax the largest s^2.
        float umax = 0.f;
        auto speculate = [&](auto mode_c, auto mask_c) -> float {
          constexpr int kMode = decltype(mode_c)::value;
          constexpr bool kMask = decltype(mask_c)::value;
          f32x2 ls[2] = {0ull, 0ull};
          float um[2] = {0.f, 0.f};
          const float bs = kBias ? (below ? slope2 : -slope2) : 0.f;
          const float ref = m_used == -INFINITY ? 0.f : m_used;
          const float bb = kBias ? fmaf(-bs, static_cast<float>(dq), -ref) : -ref;
          const f32x2 bs2 = pair(bs, bs), bb2 = pair(bb, bb), sl22 = pair(sl2, sl2);
          uint32_t buf[2][16];
          tmem_ld16(t_s, buf[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t(&sr)[16] = buf[c & 1];
            tmem_wait_ld();
            tmem_pin(sr);
            if (c < 7) tmem_ld16(t_s + (c + 1) * 16, buf[(c + 1) & 1]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int col = 16 * c + 2 * e;
              const bool on0 = !kMask || ((on[c >> 1] >> (col & 31)) & 1u);
              const bool on1 = !kMask || ((on[c >> 1] >> ((col & 31) + 1)) & 1u);
              f32x2 s2 = pair_u(sr[2 * e], sr[2 * e + 1]), fac = sl22;
              if constexpr (kMode >= 3) {
                if (kMask) s2 = pair_u(on0 ? sr[2 * e] : 0u, on1 ? sr[2 * e + 1] : 0u);
                const f32x2 u2 = mul_x2(s2, s2);
                float u0, u1;
                split(u2, u0, u1);
                um[e & 1] = fmax3(um[e & 1], u0, u1);
                fac = cap_poly<kMode>(cc, u2);
              }
              const f32x2 x2 = fma_x2(s2, fac, kBias ? fma_x2(bs2, columns(col), bb2) : bb2);
              float x0, x1;
              split(x2, x0, x1);
              if (kMask) {
                x0 = on0 ? x0 : -INFINITY;
                x1 = on1 ? x1 : -INFINITY;
              }
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              pk[8 * c + e] = pack_bf16x2(p0, p1);
              ls[e & 1] = add_x2(ls[e & 1], pair(p0, p1));
            }
          }
          umax = fmaxf(um[0], um[1]);
          float l0, l1;
          split(add_x2(ls[0], ls[1]), l0, l1);
          return l0 + l1;
        };
        float f = 1.f, lsum = INFINITY;
        bool fits = false;
        // speculatively with the reference that the row has (0 before it has one):
        // any will do that keeps its sums far from overflow, which a row sum
        // within 2^20 and those before within 2^26 prove (every P is at most that),
        // and from underflow, where the first sum is above 2^-20; and s^2 within the
        // polynomial's range
        const bool none = masked && (on[0] | on[1] | on[2] | on[3]) == 0u;
        auto holds = [&](float sum) {
          return sum <= kSumMost && l <= kTotalMost && (m_used != -INFINITY || sum >= 1.f / kSumMost || none);
        };
        if (!kBias || below || above) {
          using std::integral_constant;
          if constexpr (kCap) {
            if (level == 0) {
              lsum = masked ? speculate(integral_constant<int, 3>{}, std::true_type{})
                            : speculate(integral_constant<int, 3>{}, std::false_type{});
              fits = holds(lsum) && umax <= cc.u3;
            } else if (level == 1 && !masked) {
              lsum = speculate(integral_constant<int, 6>{}, std::false_type{});
              fits = holds(lsum) && umax <= cc.u6;
            }
          } else if (level == 0) {
            lsum = masked ? speculate(integral_constant<int, 1>{}, std::true_type{})
                          : speculate(integral_constant<int, 1>{}, std::false_type{});
            fits = holds(lsum);
          }
        }
        if (__all_sync(0xffffffffu, fits)) {
          tmem_st32(t_s, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
          tmem_st32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
          m_used = m_used == -INFINITY && !none ? 0.f : m_used;
        } else {
          // exactly, 32 columns at a time: scores in log2 units back over S and
          // their maximum; move to it if it grew by more than 2^8 (and by 2^26 at
          // least where the sum has reached that), rescaling O
          // and l by the same factor (O is idle here: PV of the previous tile
          // completed before S of this tile was committed, and PV of this tile
          // waits for P); then P. Columns [16 c, 16 c + 16) of P lie over
          // columns of S that have been read. A row that has seen no key keeps
          // m = -inf and P = 0.
          float mxs = -INFINITY, um = 0.f;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t sr[32];
            tmem_ld32(t_s + c * 32, sr);
            tmem_wait_ld();
            tmem_pin(sr);
            const uint32_t onw = c == 0 ? on[0] : c == 1 ? on[1] : c == 2 ? on[2] : on[3];
            const f32x2 sl22 = pair(sl2, sl2);
            bool poly = false;  // (a masked place may only cost the polynomial)
            if (kCap) {
              float u = 0.f;
#pragma unroll
              for (int e = 0; e < 32; e += 2) u = fmax3(u, fabsf(u2f(sr[e])), fabsf(u2f(sr[e + 1])));
              um = fmaxf(um, u * u);
              poly = __all_sync(0xffffffffu, u * u <= cc.u3);
            }
            const float dc = static_cast<float>(dq - 32 * c);
            if (kBias && !kCap) {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                float x = fmaf(-slope2, fabsf(dc - static_cast<float>(e)), u2f(sr[e]) * sl2);
                x = (onw >> e) & 1u ? x : -INFINITY;
                mxs = fmaxf(mxs, x);
                sr[e] = __float_as_uint(x);
              }
            } else {
              if (!kCap || poly) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  const f32x2 s2 = pair_u(sr[e], sr[e + 1]);
                  float x0, x1;
                  split(mul_x2(s2, kCap ? cap_poly<3>(cc, mul_x2(s2, s2)) : sl22), x0, x1);
                  sr[e] = __float_as_uint(x0);
                  sr[e + 1] = __float_as_uint(x1);
                }
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) sr[e] = __float_as_uint(cap_exact(cc, u2f(sr[e])));
              }
              if (kBias) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  sr[e] = __float_as_uint(fmaf(-slope2, fabsf(dc - static_cast<float>(e)), u2f(sr[e])));
              }
              if (masked) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!((onw >> e) & 1u)) sr[e] = __float_as_uint(-INFINITY);
              }
#pragma unroll
              for (int e = 0; e < 32; e += 2) mxs = fmax3(mxs, u2f(sr[e]), u2f(sr[e + 1]));
            }
            __syncwarp();  // (tensor-memory accesses want the warp converged, here and below)
            tmem_st32(t_s + c * 32, sr);
          }
          tmem_wait_st();
          level = 0;
          if (kCap) {
            const float w = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(um)));
            level = w <= cc.u3 ? 0 : w <= cc.u6 ? 1 : 2;
          }
          const bool full = l > kTotalMost;
          const bool need = full || mxs > m_used + kRescaleThreshold || (m_used == -INFINITY && mxs > -INFINITY);
          if (need) {
            const float to = full ? fmaxf(mxs, m_used + 26.f) : mxs;
            f = ex2_approx(m_used - to);
            m_used = to;
          }
          __syncwarp();
          const float nm = m_used == -INFINITY ? 0.f : -m_used;
          f32x2 ls[2] = {0ull, 0ull};
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t sr[32], pw[16];
            tmem_ld32(t_s + c * 32, sr);
            tmem_wait_ld();
            tmem_pin(sr);
            const f32x2 nm2 = pair(nm, nm);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x0, x1;
              split(add_x2(pair_u(sr[2 * e], sr[2 * e + 1]), nm2), x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              pw[e] = pack_bf16x2(p0, p1);
              ls[e & 1] = add_x2(ls[e & 1], pair(p0, p1));
            }
            tmem_st16(t_s + c * 16, pw);
          }
          float l0, l1;
          split(add_x2(ls[0], ls[1]), l0, l1);
          lsum = l0 + l1;
          if (it > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(t_o + c * 32, o);
              tmem_wait_ld();
              tmem_pin(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(u2f(o[e]) * f);
              tmem_st32(t_o + c * 32, o);
            }
          }
        }
        l = l * f + lsum;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPFull + i));
        cur.next();
      }
      // l = 0: no key -> out 0, lse -inf (found while the last product runs)
      const float inv_l = l != 0.f ? 1.f / l : 0.f;
      const float lse_v = l != 0.f ? (m_used + log2f(l)) * kLn2 : -INFINITY;
      if (ok && NT > 0) ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarOFull + i), oc & 1, abort_flag, a.err, tmo));
      pc += NT;
      oc += NT > 0;
      const int h = item->h, b = item->b, tok0 = item->row0 + i * kTileM;
      const int rows_valid = a.Sq - tok0;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarItemEmpty + (n & 1)));
      if (ok) {
        tc_fence_after();
        if (cs > 1)
          *reinterpret_cast<float2*>(smem + L::kOffStat + (i * kTileM + row) * 8) = make_float2(m_used, l);
        else if (row < rows_valid)
          a.lse[(static_cast<int64_t>(b) * a.H + h) * a.Sq + tok0 + row] = lse_v;
        __syncwarp();
        // 32 rows x 128 bytes (64 columns in bf16, 32 in fp32) are staged in this
        // warp's buffer, 128-byte swizzled, and stored by TMA, which cuts the rows
        // past the end: the stores of all multiprocessors come at about the same
        // time, and ordinary ones would hold up this warp's next item behind them
        const uint32_t stage = sb + L::kOffStage + (warp - 2) * 4096;
        auto place = [&](int q4, uint32_t x, uint32_t y, uint32_t z, uint32_t u) {
          *reinterpret_cast<uint4*>(smem + L::kOffStage + (warp - 2) * 4096 + lane * 128 + ((q4 ^ (lane & 7)) * 16)) =
              make_uint4(x, y, z, u);
        };
        auto stage_free = [&]() {
          if (lane == 0) tma_store_wait_read();
          __syncwarp();
        };
        auto flush = [&](int col) {
          fence_async();
          __syncwarp();
          if (lane == 0 && wq * 32 < rows_valid) tma_store_4d(&to, stage, col, h, tok0 + wq * 32, b);
        };
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (NT > 0) {
            tmem_ld32(t_o + c * 32, o);
            tmem_wait_ld();
            tmem_pin(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          auto w = [&](int e) { return __float_as_uint(u2f(o[e]) * inv_l); };
          auto w2 = [&](int e) { return pack_bf16x2(u2f(o[e]) * inv_l, u2f(o[e + 1]) * inv_l); };
          if (cs > 1) {
            // this CTA's part over the idle tiles: [256 rows][D], 16-byte pieces permuted by row
            const int r = i * kTileM + row;
            float* part = reinterpret_cast<float*>(smem) + r * D;
#pragma unroll
            for (int x = 0; x < 8; ++x)
              *reinterpret_cast<uint4*>(part + (((c * 8 + x) ^ (r & 7)) * 4)) =
                  make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          } else if (a.out_bf16) {
            if ((c & 1) == 0) stage_free();
#pragma unroll
            for (int x = 0; x < 4; ++x)
              place((c & 1) * 4 + x, w2(8 * x), w2(8 * x + 2), w2(8 * x + 4), w2(8 * x + 6));
            if (c & 1) flush((c >> 1) * 64);
          } else {
            stage_free();
#pragma unroll
            for (int x = 0; x < 8; ++x) place(x, w(4 * x), w(4 * x + 1), w(4 * x + 2), w(4 * x + 3));
            flush(c * 64);
          }
        }
      }
    }
    if (lane == 0) tma_store_wait_read();
  }
  if (cs > 1) {
    static_assert(2 * kTileM * D * 4 <= L::kOffStage, "the parts lie over the tiles");
    const int h = static_cast<int>(blockIdx.x) >> (__ffs(cs) - 1), b = blockIdx.y;
    const int row0 = (static_cast<int>(gridDim.z) - 1 - static_cast<int>(blockIdx.z)) * 2 * kTileM;
    const int nrows = min(2 * kTileM, a.Sq - row0);
    cluster_sync();
    // a row's D / 4 pieces on neighbouring lanes, kIn rows a thread at once: every
    // load of a step is under way before the first is used
    auto join = [&](auto cs_c) {
      constexpr int kCs = decltype(cs_c)::value, kIn = 16 / kCs;
      constexpr int kStep = kThreads / (D / 4);  // rows side by side
      const int share = 2 * kTileM / kCs, x = threadIdx.x % (D / 4);
      for (int r0 = threadIdx.x / (D / 4); r0 < share; r0 += kStep * kIn) {
        float2 ml[kIn][kCs];
        float4 y[kIn][kCs];
#pragma unroll
        for (int u = 0; u < kIn; ++u) {
          const int r = rank * share + min(r0 + u * kStep, share - 1);
#pragma unroll
          for (int c = 0; c < kCs; ++c) {
            ml[u][c] = ld_peer2(cluster_peer(sb + L::kOffStat + r * 8, c));
            y[u][c] = ld_peer4(cluster_peer(sb + (r * D + ((x ^ (r & 7)) * 4)) * 4, c));
          }
        }
#pragma unroll
        for (int u = 0; u < kIn; ++u) {
          const int r = rank * share + r0 + u * kStep;
          if (r0 + u * kStep >= share || r >= nrows) break;
          float mx = -INFINITY, sum = 0.f;
#pragma unroll
          for (int c = 0; c < kCs; ++c) mx = fmaxf(mx, ml[u][c].x);
          const float base = mx == -INFINITY ? 0.f : mx;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int c = 0; c < kCs; ++c) {
            const float f = ex2_approx(ml[u][c].x - base);
            sum = fmaf(ml[u][c].y, f, sum);
            o = make_float4(fmaf(y[u][c].x, f, o.x), fmaf(y[u][c].y, f, o.y), fmaf(y[u][c].z, f, o.z),
                            fmaf(y[u][c].w, f, o.w));
          }
          const float inv = sum != 0.f ? 1.f / sum : 0.f;
          const int64_t at = ((static_cast<int64_t>(b) * a.Sq + row0 + r) * a.H + h) * D + x * 4;
          if (a.out_bf16) {
            uint2 v;
            v.x = pack_bf16x2(o.x * inv, o.y * inv);
            v.y = pack_bf16x2(o.z * inv, o.w * inv);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) = v;
          } else {
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) =
                make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
          }
          if (x == 0)
            a.lse[(static_cast<int64_t>(b) * a.H + h) * a.Sq + row0 + r] =
                sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
        }
      }
    };
    if (cs == 2)
      join(std::integral_constant<int, 2>{});
    else if (cs == 4)
      join(std::integral_constant<int, 4>{});
    else
      join(std::integral_constant<int, 8>{});
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }

  // ---- teardown: every thread of the CTA arrives here, aborted or not ----
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool kCap, bool kBias>
cudaError_t launch_rule(const ScoreArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const CUtensorMap& to, cudaStream_t s) {
  using L = Smem<D>;
  static_assert(L::kAlloc <= 227 * 1024, "shared memory budget");
  cudaError_t e = allow_smem<score_fwd_tc_kernel<D, kCap, kBias>>(L::kAlloc);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>((a.Sq + 2 * kTileM - 1) / (2 * kTileM)) * a.H * a.B;
  // steps: key tiles; some 8 of them go by before the first and after the last
  const int cs = cluster_for(8.0, items, (a.Skv + kTileN - 1) / kTileN, 0, 0, a.causal ? 0.5 : 1.0, true, a.sms);
  return launch_clusters(score_fwd_tc_kernel<D, kCap, kBias>, a.H, a.B, (a.Sq + 2 * kTileM - 1) / (2 * kTileM), cs, kThreads, L::kAlloc, a.qdoc != nullptr, s, tq, tk,
                         tv, to, a, make_cap_coef(a.scale, a.cap, false));
}

template <int D>
cudaError_t launch_d(const ScoreArgs& a, cudaStream_t s) {
  CUtensorMap tq, tk, tv, to;
  // without keys the maps of k and v are never read through
  const bool none = a.Skv == 0;
  if (!host_tmap_bf16(&tq, a.q, D, a.H, a.Sq, a.B, kTileM) ||
      !host_tmap_bf16(&tk, none ? a.q : a.k, D, none ? a.H : a.Hkv, none ? a.Sq : a.Skv, a.B, kTileN) ||
      !host_tmap_bf16(&tv, none ? a.q : a.v, D, none ? a.H : a.Hkv, none ? a.Sq : a.Skv, a.B, kTileN) ||
      // fp32 rows as twice as many 16-bit columns
      !host_tmap_bf16(&to, a.out, a.out_bf16 ? D : 2 * D, a.H, a.Sq, a.B, 32))
    return cudaErrorInvalidValue;
  if (a.cap > 0.f) return a.slopes ? launch_rule<D, true, true>(a, tq, tk, tv, to, s) : launch_rule<D, true, false>(a, tq, tk, tv, to, s);
  return a.slopes ? launch_rule<D, false, true>(a, tq, tk, tv, to, s) : launch_rule<D, false, false>(a, tq, tk, tv, to, s);
}

}  // namespace

cudaError_t launch_score_fwd_tc(const ScoreArgs& a, int D, cudaStream_t s) {
  return D == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace cp
