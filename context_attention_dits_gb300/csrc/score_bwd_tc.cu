// score_bwd_tc.cu — backward of attention with a score rule on the
// 5th-generation tensor cores (tcgen05, bf16 operands, fp32 accumulators in
// tensor memory). With y = the capped score, x = y less the bias:
//   p_ij = exp(x_ij - lse_i), ds_ij = p_ij (dout_i.v_j - delta_i) (1 - (y_ij / cap)^2),
//   dv_j = sum p_ij dout_i, dk_j = scale sum ds_ij q_i (over rows i and the
//   query heads that share the key/value head), dq_i = scale sum_j ds_ij k_j.
//
// Two kinds of CTA in one launch, neither with atomics, as in the plain
// backward: dk/dv CTAs (128 keys of one key/value head; 64-row query sub-tiles
// of each of its query heads stream by) and then dq CTAs (128 query rows; 64-key
// sub-tiles stream by). S and dP are formed in both, 14 D flop a pair instead
// of 10, in exchange for no reduction of dq across key tiles. TMEM and
// shared-memory layout, the two TMEM slots that let the row pass of one
// sub-step run beside the products of the other, and the issue order are those
// of the plain backward. What the rule adds:
//   * only the sub-tiles that hold a pair are walked: causal and prefix give a
//     range, documents a bitmap built from the ranges of 64-row blocks;
//   * the row pass, a thread per row and column half, masks the sub-tiles that
//     a limit or a document border cuts, and forms y and its derivative by the
//     cap's polynomial (score_math.cuh) while the warp's scores stay in its
//     range, exactly otherwise;
//   * -lse log2e and delta come from copies padded to 64 rows a (batch entry,
//     head), written by the delta kernel, so that a sub-tile's are one aligned
//     bulk copy. Rows past the end, and rows that saw no key, hold -inf: p = 0.
// P and dS are rounded to bf16 for their products; all sums are fp32.
// Warp roles: 0 = TMA producer, 1 = MMA issuer, then the row warps.
// The longest CTAs of each kind are launched first.
// What bounds it: the tensor pipe and what feeds it. At D = 128 a dk/dv sub-step
// takes 1464 cycles, of which the pipe needs 1280 (S^T and dP^T, 64 columns wide
// with both operands in shared memory, are bound by its reads: 48 cycles a K step
// in place of 32); a dq sub-step 919, of which 768. Starts and ends are 12000
// cycles of a dk/dv CTA and 9000 of a dq CTA. With a cap the row pass of D = 64 is
// as long as the products. Measured, 4608 tokens, 24 heads on 8, D = 128: plain
// 581 us (1123 TFLOP/s of 10 D flop a pair), causal 316, cap 50 744, causal with it
// 397, slopes 584, causal with them 320, causal with both 425; documents of 512
// 97 (24 heads on 24: 117). D = 64: 409, 222, 607, 322, 444, 240, 361.
// Every wait is bounded; on
// expiry the CTA records a timeout, lets its copies land, frees its tensor
// memory and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "cp_internal.h"
#include "cp_ptx.cuh"
#include "cp_score.h"
#include "score_math.cuh"

namespace cp {
namespace {

// Row warps come in groups of 8: two per TMEM lane quarter, one per 32-column
// half of a sub-step. At D = 64 two groups take the sub-steps in turn, so that the
// waits and tensor-memory latencies of one group's pass go by under the other's
// (4608 tokens, 24 heads: plain 442 -> 412 us, cap 50 704 -> 607). At D = 128, where
// the tensor cores set the pace, one group is faster (567 us against 588): its warps
// have the registers for 32 columns at once.
constexpr int kGroupWarps = 8;
template <int D>
struct Rows {
  static constexpr int kGroups = D == 64 ? 2 : 1;
  static constexpr int kWarps = kGroups * kGroupWarps;
  static constexpr int kThreads = 64 + 32 * kWarps;
  static constexpr int kN = 32 / kGroups;  // columns of a row pass
};
constexpr uint32_t kTmemColsB = 512;
constexpr int kT = 128;         // keys per dk/dv CTA, query rows per dq CTA
constexpr int kSub = 64;        // rows of a streamed sub-tile: query rows (dk/dv) or keys (dq) per sub-step

// Depth of the rings. A TMEM slot holds a sub-step's S and dP, and the row pass of
// one sub-step runs while the tensor cores work on the others': two slots are what
// 512 columns leave at D = 128. At D = 64, where the products take half as long and
// a sub-step's chain (S, row pass, gradients) would set the pace, there are three.
template <int D>
struct Ring {
  static constexpr int kTS = D == 64 ? 3 : 2;     // TMEM slots of 128 columns
  static constexpr int kSlots = D == 64 ? 6 : 4;  // dk/dv: streamed query sub-tiles in shared memory (a multiple of kTS)
  static constexpr int kAcc = kTS * 128;          // TMEM column of the accumulators
  static_assert(kSlots % kTS == 0 && kAcc + 2 * D <= 512, "the TMEM slot is the smem slot modulo kTS");
};

// f(0) && f(1) && ... with the indexes as constants
template <typename F, int... I>
__device__ __forceinline__ bool each(std::integer_sequence<int, I...>, F&& f) {
  return (f(std::integral_constant<int, I>{}) && ...);
}
constexpr int kMapWords = kScoreMaxTokens / kSub / 32;  // bitmap of sub-tiles
static_assert(kSub == kDocBlock, "a sub-tile is a block of document ranges");

// K-major operand of 128 rows: 16-element K steps within a 64-column box,
// then the next box (boxes of 128 rows x 128 bytes)
__device__ __forceinline__ uint32_t kstep128(int kk) {
  return static_cast<uint32_t>(((kk >> 2) * (kT * 128) + (kk & 3) * 32) >> 4);
}
// the same for a 64-row sub-tile (boxes of 64 rows x 128 bytes)
__device__ __forceinline__ uint32_t kstep64(int kk) {
  return static_cast<uint32_t>(((kk >> 2) * (kSub * 128) + (kk & 3) * 32) >> 4);
}

template <int D>
struct BSmem {
  static constexpr int kSlots = Ring<D>::kSlots;
  static constexpr int kTile = kT * D * 2;    // one bf16 128-row tile (K or V)
  static constexpr int kSubT = kSub * D * 2;  // one bf16 64-row sub-tile (Q or dO)
  static constexpr int kHalfS = kSub * 128;   // one 64-column box of a sub-tile
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kTile;
  static constexpr int kOffQ = kOffV + kTile;            // kSlots sub-tiles
  static constexpr int kOffO = kOffQ + kSlots * kSubT;   // dO, kSlots sub-tiles
  static constexpr int kOffLse = kOffO + kSlots * kSubT;     // kSlots x 64 floats: -lse log2 e
  static constexpr int kOffDlt = kOffLse + kSlots * kSub * 4; // kSlots x 64 floats: delta
  static constexpr int kOffBar = kOffDlt + kSlots * kSub * 4;
  static constexpr int kNumBars = 21;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffMap = kOffMisc + 16;  // which sub-tiles are walked, and which are mixed
  static constexpr int kBytes = kOffMap + 2 * kMapWords * 4;
  // + room to align the base to 1024 bytes, as much as the 227 KB budget leaves
  static constexpr int kMax = 227 * 1024;
  static constexpr int kAlloc = kBytes + 1024 <= kMax ? kBytes + 1024 : kMax;
};

enum : int {
  kBarKV = 0,      // K and V tiles landed
  kBarQFull = 1,   // +slot (6): Q, dO, lse, delta of a sub-tile landed (TMA bytes)
  kBarQEmpty = 7,  // +slot (6): MMAs done with the slot
  kBarSFull = 13,  // +TMEM slot (3): S^T and dP^T of the sub-step in TMEM
  kBarPFull = 16,  // +TMEM slot (3): P^T, dS^T written (every row warp arrives)
  kBarDone = 19,   // every MMA of the CTA done: dK, dV final
  kBarDrain = 20,
};

// TMEM column (within S's or dP's 64) of the bf16 A operand for K step kk of
// a sub-step: rows [32 h, 32 h + 32) of the sub-step (written by the row warps
// of column half h) sit in columns [32 h, 32 h + 16), 8 columns per K step
__device__ __forceinline__ uint32_t pcol(int kk) { return static_cast<uint32_t>((kk >> 1) * 32 + (kk & 1) * 8); }

__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[32]) { tmem_ld32(t, r); }
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[16]) { tmem_ld16(t, r); }
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&r)[16]) { tmem_st16(t, r); }
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&r)[8]) { tmem_st8(t, r); }

// The sub-tiles of [t0, t1) that meet the CTA's rows' documents (own: their
// range), into the bitmaps act and mixed; returns how many. All threads call it.
__device__ __forceinline__ int walk_map(const DocRange* other, int nblk, const DocRange& own, int t0, int t1,
                                        uint32_t* act, uint32_t* count) {
  uint32_t* mixed = act + kMapWords;
  if (threadIdx.x == 0) *count = 0;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int w0 = (t0 & ~31) + warp * 32; w0 < t1; w0 += static_cast<int>(blockDim.x)) {
    const int t = w0 + lane;
    const DocRange r = doc_span(other, nblk, t, 1);
    const uint32_t w = __ballot_sync(0xffffffffu, t >= t0 && t < t1 && docs_meet(own, r));
    const uint32_t m = __ballot_sync(0xffffffffu, !docs_same(own, r));
    if (lane == 0) {
      act[w0 >> 5] = w;
      mixed[w0 >> 5] = m;
      atomicAdd(count, __popc(w));
    }
  }
  __syncthreads();
  return static_cast<int>(*count);
}

// N scores of a row pass: p in place of s and -ds in place of dp, packed as
// bf16 pairs. Element e has the distance |d0 + step e| (step +1 or -1);
// nl(e) = -lse log2e and dl(e) = delta of its row; on: the pairs that take part.
// The signs are such that no packed operand has to be negated (an instruction
// each): -ds = p (delta - dp), or with a cap p (delta - dp)(1 - tanh^2) from
// p (dp - delta)(tanh^2 - 1); the epilogues multiply by -scale.
template <bool kCap, bool kBias, int kStep, int N, typename NL, typename ND>
__device__ __forceinline__ void row_pass(const uint32_t (&sr)[N], const uint32_t (&dr)[N], const CapCoef& cc,
                                         float c2, float capl2, float slope2, float d0, uint32_t on, NL nl, ND dl,
                                         uint32_t (&pp)[N / 2], uint32_t (&dd)[N / 2]) {
  const f32x2 c22 = pair(c2, c2), cap2 = pair(capl2, capl2), minus = pair(-1.f, -1.f);
  // kHow: 0 no cap, 3 and 6 the polynomials, 1 exact
  auto pass = [&](auto how_c) {
    constexpr int kHow = decltype(how_c)::value;
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const f32x2 s2 = pair_u(sr[e], sr[e + 1]);
      f32x2 b2 = nl(e);
      if constexpr (kBias) {
        const float a0 = fabsf(d0 + static_cast<float>(kStep * e)), a1 = fabsf(d0 + static_cast<float>(kStep * (e + 1)));
        b2 = fma_x2(pair(-slope2, -slope2), pair(a0, a1), b2);
      }
      const f32x2 dp2 = pair_u(dr[e], dr[e + 1]);
      f32x2 t2, q2;
      if constexpr (kHow == 0) {
        t2 = fma_x2(s2, c22, b2);
        q2 = fma_x2(dp2, minus, dl(e));
      } else {
        f32x2 th, nd;  // tanh, tanh^2 - 1
        if constexpr (kHow >= 3) {
          th = mul_x2(s2, cap_poly<kHow>(cc, mul_x2(s2, s2)));
          nd = fma_x2(th, th, minus);
        } else {
          float h0, h1, n0, n1;
          tanh_exact(cc, u2f(sr[e]), h0, n0);
          tanh_exact(cc, u2f(sr[e + 1]), h1, n1);
          th = pair(h0, h1);
          nd = pair(n0, n1);
        }
        t2 = fma_x2(th, cap2, b2);
        q2 = mul_x2(fma_x2(dl(e), minus, dp2), nd);
      }
      float t0, t1;
      split(t2, t0, t1);
      const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
      q2 = mul_x2(pair(p0, p1), q2);
      float q0, q1;
      split(q2, q0, q1);
      pp[e >> 1] = pack_bf16x2(p0, p1);
      dd[e >> 1] = pack_bf16x2(q0, q1);
    }
  };
  if constexpr (kCap) {
    float um = 0.f;
#pragma unroll
    for (int e = 0; e < N; e += 4) um = fmax3(um, fmaxf(fabsf(u2f(sr[e])), fabsf(u2f(sr[e + 1]))), fmaxf(fabsf(u2f(sr[e + 2])), fabsf(u2f(sr[e + 3]))));
    um *= um;
    if (__all_sync(0xffffffffu, um <= cc.u3))
      pass(std::integral_constant<int, 3>{});
    else if (__all_sync(0xffffffffu, um <= cc.u6))
      pass(std::integral_constant<int, 6>{});
    else
      pass(std::integral_constant<int, 1>{});
  } else {
    pass(std::integral_constant<int, 0>{});
  }
  if (__any_sync(0xffffffffu, (on | ~(~0u >> (32 - N))) != ~0u)) {
#pragma unroll
    for (int x = 0; x < N / 2; ++x) {
      const uint32_t keep = ((on >> (2 * x)) & 1u ? 0x0000ffffu : 0u) | ((on >> (2 * x + 1)) & 1u ? 0xffff0000u : 0u);
      pp[x] &= keep;
      dd[x] &= keep;
    }
  }
}

// A warp's 32 rows (a lane each) of kP 16-byte pieces to dst, `pitch` bytes from
// row to row, the first `rows` of them: through 512 kP bytes of shared memory,
// so that a warp instruction stores whole lines (a lane storing its own row
// took 7000 cycles a dk/dv tile, this 2900).
template <int kP>
__device__ __forceinline__ void store_rows(uint8_t* stage, int lane, const uint4 (&v)[kP], uint8_t* dst, int64_t pitch,
                                           int rows) {
#pragma unroll
  for (int q = 0; q < kP; ++q)
    *reinterpret_cast<uint4*>(stage + lane * kP * 16 + ((q ^ (lane & (kP - 1))) * 16)) = v[q];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const int r = (i * 32 + lane) / kP, q = lane % kP;
    const uint4 x = *reinterpret_cast<const uint4*>(stage + r * kP * 16 + ((q ^ (r & (kP - 1))) * 16));
    if (r < rows) *reinterpret_cast<uint4*>(dst + r * pitch + q * 16) = x;
  }
  __syncwarp();  // the stage is read before it is filled again
}

// kCols2 columns from TMEM column t_acc of a warp's rows, times mul, to dst (fp32
// or bf16, element `at` of the first row, `pitch` elements from row to row);
// none: there are zeros instead.
template <int kCols2>
__device__ __forceinline__ void store_acc(uint32_t t_acc, bool none, float mul, uint8_t* stage, int lane, void* dst,
                                          int64_t at, int64_t pitch, int rows, bool bf16) {
  if (bf16) {
    constexpr int kStep = kCols2 < 64 ? kCols2 : 64;  // columns of a pass
#pragma unroll 1
    for (int c = 0; c < kCols2; c += kStep) {
      uint4 v[kStep / 8];
#pragma unroll
      for (int u = 0; u < kStep / 32; ++u) {
        uint32_t r[32];
        tmem_ld32(t_acc + c + u * 32, r);
        tmem_wait_ld();
        tmem_pin(r);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float m = none ? 0.f : mul;
          auto w = [&](int e) { return none ? 0u : pack_bf16x2(u2f(r[8 * x + e]) * m, u2f(r[8 * x + e + 1]) * m); };
          v[u * 4 + x] = make_uint4(w(0), w(2), w(4), w(6));
        }
      }
      store_rows<kStep / 8>(stage, lane, v, static_cast<uint8_t*>(dst) + (at + c) * 2, pitch * 2, rows);
    }
  } else {
#pragma unroll 1
    for (int c = 0; c < kCols2; c += 32) {
      uint32_t r[32];
      tmem_ld32(t_acc + c, r);
      tmem_wait_ld();
      tmem_pin(r);
      uint4 v[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        auto w = [&](int e) { return none ? 0u : __float_as_uint(u2f(r[4 * x + e]) * mul); };
        v[x] = make_uint4(w(0), w(1), w(2), w(3));
      }
      store_rows<8>(stage, lane, v, static_cast<uint8_t*>(dst) + (at + c) * 4, pitch * 4, rows);
    }
  }
}

// One dk/dv CTA: key tile bx of key/value head hk, batch entry b. The maps have
// 64-row boxes; smem_raw holds alloc bytes of dynamic shared memory. The cs CTAs of a cluster take equal
// ranges of the sub-steps, and each sums the rows of its share over all of them
// (in the order of their ranks) through distributed shared memory.
template <int D, bool kCap, bool kBias>
__device__ __forceinline__ void dkdv_cta(const CUtensorMap& tq64, const CUtensorMap& tk64, const CUtensorMap& tv64,
                                         const CUtensorMap& to64, const ScoreArgs& a, const CapCoef& cc,
                                         uint8_t* smem_raw, int alloc, int cs, int rank, int bx, int hk, int b) {
  using L = BSmem<D>;
  constexpr int kSlots = Ring<D>::kSlots, kTS = Ring<D>::kTS, kAcc = Ring<D>::kAcc;
  constexpr int kGroups = Rows<D>::kGroups, kN = Rows<D>::kN, kThreadsB = Rows<D>::kThreads;
  // the swizzled tiles need a 1024-byte aligned base; a base that would need
  // more padding than the allocation holds is reported (uniformly, before any
  // barrier or TMEM use) instead of used
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  if (pad > static_cast<uint32_t>(alloc - L::kBytes)) {
    if (threadIdx.x == 0) atomicOr(a.err, kDevErrLayout);
    return;
  }
  uint8_t* smem = smem_raw + pad;
  const uint32_t sb = smem_addr(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);  // [0] TMEM base, [1] abort flag, [2] count
  volatile uint32_t* abort_flag = misc + 1;
  auto bar = [&](int i) -> uint32_t { return sb + L::kOffBar + 8 * i; };
  float* s_lse = reinterpret_cast<float*>(smem + L::kOffLse);
  float* s_dlt = reinterpret_cast<float*>(smem + L::kOffDlt);

  const int key0 = bx * kT;
  const int nk = min(kT, a.Skv - key0);
  const int plim = prefix_limit(a, b);
  // query sub-tiles that reach a key of the tile: all, if it holds a prefix key
  // or there is no causal rule, else from the first key's position on
  const int ntq = (a.Sq + kSub - 1) / kSub;
  const int t0 = a.causal && key0 >= plim ? min(ntq, max(0, key0 - a.rel) / kSub) : 0;
  const int nqb = ntq, nkb = (a.Skv + kDocBlock - 1) / kDocBlock;
  uint32_t* act = reinterpret_cast<uint32_t*>(smem + L::kOffMap);
  const uint32_t* bits = a.qdoc ? act : nullptr;
  int per_head = ntq - t0;
  if (a.qdoc)
    per_head = walk_map(a.qrange + static_cast<int64_t>(b) * nqb, nqb,
                        doc_span(a.krange + static_cast<int64_t>(b) * nkb, nkb, bx * 2, 2), t0, ntq, act, misc + 2);
  // sub-steps: the sub-tiles of every query head, head by head; this CTA's part of them
  const int all = per_head * a.G, j0 = cluster_part(all, rank, cs), NJ = cluster_part(all, rank + 1, cs) - j0;
  struct HeadWalk {
    TileWalk<> first, w;
    int h;
    __device__ __forceinline__ HeadWalk(const uint32_t* bits, int t0, int t1, int per_head, int h0, int j)
        : first(bits, t0, t1, t0 - 1), w(first), h(h0) {
      if (per_head > 0) {
        h += j / per_head;
        for (int i = j % per_head; i > 0; --i) w.next();
      }
    }
    __device__ __forceinline__ void next() {
      w.next();
      if (w.done()) {
        w = first;
        ++h;
      }
    }
  };

  // No copy, product or wait meets a barrier before this: initialised, the
  // initialisation fenced for the cluster and for the async proxy (the copies' and
  // the commits' arrivals), then the CTA's barrier. No peer's shared memory is
  // touched before the first cluster_sync.
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      mbar_init(bar(i), i >= kBarPFull && i < kBarDone ? kGroupWarps : 1);
    }
    misc[1] = 0;
    fence_mbar_init();
    fence_async();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(misc), kTmemColsB);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const uint64_t tmo = a.timeout_ns;

  if (warp == 0) {
    // ===================== TMA producer =====================
    const bool leader = elect_one();
    if (leader) {
      tma_prefetch_desc(&tq64);
      tma_prefetch_desc(&tk64);
      tma_prefetch_desc(&tv64);
      tma_prefetch_desc(&to64);
      mbar_arrive_expect_tx(bar(kBarKV), 2 * L::kTile);
      for (int c = 0; c < D / 64; ++c)
        for (int r = 0; r < kT; r += kSub) {  // two boxes of 64 rows lie as one of 128 would
          tma_load_4d(sb + L::kOffK + c * (kT * 128) + r * 128, &tk64, bar(kBarKV), c * 64, hk, key0 + r, b);
          tma_load_4d(sb + L::kOffV + c * (kT * 128) + r * 128, &tv64, bar(kBarKV), c * 64, hk, key0 + r, b);
        }
    }
    int issued[kSlots] = {};
    HeadWalk cur(bits, t0, ntq, per_head, hk * a.G, j0);
    for (int j = 0; j < NJ; ++j) {
      const int s = j % kSlots;
      const uint32_t ph = (j / kSlots) & 1;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarQEmpty + s), ph ^ 1, abort_flag, a.err, tmo))) break;
      const int q0 = cur.w.t * kSub, h = cur.h;
      if (leader) {
        mbar_arrive_expect_tx(bar(kBarQFull + s), 2 * L::kSubT + 2 * kSub * 4);
        for (int c = 0; c < D / 64; ++c) {
          tma_load_4d(sb + L::kOffQ + s * L::kSubT + c * L::kHalfS, &tq64, bar(kBarQFull + s), c * 64, h, q0, b);
          tma_load_4d(sb + L::kOffO + s * L::kSubT + c * L::kHalfS, &to64, bar(kBarQFull + s), c * 64, h, q0, b);
        }
        const int64_t pr = ((static_cast<int64_t>(b) * a.H + h) * ntq + cur.w.t) * kSub;
        bulk_g2s(smem_addr(s_lse + s * kSub), a.lse2p + pr, kSub * 4, bar(kBarQFull + s));
        bulk_g2s(smem_addr(s_dlt + s * kSub), a.dltp + pr, kSub * 4, bar(kBarQFull + s));
      }
      __syncwarp();
      ++issued[s];
      cur.next();
    }
    if (*abort_flag) {
      // let every issued copy land before the CTA's shared memory goes away
      drain_wait(bar(kBarKV), 0, tmo);
      for (int s = 0; s < kSlots; ++s)
        if (issued[s]) drain_wait(bar(kBarQFull + s), (issued[s] - 1) & 1, tmo);
    }
  } else if (warp == 1) {
    // ===================== MMA issuer =====================
    const bool leader = elect_one();
    constexpr uint32_t idesc_s = idesc_bf16_f32(kT, kSub, false, false);  // S^T, dP^T: M = keys, N = 64 queries
    constexpr uint32_t idesc_g = idesc_bf16_f32(kT, D, false, true);      // dV, dK: A in TMEM, B MN-major
    const uint64_t k_km = smem_desc_sw128(sb + L::kOffK, 16, 1024);
    const uint64_t v_km = smem_desc_sw128(sb + L::kOffV, 16, 1024);
    const uint64_t q_km = smem_desc_sw128(sb + L::kOffQ, 16, 1024);
    const uint64_t o_km = smem_desc_sw128(sb + L::kOffO, 16, 1024);
    const uint64_t q_mn = smem_desc_sw128(sb + L::kOffQ, L::kHalfS, 1024);
    const uint64_t o_mn = smem_desc_sw128(sb + L::kOffO, L::kHalfS, 1024);
    const uint32_t km_hi = static_cast<uint32_t>(k_km >> 32), mn_hi = static_cast<uint32_t>(q_mn >> 32);
    const uint32_t k_km_lo = static_cast<uint32_t>(k_km), v_km_lo = static_cast<uint32_t>(v_km);
    const uint32_t q_km_lo = static_cast<uint32_t>(q_km), o_km_lo = static_cast<uint32_t>(o_km);
    const uint32_t q_mn_lo = static_cast<uint32_t>(q_mn), o_mn_lo = static_cast<uint32_t>(o_mn);
    auto commit = [&](uint32_t bar_addr) {
      if (leader) mma_commit(bar_addr);
    };
    // S^T and dP^T of the sub-tile in smem slot q, into TMEM slot ts
    auto issue_sdp = [&](int q, int ts) {
      const uint32_t slot = static_cast<uint32_t>((q * L::kSubT) >> 4);
      const uint32_t d = tmem + ts * 128;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        if (leader) mma_ss_lohi(d, k_km_lo + kstep128(kk), km_hi, q_km_lo + slot + kstep64(kk), km_hi, idesc_s, kk > 0);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        if (leader)
          mma_ss_lohi(d + kSub, v_km_lo + kstep128(kk), km_hi, o_km_lo + slot + kstep64(kk), km_hi, idesc_s, kk > 0);
    };
    // dV += P^T dO and dK += dS^T Q over the sub-tile's 64 query rows (K = rows:
    // 16 rows = 2048 bytes of an MN-major sub-tile; the bf16 P^T / dS^T of
    // rows [32 h, 32 h + 32) sit in TMEM columns [32 h, 32 h + 16) of theirs)
    auto issue_g = [&](int q, int ts, bool acc) {
      const uint32_t slot = static_cast<uint32_t>((q * L::kSubT) >> 4);
      const uint32_t pa = tmem + ts * 128;
#pragma unroll
      for (int kk = 0; kk < kSub / 16; ++kk)
        if (leader) mma_ts_lohi(tmem + kAcc, pa + pcol(kk), o_mn_lo + slot + ((kk * 2048) >> 4), mn_hi, idesc_g,
                                (acc || kk > 0) ? 1u : 0u);
#pragma unroll
      for (int kk = 0; kk < kSub / 16; ++kk)
        if (leader) mma_ts_lohi(tmem + kAcc + D, pa + kSub + pcol(kk), q_mn_lo + slot + ((kk * 2048) >> 4), mn_hi,
                                idesc_g, (acc || kk > 0) ? 1u : 0u);
    };
    auto wait_q = [&](int j) -> bool {
      return mbar_wait_bounded(bar(kBarQFull + j % kSlots), (j / kSlots) & 1, abort_flag, a.err, tmo);
    };
    bool ok = mbar_wait_bounded(bar(kBarKV), 0, abort_flag, a.err, tmo);
    // prologue: S^T, dP^T of the first kTS sub-steps
    for (int j = 0; ok && j < kTS && j < NJ; ++j) {
      if (!wait_q(j)) {
        ok = false;
        break;
      }
      tc_fence_after();
      issue_sdp(j, j);
      commit(bar(kBarSFull + j));
    }
    // sub-step j: once P^T, dS^T are in TMEM slot j mod kTS, dV and dK consume
    // them and S^T, dP^T of sub-step j + kTS go into the same slot; the step is
    // instantiated per smem slot so every operand offset is a constant
    auto step = [&](auto q_c, int j) -> bool {
      constexpr int q = decltype(q_c)::value;
      constexpr int ts = q % kTS;
      if (!mbar_wait_bounded(bar(kBarPFull + ts), (j / kTS) & 1, abort_flag, a.err, tmo)) return false;
      tc_fence_after();
      issue_g(q, ts, j > 0);
      commit(bar(kBarQEmpty + q));
      if (j + kTS < NJ) {
        if (!wait_q(j + kTS)) return false;
        tc_fence_after();
        issue_sdp((q + kTS) % kSlots, ts);
        commit(bar(kBarSFull + ts));
      }
      return true;
    };
    for (int j = 0; ok && j < NJ; j += kSlots)
      ok = each(std::make_integer_sequence<int, kSlots>{}, [&](auto q) { return j + q >= NJ || step(q, j + q); });
    if (ok) {
      commit(bar(kBarDone));
    } else {
      commit(bar(kBarDrain));
      drain_wait(bar(kBarDrain), 0, tmo);
    }
  } else {
    // ===================== row pass: one thread per key row and column half =====================
    const int wq = warp & 3;
    const int group = (warp - 2) / kGroupWarps;  // takes the sub-steps j = group mod kGroups
    const int hc = ((warp - 2) >> 2) & 1;        // this warp's 32 query columns of each
    const int key = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const bool kvalid = key < nk;
    const float c2 = a.scale * kLog2e, capl2 = a.cap * kLog2e;
    const int jkey = key0 + key;
    const bool open = !a.causal || jkey < plim;  // every row may see this key
    const int kd = a.qdoc && kvalid ? a.kdoc[static_cast<int64_t>(b) * a.Skv + jkey] : -1;
    const int* qdoc = a.qdoc + static_cast<int64_t>(b) * a.Sq;
    bool ok = true;
    HeadWalk cur(bits, t0, ntq, per_head, hk * a.G, j0 + group);
    for (int j = group; j < NJ; j += kGroups) {
      const int q = j % kSlots, ts = j % kTS;
      const float slope2 = kBias ? __ldg(a.slopes + cur.h) * kLog2e : 0.f;
      const int i0 = cur.w.t * kSub + hc * 32;  // the query row of this warp's first column
      const int d0 = a.rel + i0 - jkey;       // its position less the key's
      uint32_t on = !kvalid ? 0u : open || d0 >= 0 ? ~0u : d0 <= -32 ? 0u : ~0u << -d0;
      if (bits != nullptr && ((act[kMapWords + (cur.w.t >> 5)] >> (cur.w.t & 31)) & 1u)) {
        const int ids[1] = {i0 + lane < a.Sq ? __ldg(qdoc + i0 + lane) : -1};
        uint32_t same[1];
        same_docs<1>(kd, ids, same);
        on &= same[0];
      }
      ok = __all_sync(0xffffffffu,
                      mbar_wait_bounded(bar(kBarQFull + q), (j / kSlots) & 1, abort_flag, a.err, tmo) &&
                          mbar_wait_bounded(bar(kBarSFull + ts), (j / kTS) & 1, abort_flag, a.err, tmo));
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_s = tmem + lane_off + ts * 128 + hc * 32, t_dp = t_s + kSub;
      const float* nlse2 = s_lse + q * kSub + hc * 32;
      const float* dlt = s_dlt + q * kSub + hc * 32;
      // P^T over the first half of this warp's S^T columns, dS^T over those of
      // dP^T, kN columns at a time, the next ones' loads under way meanwhile
      uint32_t sr[kGroups][kN], dr[kGroups][kN], pp[kN / 2], dd[kN / 2];
      tmem_ld(t_s, sr[0]);
      tmem_ld(t_dp, dr[0]);
#pragma unroll
      for (int c = 0; c < kGroups; ++c) {
        tmem_wait_ld();
        tmem_pin(sr[c]);
        tmem_pin(dr[c]);
        if (c + 1 < kGroups) {
          tmem_ld(t_s + (c + 1) * kN, sr[(c + 1) % kGroups]);
          tmem_ld(t_dp + (c + 1) * kN, dr[(c + 1) % kGroups]);
        }
        row_pass<kCap, kBias, 1>(
            sr[c], dr[c], cc, c2, capl2, slope2, static_cast<float>(d0 + kN * c), on >> (kN * c),
            [&](int e) { return *reinterpret_cast<const f32x2*>(nlse2 + kN * c + e); },
            [&](int e) { return *reinterpret_cast<const f32x2*>(dlt + kN * c + e); }, pp, dd);
        tmem_st(t_s + kN / 2 * c, pp);
        tmem_st(t_dp + kN / 2 * c, dd);
      }
#pragma unroll
      for (int c = 0; c < kGroups; ++c) cur.next();
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarPFull + ts));
    }
    // ---- dk, dv of this CTA's keys ----
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarDone), 0, abort_flag, a.err, tmo));
    if (ok) {
      tc_fence_after();
      const int g = hc;  // column half 0 writes dv, half 1 dk; NJ == 0: no row reaches these keys
      if (cs > 1) {  // this CTA's part, over the idle tiles: [dv, dk][key][D], 16-byte pieces permuted by row
        float* part = reinterpret_cast<float*>(smem) + (g * kT + key) * D;
#pragma unroll 1
        for (int c = group * (D / 32 / kGroups); c < (group + 1) * (D / 32 / kGroups); ++c) {
          uint32_t r[32];
          tmem_ld32(tmem + lane_off + kAcc + g * D + c * 32, r);
          tmem_wait_ld();
          tmem_pin(r);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            *reinterpret_cast<float4*>(part + (((c * 8 + x) ^ (key & 7)) * 4)) =
                NJ == 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                        : make_float4(u2f(r[4 * x]), u2f(r[4 * x + 1]), u2f(r[4 * x + 2]), u2f(r[4 * x + 3]));
        }
      } else {
        constexpr int kCols = D / kGroups;
        const int c = group * kCols;
        store_acc<kCols>(tmem + lane_off + kAcc + g * D + c, NJ == 0, g == 0 ? 1.f : -a.scale,
                     smem + L::kOffQ + (warp - 2) * 4096, lane, g == 0 ? a.dv : a.dk,
                     ((static_cast<int64_t>(b) * a.Skv + key0 + wq * 32) * a.Hkv + hk) * D + c,
                     static_cast<int64_t>(a.Hkv) * D, nk - wq * 32, a.grad_bf16);
      }
    }
  }
  if (cs > 1) {
    static_assert(2 * kT * D * 4 <= L::kOffLse, "the parts lie over the tiles");
    cluster_sync();
    // a row's D / 4 pieces on neighbouring lanes, kIn rows a thread at once: every
    // load of a step is under way before the first is used
    auto join = [&](auto cs_c) {
      constexpr int kCs = decltype(cs_c)::value, kIn = 16 / kCs;
      constexpr int kStep = kThreadsB / (D / 4);  // rows side by side
      const int share = kT / kCs, p = threadIdx.x % (D / 4);
      for (int e0 = threadIdx.x / (D / 4); e0 < 2 * share; e0 += kStep * kIn) {  // dv's rows, then dk's
        float4 y[kIn][kCs];
#pragma unroll
        for (int u = 0; u < kIn; ++u) {
          const int e = min(e0 + u * kStep, 2 * share - 1), g = e / share, k = rank * share + e % share;
#pragma unroll
          for (int c = 0; c < kCs; ++c)
            y[u][c] = ld_peer4(cluster_peer(sb + static_cast<uint32_t>(((g * kT + k) * D + ((p ^ (k & 7)) * 4)) * 4), c));
        }
#pragma unroll
        for (int u = 0; u < kIn; ++u) {
          const int e = e0 + u * kStep, g = e / share, k = rank * share + e % share;
          if (e >= 2 * share) break;
          if (k >= nk) continue;
          float4 x = y[u][0];
#pragma unroll
          for (int c = 1; c < kCs; ++c) x = make_float4(x.x + y[u][c].x, x.y + y[u][c].y, x.z + y[u][c].z, x.w + y[u][c].w);
          const float mul = g == 0 ? 1.f : -a.scale;
          void* dst = g == 0 ? a.dv : a.dk;
          const int64_t o = ((static_cast<int64_t>(b) * a.Skv + key0 + k) * a.Hkv + hk) * D + p * 4;
          if (a.grad_bf16) {
            uint2 v;
            v.x = pack_bf16x2(x.x * mul, x.y * mul);
            v.y = pack_bf16x2(x.z * mul, x.w * mul);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(dst) + o) = v;
          } else {
            *reinterpret_cast<float4*>(static_cast<float*>(dst) + o) =
                make_float4(x.x * mul, x.y * mul, x.z * mul, x.w * mul);
          }
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
    tmem_dealloc(tmem, kTmemColsB);
  }
}

// ----------------------------------------------------------------------------
// dq: one CTA per 128 query rows of one (batch entry, head). The row warps
// load the CTA's Q and dO rows once into TMEM (bf16 pairs, the A-operand
// layout: D columns behind dQ); 64-key K and V
// sub-tiles that the rows reach stream through kDqSlots shared-memory slots. Per sub-tile three MMAs (M = 128 rows):
//   S  = Q K^T    (TS: Q in TMEM, K K-major; N = 64) -> TMEM slot j mod kTS, [0, 64)
//   dP = dO V^T   (TS)                               -> the same slot, [64, 128)
//   dQ += dS K    (TS: dS over S's first 32 columns, K read MN-major)
//                                                    -> TMEM [kAcc, kAcc + D)
// Only K and V come from shared memory. S and dP of sub-step j + kTS are issued
// right after dQ of sub-step j, so they run while the row warps (one thread
// per query row and column half, lse and delta in registers) form
// dS = p (dp - delta) of sub-step j + 1. dq is stored once, without atomics.
// ----------------------------------------------------------------------------
constexpr int kDqSlots = 6;  // K/V sub-tile slots of the dq kernel

template <int D>
struct DqSmem {
  static constexpr int kSubT = kSub * D * 2;  // a K or V sub-tile: 64 keys
  static constexpr int kHalfS = kSub * 128;
  static constexpr int kOffK = 0;                          // kDqSlots sub-tiles
  static constexpr int kOffV = kOffK + kDqSlots * kSubT;   // kDqSlots sub-tiles
  static constexpr int kOffBar = kOffV + kDqSlots * kSubT;
  static constexpr int kNumBars = 1 + 2 * kDqSlots + 9;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffMap = kOffMisc + 16;
  static constexpr int kBytes = kOffMap + 2 * kMapWords * 4;
  static constexpr int kMax = 227 * 1024;
  static constexpr int kAlloc = kBytes + 1024 <= kMax ? kBytes + 1024 : kMax;
};

enum : int {
  kDqBarQ = 0,                             // Q and dO in TMEM (every row warp arrives)
  kDqBarKVFull = 1,                        // +slot: K and V sub-tiles landed
  kDqBarKVEmpty = 1 + kDqSlots,            // +slot: MMAs done with the slot
  kDqBarSFull = 1 + 2 * kDqSlots,          // +TMEM slot (3): S and dP in TMEM
  kDqBarPFull = kDqBarSFull + 3,           // +TMEM slot (3): dS written (every row warp arrives)
  kDqBarDone = kDqBarPFull + 3,            // every MMA done: dQ final
  kDqBarDrain = kDqBarDone + 1,
  kDqBarLoad = kDqBarDrain + 1,            // Q and dO landed in the last two slots
};

// One dq CTA: query tile bx of head h, batch entry b.
template <int D, bool kCap, bool kBias>
__device__ __forceinline__ void dq_cta(const CUtensorMap& tq64, const CUtensorMap& to64, const CUtensorMap& tk64,
                                       const CUtensorMap& tv64, const ScoreArgs& a,
                                       const CapCoef& cc, uint8_t* smem_raw, int alloc, int bx, int h, int b) {
  using L = DqSmem<D>;
  // TMEM: the slots, dQ, then Q and dO (D / 2 columns each)
  constexpr int kTS = Ring<D>::kTS, kAcc = Ring<D>::kAcc, kOp = kAcc + D;
  constexpr int kGroups = Rows<D>::kGroups, kN = Rows<D>::kN;
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  if (pad > static_cast<uint32_t>(alloc - L::kBytes)) {
    if (threadIdx.x == 0) atomicOr(a.err, kDevErrLayout);
    return;
  }
  uint8_t* smem = smem_raw + pad;
  const uint32_t sb = smem_addr(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);  // [0] TMEM base, [1] abort flag, [2] count
  volatile uint32_t* abort_flag = misc + 1;
  auto bar = [&](int i) -> uint32_t { return sb + L::kOffBar + 8 * i; };

  const int hk = h / a.G;
  const int q0 = bx * kT;
  const int nq = min(kT, a.Sq - q0);
  const int plim = prefix_limit(a, b);
  // key sub-tiles that the last row (the largest limit) reaches
  const int ntk = (max(0, min(a.Skv, key_limit(a, plim, q0 + nq - 1))) + kSub - 1) / kSub;
  const int nqb = (a.Sq + kDocBlock - 1) / kDocBlock, nkb = (a.Skv + kDocBlock - 1) / kDocBlock;
  uint32_t* act = reinterpret_cast<uint32_t*>(smem + L::kOffMap);
  const uint32_t* bits = a.qdoc ? act : nullptr;
  int NJ = ntk;
  if (a.qdoc)
    NJ = walk_map(a.krange + static_cast<int64_t>(b) * nkb, nkb,
                  doc_span(a.qrange + static_cast<int64_t>(b) * nqb, nqb, bx * 2, 2), 0, ntk, act, misc + 2);

  if (threadIdx.x == 0) {  // (in the order that dkdv_cta states)
    for (int i = 0; i < L::kNumBars; ++i)
      mbar_init(bar(i), i == kDqBarQ ? Rows<D>::kWarps : i >= kDqBarPFull && i < kDqBarDone ? kGroupWarps : 1);
    misc[1] = 0;
    fence_mbar_init();
    fence_async();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(misc), kTmemColsB);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const uint64_t tmo = a.timeout_ns;

  if (warp == 0) {
    // ===================== TMA producer =====================
    const bool leader = elect_one();
    // Q and dO first, through the last two K and the last two V slots: the row
    // warps take them to TMEM before those are needed
    if (leader) {
      mbar_arrive_expect_tx(bar(kDqBarLoad), 2 * kT * D * 2);
      for (int c = 0; c < D / 64; ++c)
        for (int r = 0; r < kT; r += kSub) {
          const uint32_t at = (kDqSlots - 2) * L::kSubT + c * (kT * 128) + r * 128;
          tma_load_4d(sb + L::kOffK + at, &tq64, bar(kDqBarLoad), c * 64, h, q0 + r, b);
          tma_load_4d(sb + L::kOffV + at, &to64, bar(kDqBarLoad), c * 64, h, q0 + r, b);
        }
    }
    int issued[kDqSlots] = {};
    TileWalk<> cur(bits, 0, ntk, -1);
    for (int j = 0; j < NJ; ++j) {
      const int s = j % kDqSlots;
      const uint32_t ph = (j / kDqSlots) & 1;
      if (j == kDqSlots - 2 && !__all_sync(0xffffffffu, mbar_wait_bounded(bar(kDqBarQ), 0, abort_flag, a.err, tmo))) break;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar(kDqBarKVEmpty + s), ph ^ 1, abort_flag, a.err, tmo)))
        break;
      if (leader) {
        mbar_arrive_expect_tx(bar(kDqBarKVFull + s), 2 * L::kSubT);
        for (int c = 0; c < D / 64; ++c) {
          tma_load_4d(sb + L::kOffK + s * L::kSubT + c * L::kHalfS, &tk64, bar(kDqBarKVFull + s), c * 64, hk,
                      cur.t * kSub, b);
          tma_load_4d(sb + L::kOffV + s * L::kSubT + c * L::kHalfS, &tv64, bar(kDqBarKVFull + s), c * 64, hk,
                      cur.t * kSub, b);
        }
      }
      ++issued[s];
      cur.next();
    }
    if (*abort_flag) {
      // let every issued copy land before the CTA's shared memory goes away
      drain_wait(bar(kDqBarLoad), 0, tmo);
      for (int s = 0; s < kDqSlots; ++s)
        if (issued[s]) drain_wait(bar(kDqBarKVFull + s), (issued[s] - 1) & 1, tmo);
    }
  } else if (warp == 1) {
    // ===================== MMA issuer =====================
    const bool leader = elect_one();
    constexpr uint32_t idesc_s = idesc_bf16_f32(kT, kSub, false, false);  // S, dP: M = query rows, N = 64 keys
    constexpr uint32_t idesc_q = idesc_bf16_f32(kT, D, false, true);      // dQ: A (dS) in TMEM, B (K) MN-major
    const uint64_t k_km = smem_desc_sw128(sb + L::kOffK, 16, 1024);
    const uint64_t v_km = smem_desc_sw128(sb + L::kOffV, 16, 1024);
    const uint64_t k_mn = smem_desc_sw128(sb + L::kOffK, L::kHalfS, 1024);
    const uint32_t km_hi = static_cast<uint32_t>(k_km >> 32), mn_hi = static_cast<uint32_t>(k_mn >> 32);
    const uint32_t k_lo = static_cast<uint32_t>(k_km), v_lo = static_cast<uint32_t>(v_km);
    const uint32_t k_mn_lo = static_cast<uint32_t>(k_mn);
    const uint32_t t_q = tmem + kOp, t_o = tmem + kOp + D / 2;  // Q and dO rows in TMEM (8 columns per K step)
    auto commit = [&](uint32_t bar_addr) {
      if (leader) mma_commit(bar_addr);
    };
    // S and dP of the K/V sub-tile in smem slot q, into TMEM slot ts
    auto issue_sdp = [&](int q, int ts) {
      const uint32_t slot = static_cast<uint32_t>((q * L::kSubT) >> 4);
      const uint32_t d = tmem + ts * 128;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        if (leader) mma_ts_lohi(d, t_q + kk * 8, k_lo + slot + kstep64(kk), km_hi, idesc_s, kk > 0 ? 1u : 0u);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        if (leader) mma_ts_lohi(d + kSub, t_o + kk * 8, v_lo + slot + kstep64(kk), km_hi, idesc_s, kk > 0 ? 1u : 0u);
    };
    auto wait_kv = [&](int j) -> bool {
      return mbar_wait_bounded(bar(kDqBarKVFull + (j % kDqSlots)), (j / kDqSlots) & 1, abort_flag, a.err, tmo);
    };
    bool ok = mbar_wait_bounded(bar(kDqBarQ), 0, abort_flag, a.err, tmo);
    for (int j = 0; ok && j < kTS && j < NJ; ++j) {
      if (!wait_kv(j)) {
        ok = false;
        break;
      }
      tc_fence_after();
      issue_sdp(j, j);
      commit(bar(kDqBarSFull + j));
    }
    // sub-step j: dQ += dS K once dS is in TMEM slot j mod kTS (K = keys: 16 key
    // rows = 2048 bytes of the MN-major sub-tile), then S, dP of sub-step j + kTS
    // into the same slot; instantiated per smem slot (a multiple of kTS of them, so
    // the TMEM slot is the smem slot modulo kTS)
    static_assert(kDqSlots % kTS == 0, "TMEM slot = smem slot modulo kTS");
    auto step = [&](auto q_c, int j) -> bool {
      constexpr int q = decltype(q_c)::value;
      constexpr int ts = q % kTS;
      if (!mbar_wait_bounded(bar(kDqBarPFull + ts), (j / kTS) & 1, abort_flag, a.err, tmo)) return false;
      tc_fence_after();
      const uint32_t slot = static_cast<uint32_t>((q * L::kSubT) >> 4);
#pragma unroll
      for (int kk = 0; kk < kSub / 16; ++kk)
        if (leader) mma_ts_lohi(tmem + kAcc, tmem + ts * 128 + pcol(kk), k_mn_lo + slot + ((kk * 2048) >> 4), mn_hi,
                                idesc_q, (j > 0 || kk > 0) ? 1u : 0u);
      commit(bar(kDqBarKVEmpty + q));
      if (j + kTS < NJ) {
        if (!wait_kv(j + kTS)) return false;
        tc_fence_after();
        issue_sdp((q + kTS) % kDqSlots, ts);
        commit(bar(kDqBarSFull + ts));
      }
      return true;
    };
    for (int j = 0; ok && j < NJ; j += kDqSlots)
      ok = each(std::make_integer_sequence<int, kDqSlots>{}, [&](auto q) { return j + q >= NJ || step(q, j + q); });
    if (ok) {
      commit(bar(kDqBarDone));
    } else {
      commit(bar(kDqBarDrain));
      drain_wait(bar(kDqBarDrain), 0, tmo);
    }
  } else {
    // ===================== dS: one thread per query row and column half =====================
    const int wq = warp & 3;
    const int group = (warp - 2) / kGroupWarps;  // takes the sub-steps j = group mod kGroups
    const int hc = ((warp - 2) >> 2) & 1;        // this warp's 32 key columns of each
    const int row = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const float c2 = a.scale * kLog2e, capl2 = a.cap * kLog2e;
    // the row's -lse log2e and delta, from the padded copies (a row past the end holds -inf, 0)
    float nl2 = -INFINITY, dlt = 0.f;
    if (row < nq) {
      const int64_t o = (static_cast<int64_t>(b) * a.H + h) * nqb * kDocBlock + q0 + row;
      nl2 = a.lse2p[o];
      dlt = a.dltp[o];
    }
    // this row's Q (column half 0) or dO (half 1) into TMEM as the A operand
    // of S and dP: column c holds elements 2c and 2c + 1 of the row, which is
    // the row's memory read as 32-bit words; rows past the end were filled with
    // zeros (read from global memory a row a lane, this took 7000 cycles)
    bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kDqBarLoad), 0, abort_flag, a.err, tmo));
    if (ok) {
      const uint8_t* src = smem + (hc == 0 ? L::kOffK : L::kOffV) + (kDqSlots - 2) * L::kSubT + row * 128;
#pragma unroll 1
      for (int c = group; c < D / 64; c += kGroups) {
        uint32_t w[32];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const uint4 u = *reinterpret_cast<const uint4*>(src + c * (kT * 128) + ((x ^ (row & 7)) * 16));
          w[4 * x] = u.x;
          w[4 * x + 1] = u.y;
          w[4 * x + 2] = u.z;
          w[4 * x + 3] = u.w;
        }
        tmem_st32(tmem + lane_off + kOp + hc * (D / 2) + c * 32, w);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kDqBarQ));
    }
    const int lim = min(a.Skv, key_limit(a, plim, q0 + row));
    const int qd = a.qdoc && row < nq ? a.qdoc[static_cast<int64_t>(b) * a.Sq + q0 + row] : -1;
    const int* kdoc = a.kdoc + static_cast<int64_t>(b) * a.Skv;
    const float slope2 = kBias ? a.slopes[h] * kLog2e : 0.f;
    TileWalk<> cur(bits, 0, ntk, -1);
    if (group == 1) cur.next();
    for (int j = group; ok && j < NJ; j += kGroups) {
      const int ts = j % kTS;
      const int j0 = cur.t * kSub + hc * 32;  // the key of this warp's first column
      const int n = lim - j0;
      uint32_t on = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
      if (bits != nullptr && ((act[kMapWords + (cur.t >> 5)] >> (cur.t & 31)) & 1u)) {
        const int ids[1] = {j0 + lane < a.Skv ? __ldg(kdoc + j0 + lane) : -1};
        uint32_t same[1];
        same_docs<1>(qd, ids, same);
        on &= same[0];
      }
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kDqBarSFull + ts), (j / kTS) & 1, abort_flag, a.err, tmo));
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_s = tmem + lane_off + ts * 128 + hc * 32, t_dp = t_s + kSub;  // this sub-step's slot
      uint32_t sr[kGroups][kN], dr[kGroups][kN], pp[kN / 2], dd[kN / 2];
      tmem_ld(t_s, sr[0]);
      tmem_ld(t_dp, dr[0]);
#pragma unroll
      for (int c = 0; c < kGroups; ++c) {
        tmem_wait_ld();
        tmem_pin(sr[c]);
        tmem_pin(dr[c]);
        if (c + 1 < kGroups) {
          tmem_ld(t_s + (c + 1) * kN, sr[(c + 1) % kGroups]);
          tmem_ld(t_dp + (c + 1) * kN, dr[(c + 1) % kGroups]);
        }
        row_pass<kCap, kBias, -1>(
            sr[c], dr[c], cc, c2, capl2, slope2, static_cast<float>(a.rel + q0 + row - j0 - kN * c), on >> (kN * c),
            [&](int) { return pair(nl2, nl2); }, [&](int) { return pair(dlt, dlt); }, pp, dd);
        tmem_st(t_s + kN / 2 * c, dd);  // dS over the first half of this warp's S columns
      }
#pragma unroll
      for (int c = 0; c < kGroups; ++c) cur.next();
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kDqBarPFull + ts));
    }
    // ---- dq of this CTA's rows ----
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kDqBarDone), 0, abort_flag, a.err, tmo));
    if (ok) {
      tc_fence_after();
      // half the columns by each column half (of the first group); NJ == 0: these rows reach no key
      if (group == 0)
        store_acc<D / 2>(tmem + lane_off + kAcc + hc * (D / 2), NJ == 0, -a.scale, smem + L::kOffK + (warp - 2) * 4096, lane,
                         a.dq, ((static_cast<int64_t>(b) * a.Sq + q0 + wq * 32) * a.H + h) * D + hc * (D / 2),
                         static_cast<int64_t>(a.H) * D, nq - wq * 32, a.grad_bf16);
    }
  }

  // ---- teardown: every thread of the CTA arrives here, aborted or not ----
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemColsB);
  }
}

template <int D>
__host__ __device__ constexpr int bwd_alloc() {
  return BSmem<D>::kAlloc > DqSmem<D>::kAlloc ? BSmem<D>::kAlloc : DqSmem<D>::kAlloc;
}

// Both kinds of CTA in one launch: the dk/dv items from the first keys (which
// the most causal rows reach), each taken by the CTAs of one cluster; then the
// dq CTAs from the last rows, heads fastest, so that long CTAs start first and
// short ones fill the end.
template <int D, bool kCap, bool kBias>
__global__ void __launch_bounds__(Rows<D>::kThreads, 1)
    score_bwd_tc_kernel(const __grid_constant__ CUtensorMap tq64, const __grid_constant__ CUtensorMap to64,
                        const __grid_constant__ CUtensorMap tk64, const __grid_constant__ CUtensorMap tv64,
                        const __grid_constant__ ScoreArgs a, const __grid_constant__ CapCoef cc) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int cs = static_cast<int>(cluster_size());
  const int nkv = (a.Skv + kT - 1) / kT, nq = (a.Sq + kT - 1) / kT;
  const int kv_ctas = nkv * a.Hkv * a.B * cs;
  const int id = static_cast<int>(blockIdx.x);
  grid_wait();  // the delta kernel's results
  if (id < kv_ctas) {
    const int item = id / cs, bh = item % (a.Hkv * a.B);
    dkdv_cta<D, kCap, kBias>(tq64, tk64, tv64, to64, a, cc, smem_raw, bwd_alloc<D>(), cs, id % cs, item / (a.Hkv * a.B),
                             bh % a.Hkv, bh / a.Hkv);
  } else {
    const int i = id - kv_ctas, bh = i % (a.H * a.B);
    if (i < nq * a.H * a.B)  // the last cluster may have CTAs without work
      dq_cta<D, kCap, kBias>(tq64, to64, tk64, tv64, a, cc, smem_raw, bwd_alloc<D>(), nq - 1 - i / (a.H * a.B), bh % a.H, bh / a.H);
  }
}

// delta_i = out_i . dout_i and -lse_i log2e, 64 rows of one (batch entry, head) a
// CTA, into copies padded to 64 rows: -inf and 0 past the end, -inf for a row
// that saw no key. Bound by HBM (out and dout are read once).
template <int D, bool kOutBf16>
__global__ void __launch_bounds__(256) score_delta_tc_kernel(const __grid_constant__ ScoreArgs a) {
  constexpr int kLanes = D / 8;        // lanes of a row, 8 elements each
  constexpr int kRows = 256 / kLanes;  // rows a pass
  grid_release();
  const int sub = threadIdx.x % kLanes;
  const int blk = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int64_t pad0 = ((static_cast<int64_t>(b) * a.H + h) * gridDim.x + blk) * kSub;
#pragma unroll
  for (int r0 = 0; r0 < kSub; r0 += kRows) {
    const int r = r0 + threadIdx.x / kLanes, row = blk * kSub + r;
    float sum = 0.f;
    if (row < a.Sq) {
      const int64_t at = ((static_cast<int64_t>(b) * a.Sq + row) * a.H + h) * D + sub * 8;
      const uint4 g = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.dout) + at);
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
      float o[8];
      if constexpr (kOutBf16) {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.o) + at);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[2 * i] = __uint_as_float(w[i] << 16);
          o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      } else {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.o) + at);
        const float4 x = p[0], y = p[1];
        o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
        o[4] = y.x; o[5] = y.y; o[6] = y.z; o[7] = y.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum = fmaf(__uint_as_float(gw[i] << 16), o[2 * i], sum);
        sum = fmaf(__uint_as_float(gw[i] & 0xffff0000u), o[2 * i + 1], sum);
      }
    }
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    if (sub == 0) {
      const float l = row < a.Sq ? a.lse[(static_cast<int64_t>(b) * a.H + h) * a.Sq + row] : -INFINITY;
      a.lse2p[pad0 + r] = l == -INFINITY ? -INFINITY : -l * kLog2e;
      a.dltp[pad0 + r] = row < a.Sq ? sum : 0.f;
    }
  }
}

struct BwdMaps {
  CUtensorMap q64, o64, k64, v64;
};

template <int D, bool kCap, bool kBias>
cudaError_t launch_rule(const ScoreArgs& a, const BwdMaps& m, cudaStream_t s) {
  constexpr int kAlloc = bwd_alloc<D>();
  static_assert(kAlloc <= 227 * 1024, "shared memory budget");
  cudaError_t e = allow_smem<score_bwd_tc_kernel<D, kCap, kBias>>(kAlloc);
  if (e != cudaSuccess) return e;
  const int64_t ntq = (a.Sq + kSub - 1) / kSub, ntk = (a.Skv + kSub - 1) / kSub;
  const int64_t kv_items = static_cast<int64_t>((a.Skv + kT - 1) / kT) * a.Hkv * a.B;
  const int64_t q_ctas = static_cast<int64_t>((a.Sq + kT - 1) / kT) * a.H * a.B;
  // sub-steps: a dq CTA's take 3/4 of a dk/dv CTA's; some 8 of them go by before
  // the first and after the last
  const int cs = cluster_for(8.0, kv_items, ntq * a.G, q_ctas, ntk * 3 / 4, a.causal ? 0.5 : 1.0, false, a.sms);
  const int64_t ctas = kv_items * cs + (q_ctas + cs - 1) / cs * cs;
  return launch_clusters(score_bwd_tc_kernel<D, kCap, kBias>, ctas / cs, 1, 1, cs, Rows<D>::kThreads, kAlloc, a.Sq > 0, s, m.q64,
                         m.o64, m.k64, m.v64, a, make_cap_coef(a.scale, a.cap, true));
}

template <int D>
cudaError_t launch_d(const ScoreArgs& a, cudaStream_t s) {
  if (a.Sq > 0) {
    const dim3 grid((a.Sq + kSub - 1) / kSub, a.H, a.B);
    if (a.out_bf16)
      score_delta_tc_kernel<D, true><<<grid, 256, 0, s>>>(a);
    else
      score_delta_tc_kernel<D, false><<<grid, 256, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // one side may be empty: its maps stand on the other's memory and are never read through
  const bool noq = a.Sq == 0, nok = a.Skv == 0;
  const void *q = noq ? a.k : a.q, *o = noq ? a.k : a.dout, *k = nok ? a.q : a.k, *v = nok ? a.q : a.v;
  const int hq = noq ? a.Hkv : a.H, sq = noq ? a.Skv : a.Sq, hk = nok ? a.H : a.Hkv, sk = nok ? a.Sq : a.Skv;
  BwdMaps m;
  if (!host_tmap_bf16(&m.q64, q, D, hq, sq, a.B, kSub) || !host_tmap_bf16(&m.o64, o, D, hq, sq, a.B, kSub) ||
      !host_tmap_bf16(&m.k64, k, D, hk, sk, a.B, kSub) || !host_tmap_bf16(&m.v64, v, D, hk, sk, a.B, kSub))
    return cudaErrorInvalidValue;
  if (a.cap > 0.f) return a.slopes ? launch_rule<D, true, true>(a, m, s) : launch_rule<D, true, false>(a, m, s);
  return a.slopes ? launch_rule<D, false, true>(a, m, s) : launch_rule<D, false, false>(a, m, s);
}

}  // namespace

cudaError_t launch_score_bwd_tc(const ScoreArgs& a, int D, cudaStream_t s) {
  return D == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace cp
