// cp_score_api.cu — the C ABI of score-rule attention and of the paged cache
// (declared in include/cp_attn.h): argument checks, workspace layout and
// launches.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "cp_attn.h"
#include "cp_score.h"

namespace {

using cp::DocRange;
using cp::PagedArgs;
using cp::ScoreArgs;

constexpr uint64_t kWaitTimeoutNs = 1000000000ull;  // 1 s per device-side wait
constexpr int64_t kMaxPos = 1 << 30;                // positions stay within 31 bits
constexpr int kMaxGrid = 65535;                     // batch entries, heads

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool known(cp_dtype t) { return t == CP_BF16 || t == CP_F32; }

// An output is fp32 or of the inputs' type.
bool out_type_ok(cp_dtype out, cp_dtype in) { return known(out) && (out == CP_F32 || out == in); }

// A scale and a cap whose quotient, products with log2 e and coefficients fp32 holds.
bool scores_ok(float scale, float softcap) {
  if (!(std::fabs(scale) <= 1e30f) || !(softcap >= 0.f && softcap <= 1e30f)) return false;
  return softcap == 0.f || (softcap >= 1e-30f && softcap >= std::fabs(scale) * 1e-30f);
}

const cp_score_rule kPlainRule = {0.f, nullptr, 0, nullptr, nullptr, nullptr, 0, 0};

int64_t doc_blocks(int S) { return (static_cast<int64_t>(S) + cp::kDocBlock - 1) / cp::kDocBlock; }

// Workspace of the forward: the document ranges of q and k. The backward has
// lse log2e and delta in front, each (batch entry, head) padded to 64 rows
// (fp32 inputs use delta alone, unpadded).
struct ScoreWs {
  size_t lse = 0, delta = 0, qr = 0, kr = 0, total = 0;
};
ScoreWs score_ws(int B, int H, int Sq, int Skv, bool docs, bool bwd) {
  ScoreWs w;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = round_up(o + bytes, 256);
    return at;
  };
  if (bwd) {
    const size_t rows = static_cast<size_t>(B) * H * doc_blocks(Sq) * cp::kDocBlock;
    w.lse = take(rows * 4);
    w.delta = take(rows * 4);
  }
  if (docs) {
    w.qr = take(static_cast<size_t>(B) * doc_blocks(Sq) * sizeof(DocRange));
    w.kr = take(static_cast<size_t>(B) * doc_blocks(Skv) * sizeof(DocRange));
  }
  w.total = o;
  return w;
}

cp_status fill_args(ScoreArgs* a, const cp_score_rule& r, const void* q, const void* k, const void* v, int B, int H,
                    int Hkv, int Sq, int Skv, float scale, char* ws, const ScoreWs& w) {
  std::memset(a, 0, sizeof(*a));
  a->B = B;
  a->H = H;
  a->Hkv = Hkv;
  a->G = H / Hkv;
  a->Sq = Sq;
  a->Skv = Skv;
  a->scale = scale;
  a->cap = r.softcap;
  a->slopes = r.slopes;
  a->causal = r.causal != 0;
  a->rel = static_cast<int>(r.q_pos0 - r.kv_pos0);
  a->prefix = r.prefix_lens;
  a->kv_pos0 = static_cast<int>(r.kv_pos0);
  a->qdoc = r.q_docs;
  a->kdoc = r.kv_docs;
  a->q = q;
  a->k = k;
  a->v = v;
  if (r.q_docs) {
    a->qrange = reinterpret_cast<DocRange*>(ws + w.qr);
    a->krange = reinterpret_cast<DocRange*>(ws + w.kr);
  }
  a->timeout_ns = kWaitTimeoutNs;
  return static_cast<cp_status>(cp::host_device(&a->err, &a->sms));
}

}  // namespace

extern "C" {

cp_status cp_scored_attn_validate(int B, int H, int Hkv, int Sq, int Skv, int D, float scale,
                                  const cp_score_rule* rule, cp_dtype dt) {
  const cp_score_rule& r = rule ? *rule : kPlainRule;
  if (B < 0 || H < 1 || Hkv < 1 || Sq < 0 || Skv < 0 || (D != 64 && D != 128) || !known(dt)) return CP_ERR_INVALID_ARG;
  if (B > kMaxGrid || H > kMaxGrid || Sq > cp::kScoreMaxTokens || Skv > cp::kScoreMaxTokens) return CP_ERR_INVALID_ARG;
  if (!scores_ok(scale, r.softcap)) return CP_ERR_INVALID_ARG;
  if (r.q_pos0 < 0 || r.kv_pos0 < 0 || r.q_pos0 > kMaxPos || r.kv_pos0 > kMaxPos) return CP_ERR_INVALID_ARG;
  if ((r.q_docs == nullptr) != (r.kv_docs == nullptr)) return CP_ERR_INVALID_ARG;
  if (r.prefix_lens && !r.causal) return CP_ERR_UNSUPPORTED_COMBO;
  if (H % Hkv) return CP_ERR_NOT_DIVISIBLE;
  if (!aligned(r.slopes, 4) || !aligned(r.prefix_lens, 4) || !aligned(r.q_docs, 4) || !aligned(r.kv_docs, 4))
    return CP_ERR_ALIGNMENT;
  return CP_OK;
}

size_t cp_scored_attn_workspace_size(int B, int H, int Sq, int Skv, int docs) {
  if (B < 0 || H < 1 || Sq < 0 || Skv < 0) return 0;
  return score_ws(B, H, Sq, Skv, docs != 0, false).total;
}

size_t cp_scored_attn_bwd_workspace_size(int B, int H, int Sq, int Skv, int docs) {
  if (B < 0 || H < 1 || Sq < 0 || Skv < 0) return 0;
  return score_ws(B, H, Sq, Skv, docs != 0, true).total;
}

cp_status cp_scored_attn_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int B, int H, int Hkv,
                             int Sq, int Skv, int D, float scale, const cp_score_rule* rule, void* workspace,
                             size_t ws_bytes, cp_dtype dt, cp_dtype out_dt, void* stream) {
  const cp_score_rule& r = rule ? *rule : kPlainRule;
  cp_status st = cp_scored_attn_validate(B, H, Hkv, Sq, Skv, D, scale, rule, dt);
  if (st != CP_OK) return st;
  if (!out_type_ok(out_dt, dt)) return CP_ERR_INVALID_ARG;
  if (B == 0 || Sq == 0) return CP_OK;
  if (!q || !out || !lse || (Skv > 0 && (!k || !v))) return CP_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 16) || (Skv > 0 && (!aligned(k, 16) || !aligned(v, 16))))
    return CP_ERR_ALIGNMENT;
  const ScoreWs w = score_ws(B, H, Sq, Skv, r.q_docs != nullptr, false);
  if (w.total > 0 && (!workspace || ws_bytes < w.total)) return CP_ERR_WORKSPACE;
  if (w.total > 0 && !aligned(workspace, 256)) return CP_ERR_ALIGNMENT;
  ScoreArgs a;
  if ((st = fill_args(&a, r, q, k, v, B, H, Hkv, Sq, Skv, scale, static_cast<char*>(workspace), w)) != CP_OK) return st;
  a.out = out;
  a.out_bf16 = out_dt == CP_BF16;
  a.lse = lse;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.qdoc && cp::launch_doc_ranges(a, s) != cudaSuccess) return CP_ERR_CUDA;
  const cudaError_t e = dt == CP_BF16 ? cp::launch_score_fwd_tc(a, D, s) : cp::launch_score_fwd_f32(a, D, s);
  return e == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

cp_status cp_scored_attn_bwd(const void* q, const void* k, const void* v, const void* out, const void* dout,
                             const float* lse, void* dq, void* dk, void* dv, int B, int H, int Hkv, int Sq, int Skv,
                             int D, float scale, const cp_score_rule* rule, void* workspace, size_t ws_bytes,
                             cp_dtype dt, cp_dtype out_dt, cp_dtype grad_dt, void* stream) {
  const cp_score_rule& r = rule ? *rule : kPlainRule;
  cp_status st = cp_scored_attn_validate(B, H, Hkv, Sq, Skv, D, scale, rule, dt);
  if (st != CP_OK) return st;
  if (!out_type_ok(out_dt, dt) || !out_type_ok(grad_dt, dt)) return CP_ERR_INVALID_ARG;
  if (B == 0 || (Sq == 0 && Skv == 0)) return CP_OK;
  const void* qs[5] = {q, out, dout, lse, dq};
  if (Sq > 0)
    for (const void* p : qs) {
      if (!p) return CP_ERR_INVALID_ARG;
      if (!aligned(p, 16)) return CP_ERR_ALIGNMENT;
    }
  const void* ks[4] = {k, v, dk, dv};
  if (Skv > 0)
    for (const void* p : ks) {
      if (!p) return CP_ERR_INVALID_ARG;
      if (!aligned(p, 16)) return CP_ERR_ALIGNMENT;
    }
  const ScoreWs w = score_ws(B, H, Sq, Skv, r.q_docs != nullptr, true);
  if (w.total > 0 && (!workspace || ws_bytes < w.total)) return CP_ERR_WORKSPACE;
  if (w.total > 0 && !aligned(workspace, 256)) return CP_ERR_ALIGNMENT;
  char* ws = static_cast<char*>(workspace);
  ScoreArgs a;
  if ((st = fill_args(&a, r, q, k, v, B, H, Hkv, Sq, Skv, scale, ws, w)) != CP_OK) return st;
  a.o = out;
  a.out_bf16 = out_dt == CP_BF16;
  a.dout = dout;
  a.lse = const_cast<float*>(lse);
  a.delta = reinterpret_cast<float*>(ws + w.delta);
  a.lse2p = reinterpret_cast<float*>(ws + w.lse);
  a.dltp = a.delta;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.grad_bf16 = grad_dt == CP_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.qdoc && cp::launch_doc_ranges(a, s) != cudaSuccess) return CP_ERR_CUDA;
  const cudaError_t e = dt == CP_BF16 ? cp::launch_score_bwd_tc(a, D, s) : cp::launch_score_bwd_f32(a, D, s);
  return e == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// the paged cache
// ---------------------------------------------------------------------------
static cp_status check_paged(int B, int Hkv, int D, int num_pages, int page_size, int max_pages, cp_dtype dt,
                             int* shift) {
  if (B < 0 || Hkv < 1 || (D != 64 && D != 128) || num_pages < 1 || max_pages < 0 || !known(dt))
    return CP_ERR_INVALID_ARG;
  if (B > cp::kPagedMaxBatch || Hkv > kMaxGrid || page_size < 1 || page_size > 65536 || (page_size & (page_size - 1)))
    return CP_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_pages) * page_size > INT_MAX) return CP_ERR_INVALID_ARG;
  *shift = 0;
  while ((1 << *shift) < page_size) ++*shift;
  return CP_OK;
}

cp_status cp_paged_kv_append(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                             const int32_t* block_table, const int32_t* seq_lens, const int32_t* new_lens, int B, int T,
                             int Hkv, int D, int num_pages, int page_size, int max_pages, cp_dtype dt, void* stream) {
  PagedArgs a;
  std::memset(&a, 0, sizeof(a));
  cp_status st = check_paged(B, Hkv, D, num_pages, page_size, max_pages, dt, &a.page_shift);
  if (st != CP_OK) return st;
  if (T < 0 || static_cast<int64_t>(B) * T > INT_MAX) return CP_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return CP_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !block_table || !seq_lens) return CP_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(new_lens, 4))
    return CP_ERR_ALIGNMENT;
  a.B = B;
  a.T = T;
  a.Hkv = Hkv;
  a.D = D;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  const int64_t positions = static_cast<int64_t>(max_pages) * page_size;
  a.positions = static_cast<uint32_t>(positions < (int64_t{1} << 31) ? positions : int64_t{1} << 31);
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.k_new = k_new;
  a.v_new = v_new;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  if ((st = static_cast<cp_status>(cp::host_device(&a.err, &a.sms))) != CP_OK) return st;
  return cp::launch_paged_append(a, dt == CP_BF16 ? 2 : 4, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? CP_OK
             : CP_ERR_CUDA;
}

// Partials of the CTAs, then which of them make up each unit.
static size_t paged_partial_bytes(int G, int D, cp_dtype dt) {
  const int rows = cp::paged_rows(dt == CP_BF16);
  return round_up(static_cast<size_t>(cp::kPagedCtas) * 2 * (G < rows ? G : rows) * (D + 2) * 4, 256);
}

size_t cp_paged_attn_workspace_size(int B, int H, int Hkv, int D, cp_dtype dt) {
  if (B < 1 || H < 1 || Hkv < 1 || D < 1 || H % Hkv) return 0;
  const int rows = cp::paged_rows(dt == CP_BF16);
  const size_t groups = (H / Hkv + rows - 1) / rows;
  return paged_partial_bytes(H / Hkv, D, dt) + round_up(static_cast<size_t>(B) * Hkv * groups * sizeof(int2), 256);
}

size_t cp_paged_attn_workspace_size_for(int B, int H, int Hkv, int D, int page_size, int max_pages, cp_dtype dt) {
  if (page_size < 1 || page_size > 65536 || max_pages < 0) return 0;
  const size_t most = cp_paged_attn_workspace_size(B, H, Hkv, D, dt);
  int shift = 0;
  while ((2 << shift) <= page_size) ++shift;
  return most && cp::paged_cluster(D, dt == CP_BF16, B, Hkv, H / Hkv, max_pages, shift) > 0 ? 0 : most;
}

cp_status cp_paged_attn_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                               const int32_t* seq_lens, void* out, float* lse, int B, int H, int Hkv, int D,
                               int num_pages, int page_size, int max_pages, float scale, float softcap,
                               const float* slopes, void* workspace, size_t ws_bytes, cp_dtype dt, cp_dtype out_dt,
                               void* stream) {
  PagedArgs a;
  std::memset(&a, 0, sizeof(a));
  cp_status st = check_paged(B, Hkv, D, num_pages, page_size, max_pages, dt, &a.page_shift);
  if (st != CP_OK) return st;
  if (H < 1 || H > kMaxGrid || !out_type_ok(out_dt, dt)) return CP_ERR_INVALID_ARG;
  if (!scores_ok(scale, softcap)) return CP_ERR_INVALID_ARG;
  if (H % Hkv) return CP_ERR_NOT_DIVISIBLE;
  const int rows = cp::paged_rows(dt == CP_BF16), groups = (H / Hkv + rows - 1) / rows;
  // the list of 64-key blocks is indexed in 32 bits
  const int64_t blocks = (static_cast<int64_t>(max_pages) * page_size + cp::kPagedBlock - 1) / cp::kPagedBlock;
  if (static_cast<int64_t>(max_pages) * page_size > INT_MAX || blocks * Hkv * groups * (B > 0 ? B : 1) > INT_MAX / 2)
    return CP_ERR_INVALID_ARG;
  if (B == 0) return CP_OK;
  if (!q || !k_cache || !v_cache || (max_pages > 0 && !block_table) || !seq_lens || !out || !lse)
    return CP_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(slopes, 4))
    return CP_ERR_ALIGNMENT;
  const size_t need = cp_paged_attn_workspace_size_for(B, H, Hkv, D, page_size, max_pages, dt);
  if (need && (!workspace || ws_bytes < need)) return CP_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return CP_ERR_ALIGNMENT;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.D = D;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.k_cache = const_cast<void*>(k_cache);
  a.v_cache = const_cast<void*>(v_cache);
  a.q = q;
  a.out = out;
  a.out_bf16 = out_dt == CP_BF16;
  a.lse = lse;
  a.scale = scale;
  a.cap = softcap;
  a.slopes = slopes;
  if (need) {
    a.partial = static_cast<float*>(workspace);
    a.info = reinterpret_cast<int2*>(static_cast<char*>(workspace) + paged_partial_bytes(a.G, D, dt));
  }
  if ((st = static_cast<cp_status>(cp::host_device(&a.err, &a.sms))) != CP_OK) return st;
  return cp::launch_paged_decode(a, dt == CP_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CP_OK
                                                                                                       : CP_ERR_CUDA;
}

}  // extern "C"
