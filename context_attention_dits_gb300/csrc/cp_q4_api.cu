// cp_q4_api.cu — the C ABI of the paged cache in 4 bits (declared in
// include/cp_attn.h): argument checks, workspace and launches.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "cp_attn.h"
#include "cp_score.h"

namespace {

using cp::PagedArgs;

constexpr uint64_t kWaitTimeoutNs = 1000000000ull;  // 1 s per device-side wait
constexpr int kMaxGrid = 65535;                     // heads

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Sizes and the cache's arrays, shared by the three calls.
cp_status take_cache(PagedArgs* a, const cp_q4_cache* c, int B, int Hkv, int D, cp_dtype dt, bool used) {
  std::memset(a, 0, sizeof(*a));
  if (!c || B < 0 || B > cp::kPagedMaxBatch || Hkv < 1 || Hkv > kMaxGrid || (D != 64 && D != 128)) return CP_ERR_INVALID_ARG;
  if (dt != CP_BF16 && dt != CP_F32) return CP_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->max_pages < 0 || c->page_size < cp::kQ4MinPage || c->page_size > 65536 ||
      (c->page_size & (c->page_size - 1)))
    return CP_ERR_INVALID_ARG;
  if (static_cast<int64_t>(c->num_pages) * c->page_size > INT_MAX) return CP_ERR_INVALID_ARG;
  while ((1 << a->page_shift) < c->page_size) ++a->page_shift;
  if (used) {
    const void* arrays[4] = {c->k_codes, c->k_scales, c->v_codes, c->v_scales};
    for (const void* p : arrays) {
      if (!p) return CP_ERR_INVALID_ARG;
      if (!aligned(p, 16)) return CP_ERR_ALIGNMENT;
    }
    if (c->max_pages > 0 && !c->block_table) return CP_ERR_INVALID_ARG;
    if (!aligned(c->block_table, 4)) return CP_ERR_ALIGNMENT;
  }
  a->B = B;
  a->Hkv = Hkv;
  a->D = D;
  a->num_pages = c->num_pages;
  a->max_pages = c->max_pages;
  const int64_t positions = static_cast<int64_t>(c->max_pages) * c->page_size;
  a->positions = static_cast<uint32_t>(positions < (int64_t{1} << 31) ? positions : int64_t{1} << 31);
  a->table = c->block_table;
  a->k_cache = c->k_codes;
  a->k_scales = c->k_scales;
  a->v_cache = c->v_codes;
  a->v_scales = c->v_scales;
  a->timeout_ns = kWaitTimeoutNs;
  cp::divide_by(Hkv, &a->hkv_mul, &a->hkv_shift);
  return CP_OK;
}

cp_status ran(cudaError_t e) { return e == cudaSuccess ? CP_OK : CP_ERR_CUDA; }

size_t partial_bytes(int G, int D, cp_dtype dt) {
  const int rows = cp::q4_rows(dt == CP_BF16, G);
  const int workers = 4 * 152 * cp::q4_per_sm(dt == CP_BF16, rows, cp::q4_chunk(dt == CP_BF16, rows));
  return round_up(static_cast<size_t>(workers) * 2 * (G < rows ? G : rows) * (D + 2) * 4, 256);
}

}  // namespace

extern "C" {

cp_status cp_paged_kv_append_q4(const void* k_new, const void* v_new, const cp_q4_cache* cache, const int32_t* seq_lens,
                                const int32_t* new_lens, int B, int T, int Hkv, int D, cp_dtype dt, void* stream) {
  PagedArgs a;
  cp_status st = take_cache(&a, cache, B, Hkv, D, dt, B > 0 && T > 0);
  if (st != CP_OK) return st;
  if (T < 0 || static_cast<int64_t>(B) * T > INT_MAX || static_cast<int64_t>(T) * Hkv > INT_MAX - 65536)
    return CP_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return CP_OK;
  if (!k_new || !v_new || !seq_lens) return CP_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(seq_lens, 4) || !aligned(new_lens, 4)) return CP_ERR_ALIGNMENT;
  a.T = T;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.k_new = k_new;
  a.v_new = v_new;
  if ((st = static_cast<cp_status>(cp::host_device(&a.err, &a.sms))) != CP_OK) return st;
  return ran(cp::launch_q4_append(a, dt == CP_BF16, static_cast<cudaStream_t>(stream)));
}

cp_status cp_paged_kv_read_q4(const cp_q4_cache* cache, const int32_t* seq_lens, void* k_out, void* v_out, int B, int T,
                              int Hkv, int D, cp_dtype out_dt, void* stream) {
  PagedArgs a;
  cp_status st = take_cache(&a, cache, B, Hkv, D, out_dt, B > 0 && T > 0);
  if (st != CP_OK) return st;
  if (T < 0 || static_cast<int64_t>(B) * T > INT_MAX || static_cast<int64_t>(T) * Hkv > INT_MAX - 65536)
    return CP_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return CP_OK;
  if (!k_out || !v_out || !seq_lens) return CP_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(seq_lens, 4)) return CP_ERR_ALIGNMENT;
  a.T = T;
  a.seq_lens = seq_lens;
  a.k_out = k_out;
  a.v_out = v_out;
  if ((st = static_cast<cp_status>(cp::host_device(&a.err, &a.sms))) != CP_OK) return st;
  return ran(cp::launch_q4_read(a, out_dt == CP_BF16, static_cast<cudaStream_t>(stream)));
}

size_t cp_paged_attn_q4_workspace_size(int B, int H, int Hkv, int D, int page_size, int max_pages, cp_dtype dt) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || D < 1 || page_size < cp::kQ4MinPage || page_size > 65536 || max_pages < 0) return 0;
  const int G = H / Hkv, rows = cp::q4_rows(dt == CP_BF16, G);
  int shift = 0;
  while ((2 << shift) <= page_size) ++shift;
  if (cp::q4_cluster(dt == CP_BF16, B, Hkv, G, max_pages, shift) > 0) return 0;
  const size_t units = static_cast<size_t>(B) * Hkv * ((G + rows - 1) / rows);
  return partial_bytes(G, D, dt) + round_up(units * sizeof(int2), 256);
}

cp_status cp_paged_attn_decode_q4(const void* q, const cp_q4_cache* cache, const int32_t* seq_lens, void* out, float* lse,
                                  int B, int H, int Hkv, int D, float scale, float softcap, const float* slopes,
                                  void* workspace, size_t ws_bytes, cp_dtype dt, cp_dtype out_dt, void* stream) {
  PagedArgs a;
  cp_status st = take_cache(&a, cache, B, Hkv, D, dt, B > 0);
  if (st != CP_OK) return st;
  if (H < 1 || H > kMaxGrid || (out_dt != dt && out_dt != CP_F32)) return CP_ERR_INVALID_ARG;
  if (!(std::fabs(scale) <= 1e30f) || !(softcap >= 0.f && softcap <= 1e30f) ||
      (softcap > 0.f && (softcap < 1e-30f || softcap < std::fabs(scale) * 1e-30f)))
    return CP_ERR_INVALID_ARG;
  if (H % Hkv) return CP_ERR_NOT_DIVISIBLE;
  const int G = H / Hkv, rows = cp::q4_rows(dt == CP_BF16, G), groups = (G + rows - 1) / rows;
  // the list of blocks is indexed in 32 bits
  const int64_t keys = static_cast<int64_t>(cache->max_pages) * cache->page_size;
  const int block = cp::q4_chunk(dt == CP_BF16, rows);
  const int64_t blocks = (keys + block - 1) / block;
  if (keys > INT_MAX || blocks * Hkv * groups * (B > 0 ? B : 1) > INT_MAX / 2) return CP_ERR_INVALID_ARG;
  if (B == 0) return CP_OK;
  if (!q || !seq_lens || !out || !lse) return CP_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(seq_lens, 4) || !aligned(slopes, 4))
    return CP_ERR_ALIGNMENT;
  const size_t need = cp_paged_attn_q4_workspace_size(B, H, Hkv, D, cache->page_size, cache->max_pages, dt);
  if (need && (!workspace || ws_bytes < need)) return CP_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return CP_ERR_ALIGNMENT;
  a.H = H;
  a.G = G;
  a.seq_lens = seq_lens;
  a.q = q;
  a.out = out;
  a.out_bf16 = out_dt == CP_BF16;
  a.lse = lse;
  a.scale = scale;
  a.cap = softcap;
  a.slopes = slopes;
  if (need) {
    a.partial = static_cast<float*>(workspace);
    a.info = reinterpret_cast<int2*>(static_cast<char*>(workspace) + partial_bytes(G, D, dt));
  }
  if ((st = static_cast<cp_status>(cp::host_device(&a.err, &a.sms))) != CP_OK) return st;
  return ran(cp::launch_q4_decode(a, dt == CP_BF16, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
