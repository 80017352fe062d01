// cp_rope_api.cu — the C ABI of the head norm with rotary positions (declared
// in include/cp_attn.h): argument checks, workspace and launches.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <utility>

#include "cp_attn.h"
#include "cp_rope.h"
#include "cp_score.h"

namespace {

using cp::RopeArgs;
using cp::RopeRows;

constexpr uint64_t kWaitTimeoutNs = 1000000000ull;  // 1 s per device-side wait

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// One tensor's address and strides (batch, token, head; dense without them). Sizes
// of 1 need no stride; others are whole 16-byte pieces, and rows that are written
// lie apart.
cp_status take_rows(RopeRows* r, const void* p, const int64_t* strides, int B, int S, int H, int D, int elem,
                    bool written) {
  r->p = const_cast<void*>(p);
  int64_t st[3] = {static_cast<int64_t>(S) * H * D, static_cast<int64_t>(H) * D, D};
  const int n[3] = {B, S, H};
  if (strides)
    for (int i = 0; i < 3; ++i) st[i] = n[i] > 1 ? strides[i] : 0;
  for (int i = 0; i < 3; ++i)
    if (st[i] < 0 || st[i] > (int64_t{1} << 40)) return CP_ERR_INVALID_ARG;
  r->sb = st[0];
  r->ss = st[1];
  r->sh = st[2];
  if (!p) return CP_ERR_INVALID_ARG;
  if (!aligned(p, 16)) return CP_ERR_ALIGNMENT;
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && st[i] * elem % 16) return CP_ERR_ALIGNMENT;
  if (written) {  // from the narrowest stride on, each steps over all that lies within
    int at[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (st[at[j]] > st[at[j + 1]]) std::swap(at[j], at[j + 1]);
    int64_t extent = D;
    for (int i : at) {
      if (n[i] <= 1) continue;
      if (st[i] < extent) return CP_ERR_INVALID_ARG;
      extent += st[i] * (n[i] - 1);
    }
  }
  return CP_OK;
}

cp_status take_rule(RopeArgs* a, const cp_qk_rule* r, int B, int S, int H, int Hkv, int D, cp_dtype dt) {
  std::memset(a, 0, sizeof(*a));
  if (!r || B < 0 || S < 0 || H < 1 || Hkv < 0 || (D != 64 && D != 128) || (dt != CP_BF16 && dt != CP_F32))
    return CP_ERR_INVALID_ARG;
  if (H > 65535 || Hkv > 65535 || static_cast<int64_t>(B) * S > INT_MAX / 64) return CP_ERR_INVALID_ARG;
  if (r->norm && !(r->eps >= 0.f && r->eps <= 1e30f)) return CP_ERR_INVALID_ARG;
  if ((r->q_weight || r->k_weight) && (!r->norm || (r->weight_dt != dt && r->weight_dt != CP_F32)))
    return CP_ERR_INVALID_ARG;
  if (r->pairs < 0 || r->pairs > D / 2 || r->pairs % 4) return CP_ERR_INVALID_ARG;
  if (r->pairs && (r->axes < 1 || r->axes > cp::kRopeMaxAxes)) return CP_ERR_INVALID_ARG;
  if (r->pairs && r->pair_axis)
    for (int i = 0; i < r->pairs; ++i) {
      if (r->pair_axis[i] >= r->axes) return CP_ERR_INVALID_ARG;
      a->axis[i] = r->pair_axis[i];
    }
  if (!aligned(r->freqs, 8) || !aligned(r->positions, 4) || !aligned(r->q_weight, 2) || !aligned(r->k_weight, 2) ||
      (r->weight_dt == CP_F32 && (!aligned(r->q_weight, 4) || !aligned(r->k_weight, 4))))
    return CP_ERR_ALIGNMENT;
  a->timeout_ns = kWaitTimeoutNs;
  a->S = S;
  a->H = H;
  a->Hkv = Hkv;
  a->tokens = B * S;
  a->norm = r->norm != 0;
  a->eps = r->eps;
  a->wq = r->q_weight;
  a->wk = r->k_weight;
  a->w_f32 = r->weight_dt == CP_F32;
  a->pairs = r->pairs;
  a->freqs = r->freqs;
  a->pos = r->positions;
  a->axes = r->axes;
  a->pos_sb = r->positions_shared ? 0 : static_cast<int64_t>(S) * r->axes;
  return CP_OK;
}

// What a call that has tokens needs of the rule's tensors.
bool rule_there(const RopeArgs& a) { return !a.pairs || (a.freqs && a.pos); }

}  // namespace

extern "C" {

cp_status cp_qk_norm_rope_fwd(const void* q, const void* k, void* q_out, void* k_out, const int64_t* strides, int B,
                              int S, int H, int Hkv, int D, const cp_qk_rule* rule, cp_dtype dt, void* stream) {
  RopeArgs a;
  cp_status st = take_rule(&a, rule, B, S, H, Hkv, D, dt);
  if (st != CP_OK) return st;
  if (a.tokens == 0) return CP_OK;
  if (!rule_there(a)) return CP_ERR_INVALID_ARG;
  const int e = dt == CP_BF16 ? 2 : 4;
  auto at = [&](int i) { return strides ? strides + 3 * i : nullptr; };
  if ((st = take_rows(&a.q, q, at(0), B, S, H, D, e, false)) != CP_OK) return st;
  if ((st = take_rows(&a.qo, q_out, at(2), B, S, H, D, e, true)) != CP_OK) return st;
  if (Hkv > 0) {
    if ((st = take_rows(&a.k, k, at(1), B, S, Hkv, D, e, false)) != CP_OK) return st;
    if ((st = take_rows(&a.ko, k_out, at(3), B, S, Hkv, D, e, true)) != CP_OK) return st;
  }
  int sms;
  if ((st = static_cast<cp_status>(cp::host_device(&a.err, &sms))) != CP_OK) return st;
  return cp::launch_rope_fwd(a, D, dt == CP_BF16, rule->interleaved != 0, sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? CP_OK
             : CP_ERR_CUDA;
}

size_t cp_qk_norm_rope_bwd_workspace_size(int D) {
  return D == 64 || D == 128 ? static_cast<size_t>(cp::kRopeCtas) * D * sizeof(float) : 0;
}

cp_status cp_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out, void* dq, void* dk,
                              float* dq_weight, float* dk_weight, const int64_t* strides, int B, int S, int H, int Hkv,
                              int D, const cp_qk_rule* rule, void* workspace, size_t ws_bytes, cp_dtype dt,
                              cp_dtype grad_dt, void* stream) {
  RopeArgs a;
  cp_status st = take_rule(&a, rule, B, S, H, Hkv, D, dt);
  if (st != CP_OK) return st;
  if (grad_dt != dt && grad_dt != CP_F32) return CP_ERR_INVALID_ARG;
  const bool weights = dq_weight || dk_weight;
  if ((weights && !a.norm) || (dk_weight && Hkv == 0)) return CP_ERR_INVALID_ARG;
  if (a.tokens == 0 && !weights) return CP_OK;
  if (a.tokens > 0) {
    if (!rule_there(a)) return CP_ERR_INVALID_ARG;
    const int e = dt == CP_BF16 ? 2 : 4, ge = grad_dt == CP_BF16 ? 2 : 4;
    auto at = [&](int i) { return strides ? strides + 3 * i : nullptr; };
    // without a norm the rows themselves are not read
    if (a.norm && (st = take_rows(&a.q, q, at(0), B, S, H, D, e, false)) != CP_OK) return st;
    if ((st = take_rows(&a.qo, dq_out, at(2), B, S, H, D, ge, false)) != CP_OK) return st;
    if ((st = take_rows(&a.dq, dq, at(4), B, S, H, D, e, true)) != CP_OK) return st;
    if (Hkv > 0) {
      if (a.norm && (st = take_rows(&a.k, k, at(1), B, S, Hkv, D, e, false)) != CP_OK) return st;
      if ((st = take_rows(&a.ko, dk_out, at(3), B, S, Hkv, D, ge, false)) != CP_OK) return st;
      if ((st = take_rows(&a.dk, dk, at(5), B, S, Hkv, D, e, true)) != CP_OK) return st;
    }
  }
  if (weights) {
    if (!workspace || ws_bytes < cp_qk_norm_rope_bwd_workspace_size(D)) return CP_ERR_WORKSPACE;
    if (!aligned(workspace, 256) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return CP_ERR_ALIGNMENT;
    a.partial = static_cast<float*>(workspace);
    a.dwq = dq_weight;
    a.dwk = dk_weight;
  }
  int sms;
  if ((st = static_cast<cp_status>(cp::host_device(&a.err, &sms))) != CP_OK) return st;
  return cp::launch_rope_bwd(a, D, dt == CP_BF16, grad_dt == CP_F32, rule->interleaved != 0, sms,
                             static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? CP_OK
             : CP_ERR_CUDA;
}

}  // extern "C"
