// cp_rope.h — launch parameters of the head norm with rotary positions, shared
// by its kernels and entry points. Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace cp {

constexpr int kRopeMaxPairs = 64;  // D / 2 at most
constexpr int kRopeMaxAxes = 4;
constexpr int kRopeWarps = 8;      // of a CTA
// CTAs of a launch at most: the backward leaves a partial of the weights' gradients each.
constexpr int kRopeCtas = 152 * 4;

// Rows of heads: element (b, s, h, d) at b * sb + s * ss + h * sh + d.
struct RopeRows {
  void* p;
  int64_t sb, ss, sh;
};

struct RopeArgs {
  int S, H, Hkv;    // Hkv = 0: no keys
  int tokens;       // B * S
  int parts, parts_q;  // each token's heads are cut into parts, the first parts_q of q
  RopeRows q, k;    // the rows before
  RopeRows qo, ko;  // forward: the rows after; backward: their gradients
  RopeRows dq, dk;  // backward: the gradients of q and k
  const void *wq, *wk;  // [D], or nullptr
  int w_f32;            // type of the weights: float32, or that of the rows
  int norm;
  float eps;
  const double* freqs;  // [pairs]
  int pairs;
  const int* pos;  // [B, S, axes], or [S, axes] with pos_sb = 0
  int64_t pos_sb;
  int axes;
  float* partial;  // backward: [CTAs][D], or nullptr
  float *dwq, *dwk;
  uint32_t* err;        // device error word, and the bound on each wait
  uint64_t timeout_ns;
  uint32_t stall;       // 0; in tests, warps of each CTA (a bit each) whose copies never count as done
  uint8_t axis[kRopeMaxPairs];  // of each pair
};

cudaError_t launch_rope_fwd(RopeArgs& a, int D, bool bf16, bool interleaved, int sms, cudaStream_t s);
// g_f32: the gradients qo, ko are float32 (else of the rows' type).
cudaError_t launch_rope_bwd(RopeArgs& a, int D, bool bf16, bool g_f32, bool interleaved, int sms, cudaStream_t s);

}  // namespace cp
