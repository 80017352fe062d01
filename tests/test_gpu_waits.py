"""Waits that run out in the kernels with rows on their way through shared memory: the norm with rotation, and decode from
the cache in 4 bits.

A barrier that awaits one arrival more than its copies bring is never done, so the wait ends by its limit (a few
milliseconds); the copies themselves land. The kernels return, cp_check_device_status reports the timeout, and the next
call is right. Launches go through the library's internal interface, whose arguments name the warps concerned.
"""
import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F4 = torch.bfloat16, torch.float32
TIMEOUT = -6   # CP_ERR_TIMEOUT
SHIM = r"""
#include <cstring>
#include "cp_rope.h"
#include "cp_score.h"
extern "C" int stalled_decode(void* const* p, int B, int H, int Hkv, int D, int pages, int page_shift, int max_pages, int bf16,
                              long partial_bytes, unsigned warps, long limit_us) {
  cp::PagedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.B = B, a.H = H, a.Hkv = Hkv, a.G = H / Hkv, a.D = D;
  a.num_pages = pages, a.page_shift = page_shift, a.max_pages = max_pages;
  a.q = p[0], a.k_cache = p[1], a.k_scales = p[2], a.v_cache = p[3], a.v_scales = p[4];
  a.table = static_cast<const int*>(p[5]), a.seq_lens = static_cast<const int*>(p[6]);
  a.out = p[7], a.lse = static_cast<float*>(p[8]), a.scale = 0.1f, a.out_bf16 = bf16;
  a.partial = static_cast<float*>(p[9]), a.info = reinterpret_cast<int2*>(static_cast<char*>(p[9]) + partial_bytes);
  a.timeout_ns = limit_us * 1000, a.stall = warps;
  cp::divide_by(Hkv, &a.hkv_mul, &a.hkv_shift);
  const int st = cp::host_device(&a.err, &a.sms);
  return st ? st : static_cast<int>(cp::launch_q4_decode(a, bf16, nullptr));
}
extern "C" int stalled_rope(void* const* p, int tokens, int H, int Hkv, int D, int bf16, int backward, unsigned warps, long limit_us) {
  cp::RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.S = a.tokens = tokens, a.H = H, a.Hkv = Hkv, a.norm = 1, a.eps = 1e-6f, a.axes = 1;
  cp::RopeRows* rows[6] = {&a.q, &a.k, &a.qo, &a.ko, &a.dq, &a.dk};
  for (int i = 0; i < 6; ++i) *rows[i] = {p[i], 0, static_cast<int64_t>(i & 1 ? Hkv : H) * D, D};
  a.partial = static_cast<float*>(p[6]), a.dwq = static_cast<float*>(p[7]), a.dwk = static_cast<float*>(p[8]);
  a.timeout_ns = limit_us * 1000, a.stall = warps;
  int sms;
  const int st = cp::host_device(&a.err, &sms);
  if (st) return st;
  return static_cast<int>(backward ? cp::launch_rope_bwd(a, D, bf16, !bf16, true, sms, nullptr)
                                   : cp::launch_rope_fwd(a, D, bf16, true, sms, nullptr));
}
"""


def cpa():
    import context_attention_dits_gb300 as m
    return m


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from context_attention_dits_gb300 import build
    build.build()
    cpa().lib()
    at = tmp_path_factory.mktemp("shim")
    (at / "shim.cu").write_text(SHIM)
    subprocess.run([build.nvcc_path(), *build.ARCH, "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", build.CSRC, "-I",
                    build.INCLUDE, "-o", str(at / "libshim.so"), str(at / "shim.cu"), build.LIB, "-Xlinker", "-rpath",
                    "-Xlinker", build.LIBDIR], check=True)
    return ctypes.CDLL(str(at / "libshim.so"))


def pointers(tensors):
    return (ctypes.c_void_p * len(tensors))(*(t.data_ptr() for t in tensors))


# tables that clusters take (of 1, 4 and 16 CTAs), and two of the list, in which a warp has one sequence's part and many
@pytest.mark.parametrize("lens,most,G,D,dt", [
    ([100], 128, 4, 64, BF), ([1000, 0, 77], 1024, 3, 128, BF), ([4000], 4096, 2, 64, F4),
    ([200000], 1 << 18, 8, 128, BF), ([70] * 2000 + [0, 3000], 1 << 13, 12, 64, BF), ([100000, 500], 1 << 17, 2, 128, F4),
])
@pytest.mark.parametrize("warps", [2, 15])
def test_decode_waits_run_out(shim, lens, most, G, D, dt, warps):
    Hkv, page = 2, 64
    B, H, g = len(lens), Hkv * G, torch.Generator(device="cuda").manual_seed(1)
    pages = 64
    q = torch.randn((B, H, D), generator=g, device="cuda").to(dt)
    cache = []
    for _ in range(2):
        cache.append(torch.randint(0, 256, (pages, Hkv, page, D // 2), generator=g, device="cuda", dtype=torch.uint8))
        cache.append(torch.rand((pages, Hkv, page, D // 64, 2), generator=g, device="cuda").to(BF))
    table = torch.randint(0, pages, (B, most // page), generator=g, device="cuda", dtype=torch.int32)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    size = cpa().cp_paged_attn_q4_workspace_size(B, H, Hkv, D, page, most // page, dt)
    assert (size > 0) == (most > 4096)
    units = -(-B * Hkv * -(-G // (16 if dt == BF and G > 8 else 8)) * 8 // 256) * 256
    ws = torch.full((max(size, 256),), 255, dtype=torch.uint8, device="cuda")

    def call():
        out, lse = torch.empty_like(q), torch.empty((B, H), device="cuda")
        cpa().cp_paged_attn_decode_q4(q, *cache, table, n, out, lse, 0.1, workspace=ws)
        assert cpa().cp_check_device_status() == 0
        return out, lse

    want = call()
    out, lse = torch.empty_like(q), torch.empty((B, H), device="cuda")
    p = pointers([q, *cache, table, n, out, lse, ws])
    torch.cuda.synchronize()
    assert shim.stalled_decode(p, B, H, Hkv, D, pages, 6, most // page, int(dt == BF), ctypes.c_long(max(size - units, 0)), warps,
                               ctypes.c_long(2000)) == 0
    torch.cuda.synchronize()
    assert cpa().cp_check_device_status() == TIMEOUT and cpa().cp_check_device_status() == 0
    got = call()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("D,dt,warps", [(64, BF, 255), (128, BF, 2), (128, F4, 96)])
@pytest.mark.parametrize("backward", [False, True])
def test_rows_waits_run_out(shim, D, dt, warps, backward):
    tokens, H, Hkv, g = 3000, 20, 3, torch.Generator(device="cuda").manual_seed(2)
    q, k, gq, gk = (torch.randn((1, tokens, h, D), generator=g, device="cuda").to(dt) for h in (H, Hkv, H, Hkv))
    ws = torch.empty(cpa().cp_qk_norm_rope_bwd_workspace_size(D), dtype=torch.uint8, device="cuda")

    def call():
        a, b, w = torch.empty_like(q), torch.empty_like(k), torch.empty((2, D), device="cuda")
        if backward:
            cpa().cp_qk_norm_rope_bwd(q, k, gq, gk, a, b, eps=1e-6, dq_weight=w[0], dk_weight=w[1], workspace=ws)
        else:
            w.zero_()
            cpa().cp_qk_norm_rope_fwd(q, k, a, b, eps=1e-6)
        assert cpa().cp_check_device_status() == 0
        return a, b, w

    want = call()
    a, b, w = torch.empty_like(q), torch.empty_like(k), torch.empty((2, D), device="cuda")
    p = pointers([q, k, gq, gk, a, b, ws, w[0], w[1]] if backward else [q, k, a, b, a, b, ws, w[0], w[1]])
    torch.cuda.synchronize()
    assert shim.stalled_rope(p, tokens, H, Hkv, D, int(dt == BF), int(backward), warps, ctypes.c_long(2000)) == 0
    torch.cuda.synchronize()
    assert cpa().cp_check_device_status() == TIMEOUT and cpa().cp_check_device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(call(), want))
