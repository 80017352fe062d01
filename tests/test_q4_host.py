"""Refusals and sizes of the calls on a cache in 4 bits: every call here fails its
checks on the host or has nothing to do, and none reaches a GPU."""
import ctypes
import os
import subprocess

import pytest
import torch

import context_attention_dits_gb300 as cpa
from context_attention_dits_gb300 import _lib, build

P = 1 << 20  # an aligned "device" address that is never dereferenced
BAD, ALIGN, WS, DIV = (_lib.CP_ERR_INVALID_ARG, _lib.CP_ERR_ALIGNMENT, _lib.CP_ERR_WORKSPACE, _lib.CP_ERR_NOT_DIVISIBLE)


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    build.build()


def cache(**kw):
    kw = {**dict(k_codes=P, k_scales=P, v_codes=P, v_scales=P, block_table=P, num_pages=9, page_size=16, max_pages=4), **kw}
    return ctypes.byref(_lib.Q4Cache(**kw))


def append(k=P, v=P, c=None, lens=P, new=None, B=2, T=3, Hkv=2, D=64, dt=0):
    return _lib.lib().cp_paged_kv_append_q4(k, v, c or cache(), lens, new, B, T, Hkv, D, dt, None)


def read(c=None, lens=P, k=P, v=P, B=2, T=3, Hkv=2, D=64, dt=0):
    return _lib.lib().cp_paged_kv_read_q4(c or cache(), lens, k, v, B, T, Hkv, D, dt, None)


def decode(q=P, c=None, lens=P, o=P, l=P, B=2, H=4, Hkv=2, D=64, scale=0.1, cap=0.0, slopes=None, ws=P, n=1 << 30, dt=0, odt=0):
    return _lib.lib().cp_paged_attn_decode_q4(q, c or cache(), lens, o, l, B, H, Hkv, D, scale, cap, slopes, ws, n, dt, odt,
                                              None)


@pytest.mark.parametrize("call", [append, read, decode])
def test_sizes_and_cache(call):
    for bad in (dict(D=96), dict(B=-1), dict(B=4097), dict(Hkv=0), dict(Hkv=65536), dict(dt=2)):
        assert call(**bad) == BAD, bad
    for bad in (dict(page_size=8), dict(page_size=0), dict(page_size=48), dict(page_size=131072), dict(num_pages=0),
                dict(max_pages=-1), dict(num_pages=1 << 20, page_size=4096), dict(k_codes=0), dict(k_scales=0),
                dict(v_codes=0), dict(v_scales=0), dict(block_table=0)):
        assert call(c=cache(**bad)) == BAD, bad
    for bad in (dict(k_codes=P + 8), dict(k_scales=P + 4), dict(v_codes=P + 1), dict(v_scales=P + 2), dict(block_table=P + 2)):
        assert call(c=cache(**bad)) == ALIGN, bad
    assert call(B=0) == 0 and call(B=0, c=cache(k_codes=0, block_table=0)) == 0
    assert call(lens=0) == BAD and call(lens=P + 2) == ALIGN


def test_append_and_read_tensors():
    for call in (append, read):
        assert call(k=0) == BAD and call(v=0) == BAD and call(k=P + 8) == ALIGN and call(v=P + 4) == ALIGN
        assert call(T=-1) == BAD and call(T=0) == 0 and call(B=4096, T=1 << 20) == BAD
        assert call(B=1, T=1 << 20, Hkv=2048) == BAD
    assert append(new=P + 1) == ALIGN
    assert _lib.lib().cp_paged_kv_append_q4(P, P, None, P, None, 1, 1, 1, 64, 0, None) == BAD


def test_decode_tensors_and_workspace():
    assert decode(q=0) == BAD and decode(o=0) == BAD and decode(l=0) == BAD
    assert decode(q=P + 8) == ALIGN and decode(o=P + 8) == ALIGN and decode(l=P + 2) == ALIGN and decode(slopes=P + 1) == ALIGN
    assert decode(H=0) == BAD and decode(H=65536) == BAD and decode(H=5) == DIV
    assert decode(dt=1, odt=0) == BAD and decode(odt=3) == BAD
    for bad in (dict(scale=float("nan")), dict(scale=1e31), dict(cap=-1.0), dict(cap=1e-31), dict(cap=float("nan")),
                dict(scale=1e25, cap=1e-6)):
        assert decode(**bad) == BAD, bad
    wide = cache(max_pages=4096)
    need = cpa.cp_paged_attn_q4_workspace_size(2, 4, 2, 64, 16, 4096)
    assert need > 0 and decode(c=wide, ws=0) == WS and decode(c=wide, n=need - 1) == WS
    assert decode(c=wide, ws=P + 16) == ALIGN
    assert decode(c=cache(max_pages=1 << 28)) == BAD                     # more positions than 31 bits
    size = cpa.cp_paged_attn_q4_workspace_size
    assert size(2, 4, 2, 64, 16, 4) == 0                                 # one launch
    assert size(0, 4, 2, 64, 16, 4096) == 0 and size(2, 5, 2, 64, 16, 4096) == 0 and size(2, 4, 2, 64, 8, 4096) == 0
    assert size(2, 4, 2, 64, 16, 4096, torch.float32) > 0


def test_wrapper_refuses_host_tensors():
    k = torch.zeros(1, 3, 2, 64)
    codes, scales = torch.zeros(4, 2, 16, 32, dtype=torch.uint8), torch.zeros(4, 2, 16, 1, 2, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    c = (codes, scales, codes, scales, table)
    for f in (lambda: cpa.cp_paged_kv_append_q4(k, k, *c, lens), lambda: cpa.cp_paged_kv_read_q4(*c, lens, k, k),
              lambda: cpa.cp_paged_attn_decode_q4(k[:, 0], *c, lens, k[:, 0], k[:, 0, :, 0], 0.1)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        cpa.cp_paged_kv_append_q4([1], k, *c, lens)


PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "cp_score.h"
int main(int argc, char** argv) {
  const int sms = std::atoi(argv[1]);
  for (int smem = 1 << 14; smem < 228 << 10; smem *= 2)
    for (int rows = 8; rows <= 16; rows *= 2)
      std::printf("%d ", cp::q4_ctas(true, rows, smem, sms));
  for (int bf16 = 0; bf16 < 2; ++bf16)
    for (int B = 1; B <= 512; B *= 2)
      for (int G = 1; G <= 32; G *= 2)
        for (int pages = 0; pages <= 1 << 17; pages = pages ? pages * 2 : 1) {
          const int rows = cp::q4_rows(bf16, G), cs = cp::q4_cluster(bf16, B, 8, G, pages, 4);
          const long long blocks = (16ll * pages + 127) / 128, units = 8ll * B * ((G + rows - 1) / rows);
          // powers of two up to 16, all at once on the device, a few blocks each
          if (cs < 0 || cs > 16 || (cs & (cs - 1)) || (cs && (units * cs > 608 || blocks > 8ll * cs))) return 1;
        }
  for (int d = 1; d <= 65535; d += d < 300 ? 1 : 331) {
    uint32_t mul;
    int shift;
    cp::divide_by(d, &mul, &shift);
    for (long long n : {0ll, 1ll, d - 1ll, 1ll * d, 12345ll * d - 1, (0x7fffffffll / d) * d - 1, (0x7fffffffll / d) * d, 0x7fffffffll})
      if (n >= 0 && n <= 0x7fffffffll && static_cast<long long>((static_cast<unsigned long long>(n) * mul) >> (32 + shift)) != n / d) return 2;
  }
  return 0;
}
"""


def test_launch_rules(tmp_path):
    (tmp_path / "rules.cu").write_text(PROGRAM)
    exe = str(tmp_path / "rules")
    subprocess.run([build.nvcc_path(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-o", exe,
                    os.path.join(tmp_path, "rules.cu")], check=True)
    for sms in (152, 76, 160, 2):
        got = subprocess.run([exe, str(sms)], check=True, capture_output=True, text=True).stdout.split()
        # whole multiples of the multiprocessors, no more than the workspace's partials are laid out for, one at least
        assert all(int(x) % min(sms, 152) == 0 and min(sms, 152) <= int(x) <= 608 for x in got)
