"""Refusals and sizes of the score-rule and paged-cache calls: every call here
fails its checks on the host or has nothing to do, and none reaches a GPU."""
import ctypes

import pytest
import torch

import context_attention_dits_gb300 as cpa
from context_attention_dits_gb300 import _lib

P = 1 << 20  # an aligned "device" address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    from context_attention_dits_gb300 import build
    build.build()


def rule(**kw):
    return ctypes.byref(_lib.ScoreRule(**kw))


def test_validate():
    ok = dict(B=2, H=8, Hkv=2, Sq=5, Skv=7, D=64)
    f = lambda **kw: cpa.cp_scored_attn_validate(**{**ok, **kw})
    assert f() == 0 and f(Sq=0, Skv=0, B=0) == 0 and f(softcap=30.0, causal=True, prefix=True, dtype=torch.float32) == 0
    for bad in (dict(D=96), dict(B=-1), dict(H=0), dict(Hkv=0), dict(Sq=-1), dict(Skv=-1), dict(B=65536), dict(H=65536),
                dict(Sq=(1 << 21) + 1), dict(Skv=(1 << 21) + 1), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=1e-31), dict(scale=1e25, softcap=1e-6), dict(q_pos0=-1), dict(kv_pos0=(1 << 30) + 1)):
        assert f(**bad) == _lib.CP_ERR_INVALID_ARG, bad
    assert f(H=7) == _lib.CP_ERR_NOT_DIVISIBLE
    assert f(prefix=True) == _lib.CP_ERR_UNSUPPORTED_COMBO
    L = _lib.lib()
    v = lambda r: L.cp_scored_attn_validate(2, 8, 2, 5, 7, 64, 1.0, r, 0)
    assert v(None) == 0
    assert v(rule(q_docs=P)) == _lib.CP_ERR_INVALID_ARG
    assert v(rule(q_docs=P, kv_docs=P + 2)) == _lib.CP_ERR_ALIGNMENT
    assert L.cp_scored_attn_validate(2, 8, 2, 5, 7, 64, 1.0, None, 7) == _lib.CP_ERR_INVALID_ARG


def test_scored_calls_reject_before_launch():
    L = _lib.lib()

    def fwd(q=P, k=P, o=P, l=P, B=1, Sq=64, Skv=64, D=64, r=None, ws=None, n=0, dt=0, odt=0, H=4, Hkv=2):
        return L.cp_scored_attn_fwd(q, k, P, o, l, B, H, Hkv, Sq, Skv, D, 0.1, r, ws, n, dt, odt, None)

    assert fwd(q=0) == _lib.CP_ERR_INVALID_ARG and fwd(k=0) == _lib.CP_ERR_INVALID_ARG
    assert fwd(o=0) == _lib.CP_ERR_INVALID_ARG and fwd(l=0) == _lib.CP_ERR_INVALID_ARG
    assert fwd(k=P + 8) == _lib.CP_ERR_ALIGNMENT and fwd(o=P + 4) == _lib.CP_ERR_ALIGNMENT
    assert fwd(dt=1, odt=0) == _lib.CP_ERR_INVALID_ARG            # fp32 inputs, bf16 out
    assert fwd(odt=5) == _lib.CP_ERR_INVALID_ARG
    assert fwd(D=80) == _lib.CP_ERR_INVALID_ARG and fwd(Hkv=3) == _lib.CP_ERR_NOT_DIVISIBLE
    docs = rule(q_docs=P, kv_docs=P)
    assert fwd(r=docs) == _lib.CP_ERR_WORKSPACE
    need = cpa.cp_scored_attn_workspace_size(1, 4, 64, 64, True)
    assert need >= 2 * 16 and fwd(r=docs, ws=P, n=need - 1) == _lib.CP_ERR_WORKSPACE
    assert fwd(r=docs, ws=P + 16, n=need) == _lib.CP_ERR_ALIGNMENT
    assert fwd(B=0) == 0 and fwd(Sq=0) == 0
    assert cpa.cp_scored_attn_workspace_size(1, 4, 64, 64, False) == 0

    def bwd(q=P, dk=P, Sq=64, Skv=64, r=None, ws=P, n=1 << 30, dt=0, odt=0, gdt=0, B=1):
        return L.cp_scored_attn_bwd(q, P, P, P, P, P, P, dk, P, B, 4, 2, Sq, Skv, 64, 0.1, r, ws, n, dt, odt, gdt, None)

    assert bwd(q=0) == _lib.CP_ERR_INVALID_ARG and bwd(dk=0) == _lib.CP_ERR_INVALID_ARG
    assert bwd(dk=P + 8) == _lib.CP_ERR_ALIGNMENT
    assert bwd(ws=0) == _lib.CP_ERR_WORKSPACE and bwd(n=16) == _lib.CP_ERR_WORKSPACE
    assert bwd(ws=P + 16) == _lib.CP_ERR_ALIGNMENT
    assert bwd(dt=1, gdt=0) == _lib.CP_ERR_INVALID_ARG and bwd(dt=1, odt=0, gdt=1) == _lib.CP_ERR_INVALID_ARG
    assert bwd(r=rule(prefix_lens=P)) == _lib.CP_ERR_UNSUPPORTED_COMBO
    assert bwd(B=0) == 0 and bwd(Sq=0, Skv=0) == 0
    assert cpa.cp_scored_attn_bwd_workspace_size(1, 4, 64, 64) >= 4 * 64 * 4


def test_paged_calls_reject_before_launch():
    L = _lib.lib()

    def append(k=P, c=P, t=P, B=2, T=3, Hkv=2, D=64, pages=8, page=16, most=4, dt=0):
        return L.cp_paged_kv_append(k, P, c, P, t, P, None, B, T, Hkv, D, pages, page, most, dt, None)

    inv = _lib.CP_ERR_INVALID_ARG
    assert append(k=0) == inv and append(c=0) == inv and append(t=0) == inv
    assert append(k=P + 8) == _lib.CP_ERR_ALIGNMENT and append(t=P + 2) == _lib.CP_ERR_ALIGNMENT
    for bad in (dict(page=12), dict(page=0), dict(page=1 << 17), dict(D=32), dict(pages=0), dict(T=-1), dict(B=4097),
                dict(Hkv=0), dict(dt=3), dict(pages=1 << 20, page=1 << 14), dict(most=-1)):
        assert append(**bad) == inv, bad
    assert append(B=0) == 0 and append(T=0) == 0

    def decode(q=P, o=P, B=2, H=8, Hkv=2, D=64, pages=8, page=16, most=4, cap=0.0, ws=P, n=1 << 30, dt=0, odt=0):
        return L.cp_paged_attn_decode(q, P, P, P, P, o, P, B, H, Hkv, D, pages, page, most, 0.1, cap, None, ws, n, dt,
                                      odt, None)

    assert decode(q=0) == inv and decode(o=0) == inv and decode(q=P + 2) == _lib.CP_ERR_ALIGNMENT
    assert decode(H=7) == _lib.CP_ERR_NOT_DIVISIBLE
    for bad in (dict(page=24), dict(D=96), dict(cap=-1.0), dict(cap=float("inf")), dict(dt=1, odt=0), dict(B=5000),
                dict(most=1 << 30, page=16), dict(B=4096, most=1 << 20, page=64, Hkv=8)):
        assert decode(**bad) == inv, bad
    need = cpa.cp_paged_attn_workspace_size(2, 8, 2, 64)
    assert need > 0 and decode(n=need - 1, most=4096) == _lib.CP_ERR_WORKSPACE
    assert decode(ws=0, most=4096) == _lib.CP_ERR_WORKSPACE
    # a short table takes one launch and no workspace, a long one what the size without a table says
    assert cpa.cp_paged_attn_workspace_size(2, 8, 2, 64, page_size=16, max_pages=4) == 0
    assert cpa.cp_paged_attn_workspace_size(2, 8, 2, 64, page_size=16, max_pages=4096) == need
    assert decode(ws=P + 16) == _lib.CP_ERR_ALIGNMENT
    assert decode(B=0) == 0


def test_python_wrappers_reject_host_tensors():
    q, l = torch.zeros((1, 4, 2, 64)), torch.zeros((1, 2, 4))
    with pytest.raises(ValueError):
        cpa.cp_scored_attn_fwd(q, q, q, q, l, 0.1)
    with pytest.raises(ValueError):
        cpa.cp_paged_kv_append(q, q, q, q, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        cpa.cp_paged_attn_decode(q[0], q, q, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                                 q[0], l[0], 0.1)


def test_scales_and_caps_whose_products_would_overflow():
    """cap log2 e past fp32's range made NaN of a zero score in the bf16 backward."""
    f = lambda **kw: cpa.cp_scored_attn_validate(2, 8, 2, 5, 7, 64, **kw)
    assert f(softcap=1e30) == 0 and f(scale=1e30) == 0 and f(scale=-1e30, softcap=1.0) == 0
    for bad in (dict(softcap=1.1e30), dict(softcap=3e38), dict(scale=1.1e30), dict(scale=-3e38), dict(scale=float("-inf")),
                dict(softcap=float("inf"))):
        for dt in (torch.bfloat16, torch.float32):
            assert f(**bad, dtype=dt) == _lib.CP_ERR_INVALID_ARG, bad
    L = _lib.lib()
    for scale, cap in ((0.1, 3e38), (3e38, 0.0), (float("nan"), 0.0)):
        assert L.cp_paged_attn_decode(P, P, P, P, P, P, P, 1, 2, 2, 64, 8, 16, 4, scale, cap, None, None, 0, 0, 0,
                                      None) == _lib.CP_ERR_INVALID_ARG
