"""Refusals and sizes of the head norm with rotary positions: every call here
fails its checks on the host or has nothing to do, and none reaches a GPU."""
import ctypes

import pytest
import torch

import context_attention_dits_gb300 as cpa
from context_attention_dits_gb300 import _lib

P = 1 << 20  # an aligned "device" address that is never dereferenced
BAD, COMBO, ALIGN, WS = (_lib.CP_ERR_INVALID_ARG, _lib.CP_ERR_UNSUPPORTED_COMBO, _lib.CP_ERR_ALIGNMENT,
                         _lib.CP_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    from context_attention_dits_gb300 import build
    build.build()


def rule(**kw):
    kw = {**dict(norm=1, eps=1e-6, pairs=32, freqs=P, positions=P, axes=1), **kw}
    return ctypes.byref(_lib.QkRule(**kw))


def strides(*rows):
    return (ctypes.c_int64 * (3 * len(rows)))(*(x for r in rows for x in r))


DENSE = (3 * 4 * 64, 4 * 64, 64)
KEYS = (3 * 2 * 64, 2 * 64, 64)


def fwd(q=P, k=P, qo=P, ko=P, st=None, B=2, S=3, H=4, Hkv=2, D=64, r=None, dt=0):
    return _lib.lib().cp_qk_norm_rope_fwd(q, k, qo, ko, st, B, S, H, Hkv, D, r or rule(), dt, None)


def bwd(q=P, k=P, gq=P, gk=P, dq=P, dk=P, wq=P, wk=P, st=None, B=2, S=3, H=4, Hkv=2, D=64, r=None, ws=P, n=1 << 30,
        dt=0, gdt=0):
    return _lib.lib().cp_qk_norm_rope_bwd(q, k, gq, gk, dq, dk, wq, wk, st, B, S, H, Hkv, D, r or rule(), ws, n, dt, gdt,
                                          None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_sizes_and_rule(call):
    for bad in (dict(D=96), dict(B=-1), dict(S=-1), dict(H=0), dict(Hkv=-1), dict(H=65536), dict(B=1 << 13, S=1 << 13),
                dict(dt=2)):
        assert call(**bad) == BAD, bad
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(pairs=-4), dict(pairs=36),
                dict(pairs=6), dict(axes=0), dict(axes=5), dict(weight_dt=1, norm=0, q_weight=P),
                dict(weight_dt=3, k_weight=P), dict(pair_axis=bytes([0] * 31 + [1])), dict(freqs=0), dict(positions=0)):
        assert call(r=rule(**bad)) == BAD, bad
    assert call(dt=1, r=rule(weight_dt=0, q_weight=P), **({"gdt": 1} if call is bwd else {})) == BAD   # fp32 rows, bf16 weights
    for bad in (dict(freqs=P + 4), dict(positions=P + 2), dict(q_weight=P + 1), dict(weight_dt=1, k_weight=P + 2)):
        assert call(r=rule(**bad)) == ALIGN, bad
    assert _lib.lib().cp_qk_norm_rope_fwd(P, P, P, P, None, 1, 1, 1, 1, 64, None, 0, None) == BAD


def test_forward_tensors():
    for bad in ("q", "k", "qo", "ko"):
        assert fwd(**{bad: 0}) == BAD and fwd(**{bad: P + 8}) == ALIGN, bad
    assert fwd(st=strides((DENSE[0], 252, 64), KEYS, DENSE, KEYS)) == ALIGN
    assert fwd(st=strides((DENSE[0], -256, 64), KEYS, DENSE, KEYS)) == BAD
    assert fwd(st=strides(DENSE, (1 << 41, 128, 64), DENSE, KEYS)) == BAD
    for over in ((DENSE[0], 248, 64), (DENSE[0], 256, 56), (0, 256, 64), (760, 256, 64), (256, 256, 64)):
        assert fwd(st=strides(DENSE, KEYS, over, KEYS)) == BAD, over   # rows of a result overlap
    assert fwd(B=0) == 0 and fwd(S=0, q=0) == 0
    assert fwd(B=0, r=rule(freqs=0, positions=0)) == 0


def test_backward_tensors():
    for bad in ("q", "k", "gq", "gk", "dq", "dk"):
        assert bwd(**{bad: 0}) == BAD and bwd(**{bad: P + 4}) == ALIGN, bad
    assert bwd(gdt=2) == BAD and bwd(dt=1, gdt=0) == BAD
    assert bwd(r=rule(norm=0)) == BAD                      # a weight's gradient without a norm
    assert bwd(Hkv=0) == BAD and bwd(Hkv=0, wk=None, B=0, wq=None) == 0
    need = cpa.cp_qk_norm_rope_bwd_workspace_size(64)
    assert need >= 2 * 64 * 4 and cpa.cp_qk_norm_rope_bwd_workspace_size(128) == 2 * need
    assert cpa.cp_qk_norm_rope_bwd_workspace_size(80) == 0
    assert bwd(ws=0) == WS and bwd(n=need - 1) == WS and bwd(ws=P + 16) == ALIGN and bwd(wq=P + 2) == ALIGN
    assert bwd(B=0, wq=None, wk=None, ws=0) == 0
    assert bwd(st=strides(DENSE, KEYS, DENSE, KEYS, (DENSE[0], 0, 64), KEYS)) == BAD


def test_wrapper_refuses_host_tensors():
    q, k = torch.zeros(1, 3, 4, 64), torch.zeros(1, 3, 2, 64)
    with pytest.raises(ValueError):
        cpa.cp_qk_norm_rope_fwd(q, k, q, k, eps=1e-6)
    with pytest.raises(ValueError):
        cpa.cp_qk_norm_rope_bwd(q, k, q, k, q, k, eps=1e-6)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("pairs", [1 << 30, 3 << 29, (1 << 31) - 4])
def test_more_pairs_than_half_an_int(call, pairs):
    """Twice as many are no int: refused as any other number of pairs that a head has no values for."""
    assert call(r=rule(pairs=pairs)) == BAD
