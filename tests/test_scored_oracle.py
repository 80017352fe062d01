"""Pins of the float64 score-rule oracle: closed forms, torch's softmax and
autograd, central differences, and a partition of the keys."""
import numpy as np
import pytest
import torch

from oracle import cp_oracle as co
from oracle import scored as so


def data(B, Sq, Skv, H, Hkv, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    return r(B, Sq, H, D), r(B, Skv, Hkv, D), r(B, Skv, Hkv, D), r(B, Sq, H, D)


RULES = [
    {},
    dict(softcap=1.5),
    dict(slopes=torch.tensor([0.5, 0.25, -0.1, 0.0])),
    dict(causal=True, q_pos0=2),
    dict(causal=True, prefix_lens=torch.tensor([3, 0]), softcap=2.0),
    dict(q_docs=torch.tensor([[0, 0, 1, 1, -1], [4, 4, 4, 2, 2]]), kv_docs=torch.tensor([[0, 1, 1, 1, 3, -1, 0], [2, 4, 4, 9, 9, 9, 2]]),
         slopes=torch.tensor([0.5, 0.25, 0.1, 0.0]), softcap=3.0),
]


def torch_attention(q, k, v, scale, softcap=0.0, slopes=None, causal=False, prefix_lens=None, q_docs=None,
                    kv_docs=None, q_pos0=0, kv_pos0=0):
    G = q.shape[2] // k.shape[2]
    x = torch.einsum("bihd,bjhd->bhij", q, k.repeat_interleave(G, 2)) * scale
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    i = torch.arange(q.shape[1])[:, None] + q_pos0
    j = torch.arange(k.shape[1])[None] + kv_pos0
    if slopes is not None:
        x = x - slopes.double()[None, :, None, None] * (i - j).abs()
    on = torch.ones((q.shape[0], q.shape[1], k.shape[1]), dtype=torch.bool)
    if causal:
        on &= j <= i
        if prefix_lens is not None:
            on |= j < prefix_lens[:, None, None]
    if q_docs is not None:
        on &= (q_docs[:, :, None] == kv_docs[:, None]) & (q_docs >= 0)[:, :, None]
    x = x.masked_fill(~on[:, None], -1e30)
    p = torch.softmax(x, 3) * on[:, None]
    return torch.einsum("bhij,bjhd->bihd", p, v.repeat_interleave(G, 2))


@pytest.mark.parametrize("rule", RULES)
def test_forward_and_backward_match_torch(rule):
    q, k, v, g = data(2, 5, 7, 4, 2, 8)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    want = torch_attention(*leaves, 0.4, **rule)
    out, lse = so.scored_attention(q, k, v, 0.4, **rule)
    assert np.allclose(out, want.detach().numpy(), atol=1e-12)
    want.backward(g)
    got = so.scored_attention_bwd(q, k, v, out, g, lse, 0.4, **rule)
    for x, t in zip(got, leaves):
        assert np.allclose(x, t.grad.numpy(), atol=1e-11)


@pytest.mark.parametrize("rule", RULES)
def test_gradients_match_central_differences(rule):
    q, k, v, g = data(2, 5, 7, 4, 2, 3, seed=1)
    out, lse = so.scored_attention(q, k, v, 0.4, **rule)
    grads = so.scored_attention_bwd(q, k, v, out, g, lse, 0.4, **rule)
    rng = np.random.default_rng(0)
    for which, (t, gr) in enumerate(zip((q, k, v), grads)):
        for _ in range(6):
            at = tuple(rng.integers(0, n) for n in t.shape)
            f = []
            for e in (1e-5, -1e-5):
                ts = [x.clone() for x in (q, k, v)]
                ts[which][at] += e
                f.append(np.sum(so.scored_attention(*ts, 0.4, **rule)[0] * g.numpy()))
            assert abs((f[0] - f[1]) / 2e-5 - gr[at]) < 1e-7


def test_no_rule_is_plain_attention():
    q, k, v, _ = data(2, 5, 7, 4, 4, 8)
    want = co.attention(q, k, v, 0.4)
    got = so.scored_attention(q, k, v, 0.4)
    assert np.allclose(got[0], want[0], atol=1e-13) and np.allclose(got[1], want[1], atol=1e-13)


def test_wide_cap_is_no_cap_and_scores_stay_below_it():
    q, k, v, _ = data(1, 4, 4, 2, 2, 8)
    assert np.allclose(so.scores(q, k, 0, 0, 1.0, softcap=1e7)[0], so.scores(q, k, 0, 0, 1.0)[0], atol=1e-9)
    assert np.all(np.abs(so.scores(q * 100, k, 0, 0, 1.0, softcap=2.0)[0]) <= 2.0)


def test_blocks_of_keys_merge_to_the_whole():
    rule = dict(causal=True, softcap=2.0, slopes=torch.tensor([0.5, 0.25, 0.1, 0.0]))
    q, k, v, _ = data(1, 6, 9, 4, 2, 8)
    want = so.scored_attention(q, k, v, 0.4, q_pos0=3, **rule)
    o, l = so.scored_attention(q, k[:, :4], v[:, :4], 0.4, q_pos0=3, **rule)
    o2, l2 = so.scored_attention(q, k[:, 4:], v[:, 4:], 0.4, q_pos0=3, kv_pos0=4, **rule)
    got = co.lse_merge(o, l, o2, l2)
    assert np.allclose(got[0], want[0], atol=1e-12) and np.allclose(got[1], want[1], atol=1e-12)


def test_rows_without_a_key_are_empty():
    q, k, v, g = data(1, 3, 3, 2, 1, 4)
    rule = dict(q_docs=[[0, -1, 5]], kv_docs=[[0, -1, 0]])
    out, lse = so.scored_attention(q, k, v, 1.0, **rule)
    assert np.all(out[0, 1:] == 0) and np.all(np.isneginf(lse[0, :, 1:])) and np.all(np.isfinite(lse[0, :, 0]))
    dq, dk, dv = so.scored_attention_bwd(q, k, v, out, g, lse, 1.0, **rule)
    assert np.all(dq[0, 1:] == 0) and np.all(dk[0, 1] == 0) and np.all(dv[0, 1] == 0)


def test_paged_forms_match_a_dense_cache():
    rng = np.random.default_rng(3)
    table = np.array([[5, 0, 2], [1, 4, 3]])
    lens, new = np.array([3, 0]), rng.standard_normal((2, 4, 2, 8))
    cache = rng.standard_normal((6, 4, 2, 8))
    got = so.paged_append(new, cache, table, lens, [4, 2])
    assert np.array_equal(got[5, :3], cache[5, :3]) and np.array_equal(got[5, 3], new[0, 0])
    assert np.array_equal(got[0, :3], new[0, 1:]) and np.array_equal(got[0, 3], cache[0, 3])
    assert np.array_equal(got[1, :2], new[1, :2]) and np.array_equal(got[1, 2:], cache[1, 2:])
    assert np.array_equal(got[2:5], cache[2:5])
    q = rng.standard_normal((2, 4, 8))
    out, lse = so.paged_decode(q, got, got, table, np.array([7, 0]), 0.3, softcap=2.0, slopes=np.ones(4) * 0.1)
    dense = np.concatenate([got[5], got[0]])[:7][None]
    want = so.scored_attention(q[:1, None], dense, dense, 0.3, softcap=2.0, slopes=np.ones(4) * 0.1, q_pos0=6, causal=True)
    assert np.allclose(out[0], want[0][0, 0]) and np.allclose(lse[0], want[1][0, :, 0])
    assert np.all(out[1] == 0) and np.all(np.isneginf(lse[1]))
