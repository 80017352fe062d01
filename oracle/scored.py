"""Float64 definitions of attention with a score rule and of the paged cache.

TEST INFRASTRUCTURE ONLY, as the rest of this package: plain numpy, one head at
a time, sharing no code with the library.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return x.detach().cpu().double().numpy() if hasattr(x, "detach") else np.asarray(x, dtype=np.float64)


def _int(x):
    if x is None:
        return None
    return x.detach().cpu().numpy().astype(np.int64) if hasattr(x, "detach") else np.asarray(x, dtype=np.int64)


def scores(q, k, b, h, scale, softcap=0.0, slopes=None, causal=False, prefix_lens=None, q_docs=None, kv_docs=None,
           q_pos0=0, kv_pos0=0):
    """Scores of one head: x [Sq, Skv] (-inf where a pair takes no part) and the derivative of the cap."""
    q, k = _f64(q), _f64(k)
    hk = h // (q.shape[2] // k.shape[2])
    x = scale * (q[b, :, h] @ k[b, :, hk].T)
    dcap = np.ones_like(x)
    if softcap > 0:
        t = np.tanh(x / softcap)
        x, dcap = softcap * t, 1.0 - t * t
    pi = q_pos0 + np.arange(q.shape[1])[:, None]
    pj = kv_pos0 + np.arange(k.shape[1])[None, :]
    if slopes is not None:
        x = x - _f64(slopes)[h] * np.abs(pi - pj)
    on = np.ones(x.shape, dtype=bool)
    if causal:
        on = pj <= pi
        if prefix_lens is not None:
            on = on | (pj < _int(prefix_lens)[b])
    if q_docs is not None:
        dq, dk = _int(q_docs)[b][:, None], _int(kv_docs)[b][None, :]
        on = on & (dq == dk) & (dq >= 0)
    return np.where(on, x, -np.inf), dcap


def _lse(x):
    """ln sum exp over the last axis; -inf for an empty row."""
    m = np.max(x, axis=-1, initial=-np.inf)
    base = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore"):
        return base + np.log(np.sum(np.exp(x - base[..., None]), axis=-1))


def scored_attention(q, k, v, scale, **rule):
    """(out [B, Sq, H, D], lse [B, H, Sq])."""
    v = _f64(v)
    B, Sq, H, D = q.shape
    G = H // v.shape[2]
    out, lse = np.zeros((B, Sq, H, D)), np.full((B, H, Sq), -np.inf)
    for b in range(B):
        for h in range(H):
            x, _ = scores(q, k, b, h, scale, **rule)
            lse[b, h] = _lse(x)
            p = np.exp(x - np.where(np.isneginf(lse[b, h]), 0.0, lse[b, h])[:, None])
            out[b, :, h] = p @ v[b, :, h // G]
    return out, lse


def scored_attention_bwd(q, k, v, out, dout, lse, scale, **rule):
    """(dq, dk, dv) of L = sum(out * dout), from the given out and lse."""
    qf, kf, vf, o, g, l = (_f64(t) for t in (q, k, v, out, dout, lse))
    B, Sq, H, D = qf.shape
    G = H // kf.shape[2]
    dq, dk, dv = np.zeros_like(qf), np.zeros_like(kf), np.zeros_like(vf)
    for b in range(B):
        for h in range(H):
            x, dcap = scores(q, k, b, h, scale, **rule)
            p = np.exp(x - np.where(np.isneginf(l[b, h]), np.inf, l[b, h])[:, None])
            delta = np.sum(g[b, :, h] * o[b, :, h], axis=1)
            ds = p * (g[b, :, h] @ vf[b, :, h // G].T - delta[:, None]) * dcap
            dq[b, :, h] = scale * (ds @ kf[b, :, h // G])
            dk[b, :, h // G] += scale * (ds.T @ qf[b, :, h])
            dv[b, :, h // G] += p.T @ g[b, :, h]
    return dq, dk, dv


def cached_rows(cache, table, b, n):
    """Rows 0 .. n - 1 of sequence b, [n, Hkv, D]."""
    page = cache.shape[1]
    return np.stack([cache[table[b, j // page], j % page] for j in range(n)]) if n else cache[0, :0]


def paged_decode(q, k_cache, v_cache, table, seq_lens, scale, softcap=0.0, slopes=None):
    """(out [B, H, D], lse [B, H]) of one new token per sequence, its last."""
    qf, kc, vc = _f64(q), _f64(k_cache), _f64(v_cache)
    table, lens = _int(table), _int(seq_lens)
    B, H, D = qf.shape
    out, lse = np.zeros((B, H, D)), np.full((B, H), -np.inf)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        k, v = cached_rows(kc, table, b, n), cached_rows(vc, table, b, n)
        o, l = scored_attention(qf[b][None, None], k[None], v[None], scale, softcap=softcap, slopes=slopes,
                                q_pos0=n - 1)
        out[b], lse[b] = o[0, 0], l[0, :, 0]
    return out, lse


def paged_append(new, cache, table, seq_lens, new_lens=None):
    """The cache (any numpy array [num_pages, page, Hkv, D]) with the new rows [B, T, Hkv, D] written in, as a copy."""
    cache, table, lens = np.array(cache), _int(table), _int(seq_lens)
    page = cache.shape[1]
    for b in range(new.shape[0]):
        for t in range(new.shape[1] if new_lens is None else min(new.shape[1], int(_int(new_lens)[b]))):
            pos = int(lens[b]) + t
            cache[table[b, pos // page], pos % page] = new[b, t]
    return cache


def abs_products(q, k, scale):
    """max over pairs of scale * sum_d |q_d k_d|: what the rounding of a score scales with."""
    q, k = np.abs(_f64(q)), np.abs(_f64(k))
    G = q.shape[2] // k.shape[2]
    if q.shape[1] == 0 or k.shape[1] == 0:
        return 0.0
    return max(float(np.max(q[b, :, h] @ k[b, :, h // G].T)) for b in range(q.shape[0])
               for h in range(q.shape[2])) * abs(scale) if q.shape[0] else 0.0


__all__ = ["scores", "scored_attention", "scored_attention_bwd", "paged_decode", "paged_append", "cached_rows",
           "abs_products"]
