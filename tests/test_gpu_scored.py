"""cp_scored_attn_fwd and cp_scored_attn_bwd against the float64 oracle.

Bounds, element by element, with u = 2^-24 (fp32 rounding, half a step) and
w = 2^-8 for bf16 inputs (P and dS are rounded to bf16 for their products), 0
for fp32:
  a score's error is at most d = (D + 16) u max(scale sum |q||k|) + 4 u max|x|
  (the dot product, the scale, the cap, the bias), a weight's then 2 d + 2^-21
  relative (the last term: the exponential), and a sum of n terms adds n u:
    |out - ref| <= (w + e) sum_j p |v| + r |ref|,        e = 2 (2 d + 2^-21 + n u)
    |lse - ref| <= 2 d + 2^-20 + n u + 4 u |ref|
    |dv  - ref| <= (w + e) sum_i p |dout| + r |ref|
    |dq  - ref| <= scale sum_j E |k| + r |ref|, likewise dk, where
    E = (w + e) |ds| + p (D + 8) u (sum |dout||v| + sum |dout||out|)
with r the rounding of the output (2^-8 bf16, u fp32; doubled for the sums'
own). The oracle's backward takes the same out and lse. Weights below 2^-126,
fp32's smallest normal number, may come out as 0: over the at most 2^12 terms
of a sum here, each times a factor below 2^12, that is less than 2^-100, which
every bound is given on top.
"""
import numpy as np
import pytest
import torch

from oracle import scored as so

pytestmark = pytest.mark.gpu

BF, F4 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from context_attention_dits_gb300 import build
    build.build()


def cpa():
    import context_attention_dits_gb300 as m
    return m


def draw(B, Sq, Skv, H, Hkv, D, dt, seed, qmul=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    return [(r(B, Sq, H, D) * qmul).to(dt), r(B, Skv, Hkv, D).to(dt), r(B, Skv, Hkv, D).to(dt), r(B, Sq, H, D).to(dt)]


def on_gpu(rule):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in rule.items()}


def run_fwd(q, k, v, scale, rule, out_dt):
    B, Sq, H, D = q.shape
    out = torch.full((B, Sq, H, D), 7.0, dtype=out_dt, device="cuda")
    lse = torch.full((B, H, Sq), 7.0, device="cuda")
    cpa().cp_scored_attn_fwd(q.cuda(), k.cuda(), v.cuda(), out, lse, scale, **on_gpu(rule))
    torch.cuda.synchronize()
    assert cpa().cp_check_device_status() == 0
    return out.cpu(), lse.cpu()


def run_bwd(q, k, v, out, dout, lse, scale, rule, gdt):
    grads = [torch.full(t.shape, 7.0, dtype=gdt, device="cuda") for t in (q, k, v)]
    cpa().cp_scored_attn_bwd(*[t.cuda() for t in (q, k, v, out, dout, lse)], *grads, scale, **on_gpu(rule))
    torch.cuda.synchronize()
    assert cpa().cp_check_device_status() == 0
    return [t.cpu() for t in grads]


def errors_of(q, k, scale, rule):
    """d and e of the module's bounds."""
    n = max(q.shape[1] * (q.shape[2] // k.shape[2]), k.shape[1], 1)
    big = so.abs_products(q, k, scale)
    far = 0.0
    if rule.get("slopes") is not None:
        i0, j0 = rule.get("q_pos0", 0), rule.get("kv_pos0", 0)
        far = float(rule["slopes"].abs().max()) * max(abs(i0 + q.shape[1] - j0), abs(j0 + k.shape[1] - i0))
    d = (q.shape[3] + 16) * U * big + 4 * U * (big + far)
    return d, 2 * (2 * d + 2.0 ** -21 + n * U), n


def check(got, want, bound, what):
    got = got.double().numpy()
    inf = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), inf), f"{what}: -inf rows differ"
    assert np.all(np.isfinite(got[~inf])), f"{what}: not finite"
    over = np.abs(got[~inf] - want[~inf]) - np.broadcast_to(bound, want.shape)[~inf] - 2.0 ** -100
    assert over.size == 0 or over.max() <= 0, f"{what}: past its bound by {over.max():.3e}"


def probs(q, k, lse, b, h, scale, rule):
    x, dcap = so.scores(q, k, b, h, scale, **rule)
    l = lse[b, h]
    return np.exp(x - np.where(np.isneginf(l), np.inf, l)[:, None]), dcap


def check_fwd(q, k, v, scale, rule, out, lse, what):
    want, wl = so.scored_attention(q, k, v, scale, **rule)
    d, e, n = errors_of(q, k, scale, rule)
    w = 2.0 ** -8 if q.dtype == BF else 0.0
    r = (2.0 ** -8 if out.dtype == BF else U) * 2
    mass = np.zeros_like(want)
    va = np.abs(v.double().numpy())
    G = q.shape[2] // k.shape[2]
    for b in range(q.shape[0]):
        for h in range(q.shape[2]):
            mass[b, :, h] = probs(q, k, wl, b, h, scale, rule)[0] @ va[b, :, h // G]
    check(out, want, (w + e) * mass + r * np.abs(want), what + " out")
    with np.errstate(invalid="ignore"):
        check(lse, wl, 2 * d + 2.0 ** -20 + n * U + 4 * U * np.abs(np.where(np.isinf(wl), 0, wl)), what + " lse")


def check_bwd(q, k, v, out, dout, lse, scale, rule, grads, what):
    want = so.scored_attention_bwd(q, k, v, out, dout, lse, scale, **rule)
    d, e, n = errors_of(q, k, scale, rule)
    w = 2.0 ** -8 if q.dtype == BF else 0.0
    r = (2.0 ** -8 if grads[0].dtype == BF else U) * 2
    D, G = q.shape[3], q.shape[2] // k.shape[2]
    qf, kf, vf, of, gf, lf = (t.double().numpy() for t in (q, k, v, out, dout, lse))
    bound = [np.zeros_like(x) for x in want]
    for b in range(q.shape[0]):
        for h in range(q.shape[2]):
            p, dcap = probs(q, k, lf, b, h, scale, rule)
            g, vv = gf[b, :, h], vf[b, :, h // G]
            ds = p * (g @ vv.T - np.sum(g * of[b, :, h], 1)[:, None]) * dcap
            ga = np.abs(g)
            E = (w + e) * np.abs(ds) + p * (D + 8) * U * (ga @ np.abs(vv).T + np.sum(ga * np.abs(of[b, :, h]), 1)[:, None])
            bound[0][b, :, h] = abs(scale) * (E @ np.abs(kf[b, :, h // G]))
            bound[1][b, :, h // G] += abs(scale) * (E.T @ np.abs(qf[b, :, h]))
            bound[2][b, :, h // G] += (w + e) * (p.T @ ga)
    for name, x, y, bd in zip(("dq", "dk", "dv"), grads, want, bound):
        check(x, y, bd + r * np.abs(y), f"{what} {name}")


def slopes(H):
    return torch.exp2(-8.0 * torch.arange(1, H + 1) / H)


def docs(B, S, n, pad, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.sort(torch.randint(0, n, (B, S), generator=g), 1).values.to(torch.int32)
    if pad:
        ids[:, S - pad:] = -1
    return ids


# name: (B, Sq, Skv, H, Hkv, D, rule)
CASES = {
    "one pair": (1, 1, 1, 1, 1, 64, {}),
    "plain, shared heads": (2, 70, 70, 4, 2, 64, {}),
    "cap": (1, 130, 130, 2, 2, 128, dict(softcap=30.0)),
    "tight cap": (1, 97, 97, 2, 1, 64, dict(softcap=0.75)),
    "narrow cap": (1, 140, 140, 2, 2, 128, dict(softcap=1e-3, causal=True)),
    "wide cap": (1, 300, 300, 2, 2, 128, dict(softcap=1e5, causal=True)),
    "cap without effect": (1, 140, 140, 2, 2, 64, dict(softcap=1e30)),
    "bias both ways": (1, 200, 200, 3, 3, 64, dict(slopes=slopes(3))),
    "negative slope": (1, 65, 129, 2, 2, 128, dict(slopes=torch.tensor([-0.01, 0.02]), softcap=5.0)),
    "causal": (2, 257, 257, 2, 1, 128, dict(causal=True)),
    "causal cap bias": (1, 300, 300, 8, 2, 64, dict(causal=True, softcap=15.0, slopes=slopes(8))),
    "causal chunk": (1, 33, 290, 4, 4, 128, dict(causal=True, q_pos0=257)),
    "keys ahead of the rows": (1, 150, 300, 2, 2, 64, dict(causal=True, q_pos0=100, kv_pos0=20)),
    "no key yet": (1, 100, 40, 2, 2, 64, dict(causal=True, kv_pos0=60)),
    "every key ahead": (1, 20, 20, 2, 2, 64, dict(causal=True, kv_pos0=500)),
    "prefix": (3, 270, 270, 2, 2, 128, dict(causal=True, prefix_lens=torch.tensor([0, 140, 270], dtype=torch.int32))),
    "prefix past the block": (1, 90, 140, 2, 1, 64, dict(causal=True, q_pos0=3, kv_pos0=40,
                              prefix_lens=torch.tensor([100], dtype=torch.int32), softcap=20.0)),
    "documents": (2, 400, 400, 2, 2, 64, dict(causal=True, q_docs=docs(2, 400, 5, 37, 1), kv_docs=docs(2, 400, 5, 37, 1))),
    "documents in any order": (1, 260, 190, 4, 1, 128, dict(
        q_docs=torch.randint(-1, 3, (1, 260), generator=torch.Generator().manual_seed(2)).to(torch.int32),
        kv_docs=torch.randint(-1, 4, (1, 190), generator=torch.Generator().manual_seed(3)).to(torch.int32),
        slopes=slopes(4), softcap=25.0)),
    "one document, padding between": (1, 700, 700, 1, 1, 64, dict(
        q_docs=torch.where(torch.arange(700) % 300 < 150, 2, -1)[None].to(torch.int32),
        kv_docs=torch.where(torch.arange(700) % 300 < 150, 2, -1)[None].to(torch.int32), causal=True,
        prefix_lens=torch.tensor([320], dtype=torch.int32))),
    "all padding": (1, 130, 130, 2, 1, 128, dict(q_docs=torch.full((1, 130), -1, dtype=torch.int32),
                                                   kv_docs=torch.full((1, 130), -1, dtype=torch.int32))),
    "wide": (1, 520, 1030, 6, 3, 128, dict(causal=True, q_pos0=510, softcap=50.0)),
    "five heads on one": (2, 129, 64, 5, 1, 64, dict(softcap=10.0, slopes=slopes(5))),
    "sixteen heads on one": (1, 300, 300, 16, 1, 128, dict(causal=True, softcap=20.0)),
    "sixteen heads on one, documents": (1, 260, 260, 16, 1, 64, dict(causal=True, q_docs=docs(1, 260, 3, 11, 5),
                                                                     kv_docs=docs(1, 260, 3, 11, 5), slopes=slopes(16))),
    "few rows, many keys": (1, 20, 1500, 2, 1, 128, dict(causal=True, q_pos0=1480, softcap=30.0)),
    "few rows, many keys, documents": (1, 130, 1100, 2, 2, 64, dict(causal=True, q_pos0=970, q_docs=docs(1, 1100, 3, 5, 6)[:, 970:].contiguous(),
                                                                    kv_docs=docs(1, 1100, 3, 5, 6))),
    "few rows, distance": (1, 40, 900, 3, 3, 64, dict(slopes=slopes(3), q_pos0=430)),
    "no keys": (1, 9, 0, 2, 2, 64, dict(softcap=10.0)),
}


@pytest.mark.parametrize("dt,out_dt", [(F4, F4), (BF, BF), (BF, F4)])
@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_backward(name, dt, out_dt):
    B, Sq, Skv, H, Hkv, D, rule = CASES[name]
    scale = D ** -0.5
    q, k, v, dout = draw(B, Sq, Skv, H, Hkv, D, dt, seed=Sq + Skv, qmul=2.0 if rule.get("softcap") else 1.0)
    out, lse = run_fwd(q, k, v, scale, rule, out_dt)
    check_fwd(q, k, v, scale, rule, out, lse, name)
    grads = run_bwd(q, k, v, out, dout, lse, scale, rule, out_dt)
    check_bwd(q, k, v, out, dout, lse, scale, rule, grads, name)


@pytest.mark.parametrize("dt", [F4, BF])
def test_large_scores_and_growing_maxima(dt):
    """Scores up to several hundred whose row maximum keeps growing along the keys, uncapped and capped."""
    B, S, H, D = 1, 390, 2, 64
    q, k, v, dout = draw(B, S, S, H, H, D, dt, seed=5)
    k = (k.float() * torch.linspace(0.1, 12.0, S)[None, :, None, None]).to(dt)
    for rule in ({}, dict(softcap=40.0), dict(softcap=2000.0), dict(causal=True, slopes=torch.tensor([0.3, -0.2]))):
        out, lse = run_fwd(q, k, v, 0.6, rule, dt)
        check_fwd(q, k, v, 0.6, rule, out, lse, f"growing {sorted(rule)}")
        grads = run_bwd(q, k, v, out, dout, lse, 0.6, rule, dt)
        check_bwd(q, k, v, out, dout, lse, 0.6, rule, grads, f"growing {sorted(rule)}")


MANY = {  # more items than run at once, so that CTAs go on from one to the next: rule of (B, S)
    "plain": lambda B, S: {},
    "causal, cap": lambda B, S: dict(causal=True, softcap=15.0),
    "slopes both ways": lambda B, S: dict(slopes=slopes(40)),
    "prefix, slopes, cap": lambda B, S: dict(causal=True, softcap=30.0, slopes=slopes(40),
                                             prefix_lens=(torch.arange(B, dtype=torch.int32) * 97)),
    # items without a key among the others: the whole second pair of entry 1, all of entry 2
    "documents": lambda B, S: dict(causal=True, **{n: torch.where(
        (torch.arange(B)[:, None] == 2) | ((torch.arange(B)[:, None] == 1) & (torch.arange(S)[None] >= 256)),
        -1, docs(B, S, 4, 5, 7)).to(torch.int32) for n in ("q_docs", "kv_docs")}),
}


@pytest.mark.parametrize("D,out_dt", [(64, BF), (128, BF), (128, F4)])
@pytest.mark.parametrize("name", list(MANY))
def test_more_items_than_multiprocessors(name, D, out_dt):
    B, S, H, Hkv = 4, 300, 40, 8
    rule = MANY[name](B, S)
    q, k, v, dout = draw(B, S, S, H, Hkv, D, BF, seed=D, qmul=1.5)
    out, lse = run_fwd(q, k, v, D ** -0.5, rule, out_dt)
    check_fwd(q, k, v, D ** -0.5, rule, out, lse, name)
    if D == 64:
        grads = run_bwd(q, k, v, out, dout, lse, D ** -0.5, rule, out_dt)
        check_bwd(q, k, v, out, dout, lse, D ** -0.5, rule, grads, name)
    again, al = run_fwd(q, k, v, D ** -0.5, rule, out_dt)
    assert torch.equal(out, again) and torch.equal(lse, al)


@pytest.mark.parametrize("dt", [F4, BF])
@pytest.mark.parametrize("rule", [{}, dict(causal=True), dict(causal=True, slopes=torch.tensor([0.05, -0.05])),
                                  dict(softcap=400.0)], ids=["plain", "causal", "slopes", "cap"])
def test_rows_and_tiles_at_any_level(rule, dt):
    """Scores whose level differs from row to row (within a warp) and from one stretch of keys to the next, from far
    below to far above what exp2 can hold."""
    B, S, H, D = 1, 600, 2, 64
    q, k, v, dout = draw(B, S, S, H, H, D, dt, seed=11)
    u = torch.ones(D) / 8
    rows = torch.tensor([0.0, -1.0, 1.0, -0.2, 0.2, -4.0, 4.0, 0.02])[torch.arange(S) % 8]
    tiles = torch.tensor([3.0, -3.0, 40.0, 0.0, -40.0])[torch.arange(S) // 128]
    q = (0.1 * q.float() + rows[None, :, None, None] * u).to(dt)
    k = (0.1 * k.float() + tiles[None, :, None, None] * u).to(dt)
    out, lse = run_fwd(q, k, v, 1.5, rule, dt)
    check_fwd(q, k, v, 1.5, rule, out, lse, "levels")
    grads = run_bwd(q, k, v, out, dout, lse, 1.5, rule, dt)
    check_bwd(q, k, v, out, dout, lse, 1.5, rule, grads, "levels")


@pytest.mark.parametrize("n", [262144, 262145, 600000, 1 << 21])
def test_documents_among_more_keys_than_one_bitmap_bit_each(n):
    """A few rows against very many keys of many documents, bf16, against float64 on the same GPU: (w + e) p|v| with
    the pairs that take part for n in e."""
    B, S, H, D, every = 1, 150, 2, 64, 64 * 1024
    g = torch.Generator(device="cuda").manual_seed(n)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)
    q, k, v = r(B, S, H, D), r(B, n, 1, D), r(B, n, 1, D)
    pos = torch.arange(n, device="cuda")
    # stretches of 300 keys at every 65536th of document i mod 3; the others' documents are nobody's
    kd = torch.where(pos % every < 300, (pos // every) % 3, 10 + pos // 1000).to(torch.int32)[None].contiguous()
    qd = (torch.arange(S, device="cuda") // 10 % 4).to(torch.int32)[None].contiguous()   # 3: no key at all
    out, lse = torch.empty_like(q, dtype=F4), torch.empty((B, H, S), device="cuda")
    cpa().cp_scored_attn_fwd(q, k, v, out, lse, D ** -0.5, causal=True, q_pos0=n - S, q_docs=qd, kv_docs=kd)
    assert cpa().cp_check_device_status() == 0
    at = (kd[0] < 3).nonzero()[:, 0]     # the keys that any row sees
    kf, vf = k[0, at, 0].double(), v[0, at, 0].double()
    keep = (qd[0][:, None] == kd[0, at][None]) & (at[None] <= (n - S + torch.arange(S, device="cuda"))[:, None])
    m = len(at)
    for h in range(H):
        x = (q[0, :, h].double() @ kf.T) * D ** -0.5
        big = (q[0, :, h].double().abs() @ kf.abs().T).max().item() * D ** -0.5
        x = x.masked_fill(~keep, -float("inf"))
        wl = torch.logsumexp(x, 1)
        none = torch.isneginf(wl)
        assert none.any() and torch.equal(torch.isneginf(lse[0, h]), none) and (out[0, none, h] == 0).all()
        p = torch.exp(x - torch.where(none, torch.zeros_like(wl), wl)[:, None])
        d = (D + 20) * U * big
        e = 2 * (2 * d + 2.0 ** -21 + m * U)
        over = (out[0, :, h].double() - p @ vf).abs() - (2.0 ** -8 + e) * (p @ vf.abs()) - 2 * U * (p @ vf).abs()
        assert over.max().item() <= 0
        ok = ~none
        assert ((lse[0, h].double() - wl)[ok].abs() <= 2 * d + 2.0 ** -20 + m * U + 4 * U * wl[ok].abs()).all()


@pytest.mark.parametrize("dt", [F4, BF])
def test_values_of_any_size(dt):
    """out is linear in v and the gradients are in dout: powers of two come out bit for bit."""
    B, S, H, Hkv, D = 1, 500, 4, 2, 128
    q, k, v, dout = draw(B, S, S, H, Hkv, D, dt, seed=13, qmul=2.0)
    rule = dict(causal=True, softcap=30.0, slopes=slopes(4))
    out, lse = run_fwd(q, k, v, D ** -0.5, rule, dt)
    for e in (90, -60):
        far, same = run_fwd(q, k, v * 2.0 ** e, D ** -0.5, rule, dt)
        assert torch.equal(far, out * 2.0 ** e) and torch.equal(same, lse)
    grads = run_bwd(q, k, v, out, dout, lse, D ** -0.5, rule, dt)
    for e in (60, -30):
        far = run_bwd(q, k, v, out, dout * 2.0 ** e, lse, D ** -0.5, rule, dt)
        assert all(torch.equal(x, y * 2.0 ** e) for x, y in zip(far, grads))


@pytest.mark.parametrize("rule", [{}, dict(softcap=20.0), dict(slopes=slopes(4)), dict(softcap=20.0, slopes=slopes(4))],
                         ids=["plain", "cap", "slopes", "both"])
def test_rows_of_few_keys_are_exact_to_the_rounding_of_out(rule):
    """bf16: a row of one key is that key's value bit for bit (P = 1). Rows of up to 31 keys: rounding P adds at most
    what out's own rounding is off by, in the 2-norm, less the heaviest key's part, whose P is exact: below sqrt(2)."""
    B, S, H, D = 2, 300, 4, 64
    q, k, v, _ = draw(B, S, S, H, H, D, BF, seed=17, qmul=3.0)
    own = torch.arange(S, dtype=torch.int32).repeat(B, 1)
    out, _ = run_fwd(q, k, v, D ** -0.5, dict(rule, q_docs=own, kv_docs=own), BF)
    assert torch.equal(out, v)
    out, _ = run_fwd(q, k, v, D ** -0.5, dict(rule, causal=True), BF)
    assert torch.equal(out[:, 0], v[:, 0])
    for n, ids in ((3, own // 3), (20, own // 20), (31, own // 31)):
        r = dict(rule, causal=True, q_docs=ids, kv_docs=ids)
        out, _ = run_fwd(q, k, v, D ** -0.5, r, BF)
        want = torch.from_numpy(so.scored_attention(q, k, v, D ** -0.5, **r)[0])
        assert (out.double() - want).norm() <= 2 ** 0.5 * (want.to(BF).double() - want).norm(), n


def test_gradients_match_differences():
    """fp32 gradients against central differences of the library's own forward."""
    B, S, H, Hkv, D = 1, 70, 4, 2, 64
    q, k, v, dout = draw(B, S, S, H, Hkv, D, F4, seed=8)
    rule = dict(causal=True, softcap=3.0, slopes=slopes(4))
    out, lse = run_fwd(q, k, v, 0.2, rule, F4)
    grads = run_bwd(q, k, v, out, dout, lse, 0.2, rule, F4)
    g = torch.Generator().manual_seed(1)
    for i, (t, gr) in enumerate(zip((q, k, v), grads)):
        way = torch.randn(t.shape, generator=g)
        f = []
        for e in (1e-2, -1e-2):
            ts = [q, k, v]
            ts[i] = t + e * way
            f.append((run_fwd(*ts, 0.2, rule, F4)[0].double() * dout.double()).sum().item())
        want, got = (f[0] - f[1]) / 2e-2, (gr.double() * way.double()).sum().item()
        # curvature: third derivatives of a loss of this size times e^2 / 6; and the loss's rounding over 2 e
        assert abs(got - want) <= 2e-3 * (gr.double().norm() * way.double().norm()).item()


@pytest.mark.parametrize("dt", [F4, BF])
def test_ring_of_blocks_merges_to_the_whole(dt):
    """Three ring blocks, each with its positions, joined by cp_lse_merge, then their gradients added up."""
    B, S, H, Hkv, D = 1, 330, 4, 2, 64
    scale, rule = D ** -0.5, dict(causal=True, softcap=20.0, slopes=slopes(4))
    q, k, v, dout = draw(B, S, S, H, Hkv, D, dt, seed=11)
    qd, kd, vd, gd = (t.cuda() for t in (q, k, v, dout))
    r = on_gpu(rule)
    table = cpa().cp_ring_shard_table(S, 3, True)
    acc = None
    for off, n in table:
        out, lse = torch.empty((B, S, H, D), device="cuda"), torch.empty((B, H, S), device="cuda")
        cpa().cp_scored_attn_fwd(qd, kd[:, off:off + n].contiguous(), vd[:, off:off + n].contiguous(), out, lse, scale,
                                 kv_pos0=off, **r)
        if acc is None:
            acc = out, lse
        else:
            cpa().cp_lse_merge(*acc, out, lse)
    check_fwd(q, k, v, scale, rule, acc[0].cpu(), acc[1].cpu(), "ring")
    dq = torch.zeros((B, S, H, D), device="cuda")
    dks, dvs = [], []
    for off, n in table:
        part = [torch.empty(s, device="cuda") for s in ((B, S, H, D), (B, n, Hkv, D), (B, n, Hkv, D))]
        cpa().cp_scored_attn_bwd(qd, kd[:, off:off + n].contiguous(), vd[:, off:off + n].contiguous(), acc[0], gd,
                                 acc[1], *part, scale, kv_pos0=off, **r)
        dq += part[0]
        dks.append(part[1])
        dvs.append(part[2])
    grads = [dq.cpu(), torch.cat(dks, 1).cpu(), torch.cat(dvs, 1).cpu()]
    check_bwd(q, k, v, acc[0].cpu(), dout, acc[1].cpu(), scale, rule, grads, "ring")


def test_results_repeat_and_streams_and_graphs():
    """The same bits again: on another stream, from the caller's workspace, and replayed from a graph on new inputs."""
    B, S, H, Hkv, D = 2, 200, 4, 2, 128
    ids = docs(B, S, 3, 9, 4).cuda()
    rule = dict(causal=True, softcap=20.0, q_docs=ids, kv_docs=ids)
    sets = [[t.cuda() for t in draw(B, S, S, H, Hkv, D, BF, seed=s)] for s in (21, 22)]

    def outputs():
        return [torch.empty((B, S, H, D), dtype=BF, device="cuda"), torch.empty((B, H, S), device="cuda"),
                torch.empty((B, S, H, D), dtype=BF, device="cuda")] + [
                    torch.empty((B, S, Hkv, D), dtype=BF, device="cuda") for _ in range(2)]

    def step(x, y, **kw):
        q, k, v, g = x
        cpa().cp_scored_attn_fwd(q, k, v, y[0], y[1], 0.1, **rule, **kw.get("f", {}))
        cpa().cp_scored_attn_bwd(q, k, v, y[0], g, y[1], *y[2:], 0.1, **rule, **kw.get("b", {}))

    want = []
    for x in sets:
        y = outputs()
        step(x, y)
        want.append(y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = outputs()
    fw = torch.empty(cpa().cp_scored_attn_workspace_size(B, H, S, S, True), dtype=torch.uint8, device="cuda")
    bw = torch.empty(cpa().cp_scored_attn_bwd_workspace_size(B, H, S, S, True), dtype=torch.uint8, device="cuda")
    step(sets[0], y, f=dict(stream=side, workspace=fw), b=dict(stream=side.cuda_stream, workspace=bw))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(y, want[0]))
    x, y = [t.clone() for t in sets[0]], outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x, y)
    for s, w in zip(sets[::-1], want[::-1]):
        for a, b in zip(x, s):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(y, w))


def test_wrapper_refusals():
    q = torch.zeros((1, 8, 4, 64), dtype=BF, device="cuda")
    k = torch.zeros((1, 8, 2, 64), dtype=BF, device="cuda")
    lse = torch.zeros((1, 4, 8), device="cuda")
    f = lambda q=q, k=k, v=k, o=q, l=lse, **kw: cpa().cp_scored_attn_fwd(q, k, v, o, l, 0.1, **kw)
    ids = torch.zeros((1, 8), dtype=torch.int32, device="cuda")
    for bad in (dict(k=k[:, :, :1]), dict(l=lse[:, :, :4]), dict(o=q[:, :4]), dict(q=q.transpose(1, 2)),
                dict(slopes=lse[0, 0]), dict(q_docs=ids), dict(q_docs=ids, kv_docs=ids[:, :4]),
                dict(prefix_lens=ids), dict(stream=None, workspace=torch.zeros(8)[::2])):
        if "workspace" in bad:
            bad.update(q_docs=ids, kv_docs=ids)
        with pytest.raises(ValueError):
            f(**bad)
    for bad in (dict(k=k.float()), dict(o=q.half()), dict(l=lse.half()), dict(q_docs=ids.long(), kv_docs=ids)):
        with pytest.raises(TypeError):
            f(**bad)
    with pytest.raises(cpa().CpError):
        f(prefix_lens=ids[0, :1].contiguous())
    g = [torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(k)]
    with pytest.raises(TypeError):
        cpa().cp_scored_attn_bwd(q, k, k, q, q, lse, g[0].float(), g[1], g[2], 0.1)
    with pytest.raises(ValueError):
        cpa().cp_scored_attn_bwd(q, k, k, q, q, lse, g[0], g[1][:, :4], g[2], 0.1)


@pytest.mark.parametrize("dt", [F4, BF])
@pytest.mark.parametrize("Sq,Skv,H,Hkv,D", [(1, 1500, 2, 1, 64), (5, 1100, 1, 1, 128), (1500, 3, 16, 1, 64),
                                            (700, 1, 8, 1, 128)])
def test_clusters_on_a_handful_of_rows_or_keys(Sq, Skv, H, Hkv, D, dt):
    """Clusters that join fewer rows than they have CTAs or threads."""
    rule = dict(softcap=20.0, slopes=slopes(H), q_pos0=max(Skv - Sq, 0))
    q, k, v, dout = draw(1, Sq, Skv, H, Hkv, D, dt, seed=Sq + Skv)
    out, lse = run_fwd(q, k, v, D ** -0.5, rule, dt)
    check_fwd(q, k, v, D ** -0.5, rule, out, lse, "handful")
    grads = run_bwd(q, k, v, out, dout, lse, D ** -0.5, rule, dt)
    check_bwd(q, k, v, out, dout, lse, D ** -0.5, rule, grads, "handful")


@pytest.mark.parametrize("dt", [F4, BF])
@pytest.mark.parametrize("D,slope", [(64, False), (128, True)])
@pytest.mark.parametrize("low,high", [(0.3, 1.5), (4.0, 4.0), (6.5, 6.5), (9.0, 9.0), (4.0, 9.0)])
def test_gradients_of_saturated_scores(low, high, D, slope, dt):
    """Every pair far into the cap's flat part, |x / cap| from low to high: the gradients are small there, and hold
    their digits. With y = x / cap known to (D + 20) u |y| the derivative 1 - tanh^2, whose logarithm's slope in y is
    at most 2, is off by 2 (D + 20) u |y| relative, and by 8 |y| u + 32 u for its own evaluation (an exponential of 2 |y|,
    a quotient, three products); the rest is as in the module's E, the second term times the derivative."""
    B, S, H, Hkv, cap = 1, 200, 4, 2, 2.0
    scale = D ** -0.5
    q, k, v, dout = draw(B, S, S, H, Hkv, D, dt, seed=int(10 * high) + D)
    level = torch.linspace(low, high, S)[torch.randperm(S, generator=torch.Generator().manual_seed(3))]
    sign = torch.where(torch.arange(S) % 3 == 0, -1.0, 1.0)
    q = ((level * sign * cap / (scale * D))[None, :, None, None] + 0.02 * q.float()).to(dt)
    k = (1.0 + 0.03 * k.float()).to(dt)
    rule = dict(softcap=cap, causal=True)
    if slope:
        rule["slopes"] = slopes(H)
    out, lse = run_fwd(q, k, v, scale, rule, dt)
    check_fwd(q, k, v, scale, rule, out, lse, "saturated")
    grads = run_bwd(q, k, v, out, dout, lse, scale, rule, F4)
    want = so.scored_attention_bwd(q, k, v, out, dout, lse, scale, **rule)
    d, e, n = errors_of(q, k, scale, rule)
    w = 2.0 ** -8 if dt == BF else 0.0
    qf, kf, vf, of, gf, lf = (t.double().numpy() for t in (q, k, v, out, dout, lse))
    bound = [np.zeros_like(x) for x in want[:2]]
    for h in range(H):
        p, dcap = probs(q, k, lf, 0, h, scale, rule)
        g, vv = gf[0, :, h], vf[0, :, h // 2]
        y = np.abs(scale * qf[0, :, h] @ kf[0, :, h // 2].T) / cap
        rel = 2 * (D + 20) * U * (scale * np.abs(qf[0, :, h]) @ np.abs(kf[0, :, h // 2]).T) / cap + (8 * y + 32) * U
        ds = p * (g @ vv.T - np.sum(g * of[0, :, h], 1)[:, None]) * dcap
        ga = np.abs(g)
        E = (w + e + rel) * np.abs(ds) + p * dcap * (D + 8) * U * (ga @ np.abs(vv).T + np.sum(ga * np.abs(of[0, :, h]), 1)[:, None])
        bound[0][0, :, h] = scale * (E @ np.abs(kf[0, :, h // 2]))
        bound[1][0, :, h // 2] += scale * (E.T @ np.abs(qf[0, :, h]))
    for name, x, z, bd in zip(("dq", "dk"), grads, want, bound):
        x = x.double().numpy()
        over = np.abs(x - z) - bd - 2 * U * np.abs(z)
        assert np.all(np.isfinite(x)) and over.max() <= 0, (
            f"{name}: past its bound by {over.max():.3e} of {bd.flat[over.argmax()]:.3e}")


def test_a_long_row_of_heavy_weights_and_large_values():
    """2^21 keys, each of weight 2^12.9 before the division, and v = 2^96, the largest that the header allows: the
    sum of the products would pass fp32's range with the reference of the first tile. All keys are alike, so out is v
    but for the roundings of P and of itself, and lse the score plus ln 2^21 (within the module's bound, whose n u is
    taken for the 2^14 tiles' sums of 2^7 keys each)."""
    n, D = 1 << 21, 64
    q = torch.full((1, 1, 1, D), 1.1171875, dtype=BF, device="cuda")
    k, v = torch.ones((1, n, 1, D), dtype=BF, device="cuda"), torch.full((1, n, 1, D), 2.0 ** 96, dtype=BF, device="cuda")
    out, lse = torch.empty((1, 1, 1, D), device="cuda"), torch.empty((1, 1, 1), device="cuda")
    cpa().cp_scored_attn_fwd(q, k, v, out, lse, D ** -0.5)
    assert cpa().cp_check_device_status() == 0
    x = 1.1171875 * D * D ** -0.5
    want = x + n.bit_length() * np.log(2.0) - np.log(2.0)
    d, sums = (D + 20) * U * x, (2 ** 14 + 2 ** 7) * U
    assert abs(lse.item() - want) <= 2 * d + 2.0 ** -20 + sums + 4 * U * want
    off = (out.double() / 2.0 ** 96 - 1).abs().max().item()
    assert off <= 2.0 ** -8 + 2 * (2 * d + 2.0 ** -21 + sums) + 2 * U, off


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n,at", [(300000, 150001), (600000, 393300), (1 << 21, (1 << 20) + 700), (1 << 21, 0),
                                  (1 << 21, (1 << 21) - 150)])
def test_documents_and_slopes_among_more_keys_than_one_bitmap_bit_each(n, at, causal):
    """With slopes the tiles are walked from the rows' position outwards, here with a bit of the bitmap for 2, 4 or 8
    tiles, from the middle of a group, the first key and the last; bounds as without slopes, with 4 u of the bias."""
    B, S, H, D, every = 1, 150, 2, 64, 64 * 1024
    g = torch.Generator(device="cuda").manual_seed(n + at)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)
    q, k, v = r(B, S, H, D), r(B, n, 1, D), r(B, n, 1, D)
    slope = torch.tensor([2e-6, -1e-6], device="cuda")
    pos, rows = torch.arange(n, device="cuda"), torch.arange(S, device="cuda")
    near = (pos >= at - 700) & (pos < at + 900)   # keys around the rows are of the rows' documents too
    kd = torch.where((pos % every < 300) | near, (pos // 50) % 3, 10 + pos // 1000).to(torch.int32)[None].contiguous()
    qd = (rows // 10 % 4).to(torch.int32)[None].contiguous()   # 3: no key at all
    out, lse = torch.empty_like(q, dtype=F4), torch.empty((B, H, S), device="cuda")
    cpa().cp_scored_attn_fwd(q, k, v, out, lse, D ** -0.5, slopes=slope, causal=causal, q_pos0=at, q_docs=qd, kv_docs=kd)
    assert cpa().cp_check_device_status() == 0
    keys = (kd[0] < 3).nonzero()[:, 0]
    kf, vf = k[0, keys, 0].double(), v[0, keys, 0].double()
    back = (at + rows)[:, None] - keys[None]
    keep = qd[0][:, None] == kd[0, keys][None]
    if causal:
        keep &= back >= 0
    m = len(keys)
    for h in range(H):
        x = (q[0, :, h].double() @ kf.T) * D ** -0.5 - slope[h].double() * back.abs().double()
        big = (q[0, :, h].double().abs() @ kf.abs().T).max().item() * D ** -0.5 + 2e-6 * n
        x = x.masked_fill(~keep, -float("inf"))
        wl = torch.logsumexp(x, 1)
        none = torch.isneginf(wl)
        assert none.any() and torch.equal(torch.isneginf(lse[0, h]), none) and (out[0, none, h] == 0).all()
        p = torch.exp(x - torch.where(none, torch.zeros_like(wl), wl)[:, None])
        d = (D + 20) * U * big
        e = 2 * (2 * d + 2.0 ** -21 + m * U)
        over = (out[0, :, h].double() - p @ vf).abs() - (2.0 ** -8 + e) * (p @ vf.abs()) - 2 * U * (p @ vf).abs()
        assert over.max().item() <= 0
        ok = ~none
        assert ((lse[0, h].double() - wl)[ok].abs() <= 2 * d + 2.0 ** -20 + m * U + 4 * U * wl[ok].abs()).all()


def test_two_streams_at_once():
    """Forward, backward and decode of two users on two streams at the same time: the bits of each alone."""
    D, page = 64, 16

    def user(seed, S, H, Hkv):
        x = [t.cuda() for t in draw(2, S, S, H, Hkv, D, BF, seed=seed)]
        ids = docs(2, S, 3, 9, seed).cuda()
        tab = torch.arange(2 * (-(-S // page)), dtype=torch.int32, device="cuda").view(2, -1)
        kc, vc = (torch.zeros((tab.numel(), page, Hkv, D), dtype=BF, device="cuda") for _ in range(2))
        zero, full = (torch.full((2,), n, dtype=torch.int32, device="cuda") for n in (0, S))
        return dict(x=x, rule=dict(causal=True, softcap=10.0, q_docs=ids, kv_docs=ids), tab=tab, cache=(kc, vc), zero=zero,
                    full=full)

    def step(u):
        q, k, v, g = u["x"]
        out, lse = torch.empty_like(q), torch.empty((2, q.shape[2], q.shape[1]), device="cuda")
        grads = [torch.empty_like(t) for t in (q, k, v)]
        cpa().cp_scored_attn_fwd(q, k, v, out, lse, 0.1, **u["rule"])
        cpa().cp_scored_attn_bwd(q, k, v, out, g, lse, *grads, 0.1, **u["rule"])
        cpa().cp_paged_kv_append(k, v, *u["cache"], u["tab"], u["zero"])
        o, l = torch.empty_like(q[:, -1].contiguous()), torch.empty((2, q.shape[2]), device="cuda")
        cpa().cp_paged_attn_decode(q[:, -1].contiguous(), *u["cache"], u["tab"], u["full"], o, l, 0.1, softcap=10.0)
        return [out, lse, *grads, o, l]

    users = [user(31, 700, 8, 2), user(32, 1500, 4, 4)]
    want = [step(u) for u in users]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in users]
    got = []
    for _ in range(10):
        for u, s in zip(users, streams):
            with torch.cuda.stream(s):
                got.append(step(u))
    torch.cuda.synchronize()
    assert cpa().cp_check_device_status() == 0
    for i, y in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(y, want[i % 2]))


@pytest.mark.parametrize("name", ["causal, cap", "documents"])
def test_gradients_of_more_items_than_multiprocessors_repeat(name):
    """The backward at D = 128 with more items than run at once, against its bounds, and the same bits again."""
    B, S, H, Hkv, D = 4, 300, 40, 8, 128
    rule = MANY[name](B, S)
    q, k, v, dout = draw(B, S, S, H, Hkv, D, BF, seed=D, qmul=1.5)
    out, lse = run_fwd(q, k, v, D ** -0.5, rule, BF)
    grads = run_bwd(q, k, v, out, dout, lse, D ** -0.5, rule, BF)
    check_bwd(q, k, v, out, dout, lse, D ** -0.5, rule, grads, name)
    again = run_bwd(q, k, v, out, dout, lse, D ** -0.5, rule, BF)
    assert all(torch.equal(x, y) for x, y in zip(grads, again))
