"""Head norm with rotary positions against the float64 oracle, element by element.

With u = 2^-24 and r half a step of the result's type (bf16 2^-8, fp32 u):
* 1 / sqrt(mean + eps): the sum of D squares takes 8 additions in a lane and at most 4
  by shuffles, each product and sum off by u, half of it after the root; the root itself
  by 2 steps (4 u); times x and the weight 2 u: together 14 u of |y|;
* cos and sin: the turn's 32 bits 2^-32 pi, its rounding to 24 bits and the products 4 u,
  the series' rest 2.5e-8: together below e = 3e-7, of both members of the pair; the
  rotation's own products and sum 3 u;
so |result - ref| <= (|u| + |v|) (e + 17 u) + r |ref| for a pair (u, v) of y, and r |ref|
+ 14 u |y| behind the pairs.
Backward: the rotated gradient g is off by d = (|g_u| + |g_v|) (e + 3 u); the row's sum of
g w x by sum |w x| d + 14 u sum |g w x|; and with n = 1 / sqrt(...):
  |dx - ref| <= n |w| d + n^3 |x| (sum |w x| d + 14 u sum |g w x|) / D
                + 40 u (n |g w| + n^3 |x| |sum g w x| / D) + r |ref|
  |dw - ref| <= sum over rows of |x n| d + 192 u sum |g x n|
(a lane sums at most 128 rows here, then come at most 64 more additions).
"""
import numpy as np
import pytest
import torch

from oracle import qk as oq

pytestmark = pytest.mark.gpu

BF, F4 = torch.bfloat16, torch.float32
U = 2.0 ** -24
E = 3e-7


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from context_attention_dits_gb300 import build
    build.build()


def cpa():
    import context_attention_dits_gb300 as m
    return m


def half_step(dt):
    return 2.0 ** -8 if dt == BF else U


def make(B, S, H, Hkv, D, dt, pairs, axes, seed, far=100, eps=1e-6, wdt=None, inter=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    s = dict(q=(r(B, S, H, D) * 2).to(dt), k=(r(B, S, Hkv, D) * 2).to(dt), gq=r(B, S, H, D).to(dt),
             gk=r(B, S, Hkv, D).to(dt), eps=eps, inter=inter, q_weight=None, k_weight=None,
             freqs=torch.tensor([10000.0 ** (-i / max(pairs, 1)) for i in range(pairs)], dtype=torch.float64),
             positions=torch.randint(-far, far + 1, (B, S, axes), generator=g, dtype=torch.int32),
             axes=bytes(torch.randint(0, axes, (pairs,), generator=g).tolist()))
    if wdt is not None:
        s["q_weight"], s["k_weight"] = (1 + 0.3 * r(D)).to(wdt), (1 + 0.3 * r(D)).to(wdt)
    return s


def kw(s):
    c = lambda t: None if t is None else t.cuda()
    return dict(positions=c(s["positions"]), freqs=c(s["freqs"]), axes=s["axes"], interleaved=s["inter"], eps=s["eps"],
                q_weight=c(s["q_weight"]), k_weight=c(s["k_weight"]))


def turns(s):
    p = s["positions"]
    if p.dim() == 2:
        p = p[None].expand(s["q"].shape[0], -1, -1)
    return oq.angles(p, s["freqs"], s["axes"])


def partner_sum(y, pairs, inter):
    """|u| + |v| of each value's pair (its own size behind the pairs)."""
    a = np.abs(y)
    b = a.copy()
    if inter:
        b[..., 0:2 * pairs:2] += a[..., 1:2 * pairs:2]
        b[..., 1:2 * pairs:2] += a[..., 0:2 * pairs:2]
    else:
        b[..., :pairs] += a[..., pairs:2 * pairs]
        b[..., pairs:2 * pairs] += a[..., :pairs]
    return b


def within(got, ref, bound, what):
    over = np.abs(got.detach().cpu().double().numpy() - ref) - bound
    assert np.isfinite(over).all() and over.max() <= 0, f"{what}: past its bound by {over.max():.3e}"


def check_fwd(s, x, w, got, what):
    t, pairs = turns(s), len(s["freqs"])
    y = oq.forward(x, t[:, :, :0], s["inter"], s["eps"], w)
    ref = oq.rotate(y, t, s["inter"])
    within(got, ref, partner_sum(y, pairs, s["inter"]) * (E + 17 * U) + half_step(got.dtype) * np.abs(ref), what)


def check_bwd(s, x, w, grad, got, dw, what):
    t, pairs, D = turns(s), len(s["freqs"]), x.shape[-1]
    dx, dwr = oq.backward(x, grad, t, s["inter"], s["eps"], w)
    g = oq.rotate(grad.cpu().double().numpy(), -t, s["inter"])
    d = partner_sum(g, pairs, s["inter"]) * (E + 3 * U)
    r = half_step(got.dtype)
    if s["eps"] is None:
        within(got, dx, d + r * np.abs(dx), what)
        return
    x = x.cpu().double().numpy()
    n = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + s["eps"])
    wv = np.ones(D) if w is None else w.double().numpy()
    row = lambda a: a.sum(-1, keepdims=True)
    off = row(np.abs(wv * x) * d) + 14 * U * row(np.abs(g * wv * x))
    bound = (n * np.abs(wv) * d + n ** 3 * np.abs(x) * off / D +
             40 * U * (n * np.abs(g * wv) + n ** 3 * np.abs(x) * np.abs(row(g * wv * x)) / D) + r * np.abs(dx))
    within(got, dx, bound, what)
    if dw is not None:
        all_rows = (0, 1, 2)
        within(dw, dwr, (np.abs(x * n) * d).sum(all_rows) + 192 * U * np.abs(g * x * n).sum(all_rows) + U * np.abs(dwr),
               what + " weight")


def run_fwd(s, q=None, k=None):
    q, k = s["q"].cuda() if q is None else q, s["k"].cuda() if k is None else k
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    cpa().cp_qk_norm_rope_fwd(q, k, qo, ko, **kw(s))
    torch.cuda.synchronize()
    return qo, ko


def run_bwd(s, gdt=None, weights=True):
    q, k = s["q"].cuda(), s["k"].cuda()
    gq, gk = (s[n].cuda().to(gdt or q.dtype) for n in ("gq", "gk"))
    dq, dk = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    D = q.shape[3]
    ws = [torch.full((D,), 7.0, device="cuda") for _ in range(2)] if weights and s["eps"] is not None else [None, None]
    cpa().cp_qk_norm_rope_bwd(q, k, gq, gk, dq, dk, dq_weight=ws[0], dk_weight=ws[1], **kw(s))
    torch.cuda.synchronize()
    return dq, dk, *ws


def check_all(s, what, gdt=None):
    qo, ko = run_fwd(s)
    check_fwd(s, s["q"], s["q_weight"], qo, what + " q")
    check_fwd(s, s["k"], s["k_weight"], ko, what + " k")
    dq, dk, wq, wk = run_bwd(s, gdt)
    check_bwd(s, s["q"], s["q_weight"], s["gq"], dq, wq, what + " dq")
    check_bwd(s, s["k"], s["k_weight"], s["gk"], dk, wk, what + " dk")


SIZES = {
    "one token": (1, 1, 1, 1),
    "odd heads": (2, 5, 3, 1),
    "more heads than a warp's rows": (1, 37, 24, 8),
    "token of many sequences": (65, 1, 8, 2),
    "no even part": (3, 131, 7, 7),
    "many tokens": (1, 1500, 2, 1),
}


@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("D,dt,pairs,axes,inter,wdt", [
    (128, BF, 64, 3, True, BF),
    (128, BF, 64, 3, False, F4),
    (64, BF, 32, 1, False, BF),
    (64, BF, 32, 2, True, None),
    (64, BF, 4, 4, False, BF),
    (128, BF, 20, 2, False, BF),
    (128, F4, 64, 1, False, F4),
    (64, F4, 8, 3, True, F4),
    (128, F4, 0, 1, False, None),
    (64, BF, 0, 1, True, BF),
])
def test_forward_and_backward(name, D, dt, pairs, axes, inter, wdt):
    check_all(make(*SIZES[name], D, dt, pairs, axes, seed=len(name) + D, wdt=wdt, inter=inter), name)


@pytest.mark.parametrize("dt,gdt", [(BF, BF), (BF, F4), (F4, F4)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("eps", [None, 0.0, 1e-6, 10.0])
def test_norm_or_none(eps, inter, dt, gdt):
    s = make(2, 19, 5, 2, 64, dt, 16, 2, seed=3, eps=eps, wdt=None if eps is None else dt, inter=inter)
    check_all(s, f"eps {eps}", gdt)


@pytest.mark.parametrize("dt", [BF, F4])
@pytest.mark.parametrize("inter", [False, True])
def test_far_positions(inter, dt):
    """As good at the ends of 32 bits as near 0; frequencies of whole turns, above one turn, negative, 0 and tiny."""
    s = make(1, 40, 3, 1, 64, dt, 32, 1, seed=8, inter=inter)
    s["positions"] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30, 12345678, -7], dtype=torch.int32).repeat(5).view(1, 40, 1)
    # (5e-324 counts as 0, which at these positions it is)
    s["freqs"][:11] = torch.tensor([2 * np.pi, np.pi, 100.0, -0.5, 0.0, 1e-300, -100.0, -1e-9, 6.25, 2.0 ** -60, 5e-324])
    check_all(s, "far")


def test_values_of_any_size():
    """Zero rows, rows of one value, tiny and large ones."""
    s = make(1, 6, 2, 1, 64, F4, 32, 1, seed=2)
    s["q"][0, 0] = 0
    s["q"][0, 1] *= 1e-18
    s["q"][0, 2] *= 1e15
    s["q"][0, 3, :, 1:] = 0
    s["q"][0, 4] = 3.0
    check_all(s, "sizes")
    # a row of zeros has no direction without eps: NaN there, and nowhere else
    s["eps"], s["q"][0, 1:] = 0.0, 1.0
    q, k = run_fwd(s)
    assert torch.isnan(q[0, 0]).all() and torch.isfinite(q[0, 1:]).all() and torch.isfinite(k).all()
    s["q"][0, 0] = 2.0
    s["q"][0, 3, 1, 5] = float("nan")
    s["q"][0, 4, 0, 9] = float("inf")
    q, k = run_fwd(s)
    ok = torch.ones((1, 6, 2), dtype=torch.bool, device="cuda")
    ok[0, 3, 1] = ok[0, 4, 0] = False
    assert torch.isfinite(q[ok]).all() and torch.isfinite(k).all() and not torch.isfinite(q[0, 3, 1]).any()


def packed(s, dt):
    """q, k as parts of a packed projection, and dense results' places in a wider buffer."""
    B, S, H, D = s["q"].shape
    Hkv = s["k"].shape[2]
    buf = torch.full((B, S, H + 2 * Hkv + 1, D), 7.0, dtype=dt, device="cuda")
    q, k = buf[:, :, :H], buf[:, :, H + 1:H + 1 + Hkv]
    q.copy_(s["q"])
    k.copy_(s["k"])
    return buf, q, k


@pytest.mark.parametrize("dt", [BF, F4])
@pytest.mark.parametrize("inter", [False, True])
def test_strides_in_place_and_broadcast(inter, dt):
    s = make(3, 21, 6, 2, 128, dt, 32, 2, seed=5, wdt=dt, inter=inter)
    want = run_fwd(s)
    grads = run_bwd(s)
    buf, q, k = packed(s, dt)
    got = run_fwd(s, q, k)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # heads before tokens, on both sides
    q2, k2 = (s[n].cuda().transpose(1, 2).contiguous().transpose(1, 2) for n in ("q", "k"))
    o = [torch.empty_like(x).transpose(1, 2).contiguous().transpose(1, 2) for x in (q2, k2)]
    cpa().cp_qk_norm_rope_fwd(q2, k2, *o, **kw(s))
    assert all(torch.equal(a, b) for a, b in zip(o, want))
    # in place, within the packed buffer; the rest of it stays
    cpa().cp_qk_norm_rope_fwd(q, k, q, k, **kw(s))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert (buf[:, :, 6] == 7).all() and (buf[:, :, 9:] == 7).all()
    # gradients in place of the results' gradients, and of the rows
    buf, q, k = packed(s, dt)
    gq, gk = s["gq"].cuda(), s["gk"].cuda()
    w = [torch.empty(128, device="cuda") for _ in range(2)]
    cpa().cp_qk_norm_rope_bwd(q, k, gq, gk, gq, gk, dq_weight=w[0], dk_weight=w[1], **kw(s))
    assert all(torch.equal(a, b) for a, b in zip((gq, gk, *w), grads))
    cpa().cp_qk_norm_rope_bwd(q, k, s["gq"].cuda(), s["gk"].cuda(), q, k, dq_weight=w[0], **kw(s))
    assert torch.equal(q, grads[0]) and torch.equal(k, grads[1]) and torch.equal(w[0], grads[2])
    assert (buf[:, :, 6] == 7).all() and (buf[:, :, 9:] == 7).all()
    # rows and gradients that are broadcast, positions that all batch entries share
    one = dict(s, q=s["q"][:1].cuda().expand(3, -1, -1, -1), gk=s["gk"][:, :, :1].cuda().expand(-1, -1, 2, -1),
               positions=s["positions"][1].contiguous())
    check_all(one, "broadcast")
    q = s["q"][:1].cuda().expand(3, -1, -1, -1)
    with pytest.raises(cpa().CpError):   # results that share rows
        cpa().cp_qk_norm_rope_fwd(s["q"].cuda(), s["k"].cuda(), q, torch.empty_like(k2), **kw(s))


@pytest.mark.parametrize("dt,gdt", [(BF, BF), (BF, F4), (F4, F4)])
@pytest.mark.parametrize("D,H,Hkv", [(128, 20, 9), (64, 33, 3)])
def test_many_batches_a_warp(D, H, Hkv, dt, gdt):
    """Warps that take several tokens of several batches of heads: dense, in place, and heads that do not lie side by side."""
    s = make(1, 6001, H, Hkv, D, dt, D // 4, 2, seed=9, wdt=F4)
    check_all(s, "dense", gdt)
    want, grads = run_fwd(s), run_bwd(s, gdt)
    q, k = s["q"].cuda(), s["k"].cuda()
    cpa().cp_qk_norm_rope_fwd(q, k, q, k, **kw(s))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    apart = dict(s, **{n: s[n].cuda().transpose(1, 2).contiguous().transpose(1, 2) for n in ("q", "k", "gq", "gk")})
    assert all(torch.equal(a, b) for a, b in zip(run_fwd(apart), want))
    assert all(torch.equal(a, b) for a, b in zip(run_bwd(apart, gdt), grads))
    q, k, gq, gk = (s[n].cuda() for n in ("q", "k", "gq", "gk"))
    if gdt == dt:   # over the results' gradients
        cpa().cp_qk_norm_rope_bwd(q, k, gq, gk, gq, gk, **kw(s))
        assert torch.equal(gq, grads[0]) and torch.equal(gk, grads[1])
    assert cpa().cp_check_device_status() == 0


def test_offsets_past_32_bits():
    s = make(2, 3, 4, 1, 64, BF, 32, 1, seed=8, wdt=BF)
    want, grads = run_fwd(s), run_bwd(s)
    wide = 1 << 32   # elements from one batch entry to the next
    buf = torch.empty(wide + (1 << 16), dtype=BF, device="cuda")

    def far(x, at):
        y = buf.as_strided(x.shape, (wide, *x.stride()[1:]), at)
        y.copy_(x)
        return y

    q, k, gq, gk = (far(s[n].cuda(), i << 13) for i, n in enumerate(("q", "k", "gq", "gk")))
    o = [far(torch.zeros_like(x), (4 + i) << 13) for i, x in enumerate((q.contiguous(), k.contiguous()))]
    cpa().cp_qk_norm_rope_fwd(q, k, *o, **kw(s))
    assert all(torch.equal(a, b) for a, b in zip(o, want))
    w = [torch.empty(64, device="cuda") for _ in range(2)]
    cpa().cp_qk_norm_rope_bwd(q, k, gq, gk, *o, dq_weight=w[0], dk_weight=w[1], **kw(s))
    assert all(torch.equal(a, b) for a, b in zip((*o, *w), grads))


@pytest.mark.parametrize("dt", [BF, F4])
def test_queries_alone_and_nothing_at_all(dt):
    s = make(2, 9, 3, 1, 64, dt, 32, 1, seed=6, wdt=F4)
    want, grads = run_fwd(s), run_bwd(s)
    q, gq = s["q"].cuda(), s["gq"].cuda()
    o, dq, w = torch.empty_like(q), torch.empty_like(q), torch.empty(64, device="cuda")
    cpa().cp_qk_norm_rope_fwd(q, None, o, None, **kw(s))
    cpa().cp_qk_norm_rope_bwd(q, None, gq, None, dq, None, dq_weight=w, **kw(s))
    assert torch.equal(o, want[0]) and torch.equal(dq, grads[0])
    within(w, grads[2].double().cpu().numpy(), 64 * U * 200, "weight of queries alone")
    none = dict(s, q=s["q"][:, :0], k=s["k"][:, :0], gq=s["gq"][:, :0], gk=s["gk"][:, :0], positions=s["positions"][:, :0])
    qo, ko = run_fwd(none)
    assert qo.numel() == 0 and ko.numel() == 0
    assert all((x == 0).all() for x in run_bwd(none)[2:])   # no rows, no gradient
    a, b = run_bwd(s, weights=False)[:2]
    assert torch.equal(a, grads[0]) and torch.equal(b, grads[1])


def test_gradient_by_differences():
    """Along random directions, fp32: the forward's own change, its error some 1e-6 of |result| over the step."""
    s = make(2, 30, 4, 2, 64, F4, 24, 3, seed=12, wdt=F4)
    dq, dk, wq, wk = (x.double().cpu() for x in run_bwd(s))
    g = torch.Generator().manual_seed(1)
    loss = lambda s: sum(float((o.double().cpu() * s[n].double()).sum()) for o, n in zip(run_fwd(s), ("gq", "gk")))
    for name, d in (("q", dq), ("k", dk), ("q_weight", wq), ("k_weight", wk)):
        v = torch.randn(d.shape, generator=g)
        h = 2.0 ** -6
        up, down = dict(s), dict(s)
        up[name], down[name] = s[name] + h * v, s[name] - h * v
        # rounding: 17 u |y| |g| over all values and 2 h; the third derivative: h^2 of some multiples of |v|^3
        slope, want = (loss(up) - loss(down)) / (2 * h), float((d * v.double()).sum())
        size = float(s["gq"].abs().sum() + s["gk"].abs().sum()) * 4
        assert abs(slope - want) <= size * 20 * U / h + h * h * size, name


def test_repeats_streams_and_graphs():
    s = make(1, 700, 6, 2, 128, BF, 64, 3, seed=7, wdt=BF, inter=True)
    want, grads = run_fwd(s), run_bwd(s)
    assert all(torch.equal(a, b) for a, b in zip(run_bwd(s), grads))
    q, k, gq, gk = (s[n].cuda() for n in ("q", "k", "gq", "gk"))
    rule = kw(s)
    ws = torch.full((cpa().cp_qk_norm_rope_bwd_workspace_size(128),), 255, dtype=torch.uint8, device="cuda")
    o = [torch.empty_like(x) for x in (q, k, q, k)] + [torch.empty(128, device="cuda") for _ in range(2)]

    def both(**at):
        cpa().cp_qk_norm_rope_fwd(q, k, o[0], o[1], **rule, **at)
        cpa().cp_qk_norm_rope_bwd(q, k, gq, gk, o[2], o[3], dq_weight=o[4], dk_weight=o[5], workspace=ws, **rule, **at)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, (*want, *grads)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(2):
        for x in o:
            x.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, (*want, *grads)))
    s2 = dict(s, positions=s["positions"] + 3)
    rule["positions"].add_(3)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, (*run_fwd(s2), *run_bwd(s2))))


def test_wrapper_refusals():
    s = make(2, 3, 4, 2, 64, BF, 32, 2, seed=1, wdt=BF)
    q, k = s["q"].cuda(), s["k"].cuda()
    rule = kw(s)
    f = lambda q=q, k=k, qo=q, ko=k, **over: cpa().cp_qk_norm_rope_fwd(q, k, qo, ko, **{**rule, **over})
    for bad in (dict(q=q[0]), dict(k=k[:1]), dict(qo=q[:, :2]), dict(k=None), dict(positions=None), dict(freqs=None),
                dict(freqs=rule["freqs"].float()), dict(axes=bytes(5)), dict(positions=rule["positions"][:, :2]),
                dict(positions=rule["positions"].cpu()), dict(q_weight=rule["q_weight"][:5]), dict(eps=None),
                dict(q_weight=rule["q_weight"].float()), dict(q=q.transpose(2, 3)), dict(freqs=rule["freqs"][None])):
        with pytest.raises(ValueError):
            f(**bad)
    for bad in (dict(k=k.float()), dict(qo=q.float()), dict(positions=rule["positions"].long()), dict(q=q.half(), qo=q.half())):
        with pytest.raises(TypeError):
            f(**bad)
    for bad in (dict(axes=bytes([2] * 32)), dict(freqs=rule["freqs"][:6].contiguous(), axes=None), dict(eps=-1.0),
                dict(q=torch.empty(2 * 3 * 4 * 64 + 8, dtype=BF, device="cuda")[4:-4].view(2, 3, 4, 64))):
        with pytest.raises(cpa().CpError):
            f(**bad)
    w = torch.empty(64, device="cuda")
    b = lambda **over: cpa().cp_qk_norm_rope_bwd(q, k, q, k, torch.empty_like(q), torch.empty_like(k), **{**rule, **over})
    with pytest.raises(ValueError):
        b(dq_weight=w[:5])
    with pytest.raises(TypeError):
        cpa().cp_qk_norm_rope_bwd(q, k, q.half(), k.half(), q, k, **rule)
    with pytest.raises(cpa().CpError):
        b(dq_weight=w, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(cpa().CpError):   # a weight's gradient without a norm
        b(dq_weight=w, eps=None, q_weight=None, k_weight=None)


def test_norm_and_rotation_before_attention():
    """What a transformer block does: packed projection -> norm and rotation -> attention, and all gradients back.

    Against the float64 chain; bounds: the rotated rows are off by 2^-8 of themselves (rounded to bf16), which moves
    a score by at most 2^-7 scale sum |q||k| =: m, a weight by twice that, relative; the attention's own rounding of P
    2^-8; values |v|.
    """
    from oracle import scored as so
    B, S, H, Hkv, D = 1, 150, 4, 2, 64
    s = make(B, S, H, Hkv, D, BF, 32, 3, seed=21, wdt=BF, inter=True)
    v = torch.randn((B, S, Hkv, D), generator=torch.Generator().manual_seed(3)).to(BF)
    q, k = run_fwd(s)
    out, lse = torch.empty((B, S, H, D), device="cuda"), torch.empty((B, H, S), device="cuda")
    cpa().cp_scored_attn_fwd(q, k, v.cuda(), out, lse, D ** -0.5, causal=True)
    t = turns(s)
    q8, k8 = (oq.forward(s[n], t, True, s["eps"], s[n + "_weight"]) for n in ("q", "k"))
    want, wl = so.scored_attention(q8, k8, v, D ** -0.5, causal=True)
    m = 2.0 ** -7 * 1.01 * so.abs_products(q8, k8, D ** -0.5)
    top = float(v.abs().max())
    assert np.abs(lse.cpu().double().numpy() - wl).max() <= m + 1e-5
    assert np.abs(out.cpu().double().numpy() - want).max() <= top * (2 * m * (1 + m) + 2.0 ** -8 + 1e-5)
    # gradients: the chain's own calls, by differences of the float64 chain along a direction
    dout = torch.randn((B, S, H, D), generator=torch.Generator().manual_seed(4)).to(BF)
    dq, dk, dv = (torch.empty((B, S, n, D), device="cuda") for n in (H, Hkv, Hkv))
    cpa().cp_scored_attn_bwd(q, k, v.cuda(), out, dout.cuda(), lse, dq, dk, dv, D ** -0.5, causal=True)
    gq, gk = torch.empty_like(q), torch.empty_like(k)
    w = [torch.empty(D, device="cuda") for _ in range(2)]
    cpa().cp_qk_norm_rope_bwd(s["q"].cuda(), s["k"].cuda(), dq, dk, gq, gk, dq_weight=w[0], dk_weight=w[1], **kw(s))
    g8 = so.scored_attention_bwd(q8, k8, v, want, dout, wl, D ** -0.5, causal=True)
    for got, dw, x, n, g in ((gq, w[0], s["q"], "q", g8[0]), (gk, w[1], s["k"], "k", g8[1])):
        dx, dwr = oq.backward(x, g, t, True, s["eps"], s[n + "_weight"])
        # relative 2-norm: P, dS and the rotated rows each rounded to bf16 (2^-8 at most, with room for their products)
        for a, b in ((got, dx), (dw, dwr)):
            err = np.linalg.norm(a.cpu().double().numpy() - b) / np.linalg.norm(b)
            assert err <= 6 * 2.0 ** -8, (n, err)


@pytest.mark.parametrize("dt", [BF, F4])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,pairs", [(64, 0), (64, 8), (128, 28), (128, 60)])
def test_values_behind_the_pairs_keep_their_bits(D, pairs, inter, dt):
    """Without a norm they stay what they are, whatever their neighbours are: infinities, signed zeros, the least numbers."""
    s = make(2, 9, 3, 2, D, dt, pairs, 2, seed=5, eps=None, inter=inter)
    odd = torch.tensor([float("inf"), -float("inf"), 0.0, -0.0, 1e-40, -1e38, 3.0])
    at = torch.randint(0, 14, (2, 9, 3, D), generator=torch.Generator().manual_seed(8))
    for n in ("q", "gq"):
        s[n] = torch.where(at < 7, odd[at % 7], s[n].float()).to(dt)
        s[n][..., :2 * pairs] = 1
    q, k = run_fwd(s)
    dq, dk, _, _ = run_bwd(s)
    bits = torch.int16 if dt == BF else torch.int32
    for got, want in ((q, s["q"]), (k, s["k"]), (dq, s["gq"]), (dk, s["gk"])):
        assert torch.equal(got.cpu()[..., 2 * pairs:].view(bits), want[..., 2 * pairs:].view(bits))


@pytest.mark.parametrize("dt", [BF, F4])
@pytest.mark.parametrize("eps", [0.0, 1e-38, 7e-34, 8e-34, 1e-6, 1e30])
@pytest.mark.parametrize("D,inter", [(64, False), (128, True)])
def test_rows_of_any_size_below_the_largest(D, inter, eps, dt):
    """Rows from 2^-120 to 2^56, beside ordinary ones in the same warp: the norm's direction is that of any other row.

    Sizes whose squares fp32 does not hold, where eps hides that (2^-110 is 7.7e-34) and where it does not.
    """
    s = make(2, 33, 5, 3, D, dt, 16, 1, seed=6, eps=eps, wdt=dt, inter=inter)
    e = torch.randint(-120, 57, (2, 33, 8, 1), generator=torch.Generator().manual_seed(9)).float()
    e[:, ::3] = 0
    for n, x in (("q", slice(0, 5)), ("k", slice(5, 8))):   # gradients as small, so that those of the rows stay within fp32
        s[n] = (s[n].float() * torch.exp2(e[:, :, x])).to(dt)
        s["g" + n] = (s["g" + n].float() * torch.exp2(e[:, :, x])).to(dt)
    qo, ko = run_fwd(s)
    dq, dk, wq, wk = run_bwd(s)
    t, least = turns(s), 2.0 ** -133 if dt == BF else 2.0 ** -149
    for x, w, g, y, dx, dw in ((s["q"], s["q_weight"], s["gq"], qo, dq, wq), (s["k"], s["k_weight"], s["gk"], ko, dk, wk)):
        ref = oq.forward(x, t, inter, eps, w)
        dxr, dwr = oq.backward(x, g, t, inter, eps, w)
        xs = x.double().numpy()
        n = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + eps)
        gs, wv = oq.rotate(g.double().numpy(), -t, inter), w.double().numpy()
        top = lambda a: np.abs(a).max(-1, keepdims=True)
        # fp32 throughout: 2^-18 of a row's largest terms covers its some 64 roundings each way
        r, c = half_step(dt), 2.0 ** -18
        within(y, ref, r * np.abs(ref) + c * top(xs * n * wv) + least, "forward")
        within(dx, dxr, r * np.abs(dxr) + c * n * top(gs * wv) * (1 + (n * top(xs)) ** 2) + least, "gradients")
        within(dw, dwr, c * np.abs(gs * xs * n).sum((0, 1, 2)) + least, "weights' gradients")
