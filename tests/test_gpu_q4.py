"""The paged cache in 4 bits: append bit for bit, read value for value, and decode
against the float64 oracle over the values that the cache stands for.

Bounds of decode, element by element. With u = 2^-24, t = 2^-23 (the matrix
instruction's sums may truncate), n keys, k = z + s c, and for a query head
A = scale max over keys of sum |q| (s c + |z|):
* a score is off by d = (D + 32) t A + 2^-22 A (fp32 q in two parts of 11 bits) + 4 u max|x|;
* a weight, relative, by 2 d, by 2^-21 of the exponential and by n u of the sum;
* the weights times scales are rounded by w (bf16 q: fp16, 2^-11; fp32: 2^-22) and by
  n 2^-36 max s at the least where they are small; sums of p s c and of p s, 8 of which go
  off the first, are formed 32 keys at a time by the instruction (64 t of each) and
  n / 32 times in fp32:
  |out - ref| <= (w + 2 (2 d + 2^-21 + n u)) sum_j p (|s (c - 8)| + |z + 8 s|)
                 + (64 t + n u) sum_j p s (c + 8) + n 2^-36 max s + r |ref|
  |lse - ref| <= 2 d + 2^-20 + n u + 4 u |ref|
"""
import numpy as np
import pytest
import torch

from oracle import q4
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


def make(lens, H, Hkv, D, page, dt, seed, spare=2, most=None, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages = max(1, -(-max(most or 0, *lens) // page))
    total = B * pages + spare
    s = dict(q=torch.randn((B, H, D), generator=g).to(dt), lens=torch.tensor(lens, dtype=torch.int32),
             table=torch.randperm(total, generator=g)[:B * pages].to(torch.int32).view(B, pages).contiguous())
    for x in ("k", "v"):
        size = torch.exp(spread * torch.randn((total, Hkv, page, D // 64, 1), generator=g))
        s[x + "c"] = torch.randint(0, 256, (total, Hkv, page, D // 2), generator=g, dtype=torch.uint8)
        # a normal group's scale and offset: 0.3 and -2.3 or so
        sz = torch.cat((0.2 + 0.2 * torch.rand(size.shape, generator=g), -2.3 + torch.randn(size.shape, generator=g)), -1)
        s[x + "s"] = (sz * size).to(BF)
    return s


CACHE = ("kc", "ks", "vc", "vs", "table")


def decode(s, scale, out_dt, **kw):
    B, H, D = s["q"].shape
    out = torch.full((B, H, D), 7.0, dtype=out_dt, device="cuda")
    lse = torch.full((B, H), 7.0, device="cuda")
    kw = {a: b.cuda() if isinstance(b, torch.Tensor) else b for a, b in kw.items()}
    cpa().cp_paged_attn_decode_q4(s["q"].cuda(), *(s[n].cuda() for n in CACHE), s["lens"].cuda(), out, lse, scale, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def check_decode(s, scale, out, lse, what, softcap=0.0, slopes=None):
    B, H, D = s["q"].shape
    Hkv, page = s["kc"].shape[1], s["kc"].shape[2]
    G = H // Hkv
    w = 2.0 ** -11 if s["q"].dtype == BF else 2.0 ** -22
    r = 2.0 ** -8 if out.dtype == BF else U
    got, gl, table = out.double().numpy(), lse.double().numpy(), s["table"].numpy()
    q = s["q"].double().numpy()
    for b in range(B):
        n = int(s["lens"][b])
        if n == 0:
            assert np.all(got[b] == 0) and np.all(np.isneginf(gl[b])), what
            continue
        at = np.arange(n)
        rows = {x: s[x][torch.from_numpy(table[b, at // page]).long(), :, torch.from_numpy(at % page)]
                for x in ("kc", "ks", "vc", "vs")}
        k, v = q4.values(rows["kc"], rows["ks"]), q4.values(rows["vc"], rows["vs"])
        ks, vs = (np.repeat(rows[x].double().numpy(), 64, axis=-2) for x in ("ks", "vs"))
        kbig = ks[..., 0] * q4.unpack(rows["kc"]) + np.abs(ks[..., 1])
        vbig = np.abs(vs[..., 0] * (q4.unpack(rows["vc"]) - 8)) + np.abs(vs[..., 1] + 8 * vs[..., 0])
        vsum = vs[..., 0] * (q4.unpack(rows["vc"]) + 8)
        for h in range(H):
            hk = h // G
            x, _ = so.scores(q[b][None, None], k[None], 0, h, scale, softcap=softcap, slopes=slopes, q_pos0=n - 1)
            top = x[0].max()
            wl = top + np.log(np.exp(x[0] - top).sum())
            p = np.exp(x[0] - wl)
            want = p @ v[:, hk]
            A = abs(scale) * (kbig[:, hk] @ np.abs(q[b, h])).max()
            d = (D + 32) * 2 * U * A + 2.0 ** -22 * A + 4 * U * (A + np.abs(x[0]).max())
            bound = ((w + 2 * (2 * d + 2.0 ** -21 + n * U)) * (p @ vbig[:, hk]) + (128 + n) * U * (p @ vsum[:, hk]) +
                     n * 2.0 ** -36 * vs[:, hk, :, 0].max() + r * np.abs(want))
            over = np.abs(got[b, h] - want) - bound
            assert over.max() <= 0, f"{what} b{b} h{h}: past its bound by {over.max():.3e}"
            assert abs(gl[b, h] - wl) <= 2 * d + 2.0 ** -20 + n * U + 4 * U * abs(wl), f"{what} lse b{b} h{h}"


# ---------------------------------------------------------------------------
# rows in and out
# ---------------------------------------------------------------------------
def rows_of(kind, shape, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if kind == "ties":      # multiples of half a step of many groups' scales
        x = torch.randint(-8, 9, shape, generator=g) * 0.5
    elif kind == "sizes":   # each group at a size of its own, from 2^-110 to 2^110, some of one value
        e = torch.randint(-110, 111, (*shape[:-1], shape[-1] // 64, 1), generator=g).float()
        x = (x.unflatten(-1, (-1, 64)) * torch.exp2(e))
        x = torch.where(e % 7 == 0, x[..., :1], x).flatten(-2)
    elif kind == "offset":  # far from zero: the difference to the offset is not exact in fp32
        x = x * 1e-3 + torch.randn((*shape[:-1], 1), generator=g) * 1e3
    return x.to(dt)


@pytest.mark.parametrize("kind", ["normal", "ties", "sizes", "offset"])
@pytest.mark.parametrize("dt", [BF, F4])
@pytest.mark.parametrize("B,T,Hkv,D,page,lens,new", [
    (1, 1, 1, 64, 16, [0], None),
    (3, 1, 8, 128, 16, [15, 16, 0], None),
    (2, 37, 3, 64, 32, [5, 100], None),
    (4, 50, 2, 128, 64, [0, 63, 64, 200], [50, 0, 7, 60]),   # 60 > T: all 50
    (2, 5, 1, 64, 256, [0, 251], [-1, 5]),
    (1, 300, 5, 128, 128, [77], None),
])
def test_append_and_read(B, T, Hkv, D, page, lens, new, dt, kind):
    s = make([n + T for n in lens], Hkv, Hkv, D, page, dt, seed=T)
    k, v = rows_of(kind, (B, T, Hkv, D), dt, T + 1), rows_of(kind, (B, T, Hkv, D), dt, T + 2)
    at = torch.tensor(lens, dtype=torch.int32)
    nl = None if new is None else torch.tensor(new, dtype=torch.int32)
    d = {n: s[n].cuda() for n in CACHE}
    cpa().cp_paged_kv_append_q4(k.cuda(), v.cuda(), *d.values(), at.cuda(), new_lens=None if nl is None else nl.cuda())
    assert cpa().cp_check_device_status() == 0
    for x, rows in (("k", k), ("v", v)):
        wc, ws = q4.append(rows, s[x + "c"], s[x + "s"], s["table"], lens, new)
        assert np.array_equal(d[x + "s"].double().cpu().numpy(), ws)
        assert np.array_equal(d[x + "c"].cpu().numpy(), wc)
    # read back: everything, zeros behind; a shorter and a longer buffer
    after = [n + (T if new is None else max(0, min(T, new[b]))) for b, n in enumerate(lens)]
    for T2, odt in ((max(after) + 3, dt), (max(1, max(after) // 2), F4)):
        outs = [torch.full((B, T2, Hkv, D), 7.0, dtype=odt, device="cuda") for _ in range(2)]
        al = torch.tensor([min(n, s["table"].shape[1] * page) for n in after], dtype=torch.int32)
        cpa().cp_paged_kv_read_q4(*d.values(), al.cuda(), *outs)
        assert cpa().cp_check_device_status() == 0
        for x, got in zip("kv", outs):
            vals = torch.from_numpy(q4.as_rows(q4.values(d[x + "c"], d[x + "s"]))).float().to(odt)
            want = torch.zeros_like(got, device="cpu")
            for b in range(B):
                j = torch.arange(min(T2, int(al[b])))
                want[b, :len(j)] = vals[s["table"][b, j // page].long(), j % page]
            assert torch.equal(got.cpu(), want)


def test_each_value_is_within_half_a_step():
    g = torch.Generator().manual_seed(4)
    k = torch.randn((2, 100, 4, 128), generator=g).to(BF)
    s = make([100, 100], 4, 4, 128, 16, BF, seed=1)
    d = {n: s[n].cuda() for n in CACHE}
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    cpa().cp_paged_kv_append_q4(k.cuda(), -k.cuda(), *d.values(), lens)
    out = [torch.empty((2, 100, 4, 128), device="cuda") for _ in range(2)]
    cpa().cp_paged_kv_read_q4(*d.values(), lens + 100, *out)
    for x, got in ((k.float(), out[0]), (-k.float(), out[1])):
        y = x.unflatten(-1, (2, 64))
        # a step is at most 2^-7 above (largest - offset) / 15, the offset at most 2^-7 below the least
        step = (y.amax(-1) - y.amin(-1) * (1 + 2.0 ** -7 * (y.amin(-1) < 0))) / 15 * (1 + 2.0 ** -7)
        off = (got.cpu() - x).abs().unflatten(-1, (2, 64)).amax(-1)
        assert (off <= step / 2 * (1 + 2.0 ** -20) + 2.0 ** -22 * y.abs().amax(-1)).all()


@pytest.mark.parametrize("dt", [BF, F4])
def test_values_that_are_not_finite_stay_in_their_group(dt):
    k = torch.randn((1, 3, 2, 128), generator=torch.Generator().manual_seed(1)).to(dt)
    good = k.clone()
    k[0, 0, 0, 5], k[0, 1, 1, 70], k[0, 2, 0, 127] = float("nan"), float("inf"), float("-inf")
    k[0, 2, 1, 3], k[0, 2, 1, 4] = 3e38, -3e38     # a span that fp32 does not hold
    s = make([3], 2, 2, 128, 16, dt, seed=1)
    outs = []
    for rows in (k, good):
        d = {n: s[n].cuda() for n in CACHE}
        lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        cpa().cp_paged_kv_append_q4(rows.cuda(), good.cuda(), *d.values(), lens)
        o = [torch.empty((1, 3, 2, 128), device="cuda") for _ in range(2)]
        cpa().cp_paged_kv_read_q4(*d.values(), lens + 3, *o)
        outs.append(o)
    bad = torch.zeros((1, 3, 2, 128), dtype=torch.bool)
    bad[0, 0, 0, :64] = bad[0, 1, 1, 64:] = bad[0, 2, 0, 64:] = bad[0, 2, 1, :64] = True
    got = outs[0][0].cpu()
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], outs[1][0].cpu()[~bad])
    assert torch.equal(outs[0][1], outs[1][1])


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
LENS = {
    "one token": [1],
    "short": [5, 1, 16, 17],
    "block edges": [31, 32, 33, 64, 127, 128, 129],
    "ragged with empty": [300, 0, 7, 0, 1000, 64],
    "split over many CTAs": [9000],
    "many short": [3] * 70 + [0, 40] * 10,
    "uneven": [5000, 1, 1, 1, 2500],
}
FORMS = [
    (4, 4, 64, 16, BF, BF),
    (24, 8, 128, 16, BF, F4),
    (20, 1, 128, 32, BF, BF),       # more heads than a unit's rows, two tiles
    (9, 1, 64, 64, BF, BF),         # two tiles, the second of one head
    (33, 1, 128, 16, BF, F4),
    (6, 3, 128, 32, F4, F4),
    (18, 2, 64, 128, F4, F4),       # 9 heads on one: two groups of fp32 rows
]


@pytest.mark.parametrize("name", list(LENS))
@pytest.mark.parametrize("H,Hkv,D,page,dt,out_dt", FORMS)
def test_decode(name, H, Hkv, D, page, dt, out_dt):
    s = make(LENS[name], H, Hkv, D, page, dt, seed=len(name))
    out, lse = decode(s, D ** -0.5, out_dt)
    check_decode(s, D ** -0.5, out, lse, name)
    assert cpa().cp_check_device_status() == 0


def widened(s, tokens):
    """The table with room for more tokens; the columns behind hold no page and are not read."""
    s = dict(s)
    B, pages = s["table"].shape
    extra = max(0, tokens // s["kc"].shape[2] - pages)
    s["table"] = torch.cat([s["table"], torch.full((B, extra), -1, dtype=torch.int32)], 1).contiguous()
    return s


# tables for which clusters of 1 to 16 share a unit, and one that only the list of blocks takes
@pytest.mark.parametrize("tokens", [128, 256, 512, 1024, 4096, 40000])
@pytest.mark.parametrize("H,Hkv,D,page,dt,out_dt", FORMS)
def test_decode_whatever_the_table_holds(tokens, H, Hkv, D, page, dt, out_dt):
    from context_attention_dits_gb300 import cp_paged_attn_q4_workspace_size as size
    lens = [min(tokens, n) for n in (128, 0, 1, 65, 127)]
    s = widened(make(lens, H, Hkv, D, page, dt, seed=tokens), tokens)
    if tokens <= 128 or tokens == 40000:
        assert (size(5, H, Hkv, D, page, s["table"].shape[1], dt) > 0) == (tokens == 40000)
    out, lse = decode(s, D ** -0.5, out_dt, softcap=20.0)
    check_decode(s, D ** -0.5, out, lse, f"{tokens}", 20.0)
    assert cpa().cp_check_device_status() == 0
    s["table"][3, 0] = -7   # sequence 3 loses its first page (all of it, where pages hold 65), the others nothing
    bad, bl = decode(s, D ** -0.5, out_dt, softcap=20.0)
    assert cpa().cp_check_device_status() == -1 and cpa().cp_check_device_status() == 0
    rest = [0, 1, 2, 4]
    assert torch.equal(bad[rest], out[rest]) and torch.equal(bl[rest], lse[rest])
    n = int(s["lens"][3])
    if page >= n:
        assert (bad[3] == 0).all() and torch.isneginf(bl[3]).all()
    else:
        assert (bl[3] < lse[3]).all()


def test_decode_of_an_empty_table():
    s = make([0, 0], 4, 2, 64, 16, BF, seed=0)
    s["table"] = s["table"][:, :0].contiguous()
    out, lse = decode(s, 0.1, BF)
    assert (out == 0).all() and torch.isneginf(lse).all() and cpa().cp_check_device_status() == 0


@pytest.mark.parametrize("dt", [BF, F4])
@pytest.mark.parametrize("cap,bias", [(30.0, False), (0.5, False), (0.0, True), (20.0, True), (1e5, False)])
def test_decode_score_rule(dt, cap, bias):
    H, Hkv, D = 8, 2, 64
    s = make([700, 33, 1, 200], H, Hkv, D, 16, dt, seed=3)
    slopes = torch.exp2(-torch.arange(1, H + 1).float()) if bias else None
    out, lse = decode(s, 0.3, dt, softcap=cap, slopes=slopes)
    check_decode(s, 0.3, out, lse, f"cap {cap} bias {bias}", cap, slopes)


def test_decode_scores_of_fp32_queries():
    """The scores themselves (lse of one token) are as good as fp32 products of q and the cached values, over many.

    The root mean square of the distances from float64 is compared with that of the plain form, which rounds 128 products,
    their sums and 128 values z + s c. Where codes and the upper bits of q are multiplied exactly, the rounding of q's lower
    bits and of some ten operations is left, so it should be below; twice the plain form's is the bound.
    """
    B, H, Hkv, D = 200, 32, 4, 128
    s = make([1] * B, H, Hkv, D, 16, F4, seed=6)
    _, lse = decode(s, D ** -0.5, F4)
    page = s["table"][:, 0].long()
    codes, scales = s["kc"][page, :, 0], s["ks"][page, :, 0]
    k = torch.from_numpy(q4.values(codes, scales)).repeat_interleave(H // Hkv, 1)
    want = (k * s["q"].double()).sum(2) * D ** -0.5
    sz = scales.float().repeat_interleave(64, 2).repeat_interleave(H // Hkv, 1)
    c = torch.from_numpy(q4.unpack(codes)).float().repeat_interleave(H // Hkv, 1)
    plain = ((s["q"] * (sz[..., 1] + sz[..., 0] * c)).sum(2) * D ** -0.5).double()
    rms = lambda x: float((x - want).square().mean().sqrt())
    assert rms(lse.double()) <= 2 * rms(plain)


@pytest.mark.parametrize("D", [64, 128])
def test_decode_scores_of_bf16_queries(D):
    """The same for bf16 queries, whose products with c - 8 are whole numbers of 12 bits times a power of two of q's size.

    Their sums are formed 16 at a time and cut to fp32, four times a group; then a product and a sum for each of two
    groups, of scale and of offset: no more roundings than the plain form's, of sums no larger. Twice its error is the bound.
    """
    B, H, Hkv = 200, 32, 4
    s = make([1] * B, H, Hkv, D, 16, BF, seed=6)
    _, lse = decode(s, D ** -0.5, F4)
    page = s["table"][:, 0].long()
    codes, scales = s["kc"][page, :, 0], s["ks"][page, :, 0]
    k = torch.from_numpy(q4.values(codes, scales)).repeat_interleave(H // Hkv, 1)
    want = (k * s["q"].double()).sum(2) * D ** -0.5
    sz = scales.float().repeat_interleave(64, 2).repeat_interleave(H // Hkv, 1)
    c = torch.from_numpy(q4.unpack(codes)).float().repeat_interleave(H // Hkv, 1)
    plain = ((s["q"].float() * (sz[..., 1] + sz[..., 0] * c)).sum(2) * D ** -0.5).double()
    rms = lambda x: float((x - want).square().mean().sqrt())
    assert rms(lse.double()) <= 2 * rms(plain)


@pytest.mark.parametrize("D,n", [(64, 50000), (128, 20000)])
def test_decode_answers_of_fp32_queries(D, n):
    """Errors of many keys do not lean to one side, where answers are small beside the values they are summed of.

    Weights near one another and values about zero. A weight is off by 2^-22 of the exponential, 2^-22 of its two parts and
    some 2^-22 of a score below 2, each at random: together 2^-21 at most as a root mean square, and of answers, sums of as
    many values at random, no more. What leans would count once for each key: sqrt(n) times as much beside them.
    """
    H, Hkv, scale = 4, 2, D ** -0.5 / 16
    s = make([n], H, Hkv, D, 256, F4, seed=3)
    s["vs"][..., 1] = -7.5 * s["vs"][..., 0].float()
    out, _ = decode(s, scale, F4)
    page = s["table"][0].long()
    at = lambda t: t[page].transpose(1, 2).flatten(0, 1)[:n]
    k, v = (torch.from_numpy(q4.values(at(s[x + "c"]), at(s[x + "s"]))).repeat_interleave(H // Hkv, 1) for x in "kv")
    w = torch.softmax(torch.einsum("hd,nhd->hn", s["q"][0].double(), k) * scale, 1)
    want = torch.einsum("hn,nhd->hd", w, v)
    rms = lambda x: float(x.square().mean().sqrt())
    assert rms(out[0].double() - want) <= 2.0 ** -21 * rms(want)


@pytest.mark.parametrize("H,Hkv,D", [(24, 8, 128), (32, 4, 128), (32, 2, 64)])
def test_decode_answers_of_bf16_queries(H, Hkv, D):
    """The same for bf16 queries, whose weights times scales are rounded to fp16, and for each place of a code in its word.

    A rounding is off by 2^-11 of its weight at most, spread evenly over that by 2^-11 / sqrt(3), and at random, so that
    answers of as many values at random about zero are off by 2^-11.8 of their size as a root mean square; 2^-11 is the
    bound. Values stand for z + s c = s (c - 7.5) and are summed as s (c - 8) and s / 2, so the mean of those errors over
    the values of one place (every fourth of a head) has a part that a head's values share, 0.5 / 4.6 of an error, and a
    part of each value: together sqrt(0.11^2 / H + 4 / (H D)) of 2^-11.8, of which four times is the bound. What leans adds
    up over the keys and passes it. (Weights differ by powers of e, so that a product has neighbours of other sizes.)
    """
    n, scale = 1 << 18, D ** -0.5
    s = make([n], H, Hkv, D, 256, BF, seed=3)
    s["vs"][..., 1] = -7.5 * s["vs"][..., 0].float()
    out, _ = decode(s, scale, F4)
    page = s["table"][0].long()

    def rows(x, hk):  # of a head, float64
        c, sz = (s[x + a][page, hk].cuda().flatten(0, 1)[:n] for a in "cs")
        sz = sz.double().repeat_interleave(64, 1)
        return sz[..., 1] + sz[..., 0] * torch.stack((c & 15, c >> 4), -1).flatten(1)

    want = torch.empty((H, D), dtype=torch.float64)
    for hk in range(Hkv):
        at = slice(hk * H // Hkv, (hk + 1) * H // Hkv)
        x = s["q"][0, at].double().cuda() @ rows("k", hk).T * scale
        want[at] = (torch.softmax(x, 1) @ rows("v", hk)).cpu()
    off = out[0].double() - want
    rms = lambda x: float(x.square().mean().sqrt())
    assert rms(off) <= 2.0 ** -11 * rms(want)
    lean = off.unflatten(1, (-1, 4)).mean((0, 1)).abs().max()
    assert float(lean) <= 4 * (0.11 ** 2 / H + 4 / (H * D)) ** 0.5 * 2.0 ** -11.8 * rms(want)


@pytest.mark.parametrize("dt", [BF, F4])
@pytest.mark.parametrize("H,Hkv", [(4, 2), (10, 1)])
def test_decode_scales_and_queries_of_any_size(dt, H, Hkv):
    """Values' scales that differ by powers of ten from row to row and grow along the keys; queries of 1e-20 to 1e20
    in one batch, with zeros and one that is zero."""
    s = make([900, 500, 333, 40, 64], H, Hkv, 128, 32, dt, seed=9, spread=2.0)
    s["vs"] = (s["vs"].float() * torch.exp(12 * torch.rand(s["vs"].shape[:3], generator=torch.Generator().manual_seed(2)))[..., None, None]).to(BF)
    s["q"][1] *= 1e-20
    s["q"][2, 0] = 0
    s["q"][2, 1, ::3] = 0
    out, lse = decode(s, 0.02, dt)
    check_decode(s, 0.02, out, lse, "sizes")
    for f, scale in ((1e20, 2e-22), (1e-20, 2e18)):
        big = dict(s, q=(s["q"].float() * f).to(dt))
        big["q"][1] = big["q"][0]
        out, lse = decode(big, scale, dt)
        check_decode(big, scale, out, lse, "sizes of q")
    # offsets and scales near the ends of what append writes
    for f in (2.0 ** -90, 2.0 ** 90):
        far = dict(s, vs=(s["vs"].float() * f).to(BF))
        out, lse = decode(far, 0.02, F4)
        check_decode(far, 0.02, out, lse, f"values times {f}")


@pytest.mark.parametrize("dt", [BF, F4])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_with_garbage_behind(dt, D):
    """NaN scales in every row of the cache that no sequence holds, and in the pages that a table names behind the end."""
    s = make([777, 100, 16], 4, 2, D, 32, dt, seed=9, most=900)
    used = torch.zeros((s["kc"].shape[0], s["kc"].shape[2]), dtype=torch.bool)
    for b, n in enumerate(s["lens"].tolist()):
        for j in range(n):
            used[s["table"][b, j // 32].long(), j % 32] = True
    for c in ("ks", "vs"):
        s[c].transpose(1, 2)[~used] = float("nan")
    out, lse = decode(s, 0.5, dt)
    check_decode(s, 0.5, out, lse, "garbage behind")


def test_decode_growing_scores():
    s = make([2000], 4, 2, 64, 32, BF, seed=9)
    page = torch.zeros(s["ks"].shape[0])
    page[s["table"][0].long()] = torch.linspace(0.1, 30.0, s["table"].shape[1])
    s["ks"] = (s["ks"].float() * page[:, None, None, None, None]).to(BF)
    for dt in (BF, F4):
        out, lse = decode(s, 0.2, dt)
        check_decode(s, 0.2, out, lse, "growing")


def test_long_offsets():
    """Codes past 2^31 bytes into the cache are appended, read and attended to; sequences share pages."""
    D, Hkv, page = 128, 8, 256
    pages = (1 << 31) // (page * Hkv * D // 2) + 8
    g = torch.Generator().manual_seed(5)
    d = dict(kc=torch.zeros((pages, Hkv, page, D // 2), dtype=torch.uint8, device="cuda"),
             ks=torch.zeros((pages, Hkv, page, 2, 2), dtype=BF, device="cuda"))
    d["vc"], d["vs"] = torch.zeros_like(d["kc"]), torch.zeros_like(d["ks"])
    d["table"] = torch.tensor([[pages - 1, 2, pages - 3]] * 2, dtype=torch.int32, device="cuda")
    new = torch.randn((2, 600, Hkv, D), generator=g).to(BF)
    new[1] = new[0]
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    cpa().cp_paged_kv_append_q4(new[:1].cuda(), -new[:1].cuda(), *list(d.values())[:4], d["table"][:1].contiguous(), lens[:1])
    q = torch.randn((1, 16, D), generator=g).to(BF).repeat(2, 1, 1)
    small = {n: d[n][[pages - 1, 2, pages - 3]].cpu() for n in ("kc", "ks", "vc", "vs")}
    small |= dict(q=q, table=torch.tensor([[0, 1, 2]] * 2, dtype=torch.int32), lens=torch.tensor([600, 600], dtype=torch.int32))
    wc, ws = q4.append(new[:1], torch.zeros_like(small["kc"]), torch.zeros_like(small["ks"]), [[0, 1, 2]], [0])
    assert np.array_equal(small["kc"].numpy(), wc) and np.array_equal(small["ks"].double().numpy(), ws)
    out, lse = torch.empty((2, 16, D), dtype=BF, device="cuda"), torch.empty((2, 16), device="cuda")
    cpa().cp_paged_attn_decode_q4(q.cuda(), *d.values(), lens + 600, out, lse, 0.1)
    check_decode(small, 0.1, out.cpu(), lse.cpu(), "far pages")
    o = [torch.empty((2, 600, Hkv, D), device="cuda") for _ in range(2)]
    cpa().cp_paged_kv_read_q4(*d.values(), lens + 600, *o)
    want = torch.from_numpy(q4.as_rows(q4.values(small["kc"], small["ks"]))).float().flatten(0, 1)[:600]
    assert torch.equal(o[0][0].cpu(), want) and torch.equal(o[0][1].cpu(), want)


def test_bad_pages_and_lengths_are_reported_and_left_out():
    s = make([40, 40, 40], 4, 2, 64, 16, BF, seed=1)
    bad = {a: b.clone() for a, b in s.items()}
    bad["table"][1, 1] = 10 ** 6   # keys 16 .. 31 of sequence 1
    bad["table"][2, 0] = -3        # keys 0 .. 15 of sequence 2
    out, lse = decode(bad, 0.2, BF)
    assert cpa().cp_check_device_status() == -1 and cpa().cp_check_device_status() == 0
    o0, l0 = decode(s, 0.2, BF)
    assert torch.equal(out[0], o0[0]) and torch.equal(lse[0], l0[0])
    k, v = (q4.as_rows(q4.values(s[x + "c"], s[x + "s"])) for x in "kv")
    for b, keys in ((1, [*range(16), *range(32, 40)]), (2, [*range(16, 40)])):
        rows = [so.cached_rows(c, s["table"].numpy(), b, 40)[keys][None] for c in (k, v)]
        want, wl = so.scored_attention(s["q"][b][None, None], *rows, 0.2)
        assert np.abs(out[b].double().numpy() - want[0, 0]).max() <= 2.0 ** -7 * np.abs(rows[1]).max()
        assert np.abs(lse[b].double().numpy() - wl[0, :, 0]).max() <= 1e-4
    # lengths past the table are clamped, negative ones empty
    long = dict(s, lens=torch.tensor([10 ** 6, -5, 40], dtype=torch.int32))
    out, lse = decode(long, 0.2, BF)
    assert cpa().cp_check_device_status() == -1
    o1, l1 = decode(dict(s, lens=torch.tensor([48, 0, 40], dtype=torch.int32)), 0.2, BF)
    assert torch.equal(out, o1) and torch.equal(lse, l1) and cpa().cp_check_device_status() == 0
    # append: a position past the table and a bad page write nothing; read: zeros for a bad page, lengths clamped
    d = {n: s[n].cuda() for n in CACHE}
    new = torch.ones((3, 1, 2, 64), dtype=BF, device="cuda")
    lens = torch.tensor([48, 20, -1], dtype=torch.int32).cuda()
    cpa().cp_paged_kv_append_q4(new, new, *list(d.values())[:4], bad["table"].cuda(), lens)
    assert cpa().cp_check_device_status() == -1
    assert all(torch.equal(d[n].cpu().view(torch.uint8), s[n].view(torch.uint8)) for n in CACHE[:4])
    o = [torch.full((3, 50, 2, 64), 7.0, device="cuda") for _ in range(2)]
    cpa().cp_paged_kv_read_q4(*list(d.values())[:4], bad["table"].cuda(), torch.tensor([40, 40, 99], dtype=torch.int32).cuda(), *o)
    assert cpa().cp_check_device_status() == -1
    want = torch.zeros((3, 50, 2, 64))
    for b, n, gone in ((0, 40, []), (1, 40, range(16, 32)), (2, 48, range(16))):
        want[b, :n] = torch.from_numpy(so.cached_rows(k, s["table"].numpy(), b, n)).float()
        want[b, list(gone)] = 0
    assert torch.equal(o[0].cpu(), want)


def test_append_past_the_last_position_an_int_holds():
    """A table for more than 2^31 tokens: the token at position 2^31 - 1 is written, those behind are reported."""
    d = dict(kc=torch.zeros((2, 1, 65536, 32), dtype=torch.uint8, device="cuda"),
             ks=torch.zeros((2, 1, 65536, 1, 2), dtype=BF, device="cuda"))
    d["vc"], d["vs"] = torch.zeros_like(d["kc"]), torch.zeros_like(d["ks"])
    table = torch.zeros((2, 40000), dtype=torch.int32, device="cuda")
    table[0, 32767] = 1
    new = torch.randn((2, 3, 1, 64), generator=torch.Generator().manual_seed(1)).to(BF)
    lens = torch.tensor([2 ** 31 - 1, 7], dtype=torch.int32, device="cuda")
    cpa().cp_paged_kv_append_q4(new.cuda(), -new.cuda(), *d.values(), table, lens)
    assert cpa().cp_check_device_status() == -1 and cpa().cp_check_device_status() == 0
    c = q4.pack(q4.quantise(new)[0])
    want = np.zeros((2, 1, 65536, 32), dtype=np.uint8)
    want[1, 0, 65535], want[0, 0, 7:10] = c[0, 0, 0], c[1, :, 0]
    assert np.array_equal(d["kc"].cpu().numpy(), want)


@pytest.mark.parametrize("dt", [BF, F4])
@pytest.mark.parametrize("B,most", [(129, 400), (300, 200), (4096, 70)])
def test_decode_of_more_sequences_than_one_pass_of_the_work_list(B, most, dt):
    H, Hkv, D, page = 4, 2, 64, 16
    lens = torch.randint(1, most + 1, (B,), generator=torch.Generator().manual_seed(B))
    lens[::5] = 0
    s = widened(make(lens.tolist(), H, Hkv, D, page, dt, seed=B), 4096)
    assert cpa().cp_paged_attn_q4_workspace_size(B, H, Hkv, D, page, s["table"].shape[1], dt) > 0
    out, lse = decode(s, D ** -0.5, dt, softcap=20.0)
    check_decode(s, D ** -0.5, out, lse, f"{B} sequences", 20.0)
    assert cpa().cp_check_device_status() == 0


def test_repeat_streams_and_graph():
    s = widened(make([900, 3, 250, 0], 8, 2, 128, 16, BF, seed=6), 1 << 17)
    d = [s[n].cuda() for n in CACHE]
    q, lens = s["q"].cuda(), s["lens"].cuda()
    size = cpa().cp_paged_attn_q4_workspace_size(4, 8, 2, 128, 16, s["table"].shape[1])
    assert size > 0
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")

    def call(**kw):
        out, lse = torch.empty_like(q), torch.empty((4, 8), device="cuda")
        cpa().cp_paged_attn_decode_q4(q, *d, lens, out, lse, 0.1, **kw)
        return out, lse

    a = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = call(stream=side, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    new = torch.randn((4, 1, 2, 128), generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    start, after = lens.clone(), lens + 1
    o = [torch.empty((4, 12, 2, 128), dtype=BF, device="cuda") for _ in range(2)]
    out, lse = torch.empty_like(q), torch.empty((4, 8), device="cuda")
    fresh = [x.clone() for x in d]

    def step():
        cpa().cp_paged_kv_append_q4(new, -new, *d, start)
        cpa().cp_paged_kv_read_q4(*d, after, *o)
        cpa().cp_paged_attn_decode_q4(q, *d, after, out, lse, 0.1)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (*d, *o, out, lse)]
    for x, y in zip(d, fresh):
        x.copy_(y)
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(got, (*d, *o, out, lse)))
    start.copy_(torch.tensor([10, 800, 0, 1], dtype=torch.int32))
    after.copy_(start + 1)
    graph.replay()
    torch.cuda.synchronize()
    s2 = dict(zip(CACHE, (x.cpu() for x in d)), q=s["q"], lens=after.cpu())
    check_decode(s2, 0.1, out.cpu(), lse.cpu(), "replayed with other lengths")


def test_prompt_in_chunks_then_tokens():
    """A prompt in two chunks and then tokens: every answer equals one causal forward over the cached values.

    The first chunk attends to its own rows as the cache holds them, the second to both by the read back; tokens decode.
    Bounds: rounding of P and of results, 2^-8 of the largest value each, on both sides; lse as scores in fp32.
    """
    B, S, H, Hkv, D, page = 2, 120, 8, 2, 64, 16
    scale, cap = D ** -0.5, 20.0
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn((B, S, h, D), generator=g).to(BF).cuda() for h in (H, Hkv, Hkv))
    s = make([S, S], H, Hkv, D, page, BF, seed=2)
    d = [s[n].cuda() for n in CACHE]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    got, gl = torch.empty((B, S, H, D), dtype=BF, device="cuda"), torch.empty((B, H, S), device="cuda")
    at = 0
    for n in (50, 47):
        cpa().cp_paged_kv_append_q4(k[:, at:at + n].contiguous(), v[:, at:at + n].contiguous(), *d, lens)
        lens += n
        kc, vc = (torch.empty((B, at + n, Hkv, D), dtype=BF, device="cuda") for _ in range(2))
        cpa().cp_paged_kv_read_q4(*d, lens, kc, vc)
        o, l = torch.empty((B, n, H, D), dtype=BF, device="cuda"), torch.empty((B, H, n), device="cuda")
        cpa().cp_scored_attn_fwd(q[:, at:at + n].contiguous(), kc, vc, o, l, scale, softcap=cap, causal=True, q_pos0=at)
        got[:, at:at + n], gl[:, :, at:at + n] = o, l
        at += n
    while at < S:
        cpa().cp_paged_kv_append_q4(k[:, at:at + 1].contiguous(), v[:, at:at + 1].contiguous(), *d, lens)
        lens += 1
        o, l = torch.empty((B, H, D), dtype=BF, device="cuda"), torch.empty((B, H), device="cuda")
        cpa().cp_paged_attn_decode_q4(q[:, at].contiguous(), *d, lens, o, l, scale, softcap=cap)
        got[:, at], gl[:, :, at] = o, l
        at += 1
    assert cpa().cp_check_device_status() == 0
    kv = [q4.as_rows(q4.values(d[i], d[i + 1])) for i in (0, 2)]
    rows = [np.stack([so.cached_rows(c, s["table"].numpy(), b, S) for b in range(B)]) for c in kv]
    want, wl = so.scored_attention(q, *rows, scale, softcap=cap, causal=True)
    top = np.abs(rows[1]).max()
    # the read back rounds the cache's values to bf16 before the chunks' attention: 2^-8 of k in a score, of v in a value
    m = 2.0 ** -8 * so.abs_products(q, rows[0], scale)
    assert np.abs(got.double().cpu().numpy() - want).max() <= (3 * 2.0 ** -8 + 2 * m * (1 + m)) * top
    assert np.abs(gl.double().cpu().numpy() - wl).max() <= m + 1e-4


def test_rotated_and_cached_tokens():
    """A decoding step as a model takes it: norm and rotation of the new token, append, attention."""
    B, n, H, Hkv, D, page = 3, 40, 8, 2, 128, 16
    g = torch.Generator().manual_seed(7)
    qkv = torch.randn((B, n, H + 2 * Hkv, D), generator=g).to(BF).cuda()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(BF).cuda() for _ in range(2)]
    freqs = torch.tensor([10000.0 ** (-i / 64) for i in range(64)], dtype=torch.float64).cuda()
    pos = torch.arange(n, dtype=torch.int32).cuda()[:, None].contiguous()
    s = make([n] * B, H, Hkv, D, page, BF, seed=2)
    d = [s[x].cuda() for x in CACHE]
    rule = dict(freqs=freqs, eps=1e-6, q_weight=w[0], k_weight=w[1])
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    qs = []
    for t in range(n):
        q, k = torch.empty((B, 1, H, D), dtype=BF, device="cuda"), torch.empty((B, 1, Hkv, D), dtype=BF, device="cuda")
        one = qkv[:, t:t + 1]
        cpa().cp_qk_norm_rope_fwd(one[:, :, :H], one[:, :, H:H + Hkv], q, k, positions=pos[t:t + 1], **rule)
        cpa().cp_paged_kv_append_q4(k, one[:, :, H + Hkv:].contiguous(), *d, lens)
        lens += 1
        qs.append(q)
    out, lse = torch.empty((B, H, D), dtype=BF, device="cuda"), torch.empty((B, H), device="cuda")
    cpa().cp_paged_attn_decode_q4(qs[-1][:, 0].contiguous(), *d, lens, out, lse, D ** -0.5)
    # the same tokens at once
    q, k = torch.empty((B, n, H, D), dtype=BF, device="cuda"), torch.empty((B, n, Hkv, D), dtype=BF, device="cuda")
    cpa().cp_qk_norm_rope_fwd(qkv[:, :, :H], qkv[:, :, H:H + Hkv], q, k, positions=pos, **rule)
    assert torch.equal(q, torch.cat(qs, 1))
    d2 = [s[x].cuda() for x in CACHE]
    cpa().cp_paged_kv_append_q4(k, qkv[:, :, H + Hkv:].contiguous(), *d2, lens - n)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(d, d2))
    check_decode(dict(zip(CACHE, (x.cpu() for x in d)), q=q[:, -1].cpu(), lens=lens.cpu()), D ** -0.5, out.cpu(), lse.cpu(), "step")
    assert cpa().cp_check_device_status() == 0


@pytest.mark.parametrize("tokens", [128, 1 << 17])   # tables for clusters, and for the list and its join
def test_back_to_back_calls_see_each_other(tokens):
    """Each call reads what the one before has written, none waits for the host; the same with a wait after every call."""
    B, steps, H, Hkv, D, page = 5, 40, 8, 2, 64, 16
    g = torch.Generator().manual_seed(11)
    qk = torch.randn((B, 1, H + Hkv, D), generator=g).to(BF).cuda()
    v = torch.randn((B, 1, Hkv, D), generator=g).to(BF).cuda()
    freqs = torch.tensor([100.0 ** (-i / 32) for i in range(32)], dtype=torch.float64).cuda()
    pos = torch.arange(steps + 1, dtype=torch.int32).cuda()[:, None].contiguous()
    s = widened(make([steps] * B, H, Hkv, D, page, BF, seed=2), tokens)
    lens = [torch.full((B,), t, dtype=torch.int32, device="cuda") for t in range(steps + 1)]
    size = cpa().cp_paged_attn_q4_workspace_size(B, H, Hkv, D, page, s["table"].shape[1])
    assert (size > 0) == (tokens > 128)

    def chain(after):
        d = [s[x].cuda() for x in CACHE]
        ws = torch.full((max(size, 256),), 255, dtype=torch.uint8, device="cuda")
        ws2 = torch.full((cpa().cp_qk_norm_rope_bwd_workspace_size(D),), 255, dtype=torch.uint8, device="cuda")
        q, k, out = qk[:, :, :H].contiguous(), torch.empty_like(v), torch.empty((B, H, D), dtype=BF, device="cuda")
        dq, dk, lse = torch.empty_like(q), torch.empty_like(k), torch.empty((B, H), device="cuda")
        w = [torch.ones(D, device="cuda") for _ in range(2)]
        rows = [torch.empty((B, steps, Hkv, D), dtype=BF, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        for t in range(steps):
            rule = dict(positions=pos[t:t + 1], freqs=freqs, eps=1e-6)
            # the step's queries are the last one's answers, its weights the last one's gradients
            cpa().cp_qk_norm_rope_fwd(q, qk[:, :, H:], q, k, q_weight=w[0], k_weight=w[1], **rule)
            after()
            cpa().cp_paged_kv_append_q4(k, v, *d, lens[t])
            after()
            cpa().cp_paged_attn_decode_q4(q.view(B, H, D), *d, lens[t + 1], out, lse, D ** -0.5, workspace=ws)
            after()
            cpa().cp_qk_norm_rope_bwd(out.view(B, 1, H, D), k, q, v, dq, dk, dq_weight=w[0], dk_weight=w[1], workspace=ws2, **rule)
            after()
            cpa().cp_qk_norm_rope_fwd(dq, dk, q, k, **rule)
            after()
        cpa().cp_paged_kv_read_q4(*d, lens[steps], *rows)
        torch.cuda.synchronize()
        return q, k, out, lse, *w, *rows

    got, want = chain(lambda: None), chain(torch.cuda.synchronize)
    assert all(torch.isfinite(x).all() for x in want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert cpa().cp_check_device_status() == 0


def test_wrapper_refusals():
    s = {a: b.cuda() for a, b in make([5, 5], 4, 2, 64, 16, BF, seed=0).items()}
    out, lse = torch.empty_like(s["q"]), torch.empty((2, 4), device="cuda")

    def f(o=out, l=lse, kw={}, **over):
        x = {**s, **over}
        cpa().cp_paged_attn_decode_q4(x["q"], *(x[n] for n in CACHE), x["lens"], o, l, 0.1, **kw)

    for bad in (dict(q=s["q"][0]), dict(vc=s["vc"][:1]), dict(vs=s["vs"][:, :1]), dict(kc=s["kc"][0]), dict(table=s["table"][0]),
                dict(lens=s["lens"][:1]), dict(o=out[:1]), dict(l=lse[:1]), dict(kw=dict(slopes=lse[0, :3])),
                dict(table=s["table"].cpu()), dict(kc=s["kc"].transpose(1, 2)), dict(ks=s["ks"][..., :1])):
        with pytest.raises(ValueError):
            f(**bad)
    for bad in (dict(kc=s["kc"].int()), dict(ks=s["ks"].float()), dict(lens=s["lens"].long()), dict(o=out.half()),
                dict(l=lse.half()), dict(q=s["q"].half())):
        with pytest.raises(TypeError):
            f(**bad)
    with pytest.raises(cpa().CpError):
        f(table=s["table"].repeat(1, 4096), kw=dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")))
    c = [s[n] for n in CACHE]
    new = torch.zeros((2, 1, 2, 64), dtype=BF, device="cuda")
    for bad in ((new, new[:, :0]), (new[:1], new[:1]), (new[..., :32], new[..., :32]), (new.cpu(), new.cpu())):
        with pytest.raises(ValueError):
            cpa().cp_paged_kv_append_q4(*bad, *c, s["lens"])
        with pytest.raises(ValueError):
            cpa().cp_paged_kv_read_q4(*c, s["lens"], *bad)
    with pytest.raises(TypeError):
        cpa().cp_paged_kv_append_q4(new, new.float(), *c, s["lens"])
    with pytest.raises(cpa().CpError):   # pages of 8 rows
        small = [x[:, :, :8].contiguous() for x in c[:4]]
        cpa().cp_paged_kv_append_q4(new, new, *small, c[4], s["lens"])
