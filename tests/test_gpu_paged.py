"""The paged cache: cp_paged_kv_append (bit for bit) and cp_paged_attn_decode
against the float64 oracle, and a run of both beside cp_scored_attn_fwd.

Bounds of decode, element by element, as in the score-rule tests: with
u = 2^-24, w = 2^-8 for bf16 (P rounded for its product), a score's error
d = (D + 16) u max(scale sum |q||k|) + 4 u max|x|, n keys:
  |out - ref| <= (w + 2 (2 d + 2^-21 + n u)) sum_j p |v| + r |ref|
  |lse - ref| <= 2 d + 2^-20 + n u + 4 u |ref|
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


def make(lens, H, Hkv, D, page, dt, seed, spare=2, most=None):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages = max(1, -(-max(most or 0, *lens) // page))
    total = B * pages + spare
    r = lambda *s: torch.randn(s, generator=g).to(dt)
    table = torch.randperm(total, generator=g)[:B * pages].to(torch.int32).view(B, pages)
    return dict(q=r(B, H, D), k=r(total, page, Hkv, D), v=r(total, page, Hkv, D), table=table.contiguous(),
                lens=torch.tensor(lens, dtype=torch.int32))


def decode(s, scale, out_dt, **kw):
    B, H, D = s["q"].shape
    out = torch.full((B, H, D), 7.0, dtype=out_dt, device="cuda")
    lse = torch.full((B, H), 7.0, device="cuda")
    kw = {a: b.cuda() if isinstance(b, torch.Tensor) else b for a, b in kw.items()}
    cpa().cp_paged_attn_decode(s["q"].cuda(), s["k"].cuda(), s["v"].cuda(), s["table"].cuda(), s["lens"].cuda(), out,
                               lse, scale, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def check_decode(s, scale, out, lse, what, softcap=0.0, slopes=None):
    want, wl = so.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], scale, softcap, slopes)
    B, H, D = s["q"].shape
    Hkv = s["k"].shape[2]
    w = 2.0 ** -8 if s["q"].dtype == BF else 0.0
    r = 2 * (2.0 ** -8 if out.dtype == BF else U)
    kf, vf, table = s["k"].double().numpy(), s["v"].double().numpy(), s["table"].numpy()
    got, gl = out.double().numpy(), lse.double().numpy()
    for b in range(B):
        n = int(s["lens"][b])
        if n == 0:
            assert np.all(got[b] == 0) and np.all(np.isneginf(gl[b])), what
            continue
        k, v = so.cached_rows(kf, table, b, n), so.cached_rows(vf, table, b, n)
        q1 = s["q"][b][None, None].double().numpy()
        big = so.abs_products(q1, k[None], scale)
        far = n * float(slopes.abs().max()) if slopes is not None else 0.0
        d = (D + 16) * U * big + 4 * U * (big + far)
        for h in range(H):
            x, _ = so.scores(q1, k[None], 0, h, scale, softcap=softcap, slopes=slopes, q_pos0=n - 1)
            p = np.exp(x[0] - wl[b, h])
            bound = (w + 2 * (2 * d + 2.0 ** -21 + n * U)) * (p @ np.abs(v[:, h // (H // Hkv)])) + r * np.abs(want[b, h])
            over = np.abs(got[b, h] - want[b, h]) - bound
            assert over.max() <= 0, f"{what} b{b} h{h}: past its bound by {over.max():.3e}"
            assert abs(gl[b, h] - wl[b, h]) <= 2 * d + 2.0 ** -20 + n * U + 4 * U * abs(wl[b, h]), f"{what} lse b{b} h{h}"


LENS = {
    "one token": [1],
    "short": [5, 1, 16, 17],
    "block edges": [63, 64, 65, 128, 129],
    "ragged with empty": [300, 0, 7, 0, 1000, 64],
    "split over many CTAs": [9000],
    "many short": [3] * 70 + [0, 40] * 10,
    "uneven": [5000, 1, 1, 1, 2500],
}


@pytest.mark.parametrize("name", list(LENS))
@pytest.mark.parametrize("H,Hkv,D,page,dt,out_dt", [
    (4, 4, 64, 16, BF, BF),
    (24, 8, 128, 16, BF, F4),
    (20, 1, 128, 1, BF, BF),        # more heads than a tile has rows, one-row pages
    (8, 1, 64, 128, BF, BF),
    (6, 3, 128, 32, F4, F4),
    (18, 2, 64, 64, F4, F4),        # 9 heads on one: two groups of fp32 rows
])
def test_decode(name, H, Hkv, D, page, dt, out_dt):
    s = make(LENS[name], H, Hkv, D, page, dt, seed=len(name))
    out, lse = decode(s, D ** -0.5, out_dt)
    check_decode(s, D ** -0.5, out, lse, name)
    assert cpa().cp_check_device_status() == 0


def widened(s, tokens):
    """The table with room for more tokens; the columns behind hold no page and are not read."""
    s = dict(s)
    B, pages = s["table"].shape
    extra = max(0, tokens // s["k"].shape[1] - pages)
    s["table"] = torch.cat([s["table"], torch.full((B, extra), -1, dtype=torch.int32)], 1).contiguous()
    return s


# tables of up to 2, 4, 8, 16, 64 blocks of 64 tokens, and one that only the list of blocks takes
@pytest.mark.parametrize("tokens", [128, 256, 512, 1024, 4096, 40000])
@pytest.mark.parametrize("H,Hkv,D,page,dt,out_dt", [
    (24, 8, 128, 16, BF, BF),
    (20, 1, 128, 1, BF, F4),
    (8, 1, 64, 128, BF, BF),
    (6, 3, 128, 32, F4, F4),
    (18, 2, 64, 64, F4, F4),
])
def test_decode_whatever_the_table_holds(tokens, H, Hkv, D, page, dt, out_dt):
    from context_attention_dits_gb300 import cp_paged_attn_workspace_size as size
    lens = [min(tokens, n) for n in (128, 0, 1, 65, 127)]
    s = widened(make(lens, H, Hkv, D, page, dt, seed=tokens), tokens)
    if tokens <= 128 or tokens == 40000:
        assert (size(5, H, Hkv, D, dt, page_size=page, max_pages=s["table"].shape[1]) > 0) == (tokens == 40000)
    out, lse = decode(s, D ** -0.5, out_dt, softcap=20.0)
    check_decode(s, D ** -0.5, out, lse, f"{tokens}", 20.0)
    assert cpa().cp_check_device_status() == 0
    s["table"][3, 0] = -7   # sequence 3 loses its first page (all of it, where pages are of 128), the others nothing
    bad, bl = decode(s, D ** -0.5, out_dt, softcap=20.0)
    assert cpa().cp_check_device_status() == -1
    rest = [0, 1, 2, 4]
    assert torch.equal(bad[rest], out[rest]) and torch.equal(bl[rest], lse[rest])
    assert (bl[3] < lse[3]).all() and (page < 65 or ((bad[3] == 0).all() and torch.isneginf(bl[3]).all()))


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


@pytest.mark.parametrize("dt", [BF, F4])
def test_decode_growing_scores_and_garbage_behind(dt):
    """Maxima that grow along the keys; NaN in every row of the cache that no sequence holds."""
    s = make([777, 100], 4, 2, 64, 32, dt, seed=9, most=900)
    grow = torch.linspace(0.1, 30.0, 900)
    used = torch.zeros(s["k"].shape[:2], dtype=torch.bool)
    for b, n in enumerate(s["lens"].tolist()):
        for j in range(n):
            at = s["table"][b, j // 32].long(), j % 32
            s["k"][at] = (s["k"][at].float() * grow[j]).to(dt)
            used[at] = True
    for c in ("k", "v"):
        s[c][~used] = float("nan")
    out, lse = decode(s, 0.5, dt)
    check_decode(s, 0.5, out, lse, "growing")


def test_decode_shared_pages_and_long_offsets():
    """Sequences on the same pages give the same answer; rows past 2^31 bytes into the cache are reached."""
    D, Hkv, page = 128, 8, 256
    pages = (1 << 31) // (page * Hkv * D * 2) + 8
    k = torch.zeros((pages, page, Hkv, D), dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator().manual_seed(5)
    for at in (pages - 1, pages - 3, 2):
        k[at] = torch.randn((page, Hkv, D), generator=g).to(BF).cuda()
        v[at] = torch.randn((page, Hkv, D), generator=g).to(BF).cuda()
    full = torch.tensor([[pages - 1, 2, pages - 3]] * 2, dtype=torch.int32)
    q = torch.randn((1, 16, D), generator=g).to(BF).repeat(2, 1, 1)
    lens = torch.tensor([600, 600], dtype=torch.int32)
    out, lse = torch.empty((2, 16, D), dtype=BF, device="cuda"), torch.empty((2, 16), device="cuda")
    cpa().cp_paged_attn_decode(q.cuda(), k, v, full.cuda(), lens.cuda(), out, lse, 0.1)
    torch.cuda.synchronize()
    # the same through a small cache of the three pages
    small = dict(q=q, k=k[[pages - 1, 2, pages - 3]].cpu(), v=v[[pages - 1, 2, pages - 3]].cpu(),
                 table=torch.tensor([[0, 1, 2]] * 2, dtype=torch.int32), lens=lens)
    check_decode(small, 0.1, out.cpu(), lse.cpu(), "far pages")
    new = torch.randn((1, 2, Hkv, D), generator=g).to(BF).cuda()
    cpa().cp_paged_kv_append(new, -new, k, v, full[:1].cuda(), lens[:1].cuda())
    assert torch.equal(k[pages - 3, 88:90], new[0]) and torch.equal(v[pages - 3, 88:90], -new[0])


@pytest.mark.parametrize("dt", [BF, F4])
@pytest.mark.parametrize("B,T,Hkv,D,page,lens,new", [
    (1, 1, 1, 64, 1, [0], None),
    (3, 1, 8, 128, 16, [15, 16, 0], None),
    (2, 37, 3, 64, 8, [5, 100], None),
    (4, 50, 2, 128, 64, [0, 63, 64, 200], [50, 0, 7, 60]),   # 60 > T: all 50
    (2, 5, 1, 64, 256, [0, 251], [-1, 5]),
])
def test_append(B, T, Hkv, D, page, lens, new, dt):
    s = make([n + T for n in lens], Hkv, Hkv, D, page, dt, seed=T)
    g = torch.Generator().manual_seed(T + 1)
    kn, vn = (torch.randn((B, T, Hkv, D), generator=g).to(dt) for _ in range(2))
    at = torch.tensor(lens, dtype=torch.int32)
    nl = None if new is None else torch.tensor(new, dtype=torch.int32)
    kc, vc = s["k"].cuda(), s["v"].cuda()
    cpa().cp_paged_kv_append(kn.cuda(), vn.cuda(), kc, vc, s["table"].cuda(), at.cuda(),
                             new_lens=None if nl is None else nl.cuda())
    assert cpa().cp_check_device_status() == 0
    for got, was, x in ((kc, s["k"], kn), (vc, s["v"], vn)):
        want = so.paged_append(x.double().numpy(), was.double().numpy(), s["table"], at, nl)
        assert np.array_equal(got.cpu().double().numpy(), want)


def test_bad_pages_and_lengths_are_reported_and_left_out():
    s = make([40, 40, 40], 4, 2, 64, 16, BF, seed=1)
    good = {a: b.clone() for a, b in s.items()}
    s["table"][1, 1] = 10 ** 6   # keys 16 .. 31 of sequence 1
    s["table"][2, 0] = -3        # keys 0 .. 15 of sequence 2
    out, lse = decode(s, 0.2, BF)
    assert cpa().cp_check_device_status() == -1 and cpa().cp_check_device_status() == 0
    o0, l0 = decode(good, 0.2, BF)
    assert torch.equal(out[0], o0[0]) and torch.equal(lse[0], l0[0])
    for b, keys in ((1, [*range(16), *range(32, 40)]), (2, [*range(16, 40)])):
        rows = [so.cached_rows(good[c].double().numpy(), good["table"].numpy(), b, 40)[keys][None] for c in ("k", "v")]
        want, wl = so.scored_attention(good["q"][b][None, None], *rows, 0.2)
        assert np.abs(out[b].double().numpy() - want[0, 0]).max() <= 2.0 ** -7 * np.abs(rows[1]).max()
        assert np.abs(lse[b].double().numpy() - wl[0, :, 0]).max() <= 1e-4
    assert cpa().cp_check_device_status() == 0
    # lengths past the table are clamped, negative ones empty
    long = {a: b.clone() for a, b in good.items()}
    long["lens"] = torch.tensor([10 ** 6, -5, 40], dtype=torch.int32)
    out, lse = decode(long, 0.2, BF)
    assert cpa().cp_check_device_status() == -1
    clamped = {**good, "lens": torch.tensor([48, 0, 40], dtype=torch.int32)}
    o1, l1 = decode(clamped, 0.2, BF)
    assert torch.equal(out, o1) and torch.equal(lse, l1) and cpa().cp_check_device_status() == 0
    # append: a position past the table and a bad page write nothing
    kc, vc = good["k"].cuda(), good["v"].cuda()
    new = torch.ones((3, 1, 2, 64), dtype=BF, device="cuda")
    cpa().cp_paged_kv_append(new, new, kc, vc, s["table"].cuda(), torch.tensor([48, 20, -1], dtype=torch.int32).cuda())
    assert cpa().cp_check_device_status() == -1
    assert torch.equal(kc.cpu(), good["k"]) and torch.equal(vc.cpu(), good["v"])


def test_prompt_then_tokens_as_one_causal_sequence():
    """A prompt appended whole, then token by token: every token's decode equals its row of one causal forward."""
    B, S, P, H, Hkv, D, page = 2, 90, 70, 8, 2, 64, 16
    scale, cap = D ** -0.5, 20.0
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn((B, S, h, D), generator=g).to(BF).cuda() for h in (H, Hkv, Hkv))
    slopes = torch.exp2(-torch.arange(1, H + 1).float()).cuda()
    want, wl = torch.empty((B, S, H, D), device="cuda"), torch.empty((B, H, S), device="cuda")
    cpa().cp_scored_attn_fwd(q, k, v, want, wl, scale, softcap=cap, slopes=slopes, causal=True)
    s = make([S, S], H, Hkv, D, page, BF, seed=2)
    kc, vc, table = s["k"].cuda(), s["v"].cuda(), s["table"].cuda()
    short = torch.tensor([P, P - 13], dtype=torch.int32, device="cuda")  # the second prompt is padded
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    cpa().cp_paged_kv_append(k[:, :P].contiguous(), v[:, :P].contiguous(), kc, vc, table, lens, new_lens=short)
    lens = short.clone()
    out, lse = torch.empty((B, H, D), device="cuda"), torch.empty((B, H), device="cuda")
    rows = torch.arange(B, device="cuda")
    for _ in range(20):
        at = lens.long()
        cpa().cp_paged_kv_append(k[rows, at][:, None].contiguous(), v[rows, at][:, None].contiguous(), kc, vc, table, lens)
        lens += 1
        cpa().cp_paged_attn_decode(q[rows, at].contiguous(), kc, vc, table, lens, out, lse, scale, softcap=cap,
                                   slopes=slopes)
        # both are within 2^-8 sum p |v| <= 2^-8 max |v| of the exact value
        assert (out - want[rows, at]).abs().max() <= 2 * 2.0 ** -8 * v.abs().max().float() * 1.01
        assert (lse - wl[rows, :, at]).abs().max() <= 1e-4
    assert cpa().cp_check_device_status() == 0


def test_repeat_streams_and_graph():
    s = make([900, 3, 250, 0], 8, 2, 128, 16, BF, seed=6)
    q, k, v, table, lens = (s[n].cuda() for n in ("q", "k", "v", "table", "lens"))
    ws = torch.empty(cpa().cp_paged_attn_workspace_size(4, 8, 2, 128), dtype=torch.uint8, device="cuda")
    ws.fill_(255)

    def call(**kw):
        out, lse = torch.empty_like(q), torch.empty((4, 8), device="cuda")
        cpa().cp_paged_attn_decode(q, k, v, table, lens, out, lse, 0.1, **kw)
        return out, lse

    a = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = call(stream=side, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    out, lse = torch.empty_like(q), torch.empty((4, 8), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cpa().cp_paged_attn_decode(q, k, v, table, lens, out, lse, 0.1)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a[0]) and torch.equal(lse, a[1])
    lens.copy_(torch.tensor([10, 800, 0, 1], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    lens2 = dict(s, lens=torch.tensor([10, 800, 0, 1], dtype=torch.int32))
    check_decode(lens2, 0.1, out.cpu(), lse.cpu(), "replayed with other lengths")


def test_wrapper_refusals():
    s = {a: b.cuda() for a, b in make([5, 5], 4, 2, 64, 16, BF, seed=0).items()}
    out, lse = torch.empty_like(s["q"]), torch.empty((2, 4), device="cuda")
    f = lambda q=s["q"], k=s["k"], v=s["v"], t=s["table"], n=s["lens"], o=out, l=lse, **kw: \
        cpa().cp_paged_attn_decode(q, k, v, t, n, o, l, 0.1, **kw)
    for bad in (dict(q=s["q"][0]), dict(v=s["v"][:1]), dict(t=s["table"][0]), dict(n=s["lens"][:1]), dict(o=out[:1]),
                dict(l=lse[:1]), dict(slopes=lse[0, :3]), dict(t=s["table"].cpu()), dict(k=s["k"].transpose(1, 2))):
        with pytest.raises(ValueError):
            f(**bad)
    for bad in (dict(k=s["k"].float()), dict(n=s["lens"].long()), dict(o=out.half()), dict(l=lse.half())):
        with pytest.raises(TypeError):
            f(**bad)
    with pytest.raises(cpa().CpError):
        f(t=s["table"].repeat(1, 4096), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    new = torch.zeros((2, 1, 2, 64), dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        cpa().cp_paged_kv_append(new, new[:, :0], s["k"], s["v"], s["table"], s["lens"])
    with pytest.raises(TypeError):
        cpa().cp_paged_kv_append(new, new.float(), s["k"], s["v"], s["table"], s["lens"])
    with pytest.raises(cpa().CpError):   # a page of 12 rows
        bad = torch.zeros((4, 12, 2, 64), dtype=BF, device="cuda")
        cpa().cp_paged_kv_append(new, new, bad, bad, s["table"], s["lens"])


@pytest.mark.parametrize("dt", [BF, F4])
@pytest.mark.parametrize("H,Hkv,D", [(1, 1, 64), (3, 1, 64), (1, 1, 128)])
def test_decode_of_few_heads_by_wide_clusters(H, Hkv, D, dt):
    """A unit of one to three heads shared by 8 or 16 CTAs: most threads have nothing to join."""
    s = make([4000, 1, 0], H, Hkv, D, 16, dt, seed=H + D, most=4096)
    one = {n: (t[:1].contiguous() if n in ("q", "table", "lens") else t) for n, t in s.items()}
    for x in (one, s):
        out, lse = decode(x, D ** -0.5, dt, softcap=30.0)
        check_decode(x, D ** -0.5, out, lse, "wide clusters", 30.0)
    assert cpa().cp_check_device_status() == 0


def test_append_past_the_last_position_an_int_holds():
    """A table for more than 2^31 tokens: the token at position 2^31 - 1 is written, those behind are reported."""
    cache = torch.zeros((2, 65536, 1, 64), dtype=BF, device="cuda")
    k, v = cache.clone(), cache.clone()
    table = torch.zeros((2, 40000), dtype=torch.int32, device="cuda")
    table[0, 32767] = 1
    new = torch.randn((2, 3, 1, 64), generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    lens = torch.tensor([2 ** 31 - 1, 7], dtype=torch.int32, device="cuda")
    cpa().cp_paged_kv_append(new, -new, k, v, table, lens)
    assert cpa().cp_check_device_status() == -1 and cpa().cp_check_device_status() == 0
    for got, x in ((k, new), (v, -new)):
        want = cache.clone()
        want[1, 65535] = x[0, 0]
        want[0, 7:10] = x[1]
        assert torch.equal(got, want)


@pytest.mark.parametrize("dt", [BF, F4])
@pytest.mark.parametrize("B,most", [(129, 400), (300, 200), (4096, 70)])
def test_decode_of_more_sequences_than_one_pass_of_the_work_list(B, most, dt):
    """The list of blocks is summed 128 sequences at a time: ragged lengths, every fifth sequence empty."""
    H, Hkv, D, page = 4, 2, 64, 16
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(1, most + 1, (B,), generator=g)
    lens[::5] = 0
    s = widened(make(lens.tolist(), H, Hkv, D, page, dt, seed=B), 4096)
    assert cpa().cp_paged_attn_workspace_size(B, H, Hkv, D, dt, page_size=page, max_pages=s["table"].shape[1]) > 0
    out, lse = decode(s, D ** -0.5, dt, softcap=20.0)
    check_decode(s, D ** -0.5, out, lse, f"{B} sequences", 20.0)
    assert cpa().cp_check_device_status() == 0
