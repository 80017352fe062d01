"""Workloads of the operators around attention: what a model does to queries and keys
between their projections and the attention, and a paged cache held in 4 bits.

Five operators, each in a plain torch form and as the library's own call:

* ``fwd``    each head's query and key normalised (root mean square) and rotated by its
  position, which may have several axes (time, height, width), in one pass;
* ``bwd``    its gradients: queries, keys and the norms' weights;
* ``append`` the new tokens' keys and values into a paged cache of 4-bit codes, and the
  sequences read back as the values that the cache stands for (two operators: what a
  long prompt's next chunk does before its attention);
* ``decode`` attention of one new token per sequence over that cache.

A row of the cache (one token, one head) is cut into groups of 64 values, each held as
64 codes c of 4 bits and two bf16 numbers, a scale s and an offset z, and stands for
z + s c: z is the largest bf16 number not above the group's values, s the smallest not
below (largest value - z) / 15 nor 2^-100, c = min(15, floor((x - z) / s + 1/2)). Value
2 i of a row is the low half of its byte i, value 2 i + 1 the high half. Codes lie as
[pages, heads, rows of a page, D / 2], scales as [pages, heads, rows of a page, D / 64, 2].

Outputs of ``fwd``: queries and keys; ``bwd``: their gradients and the weights';
``append``: keys and values of the sequences, zero behind their ends; ``decode``: out and
lse.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_GROUP = 64


def listed():
    return [
        # the new token of each sequence of a serving batch, out of one packed projection
        dict(name="fwd_token", op="fwd", dtype="bf16", B=64, S=1, H=24, Hkv=8, D=128, sections="64", interleaved=False,
             norm=True, packed=True, far=4096),
        # text and image tokens of this library's headline workload: three axes of pairs 8, 28 and 28
        dict(name="fwd_image", op="fwd", dtype="bf16", B=1, S=4608, H=24, Hkv=24, D=128, sections="8,28,28",
             interleaved=True, norm=True, packed=False, far=0),
        # a video's tokens, halves rotated against each other, out of a packed projection
        dict(name="fwd_video", op="fwd", dtype="bf16", B=1, S=32768, H=24, Hkv=24, D=128, sections="16,24,24",
             interleaved=False, norm=True, packed=True, far=0),
        # fp32 without a norm, half of each head rotated, far positions: a small model's check run
        dict(name="fwd_f32", op="fwd", dtype="f32", B=2, S=387, H=4, Hkv=4, D=64, sections="16", interleaved=False,
             norm=False, packed=False, far=1 << 20),
        # gradients of a short row: latency
        dict(name="bwd_short", op="bwd", dtype="bf16", B=1, S=130, H=8, Hkv=2, D=64, sections="8,12,12",
             interleaved=True, norm=True, packed=False, far=0),
        # a training step's gradients at the headline workload's heads, odd length
        dict(name="bwd_image", op="bwd", dtype="bf16", B=1, S=4607, H=24, Hkv=24, D=128, sections="8,28,28",
             interleaved=True, norm=True, packed=True, far=0),
        # fp32 gradients, shared keys
        dict(name="bwd_f32", op="bwd", dtype="f32", B=1, S=700, H=6, Hkv=3, D=128, sections="64", interleaved=False,
             norm=True, packed=False, far=4096),
        # the new token of every sequence of a serving batch at its start, and what the cache then holds
        dict(name="append_token", op="append", dtype="bf16", B=64, T=1, Hkv=8, D=128, page=16, len=128, ragged=False),
        # chunks of prompts of different lengths, padded to the longest, behind what is cached
        dict(name="append_chunk", op="append", dtype="bf16", B=6, T=4607, Hkv=8, D=128, page=64, len=512, ragged=True),
        # one user, a short conversation: the latency of a token
        dict(name="decode_one", op="decode", dtype="bf16", B=1, H=24, Hkv=8, D=128, page=16, len=1000, ragged=False,
             cap=50.0, bias=False),
        # a serving batch whose conversations differ in length
        dict(name="decode_batch", op="decode", dtype="bf16", B=48, H=24, Hkv=8, D=128, page=64, len=8192, ragged=True,
             cap=0.0, bias=True),
        # two very long contexts
        dict(name="decode_long", op="decode", dtype="bf16", B=2, H=32, Hkv=4, D=128, page=128, len=262144, ragged=False,
             cap=50.0, bias=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "append", "decode", "decode"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 3, 4, 8])
    if op in ("fwd", "bwd"):
        pairs = D // 2 // rng.choice([1, 1, 2, 4])
        axes = rng.choice([1, 1, 2, 3])
        cuts = sorted(rng.randint(0, pairs) for _ in range(axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        S = _log_int(rng, 1, 8192 if op == "fwd" else 4608)
        B = max(1, min(rng.choice([1, 1, 2, 3, 48]), (1 << 27) // (S * (H + Hkv) * D)))
        return dict(op=op, dtype=dtype, B=B, S=S, H=H, Hkv=Hkv, D=D, sections=",".join(map(str, sections)),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.8, packed=rng.random() < 0.5,
                    far=rng.choice([0, 4096, 1 << 20]))
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "decode":
        n = _log_int(rng, 1, 65536)
        B = max(1, min(_log_int(rng, 1, 128), (1 << 27) // (n * Hkv * D)))
        return dict(op=op, dtype=dtype, B=B, H=H, Hkv=Hkv, D=D, page=page, len=n, ragged=rng.random() < 0.6,
                    cap=rng.choice([0.0, 15.0, 30.0, 50.0]), bias=rng.random() < 0.4)
    T = _log_int(rng, 1, 4096)
    n = _log_int(rng, 1, 4096)
    B = max(1, min(_log_int(rng, 1, 64), (1 << 24) // ((n + T) * Hkv * D)))
    return dict(op=op, dtype=dtype, B=B, T=T, Hkv=Hkv, D=D, page=page, len=n, ragged=rng.random() < 0.5)


def _randn(shape, g, dt, mul=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * mul).to(dt)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _positions(c, n_axes, g):
    """[B, S, axes]: a text's running positions from a random start, or the places of a grid of tokens."""
    B, S = c["B"], c["S"]
    t = torch.arange(S, device="cuda").expand(B, S)
    if n_axes > 1:  # the last axis fastest, sides about equal; an image's rows and columns, a video's frames
        side = max(1, round(S ** (1.0 / n_axes)))
        t = torch.stack([t // side ** (n_axes - 1 - a) % (side if a else S + 1) for a in range(n_axes)], 2)
    else:
        t = t[:, :, None]
    start = torch.randint(0, c["far"] + 1, (B, 1, 1), generator=g, device="cuda")
    return (t + start).to(torch.int32).contiguous()


def _freqs(sections):
    """Radians a position for each pair: a falling ladder for each axis."""
    f = [10000.0 ** (-i / n) for n in sections for i in range(n)]
    return torch.tensor(f, dtype=torch.float64, device="cuda")


def _prepare_rope(c, s, g):
    dt, B, S, H, Hkv, D = _DT[c["dtype"]], c["B"], c["S"], c["H"], c["Hkv"], c["D"]
    sections = [int(x) for x in c["sections"].split(",")]
    if c["packed"]:
        qkv = _randn((B, S, H + 2 * Hkv, D), g, dt, 1.5)
        s["q"], s["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
    else:
        s["q"], s["k"] = _randn((B, S, H, D), g, dt, 1.5), _randn((B, S, Hkv, D), g, dt, 1.5)
    s["q_weight"] = s["k_weight"] = None
    if c["norm"]:
        s["q_weight"], s["k_weight"] = ((1 + _randn((D,), g, torch.float32, 0.2)).to(dt) for _ in range(2))
    s["positions"] = _positions(c, len(sections), g)
    s["freqs"] = _freqs(sections)
    s["axes"] = bytes(a for a, n in enumerate(sections) for _ in range(n))
    s["axis"] = torch.tensor(list(s["axes"]), dtype=torch.int64, device="cuda")
    s["eps"] = 1e-6 if c["norm"] else None
    if c["op"] == "bwd":
        s["dq_out"], s["dk_out"] = _randn((B, S, H, D), g, dt), _randn((B, S, Hkv, D), g, dt)


def _prepare_cache(s, pages, Hkv, page, D, g):
    """Pages that hold quantised rows: keys with an offset to each channel, as a model's keys have, and plain values."""
    for x, spread in (("k", 1.0), ("v", 0.0)):
        at = torch.randn((Hkv, 1, D), generator=g, device="cuda") * spread
        codes = torch.empty((pages, Hkv, page, D // 2), dtype=torch.uint8, device="cuda")
        scales = torch.empty((pages, Hkv, page, D // _GROUP, 2), dtype=torch.bfloat16, device="cuda")
        step = max(1, (1 << 25) // (Hkv * page * D))
        for p in range(0, pages, step):
            rows = torch.randn((min(step, pages - p), Hkv, page, D), generator=g, device="cuda") + at
            codes[p:p + step], scales[p:p + step] = _quantised(rows.to(torch.bfloat16))
        s[x + "_codes"], s[x + "_scales"] = codes, scales


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[c["dtype"]]
    s = {"case": c}
    if c["op"] in ("fwd", "bwd"):
        _prepare_rope(c, s, g)
        return s
    B, Hkv, D, page, n = c["B"], c["Hkv"], c["D"], c["page"], c["len"]
    if c["op"] == "decode":
        s["scale"] = D ** -0.5
        s["q"] = _randn((B, c["H"], D), g, dt, 2.0 if c["cap"] else 1.0)
        s["slopes"] = None
        if c["bias"]:  # the strongest head looks about two tokens back, the weakest 256
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["H"] + 1, device="cuda", dtype=torch.float32) / c["H"])
        lens = torch.full((B,), n, device="cuda", dtype=torch.float32)
        if c["ragged"]:
            low = max(n // 16, 1)
            lens = torch.exp(torch.rand((B,), generator=g, device="cuda") * math.log(n / low)) * low
            lens[0] = n
        s["lens"] = lens.round().clamp(1, n).to(torch.int32)
    else:
        T = c["T"]
        s["k"], s["v"] = _randn((B, T, Hkv, D), g, dt), _randn((B, T, Hkv, D), g, dt)
        s["lens"] = torch.randint(0, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["new"] = None
        if c["ragged"]:
            s["new"] = torch.randint(1, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            s["new"][0] = T
        s["after"] = s["lens"] + (T if s["new"] is None else s["new"])
        n = n + T
    pages = -(-n // page)
    total = B * pages + 3
    _prepare_cache(s, total, Hkv, page, D, g)
    s["table"] = torch.randperm(total, generator=g, device="cuda")[: B * pages].to(torch.int32).view(B, pages).contiguous()
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _cos_sin(s):
    """Of each token and pair, [B, S, 1, pairs]; the angle in 64 bits."""
    angle = s["positions"].double()[:, :, s["axis"]] * s["freqs"]
    return torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]


def _rotated(x, cos, sin, interleaved):
    n = 2 * cos.shape[-1]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        y[..., 0:n:2], y[..., 1:n:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :n // 2], x[..., n // 2:n]
        y[..., :n // 2], y[..., n // 2:n] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_fwd(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    got = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.float()
        if c["norm"]:
            y = y * torch.rsqrt((y * y).mean(3, keepdim=True) + s["eps"]) * w.float()
        got.append(_rotated(y, cos, sin, c["interleaved"]).to(x.dtype))
    return got


def _plain_bwd(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    grads, weights = [], []
    for x, w, d in ((s["q"], s["q_weight"], s["dq_out"]), (s["k"], s["k_weight"], s["dk_out"])):
        g = _rotated(d.float(), cos, -sin, c["interleaved"])
        if c["norm"]:
            y = x.float()
            r = torch.rsqrt((y * y).mean(3, keepdim=True) + s["eps"])
            y = y * r
            weights.append((g * y).sum((0, 1, 2)))
            g = g * w.float()
            g = (g - y * (g * y).mean(3, keepdim=True)) * r
        grads.append(g.to(x.dtype))
    return grads + weights


def _quantised(x):
    """Rows [..., D] -> codes [..., D / 2], scales [..., D / 64, 2]."""
    v = x.float().unflatten(-1, (-1, _GROUP))
    bits = v.amin(-1).view(torch.int32)
    low = bits & 0xffff
    z = torch.where((bits < 0) & (low != 0), bits - low + 0x10000, bits - low).view(torch.float32).double()
    span = v.amax(-1).double() - z
    cut = ((span / 15).float().view(torch.int32) >> 16) << 16
    cut = torch.where(cut.view(torch.float32).double() * 15 < span, cut + 0x10000, cut)
    scale = cut.view(torch.float32).double().clamp(min=2.0 ** -100)
    code = torch.floor((v.double() - z[..., None]) / scale[..., None] + 0.5).clamp(max=15).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, torch.stack((scale, z), -1).to(torch.bfloat16)


def _values(codes, scales):
    """What codes [..., D / 2] with scales [..., D / 64, 2] stand for, float32 [..., D]."""
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (-1, _GROUP))
    scales = scales.float()
    return (scales[..., 1:] + scales[..., :1] * code.float()).flatten(-2)


def _cached(s, x, n):
    """The first n tokens of each sequence, float32 [B, n, Hkv, D]."""
    table = s["table"].long()
    v = _values(s[x + "_codes"][table], s[x + "_scales"][table])  # [B, pages, Hkv, page, D]
    return v.transpose(2, 3).flatten(1, 2)[:, :n]


def _plain_append(s):
    c = s["case"]
    t = torch.arange(c["T"], device="cuda")
    pos = s["lens"].long()[:, None] + t
    page, row = torch.gather(s["table"].long(), 1, pos // c["page"]), pos % c["page"]
    for x in ("k", "v"):
        codes, scales = _quantised(s[x])
        if s["new"] is None:
            s[x + "_codes"][page, :, row], s[x + "_scales"][page, :, row] = codes, scales
        else:
            live = t < s["new"].long()[:, None]
            p, r = page[live], row[live]
            s[x + "_codes"][p, :, r], s[x + "_scales"][p, :, r] = codes[live], scales[live]
    n = c["len"] + c["T"]
    there = (torch.arange(n, device="cuda") < s["after"].long()[:, None])[:, :, None, None]
    return [torch.where(there, _cached(s, x, n), 0.0).to(s["k"].dtype) for x in ("k", "v")]


def _plain_decode(s):
    c = s["case"]
    B, H, Hkv, D, n = c["B"], c["H"], c["Hkv"], c["D"], c["len"]
    k, v = _cached(s, "k", n), _cached(s, "v", n)
    q = s["q"].float().view(B, Hkv, H // Hkv, D)
    x = (q @ k.permute(0, 2, 3, 1)) * s["scale"]
    if c["cap"]:
        x = torch.tanh(x / c["cap"]) * c["cap"]
    back = s["lens"].long()[:, None] - 1 - torch.arange(n, device="cuda")
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, Hkv, H // Hkv, 1) * back.abs().float()[:, None, None, :]
    x = x.masked_fill((back < 0)[:, None, None, :], float("-inf"))
    m = x.amax(3, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(3, keepdim=True)
    out = (p @ v.transpose(1, 2)) / l
    return out.reshape(B, H, D).to(s["q"].dtype), (m + torch.log(l)).reshape(B, H)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import context_attention_dits_gb300 as cpa
    c = s["case"]
    if c["op"] in ("fwd", "bwd"):
        q, k = s["q"], s["k"]
        rule = dict(positions=s["positions"], freqs=s["freqs"], axes=s["axes"], interleaved=c["interleaved"],
                    eps=s["eps"], q_weight=s["q_weight"], k_weight=s["k_weight"])
        B, S, H, D = q.shape
        yq, yk = (torch.empty((B, S, n, D), dtype=q.dtype, device=q.device) for n in (H, c["Hkv"]))
        if c["op"] == "fwd":
            cpa.cp_qk_norm_rope_fwd(q, k, yq, yk, **rule)
            return [yq, yk]
        if not c["norm"]:
            cpa.cp_qk_norm_rope_bwd(q, k, s["dq_out"], s["dk_out"], yq, yk, **rule)
            return [yq, yk]
        wq, wk = (torch.empty((D,), dtype=torch.float32, device=q.device) for _ in range(2))
        cpa.cp_qk_norm_rope_bwd(q, k, s["dq_out"], s["dk_out"], yq, yk, dq_weight=wq, dk_weight=wk, **rule)
        return [yq, yk, wq, wk]
    cache = (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["table"])
    if c["op"] == "append":
        cpa.cp_paged_kv_append_q4(s["k"], s["v"], *cache, s["lens"], new_lens=s["new"])
        k, v = (torch.empty((c["B"], c["len"] + c["T"], c["Hkv"], c["D"]), dtype=s["k"].dtype, device="cuda")
                for _ in range(2))
        cpa.cp_paged_kv_read_q4(*cache, s["after"], k, v)
        return [k, v]
    q = s["q"]
    out = torch.empty_like(q)
    lse = torch.empty((c["B"], c["H"]), dtype=torch.float32, device=q.device)
    cpa.cp_paged_attn_decode_q4(q, *cache, s["lens"], out, lse, s["scale"], softcap=c["cap"], slopes=s["slopes"])
    return out, lse


def run(state):
    if own:
        return _own(state)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "append": _plain_append, "decode": _plain_decode}[
        state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _row_bytes(D):
    """A cached row of one head: codes and scales."""
    return D // 2 + D // _GROUP * 4


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] in ("fwd", "bwd"):
        tokens = c["B"] * c["S"]
        values = tokens * (c["H"] + c["Hkv"]) * c["D"]
        places = 4.0 * tokens * len(c["sections"].split(","))
        if c["op"] == "fwd":  # in, out; square and sum, scale, rotate
            return {"bytes": 2.0 * values * e + places, "flops": (7.0 if c["norm"] else 3.0) * values}
        # the gradient in and out, and the rows themselves where there is a norm
        return {"bytes": (3.0 if c["norm"] else 2.0) * values * e + places, "flops": (14.0 if c["norm"] else 3.0) * values}
    if c["op"] == "append":
        T = c["T"] * (0.5 if c["ragged"] and c["T"] > 1 else 1.0)
        rows = 2.0 * c["B"] * c["Hkv"]
        # the new rows in and their codes out; the codes of all rows in and their values, with the zeros behind, out
        n = c["len"] / 2 + T
        return {"bytes": rows * (T * (c["D"] * e + _row_bytes(c["D"])) + n * _row_bytes(c["D"]) +
                                 (c["len"] + c["T"]) * c["D"] * e), "flops": rows * c["D"] * (4.0 * T + 2.0 * n)}
    # a ragged batch: log-uniform lengths from len / 16 to len have the mean 15 / (16 ln 16) len
    mean = c["len"] * (15 / (16 * math.log(16)) if c["ragged"] and c["len"] >= 16 else 1.0)
    tokens = c["B"] * mean
    return {"bytes": tokens * (2 * c["Hkv"] * _row_bytes(c["D"]) + 4.0 / c["page"]) + c["B"] * c["H"] * (2 * c["D"] * e + 4),
            "flops": 4.0 * tokens * c["H"] * c["D"]}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_turn(s):
    """e^(i angle) of each token and pair, complex128 [B, S, pairs]."""
    at = torch.stack([s["positions"][..., a] for a in s["axes"]], -1).to(torch.float64)
    return torch.exp(1j * (at * s["freqs"].view(1, 1, -1)))


def _exact_rotate(x, turn, interleaved):
    n = turn.shape[-1]
    if interleaved:
        z = torch.view_as_complex(x[..., :2 * n].unflatten(-1, (n, 2)).contiguous())
        return torch.cat((torch.view_as_real(z * turn[:, :, None]).flatten(-2), x[..., 2 * n:]), -1)
    z = torch.complex(x[..., :n].contiguous(), x[..., n:2 * n].contiguous()) * turn[:, :, None]
    return torch.cat((z.real, z.imag, x[..., 2 * n:]), -1)


def _exact_rope(s):
    c = s["case"]
    turn = _exact_turn(s)
    outs, weights = [], []
    for x in ("q", "k"):
        v = s[x].to(torch.float64)
        w = s[x + "_weight"].to(torch.float64) if c["norm"] else None
        size = torch.sqrt(v.square().sum(-1, keepdim=True) / c["D"] + s["eps"]) if c["norm"] else None
        if c["op"] == "fwd":
            outs.append(_exact_rotate(v / size * w if c["norm"] else v, turn, c["interleaved"]))
            continue
        g = _exact_rotate(s["d" + x + "_out"].to(torch.float64), turn.conj(), c["interleaved"])
        if c["norm"]:
            unit = v / size
            weights.append(torch.einsum("bshd,bshd->d", g, unit))
            g = g * w
            g = (g - unit * torch.einsum("bshd,bshd->bsh", g, unit)[..., None] / c["D"]) / size
        outs.append(g)
    return outs + weights


def _exact_rows(s, x, b, n):
    """The first n tokens of sequence b, float64 [n, Hkv, D], from codes and scales."""
    page = s["case"]["page"]
    at = torch.arange(n, device="cuda")
    p, r = s["table"][b].long()[at // page], at % page
    byte = s[x + "_codes"][p, :, r].to(torch.float64)  # [n, Hkv, D / 2]
    high = torch.floor(byte / 16)
    code = torch.empty((*byte.shape[:2], byte.shape[2] * 2), dtype=torch.float64, device="cuda")
    code[..., 0::2], code[..., 1::2] = byte - 16 * high, high
    sz = s[x + "_scales"][p, :, r].to(torch.float64).repeat_interleave(_GROUP, 2)  # [n, Hkv, D, 2]
    return sz[..., 1] + sz[..., 0] * code


def _bf16_near(x):
    """The bf16 numbers about x, below and above it by a step or two."""
    near = x.float().to(torch.bfloat16)
    inf = torch.full_like(near, math.inf)
    down, up = torch.nextafter(near, -inf), torch.nextafter(near, inf)
    return torch.stack((down, near, up)).to(torch.float64)


def _exact_stored(rows):
    """The values that the cache holds for rows [..., D]."""
    v = rows.to(torch.float64).unflatten(-1, (-1, _GROUP))
    least, most = v.min(-1).values, v.max(-1).values
    near = _bf16_near(least)
    z = torch.where(near <= least, near, -math.inf).max(0).values
    near = _bf16_near((most - z) / 15)
    scale = torch.where(near * 15 >= most - z, near, math.inf).min(0).values.clamp(min=2.0 ** -100)
    code = torch.zeros_like(v)
    for n in range(1, 16):  # codes count the borders that a value has reached
        code += v - z[..., None] >= (n - 0.5) * scale[..., None]
    return (z[..., None] + scale[..., None] * code).flatten(-2)


def _exact_append(s):
    c = s["case"]
    outs = []
    for x in ("k", "v"):
        got = torch.zeros((c["B"], c["len"] + c["T"], c["Hkv"], c["D"]), dtype=torch.float64, device="cuda")
        for b, (n, after) in enumerate(zip(s["lens"].tolist(), s["after"].tolist())):
            got[b, :n] = _exact_rows(s, x, b, n)
            got[b, n:after] = _exact_stored(s[x][b, :after - n])
        outs.append(got)
    return outs


def _exact_decode(s):
    c = s["case"]
    B, H, Hkv, D = c["B"], c["H"], c["Hkv"], c["D"]
    out = torch.zeros((B, H, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, H), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        k, v = _exact_rows(s, "k", b, n), _exact_rows(s, "v", b, n)
        for h in range(H):
            hk = h // (H // Hkv)
            z = s["scale"] * (k[:, hk] @ s["q"][b, h].double())
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if s["slopes"] is not None:
                z = z - s["slopes"][h].double() * torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.float64)
            lse[b, h] = torch.logsumexp(z, 0)
            out[b, h] = torch.exp(z - lse[b, h]) @ v[:, hk]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"fwd": _exact_rope, "bwd": _exact_rope, "append": _exact_append, "decode": _exact_decode}[case["op"]](s)
