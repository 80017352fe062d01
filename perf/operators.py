"""Workloads of the attention operators that language models add to this library.

Four operators, each in a plain torch form and as the library's own call:

* ``fwd``    block attention with a score rule: scores capped by a tanh, a bias
  that falls with distance, a causal mask with an open prefix, a document mask,
  query heads that share key/value heads;
* ``bwd``    its gradients dq, dk, dv;
* ``decode`` attention of one new token per sequence over a paged cache;
* ``append`` the new tokens' keys and values into that cache.

Outputs of ``fwd``: out (the inputs' type) and lse (float32). ``bwd``: dq, dk, dv
in the inputs' type. ``decode``: out and lse. ``append``: both caches, whole.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a short prompt of one user: the call's latency
        dict(name="fwd_short", op="fwd", dtype="bf16", B=1, Sq=97, Skv=97, H=8, Hkv=2, D=64, cap=30.0, bias=False,
             causal=True, prefix=0, docs=0),
        # documents packed into one training row of 4608 tokens, the last places padding
        dict(name="fwd_docs", op="fwd", dtype="bf16", B=1, Sq=4608, Skv=4608, H=24, Hkv=24, D=128, cap=0.0, bias=False,
             causal=True, prefix=0, docs=9),
        # a prompt of up to 512 text tokens that sees itself whole, then a causal stretch; odd length, shared heads
        dict(name="fwd_prefix", op="fwd", dtype="bf16", B=2, Sq=4607, Skv=4607, H=24, Hkv=8, D=128, cap=0.0, bias=True,
             causal=True, prefix=512, docs=0),
        # fp32, every pair taking part, both score terms: a small model's check run
        dict(name="fwd_f32", op="fwd", dtype="f32", B=2, Sq=387, Skv=387, H=4, Hkv=4, D=64, cap=30.0, bias=True,
             causal=False, prefix=0, docs=0),
        # gradients of a short row: latency
        dict(name="bwd_short", op="bwd", dtype="bf16", B=1, Sq=130, Skv=130, H=8, Hkv=2, D=64, cap=30.0, bias=False,
             causal=True, prefix=0, docs=0),
        # the training step's backward at the length and heads of this library's headline workload
        dict(name="bwd_capped", op="bwd", dtype="bf16", B=1, Sq=4608, Skv=4608, H=24, Hkv=8, D=128, cap=50.0,
             bias=False, causal=True, prefix=0, docs=0),
        # fp32 gradients of packed documents
        dict(name="bwd_f32", op="bwd", dtype="f32", B=1, Sq=700, Skv=700, H=6, Hkv=3, D=128, cap=0.0, bias=True,
             causal=True, prefix=0, docs=3),
        # one user, a short conversation: the latency of a token
        dict(name="decode_one", op="decode", dtype="bf16", B=1, H=24, Hkv=8, D=128, page=16, len=1000, ragged=False,
             cap=50.0, bias=False),
        # a serving batch whose conversations differ in length
        dict(name="decode_batch", op="decode", dtype="bf16", B=48, H=24, Hkv=8, D=128, page=64, len=8192, ragged=True,
             cap=0.0, bias=True),
        # two very long contexts
        dict(name="decode_long", op="decode", dtype="bf16", B=2, H=32, Hkv=4, D=128, page=128, len=262144, ragged=False,
             cap=50.0, bias=False),
        # the new token of every sequence of a serving batch
        dict(name="append_token", op="append", dtype="bf16", B=64, T=1, Hkv=8, D=128, page=16, len=1024, ragged=False),
        # prompts of different lengths, padded to the longest, into the cache
        dict(name="append_chunk", op="append", dtype="bf16", B=6, T=4607, Hkv=8, D=128, page=64, len=512, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "decode", "decode", "append"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 3, 4, 8])
    cap = rng.choice([0.0, 15.0, 30.0, 50.0])
    bias = rng.random() < 0.4
    if op in ("fwd", "bwd"):
        most = {("fwd", "bf16"): 4608, ("bwd", "bf16"): 4096, ("fwd", "f32"): 800, ("bwd", "f32"): 600}[op, dtype]
        Skv = _log_int(rng, 1, most)
        causal = rng.random() < 0.7
        # a chunk of the last queries against every key so far, or all of them
        Sq = Skv if rng.random() < 0.75 else rng.randint(1, Skv)
        prefix = rng.randint(1, Skv) if causal and rng.random() < 0.3 else 0
        docs = rng.randint(1, 1 + Skv // 64) if rng.random() < 0.35 else 0
        # the work stays below the largest listed case's
        most_work = 12 * 4608 * 4608 * 128 if dtype == "bf16" else 4 * 600 * 600 * 128
        while H * Sq * Skv * D > most_work and Hkv > 1:
            H, Hkv = H // Hkv, 1
        B = max(1, min(rng.choice([1, 1, 2, 3, 5]), most_work // (H * Sq * Skv * D)))
        return dict(op=op, dtype=dtype, B=B, Sq=Sq, Skv=Skv, H=H, Hkv=Hkv, D=D, cap=cap, bias=bias, causal=causal,
                    prefix=prefix, docs=docs)
    page = rng.choice([1, 8, 16, 32, 64, 128, 256])
    if op == "decode":
        n = _log_int(rng, 1, 65536)
        B = max(1, min(_log_int(rng, 1, 128), (1 << (28 if dtype == "bf16" else 27)) // (n * Hkv * D)))
        return dict(op=op, dtype=dtype, B=B, H=H, Hkv=Hkv, D=D, page=page, len=n, ragged=rng.random() < 0.6, cap=cap,
                    bias=bias)
    T = _log_int(rng, 1, 4096)
    n = _log_int(rng, 1, 4096)
    B = max(1, min(_log_int(rng, 1, 64), (1 << 24) // ((n + T) * Hkv * D)))
    return dict(op=op, dtype=dtype, B=B, T=T, Hkv=Hkv, D=D, page=page, len=n, ragged=rng.random() < 0.5)


def _randn(shape, g, dt, mul=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * mul).to(dt)


def _slopes(c):
    """A slope per query head, 2^(-8 (h + 1) / H): the strongest head looks about two tokens back, the weakest 256."""
    h = torch.arange(1, c["H"] + 1, device="cuda", dtype=torch.float32)
    return torch.exp2(-8.0 * h / c["H"])


def _docs(c, g):
    """Ascending document ids of packed rows, [B, Skv]; the last 1 % of a row is padding (id -1)."""
    B, S, n = c["B"], c["Skv"], c["docs"]
    cuts = torch.randint(0, max(S, 1), (B, n - 1), generator=g, device="cuda").sort(1).values
    pos = torch.arange(S, device="cuda").expand(B, S).contiguous()
    ids = torch.searchsorted(cuts, pos, right=True).to(torch.int32) if n > 1 else torch.zeros_like(pos, dtype=torch.int32)
    return torch.where(pos >= S - S // 100, torch.full_like(ids, -1), ids).contiguous()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[c["dtype"]]
    s = {"case": c}
    if c["op"] in ("fwd", "bwd"):
        B, Sq, Skv, H, Hkv, D = c["B"], c["Sq"], c["Skv"], c["H"], c["Hkv"], c["D"]
        s["scale"] = D ** -0.5
        s["q"] = _randn((B, Sq, H, D), g, dt, 2.0 if c["cap"] else 1.0)
        s["k"] = _randn((B, Skv, Hkv, D), g, dt)
        s["v"] = _randn((B, Skv, Hkv, D), g, dt)
        s["slopes"] = _slopes(c) if c["bias"] else None
        s["prefix"] = None
        if c["prefix"]:
            low = max(1, c["prefix"] // 2)
            s["prefix"] = torch.randint(low, c["prefix"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["kv_docs"] = _docs(c, g) if c["docs"] else None
        s["q_docs"] = s["kv_docs"][:, Skv - Sq:].contiguous() if c["docs"] else None
        s["q_pos0"] = Skv - Sq
        if c["op"] == "bwd":
            s["dout"] = _randn((B, Sq, H, D), g, dt)
            s["out"], s["lse"] = _plain_fwd(s)
        return s
    if c["op"] == "decode":
        B, H, Hkv, D, page, n = c["B"], c["H"], c["Hkv"], c["D"], c["page"], c["len"]
        s["scale"] = D ** -0.5
        s["q"] = _randn((B, H, D), g, dt, 2.0 if c["cap"] else 1.0)
        s["slopes"] = _slopes(c) if c["bias"] else None
        lens = torch.full((B,), n, device="cuda", dtype=torch.float32)
        if c["ragged"]:
            low = max(n // 16, 1)
            lens = torch.exp(torch.rand((B,), generator=g, device="cuda") * math.log(n / low)) * low
            lens[0] = n
        s["lens"] = lens.round().clamp(1, n).to(torch.int32)
    else:
        B, Hkv, D, page, n, T = c["B"], c["Hkv"], c["D"], c["page"], c["len"], c["T"]
        s["k"] = _randn((B, T, Hkv, D), g, dt)
        s["v"] = _randn((B, T, Hkv, D), g, dt)
        s["lens"] = torch.randint(0, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["new"] = None
        if c["ragged"]:
            s["new"] = torch.randint(1, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            s["new"][0] = T
        n = n + T
    pages = -(-n // page)
    total = B * pages + 3
    s["k_cache"] = _randn((total, page, Hkv, D), g, dt)
    s["v_cache"] = _randn((total, page, Hkv, D), g, dt)
    s["table"] = torch.randperm(total, generator=g, device="cuda")[: B * pages].to(torch.int32).view(B, pages).contiguous()
    return s


def _heads_first(x, group):
    """[B, S, heads, D] -> float32 [B, heads * group, S, D], each head repeated for the query heads that share it."""
    x = x.float().transpose(1, 2)
    return x if group == 1 else x.repeat_interleave(group, 1)


def _plain_scores(s):
    """The scores after cap, bias and mask [B, H, Sq, Skv] (-inf where a pair takes no part), and the cap's tanh."""
    c = s["case"]
    x = (_heads_first(s["q"], 1) @ _heads_first(s["k"], c["H"] // c["Hkv"]).transpose(2, 3)) * s["scale"]
    t = None
    if c["cap"]:
        t = torch.tanh(x / c["cap"])
        x = t * c["cap"]
    i = torch.arange(c["Sq"], device="cuda").view(-1, 1) + s["q_pos0"]
    j = torch.arange(c["Skv"], device="cuda").view(1, -1)
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, -1, 1, 1) * (i - j).abs().float()
    allowed = None
    if c["causal"]:
        allowed = (j <= i).expand(c["B"], -1, -1)
        if s["prefix"] is not None:
            allowed = allowed | (j < s["prefix"].view(-1, 1, 1))
    if s["q_docs"] is not None:
        same = (s["q_docs"][:, :, None] == s["kv_docs"][:, None, :]) & (s["q_docs"] >= 0)[:, :, None]
        allowed = same if allowed is None else allowed & same
    if allowed is not None:
        x = x.masked_fill(~allowed[:, None], float("-inf"))
    return x, t


def _plain_fwd(s):
    c = s["case"]
    x, _ = _plain_scores(s)
    m = x.amax(3, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    l = p.sum(3, keepdim=True)
    out = (p @ _heads_first(s["v"], c["H"] // c["Hkv"])) / torch.where(l == 0, torch.ones_like(l), l)
    return out.transpose(1, 2).to(s["q"].dtype).contiguous(), (m + torch.log(l)).squeeze(3)


def _plain_bwd(s):
    c, dt = s["case"], s["q"].dtype
    B, Hkv, G, D = c["B"], c["Hkv"], c["H"] // c["Hkv"], c["D"]
    x, t = _plain_scores(s)
    lse = torch.where(s["lse"] == float("-inf"), torch.full_like(s["lse"], float("inf")), s["lse"])
    p = torch.exp(x - lse[..., None])
    do, o = _heads_first(s["dout"], 1), _heads_first(s["out"], 1)
    ds = p * (do @ _heads_first(s["v"], G).transpose(2, 3) - (do * o).sum(3, keepdim=True))
    if t is not None:
        ds = ds * (1 - t * t)
    dq = (ds @ _heads_first(s["k"], G)) * s["scale"]
    dk = (ds.transpose(2, 3) @ _heads_first(s["q"], 1)) * s["scale"]
    dv = p.transpose(2, 3) @ do
    dk, dv = (y.view(B, Hkv, G, c["Skv"], D).sum(2) for y in (dk, dv))
    return [y.transpose(1, 2).to(dt).contiguous() for y in (dq, dk, dv)]


def _plain_decode(s):
    c = s["case"]
    B, H, Hkv, D, n = c["B"], c["H"], c["Hkv"], c["D"], c["len"]
    k, v = (s[x][s["table"].long()].reshape(B, -1, Hkv, D)[:, :n].float() for x in ("k_cache", "v_cache"))
    q = s["q"].float().view(B, Hkv, H // Hkv, D)
    x = (q @ k.permute(0, 2, 3, 1)) * s["scale"]
    if c["cap"]:
        x = torch.tanh(x / c["cap"]) * c["cap"]
    j = torch.arange(n, device="cuda")
    back = s["lens"].long()[:, None] - 1 - j
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, Hkv, H // Hkv, 1) * back.abs().float()[:, None, None, :]
    x = x.masked_fill((back < 0)[:, None, None, :], float("-inf"))
    m = x.amax(3, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(3, keepdim=True)
    out = (p @ v.transpose(1, 2)) / l
    return out.reshape(B, H, D).to(s["q"].dtype), (m + torch.log(l)).reshape(B, H)


def _plain_append(s):
    c = s["case"]
    t = torch.arange(c["T"], device="cuda")
    pos = s["lens"].long()[:, None] + t
    row = torch.gather(s["table"].long(), 1, pos // c["page"]) * c["page"] + pos % c["page"]
    if s["new"] is not None:
        live = t < s["new"].long()[:, None]
        row, k, v = row[live], s["k"][live], s["v"][live]
    else:
        row, k, v = row.reshape(-1), s["k"].flatten(0, 1), s["v"].flatten(0, 1)
    s["k_cache"].flatten(0, 1)[row] = k
    s["v_cache"].flatten(0, 1)[row] = v
    return s["k_cache"], s["v_cache"]


def _own(s):
    import context_attention_dits_gb300 as cpa
    c = s["case"]
    if c["op"] == "append":
        cpa.cp_paged_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], new_lens=s["new"])
        return s["k_cache"], s["v_cache"]
    q = s["q"]
    if c["op"] == "decode":
        out = torch.empty_like(q)
        lse = torch.empty((c["B"], c["H"]), dtype=torch.float32, device=q.device)
        cpa.cp_paged_attn_decode(q, s["k_cache"], s["v_cache"], s["table"], s["lens"], out, lse, s["scale"],
                                 softcap=c["cap"], slopes=s["slopes"])
        return out, lse
    rule = dict(softcap=c["cap"], slopes=s["slopes"], causal=c["causal"], prefix_lens=s["prefix"], q_docs=s["q_docs"],
                kv_docs=s["kv_docs"], q_pos0=s["q_pos0"])
    if c["op"] == "fwd":
        out = torch.empty_like(q)
        lse = torch.empty((c["B"], c["H"], c["Sq"]), dtype=torch.float32, device=q.device)
        cpa.cp_scored_attn_fwd(q, s["k"], s["v"], out, lse, s["scale"], **rule)
        return out, lse
    dq, dk, dv = torch.empty_like(q), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    cpa.cp_scored_attn_bwd(q, s["k"], s["v"], s["out"], s["dout"], s["lse"], dq, dk, dv, s["scale"], **rule)
    return dq, dk, dv


def run(state):
    if own:
        return _own(state)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "decode": _plain_decode, "append": _plain_append}[
        state["case"]["op"]](state)


def _pairs(c):
    """Query-key pairs per head that take part (documents: equal lengths assumed, as their cuts differ by seed)."""
    Sq, Skv = c["Sq"], c["Skv"]
    n = Sq * Skv
    if c["causal"]:
        n = Sq * (Skv - Sq) + Sq * (Sq + 1) // 2
        if c["prefix"]:
            n = min(Sq * Skv, n + c["prefix"] * c["prefix"] // 2)
    if c["docs"]:
        n = max(Sq, n // c["docs"])
    return c["B"] * n


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] in ("fwd", "bwd"):
        nq, nk = c["B"] * c["Sq"] * c["H"], c["B"] * c["Skv"] * c["Hkv"]
        if c["op"] == "fwd":  # q, out, k, v, lse; two products a pair
            return {"bytes": (2 * nq + 2 * nk) * c["D"] * e + 4 * nq, "flops": 4.0 * c["H"] * c["D"] * _pairs(c)}
        # q, out, dout, dq, k, v, dk, dv, lse; five products a pair
        return {"bytes": (4 * nq + 4 * nk) * c["D"] * e + 4 * nq, "flops": 10.0 * c["H"] * c["D"] * _pairs(c)}
    if c["op"] == "decode":
        # a ragged batch: log-uniform lengths from len / 16 to len have the mean 15 / (16 ln 16) len
        mean = c["len"] * (15 / (16 * math.log(16)) if c["ragged"] and c["len"] >= 16 else 1.0)
        tokens = c["B"] * mean
        return {"bytes": tokens * (2 * c["Hkv"] * c["D"] * e + 4.0 / c["page"]) + c["B"] * c["H"] * (2 * c["D"] * e + 4),
                "flops": 4.0 * tokens * c["H"] * c["D"]}
    tokens = c["B"] * c["T"] * (0.5 if c["ragged"] and c["T"] > 1 else 1.0)
    return {"bytes": 4.0 * tokens * c["Hkv"] * c["D"] * e, "flops": 0.0}


def _exact_pair(s, b, h):
    """One head of one batch entry in 64 bits: masked scores [Sq, Skv] and the derivative of the cap."""
    c = s["case"]
    hk = h // (c["H"] // c["Hkv"])
    z = s["scale"] * torch.einsum("id,jd->ij", s["q"][b, :, h].double(), s["k"][b, :, hk].double())
    slope = torch.ones_like(z)
    if c["cap"]:
        slope = torch.cosh((z / c["cap"]).clamp(-300, 300)) ** -2
        z = c["cap"] * torch.tanh(z / c["cap"])
    pq = torch.arange(s["q_pos0"], s["q_pos0"] + c["Sq"], device="cuda", dtype=torch.float64)[:, None]
    pk = torch.arange(c["Skv"], device="cuda", dtype=torch.float64)[None, :]
    if s["slopes"] is not None:
        z = z - s["slopes"][h].double() * torch.abs(pq - pk)
    off = torch.zeros_like(z, dtype=torch.bool)
    if c["causal"]:
        off |= pk > pq
        if s["prefix"] is not None:
            off &= pk >= s["prefix"][b].double()
    if s["q_docs"] is not None:
        dq, dk = s["q_docs"][b], s["kv_docs"][b]
        off |= dq[:, None] != dk[None, :]
        off |= (dq < 0)[:, None]
    z[off] = -math.inf
    return z, slope, hk


def _exact_attn(s):
    c = s["case"]
    B, Sq, Skv, H, Hkv, D = c["B"], c["Sq"], c["Skv"], c["H"], c["Hkv"], c["D"]
    f8 = dict(dtype=torch.float64, device="cuda")
    if c["op"] == "fwd":
        out, lse = torch.zeros((B, Sq, H, D), **f8), torch.zeros((B, H, Sq), **f8)
        for b in range(B):
            for h in range(H):
                z, _, hk = _exact_pair(s, b, h)
                lse[b, h] = torch.logsumexp(z, 1)
                w = torch.exp(z - torch.where(torch.isinf(lse[b, h]), torch.zeros_like(lse[b, h]), lse[b, h])[:, None])
                out[b, :, h] = w @ s["v"][b, :, hk].double()
        return out, lse
    dq = torch.zeros((B, Sq, H, D), **f8)
    dk, dv = (torch.zeros((B, Skv, Hkv, D), **f8) for _ in range(2))
    for b in range(B):
        for h in range(H):
            z, slope, hk = _exact_pair(s, b, h)
            l = s["lse"][b, h].double()
            w = torch.exp(z - torch.where(torch.isinf(l), torch.zeros_like(l), l)[:, None])
            g, o = s["dout"][b, :, h].double(), s["out"][b, :, h].double()
            dv[b, :, hk] += torch.einsum("ij,id->jd", w, g)
            w *= torch.einsum("id,jd->ij", g, s["v"][b, :, hk].double()) - (g * o).sum(1)[:, None]
            w *= slope * s["scale"]
            dq[b, :, h] = w @ s["k"][b, :, hk].double()
            dk[b, :, hk] += torch.einsum("ij,id->jd", w, s["q"][b, :, h].double())
    return dq, dk, dv


def _exact_decode(s):
    c = s["case"]
    B, H, Hkv, D, page = c["B"], c["H"], c["Hkv"], c["D"], c["page"]
    out = torch.zeros((B, H, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, H), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        at = torch.arange(n, device="cuda")
        pages, rows = s["table"][b].long()[at // page], at % page
        for hk in range(Hkv):
            k, v = s["k_cache"][pages, rows, hk].double(), s["v_cache"][pages, rows, hk].double()
            hs = slice(hk * (H // Hkv), (hk + 1) * (H // Hkv))
            z = s["scale"] * (s["q"][b, hs].double() @ k.T)
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if s["slopes"] is not None:
                z = z - s["slopes"][hs].double()[:, None] * (n - 1 - at).double()
            lse[b, hs] = torch.logsumexp(z, 1)
            out[b, hs] = torch.exp(z - lse[b, hs, None]) @ v
    return out, lse


def _exact_append(s):
    c = s["case"]
    lens, new, table = s["lens"].tolist(), None if s["new"] is None else s["new"].tolist(), s["table"].long()
    k, v = s["k_cache"].double(), s["v_cache"].double()
    for b in range(c["B"]):
        at = torch.arange(lens[b], lens[b] + (c["T"] if new is None else new[b]), device="cuda")
        k[table[b][at // c["page"]], at % c["page"]] = s["k"][b, : len(at)].double()
        v[table[b][at // c["page"]], at % c["page"]] = s["v"][b, : len(at)].double()
    return k, v


def exact(case, seed):
    s = prepare(case, seed)
    return {"fwd": _exact_attn, "bwd": _exact_attn, "decode": _exact_decode, "append": _exact_append}[case["op"]](s)
