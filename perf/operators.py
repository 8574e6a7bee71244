"""The dense paged layer's two operators, as they are measured: appending keys and values to the paged cache with the
rotation applied on the way (csla_kv_append), and attention of each request's new tokens over that cache
(csla_kv_attend), from single-token decode to long prefill chunks.

A case's lengths come from its own fields (a seeded draw of T new tokens and a prior context per request); its tensors
from the seed given to prepare().  Pages hold 128 tokens; the pool's pages are shuffled."""
import math
import random

import torch

own = False
PAGE = 128
DEV = "cuda"
EPS = 1e-6


def _case(name, op, B, t, prior, HQ, HK, D, **kw):
    c = dict(name=name, op=op, B=B, t_lo=t[0], t_hi=t[1], p_lo=prior[0], p_hi=prior[1], lens=7, HQ=HQ, HK=HK, D=D, d_rope=64, pairs="adjacent",
             norm=True, sink=False, window=0, theta=10000.0, dtype="bf16", fused=False)
    c.update(kw)
    return c


def listed():
    return [
        # one user, one short context: the latency of a token
        _case("decode_1x900", "attend", 1, (1, 1), (900, 900), 64, 8, 128, sink=True),
        # the batch and context of this repository's decode benchmark, in a dense layer of 8 KV heads
        _case("decode_8x131072", "attend", 8, (1, 1), (131071, 131071), 64, 8, 128, sink=True),
        # a serving batch of requests of all ages
        _case("decode_64_ragged", "attend", 64, (1, 1), (0, 32767), 32, 8, 128, pairs="halves", d_rope=128, norm=False),
        # one KV head for all query heads, few long requests
        _case("decode_4x262144_one_kv_head", "attend", 4, (1, 1), (262143, 262143), 64, 1, 128, sink=True),
        # a sliding-window layer with as many KV heads as query heads
        _case("decode_32_window", "attend", 32, (1, 1), (900, 65000), 16, 16, 64, window=1000, sink=True, pairs="halves"),
        # a few tokens per request: drafts to verify
        _case("few_tokens_32", "attend", 32, (5, 5), (500, 16000), 32, 8, 128),
        # a prompt from its first token
        _case("prompt_2048", "attend", 1, (2048, 2048), (0, 0), 32, 8, 128, pairs="halves", d_rope=128),
        # one chunk of a long prompt, of the chunk length of this repository's prefill benchmark
        _case("chunk_4096_after_16384", "attend", 1, (4096, 4096), (16384, 16384), 32, 4, 128, sink=True),
        # prompts and decoding requests in one ragged batch, odd head count, q a slice of a fused projection
        _case("mixed_12", "attend", 12, (1, 1500), (0, 8000), 28, 4, 64, norm=False, pairs="halves", fused=True, lens=3),
        # the append of a decode step
        _case("append_8", "append", 8, (1, 1), (3000, 5000), 64, 8, 128),
        # the append of a long prefill chunk
        _case("append_8192", "append", 1, (8192, 8192), (0, 0), 64, 8, 128),
        # a ragged append of slices of a fused f32 projection
        _case("append_ragged_f32", "append", 24, (1, 900), (0, 3000), 8, 4, 64, norm=False, pairs="halves", dtype="f32", fused=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 2)))) - 1))


def lengths(c):
    """The requests' new tokens and contexts (new tokens included)."""
    rng = random.Random(c["lens"])
    T = [_spread(rng, c["t_lo"], c["t_hi"]) for _ in range(c["B"])]
    return T, [t + _spread(rng, c["p_lo"], c["p_hi"]) for t in T]


def _cost(c):
    """Elements of the padded scores and of the gathered keys (what the plain form holds), and the visible pairs' products."""
    T, L = lengths(c)
    return c["B"] * c["HQ"] * max(T) * max(L), c["B"] * c["HK"] * max(L) * c["D"], work(c)["flops"]


def draw(rng):
    D = rng.choice((64, 128))
    HK = rng.choice((1, 2, 3, 4, 8, 16))
    G = rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    c = _case("", "attend", 1, (1, 1), (0, 0), HK * min(G, max(1, 64 // HK)), HK, D, d_rope=rng.choice((64, D)), pairs=rng.choice(("adjacent", "halves")),
              norm=rng.random() < 0.5, sink=rng.random() < 0.5, theta=rng.choice((10000.0, 500000.0)), fused=rng.random() < 0.3)
    c["lens"] = rng.randrange(1 << 20)
    kind = rng.choice(("decode", "decode", "few", "chunk", "mixed", "append", "append"))
    if kind == "append":
        c["op"], c["dtype"] = "append", rng.choice(("bf16", "f32"))
        c["B"] = _spread(rng, 1, 32)
        c["t_hi"] = _spread(rng, 1, 8192 // c["B"])
        c["t_lo"] = rng.choice((1, c["t_hi"]))
        c["p_hi"] = _spread(rng, 0, 4000)
    else:
        c["window"] = rng.choice((0, 0, 0, _spread(rng, 100, 3000)))
        c["B"] = _spread(rng, 1, 64) if kind in ("decode", "few") else _spread(rng, 1, 3 if kind == "chunk" else 12)
        c["p_hi"] = _spread(rng, 500, 131071) if kind in ("decode", "few") else _spread(rng, 0, 16384)
        c["t_hi"] = {"decode": 1, "few": rng.randint(2, 9), "chunk": _spread(rng, 100, 4096), "mixed": _spread(rng, 10, 1500)}[kind]
        c["t_lo"] = 1 if kind == "mixed" else c["t_hi"]
        c["p_lo"] = rng.choice((0, c["p_hi"] // 2))
        while True:
            scores, keys, flops = _cost(c)
            if scores <= 2.6e9 and keys <= 1.05e9 and flops <= 1.2e12:
                break
            c["p_hi"], c["t_hi"] = int(c["p_hi"] * 0.8), max(1, int(c["t_hi"] * 0.9))
            c["p_lo"], c["t_lo"] = min(c["p_lo"], c["p_hi"]), min(c["t_lo"], c["t_hi"])
    del c["name"]
    return c


def work(case):
    T, L = lengths(case)
    HQ, HK, D, W = case["HQ"], case["HK"], case["D"], case["window"] or 1 << 40
    N = sum(T)
    if case["op"] == "append":  # K and V of the new tokens read once and written once
        return {"bytes": N * HK * D * 2 * ((4 if case["dtype"] == "f32" else 2) + 2), "flops": 0}
    pairs = kept = 0
    for t, n in zip(T, L):
        first = max(0, n - t + 1 - W)  # the first token that the request's first new token sees
        kept += n - first
        full = max(0, min(t, n - W))  # new tokens that see a whole window; the others see all before them
        pairs += full * W if full else 0
        a, b = n - t + 1, n - full  # contexts of those that see everything
        pairs += (a + b) * (b - a + 1) // 2 if b >= a else 0
    return {"bytes": kept * HK * D * 2 * 2 + N * HQ * D * 2 * 2, "flops": 4 * D * HQ * pairs}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    T, L = lengths(case)
    B, HQ, HK, D, N = case["B"], case["HQ"], case["HK"], case["D"], sum(T)
    per = [-(-n // PAGE) for n in L]
    n_pages, wide = sum(per) + 3, max(per) + 1
    ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, wide), -1, dtype=torch.int32, device=DEV)
    start = [0]
    for b in range(B):
        at = sum(per[:b])
        table[b, : per[b]] = ids[at : at + per[b]]
        start.append(start[-1] + T[b])
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    rand = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=dt)  # noqa: E731
    s = {"case": case, "B": B, "N": N, "max_new": max(T), "max_len": max(L), "HQ": HQ, "HK": HK, "D": D}
    pool = (n_pages, HK, PAGE, D)
    s["k"] = torch.randn(pool, generator=g, device=DEV, dtype=torch.bfloat16)
    s["v"] = torch.randn(pool, generator=g, device=DEV, dtype=torch.bfloat16)
    s["table"] = table
    s["slots"] = torch.arange(B, dtype=torch.int32, device=DEV)
    s["len"] = torch.tensor(L, dtype=torch.int32, device=DEV)
    s["start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
    s["uniform"] = min(T) == max(T)
    if case["fused"]:  # the projection of a layer: q, k and v of a token side by side
        x = rand(N, (HQ + 2 * HK) * D)
        s["q"], s["k_new"], s["v_new"] = (y.view(N, -1, D) for y in x.split((HQ * D, HK * D, HK * D), 1))
    elif case["op"] == "append":
        s["k_new"], s["v_new"] = rand(N, HK, D), rand(N, HK, D)
    else:
        s["q"] = rand(N, HQ, D)
    s["gamma_q"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEV) if case["norm"] else None
    s["gamma_k"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEV) if case["norm"] else None
    s["sink"] = torch.randn(HQ, generator=g, device=DEV) if case["sink"] else None
    s["out"] = torch.empty((N, HQ, D), dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------- plain form
def _rows(s):
    """Request and place in its chunk of every new token, and its position."""
    n = torch.arange(s["N"], device=DEV)
    b = torch.searchsorted(s["start"][1:].contiguous(), n.to(torch.int32), right=True)
    i = n - s["start"][b]
    ctx = s["len"][s["slots"].long()]
    new = s["start"][1:] - s["start"][:-1]
    return b, i, (ctx - new)[b] + i


def _turn(x, pos, s, gamma):
    """RMSNorm (with gamma) and rotation of the last d_rope dims of x [N, heads, D] at positions pos, in 32 bits; angles in 64."""
    c = s["case"]
    x = x.float()
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma
    R = c["d_rope"]
    inv = c["theta"] ** (-2.0 * torch.arange(R // 2, device=DEV, dtype=torch.float64) / R)
    a = pos.double()[:, None] * inv
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    keep, y = x[..., : x.shape[-1] - R], x[..., x.shape[-1] - R :]
    if c["pairs"] == "adjacent":
        u, w = y[..., 0::2], y[..., 1::2]
        y = torch.stack((u * cos - w * sin, u * sin + w * cos), -1).flatten(-2)
    else:
        u, w = y[..., : R // 2], y[..., R // 2 :]
        y = torch.cat((u * cos - w * sin, u * sin + w * cos), -1)
    return torch.cat((keep, y), -1)


def _plain_append(s):
    b, i, pos = _rows(s)
    page = s["table"][s["slots"].long()][b, pos // PAGE].long()
    s["k"][page, :, pos % PAGE] = _turn(s["k_new"], pos, s, s["gamma_k"]).to(torch.bfloat16)
    s["v"][page, :, pos % PAGE] = s["v_new"].to(torch.bfloat16)
    return {"k": s["k"], "v": s["v"]}


def _plain_attend(s):
    c, B, HQ, HK, D, t = s["case"], s["B"], s["HQ"], s["HK"], s["D"], s["max_new"]
    G, pages = HQ // HK, -(-s["max_len"] // PAGE)
    b, i, pos = _rows(s)
    q = torch.zeros((B, t, HQ, D), device=DEV)
    q[b, i] = _turn(s["q"], pos, s, s["gamma_q"])
    at = torch.full((B, t), -1, device=DEV, dtype=torch.int64)
    at[b, i] = pos.long()
    q = q.view(B, t, HK, G, D).permute(0, 2, 3, 1, 4).reshape(B, HK, G * t, D)
    ids = s["table"][s["slots"].long()][:, :pages].clamp(min=0).long()
    key = s["k"][ids].permute(0, 2, 1, 3, 4).reshape(B, HK, pages * PAGE, D).float()
    x = (q @ key.transpose(-1, -2)).mul_(D ** -0.5).view(B, HK, G, t, pages * PAGE)
    del key
    j = torch.arange(pages * PAGE, device=DEV)
    seen = j <= at[..., None]
    if c["window"]:
        seen = seen & (j > at[..., None] - c["window"])
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    if s["sink"] is not None:
        z = s["sink"].view(1, HK, G, 1, 1)
        m = torch.maximum(m, z)
    m = m.clamp(min=-1e30)  # the rows that pad a request see nothing
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(z - m)
    val = s["v"][ids].permute(0, 2, 1, 3, 4).reshape(B, HK, pages * PAGE, D).float()
    o = (x.view(B, HK, G * t, -1) @ val).view(B, HK, G, t, D) / total
    return o.permute(0, 3, 1, 2, 4).reshape(B, t, HQ, D)[b, i].to(torch.bfloat16)


# ---------------------------------------------------------------- the framework's calls
def _handle(s):
    """What a serving program keeps of a layer: its description, its cache and its workspace."""
    from compressed_sparse_long_append_b200 import csla as C

    c = s["case"]
    cfg = C.csla_kv_cfg(D=s["D"], HQ=s["HQ"], HK=s["HK"], d_rope=c["d_rope"], rope_theta=c["theta"], eps=EPS, window=c["window"],
                        rope_pairs=C.CSLA_ROPE_ADJACENT if c["pairs"] == "adjacent" else C.CSLA_ROPE_HALVES)
    kv = C.csla_kv_cache(s["k"].data_ptr(), s["v"].data_ptr(), s["table"].data_ptr(), s["len"].data_ptr(), s["table"].shape[1], s["k"].shape[0], s["B"])
    need = C.csla_kv_workspace_size(cfg, s["B"], s["N"], s["max_new"], s["max_len"])
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    # requests of equally many new tokens need no offsets
    return C, cfg, kv, ws, need, None if s["uniform"] else s["start"], C.CSLA_F32 if c["dtype"] == "f32" else C.CSLA_BF16


def run(state):
    s = state
    if not own:
        return _plain_append(s) if s["case"]["op"] == "append" else _plain_attend(s)
    if "handle" not in s:
        s["handle"] = _handle(s)
    C, cfg, kv, ws, need, start, dt = s["handle"]
    if s["case"]["op"] == "append":
        C.csla_kv_append(cfg, kv, s["slots"], s["B"], start, s["N"], s["k_new"], s["k_new"].stride(0), s["v_new"], s["v_new"].stride(0), dt, s["gamma_k"])
        return {"k": s["k"], "v": s["v"]}
    C.csla_kv_attend(cfg, kv, s["slots"], s["B"], start, s["N"], s["max_new"], s["max_len"], s["q"], dt, s["q"].stride(0), s["sink"], s["gamma_q"],
                     s["out"], C.CSLA_BF16, ws, need)
    return s["out"]


# ---------------------------------------------------------------- 64 bits, one request and KV head at a time
def exact(case, seed):
    s = prepare(case, seed)
    T, L = lengths(case)
    HQ, HK, D, R = case["HQ"], case["HK"], case["D"], case["d_rope"]
    G, table = HQ // HK, s["table"].tolist()

    def rotated(x, p, gamma):
        x = x.double()
        if gamma is not None:
            x = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS) * gamma.double()
        w = torch.exp(-math.log(case["theta"]) * torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
        turn = torch.polar(torch.ones((), device=DEV, dtype=torch.float64).expand(len(p), R // 2), p.double()[:, None] * w)[:, None]
        y = x[..., D - R :]
        if case["pairs"] == "adjacent":
            z = torch.view_as_real(torch.view_as_complex(y.reshape(*y.shape[:-1], R // 2, 2).contiguous()) * turn).flatten(-2)
        else:
            z = torch.complex(y[..., : R // 2].contiguous(), y[..., R // 2 :].contiguous()) * turn
            z = torch.cat((z.real, z.imag), -1)
        return torch.cat((x[..., : D - R], z), -1)

    if case["op"] == "append":
        out = {"k": s["k"].double(), "v": s["v"].double()}
    else:
        out = torch.zeros((s["N"], HQ, D), dtype=torch.float64, device=DEV)
    n0 = 0
    for b, (t, n) in enumerate(zip(T, L)):
        p = torch.arange(n - t, n, device=DEV)
        if case["op"] == "append":
            page = torch.tensor(table[b], device=DEV)[p // PAGE]
            out["k"][page, :, p % PAGE] = rotated(s["k_new"][n0 : n0 + t], p, s["gamma_k"])
            out["v"][page, :, p % PAGE] = s["v_new"][n0 : n0 + t].double()
        else:
            first = max(0, n - t + 1 - case["window"]) // PAGE if case["window"] else 0
            last = -(-n // PAGE)
            ids = torch.tensor(table[b][first:last], device=DEV)
            j = torch.arange(first * PAGE, last * PAGE, device=DEV)
            q = rotated(s["q"][n0 : n0 + t], p, s["gamma_q"])
            hide = j > p[:, None]
            if case["window"]:
                hide = hide | (j <= p[:, None] - case["window"])
            for h in range(HK):
                keys, vals = (x[ids, h].reshape(-1, D).double() for x in (s["k"], s["v"]))
                for i in range(0, t, 1024):  # rows at a time
                    a = torch.einsum("tgd,jd->gtj", q[i : i + 1024, h * G : h * G + G], keys) / math.sqrt(D)
                    a = a.masked_fill(hide[i : i + 1024], -math.inf)
                    if s["sink"] is not None:
                        z = s["sink"][h * G : h * G + G].double()[:, None, None].expand(-1, a.shape[1], 1)
                        a = torch.cat((a, z), -1)
                    w = torch.softmax(a, -1)[..., : len(j)]
                    out[n0 + i : n0 + min(i + 1024, t), h * G : h * G + G] = torch.einsum("gtj,jd->tgd", w, vals)
        n0 += t
    return out
