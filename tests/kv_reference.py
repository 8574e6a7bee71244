"""The dense paged layer's two operators from their formulas in 64 bits, one request and head at a time, and how far the
kernels may be from them (test infrastructure only; nothing is shared with the kernels)."""
import torch

PAGE = 128
HALF_BF16 = 2.0 ** -8    # half a bf16 step, relative to the value
HALF_F32 = 2.0 ** -24


def rotate(x, pos, d_rope, halves, theta):
    """x [n, heads, D] float64 at positions pos [n]."""
    D = x.shape[-1]
    if d_rope == 0:
        return x
    inv = theta ** (-2.0 * torch.arange(d_rope // 2, dtype=torch.float64, device=x.device) / d_rope)
    ang = pos.double()[:, None, None] * inv
    c, s = torch.cos(ang), torch.sin(ang)
    y = x.clone()
    r = y[..., D - d_rope:]
    if halves:
        u, w = r[..., :d_rope // 2].clone(), r[..., d_rope // 2:].clone()
        r[..., :d_rope // 2], r[..., d_rope // 2:] = u * c - w * s, u * s + w * c
    else:
        u, w = r[..., 0::2].clone(), r[..., 1::2].clone()
        r[..., 0::2], r[..., 1::2] = u * c - w * s, u * s + w * c
    return y


def norm(x, gamma, eps):
    return x if gamma is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double()


def append_rows(k_new, pos, shape, halves, gamma):
    """Expected K rows in float64, and how far a bf16 row may be: half a step of the value, plus the fp32
    arithmetic before it (norm: a mean over D, a root, a quotient and two products; rotation: a cosine and a sine within
    2^-21 each, two products and a sum: together below 2^-18 of the pair's magnitudes)."""
    x = norm(k_new.double(), gamma, shape.eps)
    y = rotate(x, pos, shape.d_rope, halves, shape.theta)
    mag = x.abs().amax(-1, keepdim=True) * 2
    return y, HALF_BF16 * y.abs() + (2.0 ** -18) * mag


def attend_request(q, k, v, first_pos, shape, halves, sink, gamma, q_bits=HALF_BF16):
    """One request: q [t, HQ, D], its visible cache k, v [L, HK, D] (rows 0..L-1, float64), the first new token's
    position.  Returns o [t, HQ, D] and the bound of |kernel - o| before the output's own rounding.

    The kernel rounds q' to bf16 (half a step per element), so a score is off by at most
    E = scale * sum |q'_d K_jd| (2^-8 + 2^-15) + 2^-20 |s| (fp32 sums of D terms, the norm and rotation, and the argument of
    the exponential); each weight e^s by a factor e^{+-E}, the numerator's weights also by 2^-8 (rounded to bf16) and 2^-12 (the
    exponential), the sums by 2^-12.  With A = sum p_j |V_j| / sum: |error| <= (e^{2E} (1 + 2^-8)(1 + 2^-12) / (1 - 2^-11) - 1) A.
    That is relative, so it says nothing of weights below fp32's smallest normal number 2^-126, which the exponential
    flushes to zero: a weight counts 2^8 at most before it is normalised, so L flushed ones change o by at most
    L 2^-118 max|V| (a sink of 100 over scores near 0 gives e^-100 = 2^-144)."""
    t, HQ, D = q.shape
    L, HK = k.shape[:2]
    G = HQ // HK
    scale = shape.scale or D ** -0.5
    pos = first_pos + torch.arange(t, device=q.device)
    qr = rotate(norm(q.double(), gamma, shape.eps), pos, shape.d_rope, halves, shape.theta)
    j = torch.arange(L, device=q.device)
    see = j[None] <= pos[:, None]
    if shape.window:
        see &= j[None] > pos[:, None] - shape.window
    o = torch.zeros((t, HQ, D), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    for h in range(HQ):
        K, V = k[:, h // G].double(), v[:, h // G].double()
        K = torch.where(see.any(0)[:, None], K, torch.zeros_like(K))   # rows that nobody sees may hold anything
        V = torch.where(see.any(0)[:, None], V, torch.zeros_like(V))
        s = scale * (qr[:, h] @ K.T)
        e = scale * (qr[:, h].abs() @ K.abs().T) * (q_bits + 2.0 ** -15) + s.abs() * 2.0 ** -20
        s = s.masked_fill(~see, float("-inf"))
        E = e.masked_fill(~see, 0.0).amax(-1, keepdim=True)
        m = s.amax(-1, keepdim=True)
        if sink is not None:
            m = torch.maximum(m, sink[h].double())
        p = torch.exp(s - m)
        total = p.sum(-1, keepdim=True)
        if sink is not None:
            total = total + torch.exp(sink[h].double() - m)
        o[:, h] = p @ V / total
        A = p @ V.abs() / total
        tol[:, h] = (torch.exp(2 * E) * (1 + HALF_BF16) * (1 + 2.0 ** -12) / (1 - 2.0 ** -11) - 1) * A + L * 2.0 ** -118 * V.abs().max()
    return o, tol


def with_output_step(o, tol, dtype):
    half = HALF_BF16 if dtype == torch.bfloat16 else HALF_F32
    return tol + half * (o.abs() + tol)
