"""How near a dense layer's attention is to its formula in 64 bits, as a ratio to the output's own size, so that the bound does
not outgrow the outputs of long contexts (over random values those fall as one over the root of the length).

Bound of rms(err) / rms(o) over a token's heads and dims.  A rounding to bf16 is off by d with |d| <= 2^-8 relative, evenly spread:
at most 2^-8 / sqrt(3) in the mean square.  Over values V_j of no common sign the roundings of the weights give sum p_j d_j V_j, in the
mean square at most 2^-8 / sqrt(3) of o = sum p_j V_j itself.  Rounding the output adds as much.  A query kept as one bf16
operand changes score j by scale sum_d q_d d_d K_jd, 2^-8 / sqrt(3) times the spread of the scores in the mean square, and so the weights
by as much; one kept as two changes them by 2^-16.  Independent, they add as squares.  Over n elements a mean square is within
5 sqrt(2 / n) of its expectation (5 deviations), its root within half of that, and so is that of o: a factor of (1 + x) / (1 - x), x =
2.5 sqrt(2 / n).  The fp32 parts (exponentials, sums, rotation) stay below 2^-12."""
import math

import torch

from kv_reference import norm, rotate

STEP = 2.0 ** -8 / math.sqrt(3.0)


def attend64(q, k, v, first_pos, shape, halves, sink, gamma, terms=0, weights=None):
    """o [t, HQ, D] of one request from q [t, HQ, D] and its cache k, v [L, HK, D], all in 64 bits; also the scores' spread.
    terms: the rotated query rounded to so many bf16 terms (0: not at all); weights: a dtype they are rounded to (their sum is not)."""
    t, HQ, D = q.shape
    L, HK = k.shape[:2]
    G, scale = HQ // HK, shape.scale or D ** -0.5
    pos = first_pos + torch.arange(t, device=q.device)
    x = rotate(norm(q.double(), gamma, shape.eps), pos, shape.d_rope, halves, shape.theta)
    if terms:
        hi = x.to(torch.bfloat16).double()
        x = hi + (x - hi).to(torch.bfloat16).double() if terms == 2 else hi
    j = torch.arange(L, device=q.device)
    hide = j[None] > pos[:, None]
    if shape.window:
        hide |= j[None] <= pos[:, None] - shape.window
    o, spread = torch.zeros((t, HQ, D), dtype=torch.float64, device=q.device), 0.0
    for h in range(HQ):
        s = scale * (x[:, h] @ k[:, h // G].double().T)
        spread = max(spread, float((s.masked_fill(hide, 0.0).pow(2).sum(-1) / (~hide).sum(-1)).max().sqrt()))
        s = s.masked_fill_(hide, -math.inf)
        m = s.amax(-1, keepdim=True)
        if sink is not None:
            m = torch.maximum(m, sink[h].double())
        p = s.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        if sink is not None:
            total = total + torch.exp(sink[h].double() - m)
        o[:, h] = (p if weights is None else p.to(weights).double()) @ v[:, h // G].double() / total
    return o, spread


def ratios(out, o):
    """rms(out - o) / rms(o) of each token."""
    e, y = (out.double() - o).flatten(1), o.flatten(1)
    return (e.pow(2).mean(-1) / y.pow(2).mean(-1)).sqrt()


def head_ratios(out, o):
    """The same of each token and head, flat.  Their median says little of the heads in which one key has all the weight,
    which a sum over heads is full of where scores are spread far."""
    return ratios(out.flatten(0, 1), o.flatten(0, 1))


def bound(out_dtype, terms, spread, n):
    x = 2.5 * math.sqrt(2.0 / n)
    return ((1 + x) / (1 - x) * STEP * math.sqrt(1 + (out_dtype == torch.bfloat16) + (spread ** 2 if terms == 1 else 0))
            + 2.0 ** -12)


def terms_of(rows, D):
    """Terms of the query in a request of so many rows per KV head."""
    return 1 if rows > 128 and D == 128 else 2
