"""A hybrid stack on one block table: a CSA layer, a sliding-window dense layer, an HCA layer and a full dense layer, stepped
together through their public calls.  A prompt is appended in one ragged chunk, then single tokens follow; the dense layers are checked
against their formulas at every step, the compressed ones against the same layers stepped without dense layers beside them."""
import numpy as np
import pytest
import torch

from compressed_sparse_long_append_b200 import csla as C
from compressed_sparse_long_append_b200.layer import CompressParams, DenseShape, LayerShape, LayerStack
from kv_helpers import DEV, no_device_error, randn
from kv_reference import append_rows, attend_request, with_output_step

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _params(shape, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)   # noqa: E731
    m, D, dI = shape.m, shape.D, shape.dI
    csa = shape.is_csa
    return CompressParams(1 + 0.1 * r(D), r(D) / D ** 0.5, r(m), r(dI) / dI ** 0.5 if csa else None, r(m) if csa else None, DEV)


def _compressed_step(lb, cp, slots, T, kv, ki, q, cq, W, hw, sink, gq, max_len):
    """One append of T tokens per request, then the attention of each request's latest token."""
    s, B = lb.shape, len(slots)
    cfg, st, ca = lb.cfg(), lb.state(), lb.cache()
    C.csla_compress_append(cfg, st, ca, slots, B, T, kv, ki, C.CSLA_BF16, cp.struct())
    out = torch.zeros((B, s.H, s.D), device=DEV)
    if s.is_csa:
        k, stride = 32, max(max_len // s.m, 1)
        scores = torch.zeros((B, stride), device=DEV)
        idx = torch.zeros((B, k), dtype=torch.int32, device=DEV)
        n = C.csla_workspace_size(cfg, C.CSLA_OP_INDEXER, B, max_len)
        C.csla_indexer_scores(cfg, st, ca, slots, B, max_len, cq, C.CSLA_BF16, W, C.CSLA_BF16, hw, scores, stride,
                              torch.zeros(n, dtype=torch.uint8, device=DEV), n)
        C.csla_topk_select(cfg, st, slots, B, max_len, scores, stride, k, idx)
        n = C.csla_workspace_size(cfg, C.CSLA_OP_CSA_ATTEND, B, k)
        C.csla_csa_attend(cfg, st, ca, slots, B, q, C.CSLA_BF16, idx, k, sink, gq, out, C.CSLA_F32, C.CSLA_VARIANT_AUTO,
                          torch.zeros(n, dtype=torch.uint8, device=DEV), n)
    else:
        n = C.csla_workspace_size(cfg, C.CSLA_OP_HCA_ATTEND, B, max_len)
        C.csla_hca_attend(cfg, st, ca, slots, B, max_len, q, C.CSLA_BF16, sink, gq, out, C.CSLA_F32, C.CSLA_VARIANT_AUTO,
                          torch.zeros(n, dtype=torch.uint8, device=DEV), n)
    return out


def test_dense_layers_in_a_hybrid_stack():
    shapes = [LayerShape(m=4, D=128, H=8, HI=4, dI=64, dc=128), DenseShape(D=64, HQ=8, HK=2, d_rope=64, window=150),
              LayerShape(m=128, D=128, H=8), DenseShape(D=128, HQ=12, HK=4, d_rope=128, rope_pairs=C.CSLA_ROPE_HALVES)]
    B, T0, steps = 3, 300, 3
    pages = -(-(T0 + steps) // 128)
    n_pages = B * pages + 2
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    table = torch.full((B, pages + 1), -1, dtype=torch.int32)
    for b in range(B):
        table[b, :pages] = perm[b * pages:(b + 1) * pages]
    stack = LayerStack(shapes, B, n_pages, pages + 1, DEV)
    alone = LayerStack([shapes[0], shapes[2]], B, n_pages, pages + 1, DEV)
    for st in (stack, alone):
        st.block_table.copy_(table)
    cps = {0: _params(shapes[0], 2), 2: _params(shapes[2], 3)}
    slots = torch.arange(B, dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(5)
    sinks = [randn(g, 8), randn(g, 8), randn(g, 8), randn(g, 12)]
    gammas = [1 + 0.1 * randn(g, s.D) for s in shapes]
    gk = [None, 1 + 0.1 * randn(g, 64), None, None]
    W = randn(g, 4 * 64, 128, dtype=BF)
    kept = {1: ([[] for _ in range(B)], [[] for _ in range(B)]), 3: ([[] for _ in range(B)], [[] for _ in range(B)])}
    for step in range(steps + 1):
        T = T0 if step == 0 else 1
        ctx = T0 + step
        stack.dense_len += T
        for i, s in enumerate(shapes):
            if isinstance(s, DenseShape):
                lb = stack[i]
                x = randn(g, B * T, (s.HQ + 2 * s.HK) * s.D, dtype=BF)   # one projection, q, k and v side by side
                q, k, v = x.split((s.HQ * s.D, s.HK * s.D, s.HK * s.D), 1)
                C.csla_kv_append(lb.cfg(), lb.cache(), slots, B, None, B * T, k, k.stride(0), v, v.stride(0), C.CSLA_BF16, gk[i])
                n = C.csla_kv_workspace_size(lb.cfg(), B, B * T, T, ctx)
                ws = torch.zeros(max(n, 16), dtype=torch.uint8, device=DEV)
                out = torch.zeros((B * T, s.HQ, s.D), device=DEV)
                C.csla_kv_attend(lb.cfg(), lb.cache(), slots, B, None, B * T, T, ctx, q, C.CSLA_BF16, q.stride(0), sinks[i],
                                 gammas[i], out, C.CSLA_F32, ws, n)
                no_device_error()
                halves = s.rope_pairs == C.CSLA_ROPE_HALVES
                for b in range(B):
                    pos = torch.arange(ctx - T, ctx, device=DEV)
                    y, tol = append_rows(k[b * T:(b + 1) * T].reshape(T, s.HK, s.D), pos, s, halves, gk[i])
                    page = table[b, (pos // 128).cpu().long()].to(DEV).long()
                    got = lb.k[page, :, pos % 128]
                    assert bool(((got.double() - y).abs() <= tol).all()), (step, i, b)
                    kept[i][0][b].append(got)
                    kept[i][1][b].append(v[b * T:(b + 1) * T].reshape(T, s.HK, s.D))
                    o, tol = attend_request(q[b * T:(b + 1) * T].reshape(T, s.HQ, s.D), torch.cat(kept[i][0][b]),
                                            torch.cat(kept[i][1][b]), ctx - T, s, halves, sinks[i], gammas[i])
                    err = (out[b * T:(b + 1) * T].double() - o).abs()
                    assert bool((err <= with_output_step(o, tol, torch.float32)).all()), (step, i, b)
            else:
                kv = randn(g, B, T, s.D, dtype=BF)
                ki = randn(g, B, T, 64, dtype=BF) if s.is_csa else None
                q, cq, hw = randn(g, B, s.H, s.D, dtype=BF), randn(g, B, 128, dtype=BF), randn(g, B, 4)
                a = _compressed_step(stack[i], cps[i], slots, T, kv, ki, q, cq, W, hw, sinks[i], gammas[i], ctx)
                b_ = _compressed_step(alone[i // 2], cps[i], slots, T, kv, ki, q, cq, W, hw, sinks[i], gammas[i], ctx)
                no_device_error()
                assert torch.equal(a, b_), (step, i)
    assert stack.dense_len.tolist() == [T0 + steps] * B == stack[0].len.tolist()
    assert np.array_equal(stack[0].host_view()["rows"], alone[0].host_view()["rows"])
