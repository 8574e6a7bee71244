"""Host side of the dense paged layer, without a GPU: struct layouts, refusals before any launch, workspace sizes, the
binding's buffers, and the reference the GPU tests use."""
import ctypes

import pytest
import torch

import test_abi_layout
from compressed_sparse_long_append_b200 import csla as C
from compressed_sparse_long_append_b200.layer import DenseBuffers, DenseShape, LayerShape, LayerStack
from kv_reference import attend_request, norm, rotate

FAKE = 1 << 40   # never dereferenced: every call below fails its host checks first


def test_structs_match_the_header(monkeypatch):
    monkeypatch.setattr(test_abi_layout, "STRUCTS", ("csla_kv_cfg", "csla_kv_cache"))
    test_abi_layout.test_ctypes_structs_match_the_header()


def _cfg(**kw):
    return DenseShape(**kw).cfg()


def _cache(**kw):
    f = dict(k=FAKE, v=FAKE, block_table=FAKE, len=FAKE, bt_stride=8, n_pages=16, n_slots=4)
    f.update(kw)
    return C.csla_kv_cache(**f)


def _append(cfg=None, kv=None, **kw):
    a = dict(slots=FAKE, B=2, q_start=FAKE, N=4, k=FAKE, ks=1024, v=FAKE, vs=1024, dt=C.CSLA_BF16, gamma=None)
    a.update(kw)
    cfg, kv = cfg or _cfg(), kv or _cache()
    return C._lib.csla_kv_append(ctypes.byref(cfg), ctypes.byref(kv), a["slots"], a["B"], a["q_start"], a["N"], a["k"],
                                 a["ks"], a["v"], a["vs"], a["dt"], a["gamma"], None)


def _attend(cfg=None, kv=None, **kw):
    a = dict(slots=FAKE, B=2, q_start=FAKE, N=4, mn=4, ml=100, q=FAKE, qdt=C.CSLA_BF16, qs=8192, sink=None, gamma=None,
             out=FAKE, odt=C.CSLA_BF16, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    cfg, kv = cfg or _cfg(), kv or _cache()
    return C._lib.csla_kv_attend(ctypes.byref(cfg), ctypes.byref(kv), a["slots"], a["B"], a["q_start"], a["N"], a["mn"],
                                 a["ml"], a["q"], a["qdt"], a["qs"], a["sink"], a["gamma"], a["out"], a["odt"], a["ws"],
                                 a["wsb"], None)


@pytest.mark.parametrize("bad", [dict(D=96), dict(D=256), dict(HQ=12, HK=8), dict(HK=0), dict(HQ=0), dict(HQ=2048, HK=16),
                                 dict(HQ=129, HK=1), dict(d_rope=8), dict(d_rope=144), dict(d_rope=-16),
                                 dict(rope_pairs=2)])
def test_unsupported_shapes(bad):
    assert _append(cfg=_cfg(**bad)) == C.CSLA_ERR_UNSUPPORTED
    assert _attend(cfg=_cfg(**bad)) == C.CSLA_ERR_UNSUPPORTED
    assert C.csla_kv_workspace_size(_cfg(**bad), 2, 4, 4, 100000) == 0


@pytest.mark.parametrize("bad", [dict(eps=-1.0), dict(eps=float("nan")), dict(theta=0.0), dict(window=-1), dict(scale=-1.0),
                                 dict(scale=float("inf")), dict(scale=float("nan"))])
def test_bad_numbers(bad):
    assert _append(cfg=_cfg(**bad)) == C.CSLA_ERR_ARG
    assert _attend(cfg=_cfg(**bad)) == C.CSLA_ERR_ARG


def test_null_structs():
    cfg, kv = _cfg(), _cache()
    for c, k in ((None, ctypes.byref(kv)), (ctypes.byref(cfg), None)):
        assert C._lib.csla_kv_append(c, k, FAKE, 1, None, 1, FAKE, 1024, FAKE, 1024, 1, None, None) == C.CSLA_ERR_ARG
        assert C._lib.csla_kv_attend(c, k, FAKE, 1, None, 1, 1, 1, FAKE, 1, 8192, None, None, FAKE, 1, FAKE, 1 << 40,
                                     None) == C.CSLA_ERR_ARG
    assert C._lib.csla_kv_workspace_size(None, 1, 1, 1, 1) == 0


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(block_table=None), dict(len=None), dict(bt_stride=0),
                                 dict(n_pages=0), dict(n_slots=0), dict(k=FAKE + 8), dict(v=FAKE + 2)])
def test_bad_caches(bad):
    assert _append(kv=_cache(**bad)) == C.CSLA_ERR_ARG
    assert _attend(kv=_cache(**bad)) == C.CSLA_ERR_ARG


@pytest.mark.parametrize("bad", [dict(slots=None), dict(B=0), dict(N=0), dict(q_start=None, N=5), dict(N=(1 << 30) + 1)])
def test_bad_batches(bad):
    assert _append(**bad) == C.CSLA_ERR_ARG
    assert _attend(**bad) == C.CSLA_ERR_ARG


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(k=FAKE + 2), dict(ks=1016), dict(vs=1028), dict(ks=-1024),
                                 dict(dt=2), dict(dt=-1)])
def test_bad_append_rows(bad):
    assert _append(**bad) == C.CSLA_ERR_ARG


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(q=FAKE + 4), dict(out=FAKE + 8), dict(qs=8188),
                                 dict(qs=8196), dict(qdt=2), dict(odt=3), dict(mn=0), dict(ml=0), dict(q_start=None, mn=1),
                                 dict(ml=(1 << 30) + 1)])
def test_bad_attend_rows(bad):
    assert _attend(**bad) == C.CSLA_ERR_ARG


def test_too_many_cache_rows():
    assert _attend(kv=_cache(n_pages=1 << 21)) == C.CSLA_ERR_UNSUPPORTED   # 2^21 pages x 8 heads x 128 rows


def test_workspace_is_checked():
    cfg = _cfg()
    need = C.csla_kv_workspace_size(cfg, 2, 2, 1, 100000)
    if need:
        bad = dict(N=2, mn=1, ml=100000)
        assert _attend(cfg, wsb=need - 1, **bad) == C.CSLA_ERR_ARG
        assert _attend(cfg, ws=None, **bad) == C.CSLA_ERR_ARG
        assert _attend(cfg, ws=FAKE + 8, **bad) == C.CSLA_ERR_ARG
    assert _attend(cfg, N=2, mn=1, ml=(1 << 27) + 1) == C.CSLA_ERR_ARG   # longer than a call may be
    assert C.csla_kv_workspace_size(cfg, 2, 2, 1, 1 << 27) > 0
    for args in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (1, 1, 1, (1 << 27) + 1), (1, (1 << 30) + 1, 1, 9000)):
        assert C.csla_kv_workspace_size(cfg, *args) == 0


def test_stack_holds_dense_layers():
    shapes = [LayerShape(m=4, D=128, H=8, HI=4, dI=64, dc=128), DenseShape(D=64, HQ=8, HK=2), LayerShape(m=128, D=128, H=8),
              DenseShape(D=128, HQ=4, HK=4, window=256)]
    st = LayerStack(shapes, 3, 10, 4, device="cpu")
    assert len({lb.block_table.data_ptr() for lb in st.layers}) == 1
    a, b = st[1], st[3]
    assert a.len is b.len is st.dense_len
    assert tuple(a.k.shape) == (10, 2, 128, 64) and tuple(b.v.shape) == (10, 4, 128, 128)
    kv = b.cache()
    assert (kv.k, kv.bt_stride, kv.n_pages, kv.n_slots) == (b.k.data_ptr(), 4, 10, 3)
    assert b.cfg().window == 256
    with pytest.raises(ValueError):
        DenseBuffers(shapes[1], 3, 10, 4, device="cpu", length=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        DenseBuffers(shapes[1], 3, 10, 4, device="cpu", block_table=torch.zeros((3, 4)))


# ---------------------------------------------------------------- the reference itself
def test_reference_rotation_is_relative():
    x, y = torch.randn(2, 1, 64, dtype=torch.float64), torch.randn(2, 1, 64, dtype=torch.float64)
    for halves in (False, True):
        dots = []
        for shift in (0, 1000):
            p = torch.tensor([3, 40]) + shift
            dots.append((rotate(x, p, 48, halves, 1e4) * rotate(y, p - 2, 48, halves, 1e4)).sum(-1))
        assert torch.allclose(dots[0], dots[1], atol=1e-9)
        assert torch.equal(rotate(x, torch.zeros(2, dtype=torch.long), 48, halves, 1e4), x)
        assert torch.equal(rotate(x, torch.tensor([9, 9]), 48, halves, 1e4)[..., :16], x[..., :16])


def test_reference_attention_against_a_softmax():
    sh = DenseShape(D=64, HQ=4, HK=2, d_rope=0, window=6)
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)   # noqa: E731
    q, k, v, z, gamma = r(5, 4, 64), r(9, 2, 64), r(9, 2, 64), r(4), r(64)
    o, tol = attend_request(q, k, v, 4, sh, False, z, gamma)
    qn = norm(q, gamma, sh.eps)
    for t in range(5):
        p = 4 + t
        see = list(range(max(0, p - 5), p + 1))
        for h in range(4):
            a = torch.cat([(k[see, h // 2] @ qn[t, h]) / 8.0, z[h:h + 1]])
            w = torch.softmax(a, 0)[:-1]
            assert torch.allclose(o[t, h], w @ v[see, h // 2], atol=1e-12)
    assert bool((tol > 0).all())
