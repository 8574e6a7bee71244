"""csla_kv_attend over long contexts against its formula in 64 bits, as a ratio to the output's own size (kv_accuracy.py): every way of
cutting a request's keys and of joining its parts, at lengths where a part that is lost, doubled or misweighted shows."""
import pytest
import torch

from compressed_sparse_long_append_b200 import csla as C
from compressed_sparse_long_append_b200.layer import DenseShape
from kv_accuracy import attend64, bound, head_ratios, ratios, terms_of
from kv_helpers import Batch, no_device_error

pytestmark = pytest.mark.gpu

ADJ, HALF = C.CSLA_ROPE_ADJACENT, C.CSLA_ROPE_HALVES
BF, F32 = torch.bfloat16, torch.float32

# what each is there for: (D, HQ, HK, window, T, L, more)
CASES = {
    "few, up to 8 rows, joined by blocks": (128, 8, 1, 0, [1, 1], [40000, 70001], {}),
    "few, up to 16 rows, joined by blocks": (64, 16, 1, 0, [1, 1], [65000, 100003], {}),
    "few, chunks of a batch": (128, 32, 8, 0, [1, 2, 1, 1, 4], [5000, 20011, 33000, 131072, 901], {}),
    "few, 64 dims": (64, 28, 4, 0, [1, 2, 1], [4097, 9000, 30000], {}),
    "few, long windows": (128, 16, 4, 3000, [1, 4, 2], [30000, 20011, 2990], {}),
    "one row tile, 8 KV heads, fewer chunks than SMs": (128, 32, 8, 0, [5, 20], [28500, 33000], {}),
    "one row tile, one KV head, chunks of 12 tiles": (128, 64, 1, 0, [1, 2], [230001, 3000], {}),
    "one row tile, 64 dims": (64, 8, 4, 0, [40, 64], [33000, 20011], {}),
    "one row tile, windows": (64, 16, 2, 2500, [9, 16], [20011, 9000], {}),
    "row tiles of 256, their keys cut": (128, 4, 4, 0, [300, 700], [17000, 9000], {}),
    "row tiles of 256, those left over cut": (128, 16, 16, 0, [2500], [7000], {}),
    "row tiles of 256, 64 dims, those left over cut": (64, 32, 16, 0, [1300], [9000], {}),
    "row tiles of 256, windows": (128, 8, 2, 1500, [600, 300], [9000, 300], {}),
    "a prompt": (128, 32, 8, 0, [2048], [2048], {}),
    "a chunk behind a long prefix": (128, 32, 4, 0, [4096], [20480], {}),
    "all kinds in one batch": (128, 16, 4, 0, [1, 500, 3, 30, 2], [40000, 9000, 12000, 20011, 300], {}),
    "all kinds in one batch, 64 dims": (64, 14, 2, 0, [1, 700, 2, 15], [30000, 5000, 12000, 20011], {}),
}


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_long_contexts(name, out_dtype):
    D, HQ, HK, window, T, L, more = CASES[name]
    shape = DenseShape(D=D, HQ=HQ, HK=HK, d_rope=64, rope_pairs=HALF if HK % 4 else ADJ, window=window, **more)
    b = Batch(shape, T, L, seed=len(name), sink=HK > 1, norm=D == 128)
    b.fill([max(0, n - t + 1 - window) if window else 0 for t, n in zip(T, L)])
    out = b.attend(out_dtype)
    no_device_error()
    q = b.q.reshape(b.N, HQ, D)
    for r in range(b.B):
        rows = slice(b.start_l[r], b.start_l[r + 1])
        lo = max(0, L[r] - T[r] + 1 - window) if window else 0
        k, v = (x.nan_to_num(0.0) if lo else x for x in (b.rows(r, b.lb.k), b.rows(r, b.lb.v)))
        o, spread = attend64(q[rows], k, v, L[r] - T[r], shape, b.halves, b.sink, b.gamma_q)
        most = bound(out_dtype, terms_of(T[r] * HQ // HK, D), spread, HQ * D)
        got = ratios(out[rows], o)
        assert bool((got <= most).all()), (r, int((got > most).sum()), float(got.max()), most)
        assert most < 0.02   # one page of 128 tokens more or less changes o by the root of 128 / 131072 = 0.03


@pytest.mark.parametrize("D,HQ,HK,T,L", [(128, 32, 8, 1, 20000), (64, 64, 8, 1, 20000), (128, 64, 4, 1, 20000), (64, 8, 4, 8, 20000),
                                         (128, 32, 8, 5, 20000), (128, 16, 16, 40, 9000), (64, 8, 8, 300, 9000)])
def test_requests_that_keep_the_querys_rest(D, HQ, HK, T, L):
    """Sharper scores over many keys: an error of a query rounded once to bf16 is beyond this bound (test_kv_accuracy.py)."""
    shape = DenseShape(D=D, HQ=HQ, HK=HK, d_rope=D, rope_pairs=HALF)
    b = Batch(shape, [T], [L], seed=5, norm=False)
    b.fill()
    b.q = (2.0 * b.q.float()).to(BF)
    out = b.attend(F32)
    no_device_error()
    q = b.q.reshape(b.N, HQ, D)
    o, spread = attend64(q, b.rows(0, b.lb.k), b.rows(0, b.lb.v), L - T, shape, True, b.sink, None)
    assert terms_of(T * HQ // HK, D) == 2 and spread > 1.8
    assert float(head_ratios(out, o).median()) <= bound(F32, 2, spread, T * HQ * D)
