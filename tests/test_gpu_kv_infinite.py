"""Scores of minus infinity in tokens that a row sees: by the formula such a token has no weight, and a row that sees no other is 0 / 0
without a sink (NaN) and 0 with one, however its keys are cut.  A row that sees no mapped token at all is zeros."""
import pytest
import torch

from compressed_sparse_long_append_b200 import csla as C
from compressed_sparse_long_append_b200.layer import DenseShape
from kv_helpers import Batch, no_device_error
from kv_reference import attend_request, with_output_step

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# (D, HQ, HK, T, L, window): up to 8 and up to 16 rows per KV head, one row tile, row tiles of 256; keys whole and cut
KINDS = [(128, 8, 2, 1, 90, 0), (64, 8, 2, 1, 5000, 0), (128, 8, 1, 1, 3000, 200), (64, 12, 1, 1, 90, 0), (128, 32, 2, 1, 6000, 0),
         (128, 8, 2, 9, 100, 0), (64, 20, 1, 2, 9000, 0), (64, 8, 2, 20, 700, 130), (128, 4, 1, 70, 400, 0), (64, 4, 2, 100, 5000, 0),
         (128, 16, 1, 20, 3000, 300)]


@pytest.mark.parametrize("D,HQ,HK,T,L,window", KINDS)
@pytest.mark.parametrize("sink", [False, True])
def test_rows_whose_scores_are_all_minus_infinity(D, HQ, HK, T, L, window, sink):
    # request 0: 2^100 times -2^100 in every dim overflows to -inf; request 1 is ordinary and beside it
    b = Batch(DenseShape(D=D, HQ=HQ, HK=HK, d_rope=0, window=window), [T, T], [L, L], norm=False, sink=sink, seed=90)
    b.fill()
    b.q = b.q.clone()
    b.q[:T] = 2.0 ** 100
    p = torch.arange(max(0, L - T + 1 - window) if window else 0, L)
    page, at = b.table[b.slots_l[0], p // 128].long().cuda(), (p % 128).cuda()
    b.lb.k[page, :, at] = -(2.0 ** 100)
    out = b.attend(F32)
    assert bool((out[:T] == 0).all() if sink else torch.isnan(out[:T]).all())
    ref = Batch.__new__(Batch)
    ref.__dict__.update(b.__dict__)
    ref.check_attend(torch.cat([torch.full_like(out[:T], 7.0), out[T:]]), skip={0})
    # one token of the request, the first that every row sees, scores finitely: it alone has weight
    j = max(0, L - window) if window else 0
    page, at = b.table[b.slots_l[0], j // 128].item(), j % 128
    b.lb.k[page, :, at] = 0.0
    out = b.attend(F32)
    v = b.lb.v[page, :, at].double().repeat_interleave(HQ // HK, 0)              # [HQ, D]
    z = b.sink.double() if sink else torch.full((HQ,), -float("inf"), device=v.device, dtype=torch.float64)
    o = (v / (1 + torch.exp(z))[:, None]).expand(T, HQ, D)
    # (score 0 exactly; the weight 1, its sum and the sink's exponential: 2^-20 together; V is bf16 as it is)
    assert bool(((out[:T].double() - o).abs() <= 2.0 ** -20 * o.abs()).all())
    # without any mapped page the rows are zeros, sink or not
    b.lb.block_table[b.slots_l[0]] = -1
    out = b.attend(F32)
    assert bool((out[:T] == 0).all())
    assert C.csla_device_error()[1] == C.CSLA_DEVERR_PAGE


def test_keys_of_minus_infinity_have_no_weight():
    """Every other key has -inf in a dim where the query is 1 (row tiles of 256 rows of 128 dims, whose query is one bf16 operand)."""
    T, L = 100, 400
    b = Batch(DenseShape(D=128, HQ=4, HK=1, d_rope=0), [T], [L], norm=False, seed=91)
    b.fill()
    b.q = b.q.clone().reshape(T, 4, 128)
    b.q[:, :, 0] = 1.0
    p = torch.arange(0, L, 2)
    page, at = b.table[b.slots_l[0], p // 128].long().cuda(), (p % 128).cuda()
    b.lb.k[page, 0, at, 0] = -float("inf")
    b.q = b.q.reshape(T, 512)
    out = b.attend(F32)
    no_device_error()
    k, v = b.rows(0, b.lb.k), b.rows(0, b.lb.v)
    for t in (0, 1, 57, 99):
        n = L - T + t + 1
        odd = torch.arange(1, n, 2).cuda()
        q = b.q[t:t + 1].reshape(1, 4, 128)
        o, tol = attend_request(q, k[odd], v[odd], len(odd) - 1, b.shape, False, b.sink, None)
        assert bool(((out[t:t + 1].double() - o).abs() <= with_output_step(o, tol, F32)).all()), t
