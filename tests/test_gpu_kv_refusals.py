"""The dense layer's calls with inputs that only the device can see to be wrong: what is refused is left alone, the rest is answered,
and nothing is written outside the buffers of the call."""
import pytest
import torch

from compressed_sparse_long_append_b200 import csla as C
from compressed_sparse_long_append_b200.layer import DenseShape
from kv_helpers import DEV, Batch

pytestmark = pytest.mark.gpu

F32 = torch.float32


def _bits():
    return C.csla_device_error()[1]


@pytest.mark.parametrize("T,order,kept", [
    ([2] * 40, [0, 2, 0, 2, 0, 2], [0]),                      # the same two rows again and again
    ([3, 4, 5, 6], [0, 7, 3, 12, 18], [0, 3]),                # 7..3 falls, 3..12 overlaps, 12..18 is in order again
    ([20, 1, 30], [0, 20, 10, 51], [0]),                      # longer ones
])
def test_overlapping_requests_are_refused(T, order, kept):
    """Offsets that fall and rise again: pairs that are in order alone but share rows with a request before them are skipped by both
    calls, and nothing is written behind the workspace."""
    L = [t + 3000 for t in T]
    b = Batch(DenseShape(D=64, HQ=8, HK=2, d_rope=64), T, L, seed=70)
    b.fill()
    # the same offsets over and over when there are more requests than offsets given
    starts = [order[i % len(order)] if len(T) > len(order) else order[i] for i in range(len(T) + 1)]
    if len(T) > len(order):
        b.N = 2
    b.q, b.k_new, b.v_new = b.q[:b.N], b.k_new[:b.N], b.v_new[:b.N]
    b.max_new = max(max(y - x for x, y in zip(starts, starts[1:])), 1)
    b.start = torch.tensor(starts, dtype=torch.int32, device=DEV)
    need = C.csla_kv_workspace_size(b.lb.cfg(), b.B, b.N, b.max_new, b.max_len)
    buf = torch.full((need + (1 << 20),), 77, dtype=torch.uint8, device=DEV)
    out = b.attend(F32, ws=buf)
    assert _bits() == C.CSLA_DEVERR_INDEX
    assert bool((buf[need:] == 77).all())
    rows = torch.zeros(b.N, dtype=torch.bool)
    for r in kept:
        rows[starts[r]:starts[r + 1]] = True
    assert bool((out[~rows.to(DEV)] == 7.0).all()) and bool((out[rows.to(DEV)] != 7.0).all())
    # each kept request is answered as alone
    for r in kept:
        c = Batch.__new__(Batch)
        c.__dict__.update(b.__dict__)
        c.B, c.N = 1, starts[r + 1] - starts[r]
        c.slots = b.slots[r:r + 1]
        c.q = b.q[starts[r]:starts[r + 1]]
        c.start = torch.tensor([0, c.N], dtype=torch.int32, device=DEV)
        c.max_new = c.N
        b.lb.len[c.slots.long()] = L[r]
        assert torch.equal(c.attend(F32), out[starts[r]:starts[r + 1]])
    assert _bits() == 0
    # the append writes the kept requests' tokens and no others
    b.lb.k.fill_(float("nan"))
    b.lb.v.fill_(float("nan"))
    b.append()
    assert _bits() == C.CSLA_DEVERR_INDEX
    hit = torch.zeros(b.lb.k.shape[:3], dtype=torch.bool, device=DEV)
    for r in kept:
        p = torch.arange(L[r] - (starts[r + 1] - starts[r]), L[r])
        page = b.table[b.slots_l[r], p // 128].long().to(DEV)
        hit[page, :, (p % 128).to(DEV)] = True
        v = b.v_new[starts[r]:starts[r + 1]].reshape(-1, 2, 64)
        assert torch.equal(b.lb.v[page, :, (p % 128).to(DEV)], v)
    for pool in (b.lb.k, b.lb.v):
        assert bool(torch.isnan(pool[~hit]).all()) and bool(torch.isfinite(pool[hit]).all())


def test_other_types_and_layouts_on_the_device():
    """Tensors that would be read as something else, or past their end, are refused by the binding; the call is then made right."""
    b = Batch(DenseShape(D=64, HQ=4, HK=2, d_rope=64), [3, 2], [300, 40], seed=71)
    b.fill()
    want = b.attend(F32)
    for name, bad in (("gamma_q", b.gamma_q.bfloat16()), ("gamma_q", b.gamma_q[:-1].contiguous()), ("sink", b.sink.bfloat16()),
                      ("sink", b.sink.double()), ("slots", b.slots.long()), ("slots", b.slots[:1]), ("start", b.start.long()),
                      ("start", b.start[:-1]), ("q", b.q.reshape(5, 4, 64).transpose(0, 1)), ("q", b.q[:-1]), ("slots", b.slots.cpu())):
        good = getattr(b, name)
        setattr(b, name, bad)
        with pytest.raises(ValueError):
            b.attend(F32)
        if name in ("slots", "start"):
            with pytest.raises(ValueError):
                b.append()
        setattr(b, name, good)
    with pytest.raises(ValueError):
        b.gamma_k = b.gamma_k.bfloat16()
        b.append()
    need = C.csla_kv_workspace_size(b.lb.cfg(), b.B, b.N, b.max_new, b.max_len)
    with pytest.raises(ValueError):
        b.attend(F32, ws=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    assert torch.equal(b.attend(F32), want)
    assert _bits() == 0


def test_both_bounded_waits_run_out():
    """100 ms, half for each of the library's two waits; the context stays usable."""
    b = Batch(DenseShape(D=64, HQ=4, HK=2, d_rope=64), [1, 40], [300, 400], seed=72)
    b.fill()
    want = b.attend(F32)
    assert _bits() == 0
    a, z = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    C.csla_check_wait_timeout(100000)
    z.record()
    assert C.csla_device_error() == (C.CSLA_ERR_DEVICE, C.CSLA_DEVERR_TIMEOUT)
    assert 100 <= a.elapsed_time(z) < 1000
    assert torch.equal(b.attend(F32), want) and _bits() == 0
