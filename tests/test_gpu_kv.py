"""The dense paged layer on the GPU against its formulas in 64 bits: csla_kv_append and csla_kv_attend over ragged
batches, head layouts, rotations, windows, types and strides, lengths from one token to long ones.  Every pool starts as NaN, so a
read outside what a request may see shows at once."""
import pytest
import torch

from compressed_sparse_long_append_b200 import csla as C
from compressed_sparse_long_append_b200.layer import DenseShape
from kv_helpers import DEV, Batch, no_device_error, randn

pytestmark = pytest.mark.gpu

ADJ, HALF = C.CSLA_ROPE_ADJACENT, C.CSLA_ROPE_HALVES
BF, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("D,HK,d_rope,pairs", [(128, 8, 64, ADJ), (128, 3, 128, HALF), (64, 1, 64, HALF), (64, 5, 16, ADJ),
                                               (128, 1, 0, ADJ), (128, 2, 96, HALF), (64, 16, 48, HALF), (64, 200, 32, ADJ)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,L", [([1], [1]), ([1, 1, 1], [128, 129, 300]), ([0, 5, 0, 0, 130, 1], [9, 5, 0, 128, 400, 257])])
def test_append(D, HK, d_rope, pairs, dtype, T, L):
    shape = DenseShape(D=D, HQ=HK, HK=HK, d_rope=d_rope, rope_pairs=pairs)
    b = Batch(shape, T, L, seed=D + HK, q_dtype=dtype, norm=HK % 2 == 1, extra_rows=3, pad=16)
    k, tol, v, hit = b.expected_append()
    b.append()
    no_device_error()
    assert torch.equal(b.lb.v.view(torch.int16), v.view(torch.int16))
    assert bool(torch.isnan(b.lb.k[~hit]).all())
    err = (b.lb.k.double() - k).abs()[hit]
    assert bool((err <= tol[hit]).all()), float((err / tol[hit]).max())


def test_append_long_chunk_far_positions_and_many_requests():
    # 1500 tokens ending near 2^20; then 700 requests of 0..3 tokens
    shape = DenseShape(D=128, HQ=2, HK=2, d_rope=128, rope_pairs=HALF, theta=500000.0)
    b = Batch(shape, [1500], [1 << 20], seed=3)
    k, tol, v, hit = b.expected_append()
    b.append()
    no_device_error()
    assert torch.equal(b.lb.v.view(torch.int16), v.view(torch.int16))
    assert bool(((b.lb.k.double() - k).abs()[hit] <= tol[hit]).all())
    T = [i % 4 for i in range(700)]
    b = Batch(DenseShape(D=64, HQ=2, HK=2, d_rope=64), T, [t + (37 * i) % 300 for i, t in enumerate(T)], seed=4)
    k, tol, v, hit = b.expected_append()
    b.append()
    no_device_error()
    assert torch.equal(b.lb.v.view(torch.int16), v.view(torch.int16))
    assert bool(((b.lb.k.double() - k).abs()[hit] <= tol[hit]).all()) and bool(torch.isnan(b.lb.k[~hit]).all())


@pytest.mark.parametrize("theta", [2.0 ** -7, 1.0, 1.5])
def test_small_rotation_bases(theta):
    """A base below 1 makes the later pairs the faster ones, past a whole turn per position."""
    for pairs in (ADJ, HALF):
        b = Batch(DenseShape(D=64, HQ=4, HK=2, d_rope=64, rope_pairs=pairs, theta=theta), [300, 2], [900, 300], seed=60)
        k, tol, v, hit = b.expected_append()
        b.append()
        assert bool(((b.lb.k.double() - k).abs()[hit] <= tol[hit]).all())
        b.fill()
        b.check_attend(b.attend(F32))
    no_device_error()


def test_append_keeps_special_values():
    shape = DenseShape(D=64, HQ=1, HK=1, d_rope=0)
    b = Batch(shape, [4], [6], norm=False)
    x = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0], device=DEV)
    b.k_new = x.to(BF)[:, None].expand(4, 64).contiguous()
    b.v_new = b.k_new.clone()
    b.append()
    for pool in (b.lb.k, b.lb.v):
        got = pool[b.table[1, 0].item(), 0, 2:6, 0].float()
        assert torch.isnan(got[0]) and got[1] == float("inf") and got[2] == -float("inf")
        assert got[3] == 0 and torch.signbit(got[3])


# ---------------------------------------------------------------- attention
def _run(shape, T, L, out_dtype=BF, lo=None, **kw):
    b = Batch(shape, T, L, **kw)
    b.fill(lo)
    out = b.attend(out_dtype)
    no_device_error()
    b.check_attend(out)
    return b, out


@pytest.mark.parametrize("D,HQ,HK", [(128, 1, 1), (128, 64, 8), (64, 14, 2), (64, 9, 3), (128, 5, 5), (64, 16, 1), (128, 128, 1)])
@pytest.mark.parametrize("L", [1, 2, 127, 128, 129, 255, 256, 257, 640, 1000, 1025])
def test_single_token(D, HQ, HK, L):
    _run(DenseShape(D=D, HQ=HQ, HK=HK, d_rope=64), [1], [L], seed=L, uniform=True)


@pytest.mark.parametrize("D,HQ,HK,pairs,window", [(128, 32, 8, ADJ, 0), (64, 8, 8, HALF, 0), (128, 6, 2, HALF, 100), (64, 16, 2, ADJ, 129)])
def test_ragged_decode(D, HQ, HK, pairs, window):
    L = [1, 5000, 128, 37, 2049, 130, 256, 1024, 3333, 12, 640, 4097]
    lo = [max(0, n - window) if window else 0 for n in L]
    _run(DenseShape(D=D, HQ=HQ, HK=HK, d_rope=D, rope_pairs=pairs, window=window), [1] * len(L), L, lo=lo, seed=5)


@pytest.mark.parametrize("D,HQ,HK", [(128, 4, 1), (64, 4, 4), (128, 40, 8), (64, 7, 1)])
@pytest.mark.parametrize("T,L", [([2], [2]), ([5, 3, 1, 8], [700, 3, 129, 1500]), ([33, 64, 65], [33, 300, 1000]),
                                 ([127, 128, 129], [127, 400, 129]), ([257, 0, 1, 300], [600, 77, 900, 300])])
def test_chunks(D, HQ, HK, T, L):
    _run(DenseShape(D=D, HQ=HQ, HK=HK, d_rope=64, rope_pairs=HALF), T, L, seed=len(T))


@pytest.mark.parametrize("D,HQ,HK,T", [(64, 3, 3, [7, 8, 9, 16, 17]), (128, 2, 2, [17, 9, 8, 1]), (128, 4, 2, [4, 5, 8, 9]),
                                       (64, 8, 1, [1, 2, 3]), (128, 9, 1, [1, 2]), (64, 17, 1, [1, 8])])
@pytest.mark.parametrize("window", [0, 70])
def test_rows_around_the_kinds_of_requests(D, HQ, HK, T, window):
    """8, 16 and 128 rows per KV head and one more, in one batch: each is taken by other code."""
    L = [t + 200 + 331 * i for i, t in enumerate(T)]
    lo = [max(0, n - t + 1 - window) if window else 0 for t, n in zip(T, L)]
    b, out = _run(DenseShape(D=D, HQ=HQ, HK=HK, d_rope=32, window=window), T, L, lo=lo, seed=D + window, out_dtype=F32)
    # an unmapped page (the first request's first) is masked whatever the kind, and touches nobody else's rows
    if not window:
        b.lb.block_table[b.slots_l[0], 0] = -1
        got = b.attend(F32)
        assert _bits() == C.CSLA_DEVERR_PAGE
        assert torch.equal(got[T[0]:], out[T[0]:]) and bool(torch.isfinite(got).all())
        assert not torch.equal(got[:T[0]], out[:T[0]])


@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 300])
def test_windows(window):
    T, L = [1, 260, 7, 40], [900, 260, 131, 650]
    # nothing before the first new token's window is ever read
    lo = [max(0, n - t + 1 - window) for t, n in zip(T, L)]
    _run(DenseShape(D=64, HQ=6, HK=2, d_rope=32, window=window), T, L, lo=lo, seed=window)


@pytest.mark.parametrize("q_dtype,out_dtype,norm,sink", [(BF, F32, True, False), (F32, BF, False, True), (F32, F32, True, True),
                                                         (BF, BF, False, False)])
def test_types(q_dtype, out_dtype, norm, sink):
    for D in (64, 128):
        _run(DenseShape(D=D, HQ=8, HK=2, d_rope=48, rope_pairs=HALF), [1, 70, 3], [300, 200, 1300], out_dtype=out_dtype,
             q_dtype=q_dtype, norm=norm, sink=sink, pad=24, extra_rows=5)


def test_long_contexts():
    _run(DenseShape(D=128, HQ=8, HK=1, d_rope=64), [1, 1], [40000, 70001], seed=8)
    _run(DenseShape(D=64, HQ=8, HK=4, d_rope=64, rope_pairs=HALF), [40, 4], [33000, 20011], seed=9)
    _run(DenseShape(D=128, HQ=4, HK=4, d_rope=64), [300], [17000], seed=10)


def test_many_requests():
    T = [(i * 7) % 3 for i in range(333)]
    _run(DenseShape(D=64, HQ=4, HK=2, d_rope=64), T, [t + (i * 53) % 700 for i, t in enumerate(T)], seed=11)


def test_sharp_and_scaled_scores():
    # one key dominates (scores of hundreds), all equal, and a scale of the caller's
    for scale, mul in ((0.0, 20.0), (0.5, 1.0), (0.0, 0.0)):
        b = Batch(DenseShape(D=128, HQ=8, HK=2, d_rope=64, scale=scale), [1, 9, 200], [1000, 300, 500], norm=False, seed=12)
        b.fill()
        b.q = (b.q.float() * mul).to(BF)
        out = b.attend(F32)
        no_device_error()
        b.check_attend(out)


def test_rising_scores():
    """Each key scores higher than the one before: the running maximum moves in every tile."""
    shape = DenseShape(D=64, HQ=2, HK=1, d_rope=0)
    b = Batch(shape, [1, 130], [2000, 900], norm=False, sink=False, seed=13)
    b.fill()
    for i, s in enumerate(b.slots_l):
        p = torch.arange(b.L[i])
        page = b.table[s, p // 128].long().to(DEV)
        b.lb.k[page, :, (p % 128).to(DEV), 0] = (p.float() * 0.5).to(BF).to(DEV)[:, None]
    b.q = b.q.clone()
    b.q[:, 0::64] = 2.0
    out = b.attend(F32)
    no_device_error()
    b.check_attend(out)


def test_infinite_and_masked_sinks():
    b = Batch(DenseShape(D=128, HQ=4, HK=2, d_rope=64), [1, 20], [50, 300], seed=14)
    b.fill()
    b.sink = torch.tensor([-1e30, 100.0, -float("inf"), 0.0], device=DEV)
    out = b.attend(F32)
    no_device_error()
    b.check_attend(out)


def test_batch_invariance_and_repeats():
    """A request's rows are the same bits alone, in a batch, in another order, and on every repeat."""
    shape = DenseShape(D=128, HQ=12, HK=4, d_rope=64)
    T, L = [1, 1, 300, 5, 1, 64], [9000, 40, 700, 3000, 20000, 2000]
    b = Batch(shape, T, L, seed=15)
    b.fill()
    out = b.attend()
    for _ in range(3):
        assert torch.equal(b.attend(), out)
    for order in ([5, 4, 3, 2, 1, 0], [2], [4], [3, 0], [1, 2]):
        c = Batch.__new__(Batch)
        c.__dict__.update(b.__dict__)
        c.B, c.T, c.L = len(order), [T[i] for i in order], [L[i] for i in order]
        c.slots_l = [b.slots_l[i] for i in order]
        c.slots = torch.tensor(c.slots_l, dtype=torch.int32, device=DEV)
        c.q = torch.cat([b.q[b.start_l[i]:b.start_l[i + 1]] for i in order])
        c.start_l = [0]
        for t in c.T:
            c.start_l.append(c.start_l[-1] + t)
        c.start = torch.tensor(c.start_l, dtype=torch.int32, device=DEV)
        c.N, c.max_new, c.max_len = c.start_l[-1], max(c.T) + 11, max(c.L) + 500
        got = c.attend()
        for j, i in enumerate(order):
            assert torch.equal(got[c.start_l[j]:c.start_l[j + 1]], out[b.start_l[i]:b.start_l[i + 1]]), (order, i)
    no_device_error()


# ---------------------------------------------------------------- bad inputs that only the device sees
def _bits():
    rc, bits = C.csla_device_error()
    return bits


def test_unmapped_pages_are_masked():
    shape = DenseShape(D=64, HQ=4, HK=2, d_rope=64)
    b = Batch(shape, [1, 3, 140], [700, 100, 400], seed=16)
    b.fill()
    # request 0 loses its middle page, request 1 its only one, request 2 is whole
    b.lb.block_table[b.slots_l[0], 2] = -1
    b.lb.block_table[b.slots_l[1], 0] = b.lb.n_pages
    out = b.attend(F32)
    assert _bits() == C.CSLA_DEVERR_PAGE
    assert bool((out[1:4] == 0).all())
    whole = b.attend(F32)
    assert _bits() == C.CSLA_DEVERR_PAGE
    assert torch.equal(whole, out)
    # request 0: as if the page's tokens scored -inf
    from kv_reference import attend_request, with_output_step
    k, v = b.rows(0, b.lb.k), b.rows(0, b.lb.v)
    keep = torch.cat([torch.arange(0, 256), torch.arange(384, 700)]).to(DEV)
    q = b.q.reshape(b.N, 4, 64)[:1]
    from kv_reference import norm, rotate
    qr = rotate(norm(q.double(), b.gamma_q, shape.eps), torch.tensor([699], device=DEV), 64, False, shape.theta)
    plain = DenseShape(D=64, HQ=4, HK=2, d_rope=0)
    o, tol = attend_request(qr, k[keep], v[keep], len(keep) - 1, plain, False, b.sink, None)
    assert bool(((out[:1].double() - o).abs() <= with_output_step(o, tol, F32)).all())
    # the append skips tokens in unmapped pages and writes the others
    b = Batch(shape, [140], [400], seed=17)
    k, tol, v, hit = b.expected_append()
    b.lb.block_table[b.slots_l[0], 2] = -5
    gone = b.table[b.slots_l[0], 2].long().item()
    hit[gone] = False
    b.append()
    assert _bits() == C.CSLA_DEVERR_PAGE
    assert bool(torch.isnan(b.lb.k[~hit]).all()) and bool(torch.isnan(b.lb.v[~hit]).all())
    assert bool(((b.lb.k.double() - k).abs()[hit] <= tol[hit]).all())


@pytest.mark.parametrize("what,bit", [("slot", C.CSLA_DEVERR_INDEX), ("short", C.CSLA_DEVERR_LEN), ("long", C.CSLA_DEVERR_LEN),
                                      ("order", C.CSLA_DEVERR_INDEX), ("behind", C.CSLA_DEVERR_INDEX)])
def test_bad_requests_are_skipped(what, bit):
    shape = DenseShape(D=128, HQ=4, HK=2, d_rope=64)
    b = Batch(shape, [3, 5, 2], [300, 40, 129], seed=18)
    b.fill()
    skip = {1}
    if what == "slot":
        b.slots[1] = b.n_slots
    if what == "short":
        b.lb.len[b.slots_l[1]] = 4
    if what == "long":
        b.lb.len[b.slots_l[1]] = 128 * b.lb.bt_stride + 1
    if what == "order":
        b.start[1] = 9     # request 0: rows 0..8 (its length no longer fits its context bound), request 1: 9..7
        skip = None
    if what == "behind":
        b.start[3] = b.N + 1
        skip = {2}
    out = b.attend(F32)
    assert _bits() & bit
    if skip is not None:
        b.check_attend(out, skip=skip)
    before = b.lb.k.clone()
    b.append()
    assert _bits() & bit
    if skip == {1}:
        page = b.table[b.slots_l[1], 0].item()
        assert torch.equal(b.lb.k[page].view(torch.int16), before[page].view(torch.int16))


def test_bounds_of_the_call():
    """T above max_new or len above max_len: the request is skipped, the others answered."""
    b = Batch(DenseShape(D=64, HQ=2, HK=2, d_rope=64), [1, 9, 1], [500, 20, 3], seed=19)
    b.fill()
    b.max_new = 8
    out = b.attend()
    assert _bits() == C.CSLA_DEVERR_LEN
    b.check_attend(out, skip={1})
    b.max_new, b.max_len = 9, 499
    out = b.attend()
    assert _bits() == C.CSLA_DEVERR_LEN
    b.check_attend(out, skip={0})


def test_same_request_twice_and_idle_slots():
    """Two batch entries of one slot read the same cache; entries without tokens may name any slot."""
    b = Batch(DenseShape(D=128, HQ=8, HK=2, d_rope=64), [2, 0, 1], [400, 0, 77], seed=20, slot_order=[1, 0, 2])
    b.fill()
    b.slots[1] = -1
    out = b.attend()
    no_device_error()
    b.check_attend(out)
    b.append()
    no_device_error()
    c = Batch(DenseShape(D=128, HQ=8, HK=2, d_rope=64), [1, 1], [300, 300], seed=21, slot_order=[1, 1], uniform=True)
    c.fill()
    c.q[1] = c.q[0]
    out = c.attend()
    no_device_error()
    assert torch.equal(out[0], out[1])


@pytest.mark.parametrize("T,L", [(1, [300, 1, 4097]), (5, [5, 700, 2100]), (40, [900, 41]), (300, [300, 1000])])
def test_equal_numbers_of_new_tokens_need_no_offsets(T, L):
    for D, HQ, HK in ((128, 8, 2), (64, 3, 3)):
        b, out = _run(DenseShape(D=D, HQ=HQ, HK=HK, d_rope=64, window=0 if T < 40 else 200), [T] * len(L), L, seed=T,
                      uniform=True)
        b.start = torch.tensor(b.start_l, dtype=torch.int32, device=DEV)
        assert torch.equal(b.attend(), out)


def test_long_chunk_over_a_long_context():
    """Row tiles of more than a round over the SMs, the last ones' keys cut."""
    b = Batch(DenseShape(D=128, HQ=16, HK=16, d_rope=64), [2500], [7000], seed=40)
    b.fill()
    out = b.attend(F32)
    no_device_error()
    rows = [0, 1, 127, 128, 255, 256, 300, 511, 512, 1000, 1791, 1792, 2047, 2048, 2499]   # of the first and last row tiles
    from kv_reference import attend_request, with_output_step
    k, v = b.rows(0, b.lb.k), b.rows(0, b.lb.v)
    q = b.q.reshape(b.N, 16, 128)
    for r in rows:
        n = 4500 + r + 1
        o, tol = attend_request(q[r:r + 1], k[:n], v[:n], n - 1, b.shape, False, b.sink, b.gamma_q)
        assert bool(((out[r:r + 1].double() - o).abs() <= with_output_step(o, tol, F32)).all()), r
    assert bool(torch.isfinite(out).all())


def test_a_nan_stays_in_the_rows_that_see_it():
    """NaN in one token's query, in one visible key, in one visible value: rows that see it are NaN, others are as without."""
    for T, L in (([1, 1], [700, 700]), ([40, 40], [300, 300]), ([200, 200], [500, 500])):
        b = Batch(DenseShape(D=64, HQ=4, HK=2, d_rope=0), T, L, seed=41)
        b.fill()
        clean = b.attend(F32)
        b.q = b.q.clone()
        b.q[T[0] - 1, 5] = float("nan")           # request 0, last token, head 0
        out = b.attend(F32)
        assert bool(torch.isnan(out[T[0] - 1, 0]).all())
        out[T[0] - 1, 0] = clean[T[0] - 1, 0]
        assert torch.equal(out, clean)
        b.q[T[0] - 1, 5] = 0.0
        clean = b.attend(F32)
        for pool in (b.lb.k, b.lb.v):              # request 1, its very first token, KV head 1: every row of heads 2, 3 sees it
            page = b.table[b.slots_l[1], 0].item()
            old = pool[page, 1, 0].clone()
            pool[page, 1, 0] = float("nan")
            out = b.attend(F32)
            assert bool(torch.isnan(out[T[0]:, 2:]).all())
            out[T[0]:, 2:] = clean[T[0]:, 2:]
            assert torch.equal(out, clean)
            pool[page, 1, 0] = old
    no_device_error()


def test_workspace_is_enough_and_kept_within():
    """The bytes asked for suffice at any 16-byte boundary, and nothing behind them is touched."""
    import random
    rng = random.Random(42)
    for i in range(24):
        HK = rng.choice([1, 2, 5, 10])
        G = rng.choice([1, 2, 4, 7, 16])
        B = rng.randint(1, 4)
        T = [rng.choice([0, 1, 1, 3, rng.randint(1, 40), rng.randint(1, 400)]) for _ in range(B)]
        T[0] = max(T[0], 1)
        L = [t + rng.choice([0, 50, rng.randint(0, 3000), rng.randint(0, 9000)]) for t in T]
        b = Batch(DenseShape(D=rng.choice([64, 128]), HQ=HK * G, HK=HK, d_rope=32, window=rng.choice([0, 0, 700])), T, L, seed=i)
        b.fill()
        want = b.attend()
        need = C.csla_kv_workspace_size(b.lb.cfg(), b.B, b.N, b.max_new, b.max_len)
        buf = torch.full((need + 64 + 4096,), 77, dtype=torch.uint8, device=DEV)
        for off in (0, 16, 32, 48):
            buf.fill_(77)
            out = b.attend(ws=buf[off:])
            assert torch.equal(out, want)
            assert bool((buf[:off] == 77).all()) and bool((buf[off + need:] == 77).all()), (i, off)
    no_device_error()


# ---------------------------------------------------------------- streams and graphs
def test_two_graphs_share_a_workspace_in_turn():
    """Two captured calls on one workspace, replayed one after the other, and an eager call in between."""
    bs = [Batch(DenseShape(D=128, HQ=12, HK=4, d_rope=64), T, L, seed=50 + i)
          for i, (T, L) in enumerate([([1, 1], [3000, 9000]), ([1, 20, 200], [2500, 1300, 2000])])]
    for b in bs:
        b.fill()
    want = [b.attend() for b in bs]
    need = max(C.csla_kv_workspace_size(b.lb.cfg(), b.B, b.N, b.max_new, b.max_len) for b in bs)
    ws = torch.full((max(need // 4 + 4, 4),), float("nan"), dtype=torch.float32, device=DEV)
    outs, graphs = [torch.zeros_like(w) for w in want], []
    torch.cuda.synchronize()
    for b, o in zip(bs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.attend(out=o, ws=ws)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for i in (0, 1, 1, 0):
            graphs[i].replay()
            assert torch.equal(bs[1].attend(ws=ws), want[1])
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    no_device_error()


def test_other_stream_and_two_calls_at_once():
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    bs = [Batch(DenseShape(D=128, HQ=32, HK=8, d_rope=64), [1, 200], [6000, 900], seed=22 + i) for i in range(2)]
    want = []
    for b in bs:
        b.fill()
        want.append(b.attend())
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for b, s in zip(bs, (s1, s2)):
            with torch.cuda.stream(s):
                got.append(b.attend())
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
    no_device_error()


def test_decode_steps_in_a_graph():
    """Append and attend of one decode step captured once and replayed: lengths advance on the device, every step equals
    the eager one and the formulas."""
    shape = DenseShape(D=128, HQ=12, HK=4, d_rope=64)
    L0 = [127, 1000, 2]
    steps = 4

    def make():
        b = Batch(shape, [1, 1, 1], [n + steps for n in L0], seed=30, uniform=True)
        b.fill()
        b.lb.len.zero_()
        b.lb.len[b.slots.long()] = torch.tensor(L0, dtype=torch.int32, device=DEV)
        return b

    g = torch.Generator().manual_seed(31)
    xs = [randn(g, 3, (12 + 8) * 128, dtype=BF) for _ in range(steps)]
    eager, graphed = make(), make()
    need = C.csla_kv_workspace_size(eager.lb.cfg(), 3, 3, 1, 1100)
    out = torch.empty((3, 12, 128), dtype=BF, device=DEV)
    x = xs[0].clone()
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)

    def step(b, out):
        b.max_len = 1100
        b.q, b.k_new, b.v_new = x[:, :1536], x[:, 1536:2048], x[:, 2048:]
        b.lb.len[b.slots.long()] += 1
        b.append()
        return b.attend(out=out, ws=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(graphed, out)   # warm-up
    torch.cuda.synchronize()
    graphed = make()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step(graphed, out)
    for i in range(steps):
        x.copy_(xs[i])
        gr.replay()
        got = out.clone()
        want = step(eager, torch.empty_like(out))
        assert torch.equal(got, want), i
        eager.L = [n + i + 1 for n in L0]
        eager.check_attend(want)
    assert torch.equal(graphed.lb.k.view(torch.int16), eager.lb.k.view(torch.int16))
    no_device_error()


def test_refusals_of_the_binding():
    b = Batch(DenseShape(D=64, HQ=2, HK=1, d_rope=64), [1], [5])
    b.fill()
    with pytest.raises(ValueError):
        b.attend(out=torch.empty((1, 2, 64), dtype=F32))   # a host tensor
    with pytest.raises(ValueError):
        b.attend(out=torch.empty((1, 64, 2), dtype=F32, device=DEV).transpose(1, 2))
    b.q = b.q.to(F32)
    with pytest.raises(ValueError):
        b.attend()
