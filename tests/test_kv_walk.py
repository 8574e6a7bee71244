"""The dense attention's walk over a ragged batch and its bounded wait, run on the CPU (kv_walk_host.cc: the kernels' own
header with a fiber per lane): which requests are taken, and that what they leave in the workspace stays inside the bytes
that csla_kv_workspace_size asks for, whatever the offsets hold."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from compressed_sparse_long_append_b200 import csla as C
from compressed_sparse_long_append_b200.layer import DenseShape

HERE = os.path.dirname(os.path.abspath(__file__))
ALL = 7   # every kind of request


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("kv_walk") / "kv_walk_host.so")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-shared", "-fPIC", "-I" + cuda, "-o", so,
                    os.path.join(HERE, "kv_walk_host.cc")], check=True)
    return ctypes.CDLL(so)


class Walk:
    """CTA 0's walk of `grid` over requests with the given offsets (None: N / B new tokens each) and lengths."""

    def __init__(self, host, shape, starts, lens, N, max_new, max_len, B=None, grid=4, kinds=ALL, give_up=-1, slots=None):
        B = B or len(starts) - 1
        i32 = lambda x: np.ascontiguousarray(x, dtype=np.int32)   # noqa: E731
        p = lambda x: None if x is None else x.ctypes.data_as(ctypes.c_void_p)   # noqa: E731
        st = None if starts is None else i32(starts)
        sl, ln = i32(range(B) if slots is None else slots), i32(lens)
        sh = i32([shape.D, shape.HQ, shape.HK, shape.window])
        self.join, out = np.zeros((B, 6), np.int64), np.zeros(3, np.int64)
        host.walk(p(sh), p(sl), p(st), p(ln), B, N, 0 if starts is not None else N // B, len(lens), 1 << 20, max_new, max_len,
                  grid, 0, kinds, give_up, p(self.join), p(out))
        self.items, self.err, self.part_rows = (int(x) for x in out)
        self.n0, self.rows_s, self.T, self.L, self.base = (self.join[:, i] for i in (0, 1, 3, 4, 5))
        # rows of partials in the bytes asked for (32 B per request, (m, l) and O of each row)
        need = C.csla_kv_workspace_size(shape.cfg(), B, N, max_new, max_len)
        self.room = max(0, (need - 32 * B - 16) // (8 + 4 * shape.D))


def test_overlapping_requests_are_refused(host):
    """Offsets that fall and rise again: each pair alone is a request of 2 rows, but the 32 of them share the same rows."""
    shape = DenseShape(D=128, HQ=64, HK=8)
    B, N = 64, 8
    starts = [6 + 2 * (i % 2) for i in range(B + 1)]
    w = Walk(host, shape, starts, [131072] * B, N, 2, 131072)
    assert w.err == C.CSLA_DEVERR_INDEX
    assert w.part_rows <= w.room, (w.part_rows, w.room)
    assert (w.rows_s != 0).sum() == 1 and w.rows_s[0] != 0   # the first pair, which nothing comes before


def _taken(starts, lens, slots, N, max_new, max_len):
    """Requests that the header says are answered, and the error bits of the others."""
    ok, err, top = [], 0, None
    for b in range(len(starts) - 1):
        n0, n1 = starts[b], starts[b + 1]
        if n0 < 0 or n1 < n0 or n1 > N or (top is not None and n0 < top):
            err |= C.CSLA_DEVERR_INDEX
        elif n1 > n0:
            if not 0 <= slots[b] < len(lens):
                err |= C.CSLA_DEVERR_INDEX
            elif n1 - n0 > max_new or lens[slots[b]] < n1 - n0 or lens[slots[b]] > max_len:
                err |= C.CSLA_DEVERR_LEN
            else:
                ok.append(b)
        top = n0 if top is None else max(top, n0)
    return ok, err


@pytest.mark.parametrize("broken", [False, True])
def test_random_offsets(host, broken):
    """Batches of up to 100 requests, some with offsets that fall, leave [0, N] or name bad slots: exactly those of the rule are
    taken, their rows are disjoint, and their partials fit (also those of a batch in order, at its bounds)."""
    rng = random.Random(7 + broken)
    most = 0.0
    for i in range(60):
        HK = rng.choice([1, 2, 4, 8])
        shape = DenseShape(D=rng.choice([64, 128]), HQ=HK * rng.choice([1, 4, 8, 16]), HK=HK, window=rng.choice([0, 0, 3000]))
        B = rng.choice([1, 3, 31, 32, 33, 64, 100])
        max_new = rng.choice([1, 2, 9, 700])
        starts = [0]
        for _ in range(B):
            starts.append(starts[-1] + rng.choice([0, 1, rng.randint(0, max_new), max_new]))
        N = max(starts[-1], 1)
        max_len = rng.choice([900, 20000, 131072])
        lens = [min(max_len, max_new + rng.choice([0, rng.randint(0, max_len), max_len])) for _ in range(B)]
        slots = list(range(B))
        if broken:
            for _ in range(rng.randint(1, 6)):
                j = rng.randint(0, B)
                starts[j] = rng.choice([-3, 0, N + 1, rng.randint(0, N), rng.randint(0, N), starts[rng.randint(0, B)]])
            if rng.random() < 0.3:
                slots[rng.randrange(B)] = rng.choice([-1, B])
            if rng.random() < 0.3:
                lens[rng.randrange(B)] = max_len + 1
        w = Walk(host, shape, starts, lens, N, max_new, max_len, slots=slots)
        ok, err = _taken(starts, lens, slots, N, max_new, max_len)
        assert w.err == err, (i, starts)
        assert [b for b in range(B) if w.T[b] and w.join[b, 1]] == [b for b in ok if w.join[b, 1]]
        assert not w.rows_s[[b for b in range(B) if b not in ok]].any()
        spans = sorted((starts[b], starts[b + 1]) for b in ok)
        assert all(x[1] <= y[0] for x, y in zip(spans, spans[1:]))
        if w.rows_s.any():
            assert w.part_rows <= w.room, (i, w.part_rows, w.room)
            most = max(most, w.part_rows / w.room)
    assert most > 0.3   # the bound is not out of all proportion, so the batches did reach for it


@pytest.mark.parametrize("starts", [None, [3 * i for i in range(101)]])
def test_a_role_that_gives_up_still_leaves_every_request_for_the_join(host, starts):
    """After a wait that ran out no item is taken, but the join runs all the same and reads every request's entry."""
    shape = DenseShape(D=128, HQ=16, HK=2)
    args = (host, shape, starts, [9000 + i for i in range(100)], 300, 3, 10000)
    whole = Walk(*args, B=100)
    assert whole.items > 10 and whole.err == 0 and bool((whole.rows_s > 0).all())
    for n in (0, 1, 10):
        w = Walk(*args, B=100, give_up=n)
        assert w.items == n + 1
        assert np.array_equal(w.join, whole.join)
        assert w.err == 0


@pytest.mark.parametrize("ready,stop,item,ok,took", [
    (1900, 0, 0, True, 1900), (2400, 0, 0, False, 2000),   # a tile: 2 s
    (2400, 0, 1, True, 2400),                              # 2^20 tiles of 2.3 us each, the longest item
    (9000, 0, 1, True, 9000), (17000, 0, 1, False, 16000),
    (9000, 2100, 1, False, 2100)])                         # another role of the CTA has given up
def test_waits_are_bounded(host, ready, stop, item, ok, took):
    ms, abort, err = ctypes.c_int64(), ctypes.c_int(), ctypes.c_uint()
    got = host.wait(ctypes.c_int64(ready), ctypes.c_int64(stop), item, ctypes.byref(ms), ctypes.byref(abort), ctypes.byref(err))
    assert bool(got) == ok
    assert abs(ms.value - took) <= 10
    assert (abort.value, err.value) == ((0, 0) if ok else (1, 0 if stop else C.CSLA_DEVERR_TIMEOUT))


@pytest.mark.parametrize("D,HQ,HK,T,L,rows,parts", [
    (128, 8, 1, 1, 40000, 8, 63),          # 313 tiles in 313 / 4 = 78 chunks at most, so of 5 tiles: more parts than a warp joins
    (64, 16, 1, 1, 100003, 16, 87),        # 782 in 782 / 8 = 97 at most, so of 9
    (128, 32, 8, 5, 28500, 20, 36),        # one round over the SMs: 18 chunks of 12 to 16 tiles instead of 13
    (128, 32, 8, 20, 33000, 80, 36),
    (128, 64, 1, 1, 230001, 64, 278),      # chunks of 13 tiles, two streams
    (128, 64, 1, 2, 3000, 128, 2),
    (128, 4, 4, 300, 17000, 300, 0),       # row tiles too few for the SMs: all cut (parts by row tile)
    (128, 16, 16, 2500, 7000, 256, 0),     # more row tiles than SMs: the first one of each head cut
    (64, 32, 16, 1300, 9000, 512, 0),      # the first two
    (128, 32, 8, 2048, 2048, 0, 0)])       # none
def test_how_requests_are_cut(host, D, HQ, HK, T, L, rows, parts):
    """The plan behind the cases that the GPU tests name."""
    w = Walk(host, DenseShape(D=D, HQ=HQ, HK=HK), [0, T], [L], T, T, L)
    assert (w.rows_s[0], w.join[0, 2]) == (rows, parts)
    assert w.part_rows <= w.room
