"""Batches with requests of few rows and of many in one csla_kv_attend call, whose two kernels run side by side: inputs that
change right before each call, on a stream and in a graph, and calls where the second stream is not to be had."""
import threading

import pytest
import torch

from compressed_sparse_long_append_b200 import csla as C
from compressed_sparse_long_append_b200.layer import DenseShape
from kv_helpers import DEV, Batch, no_device_error, randn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
T, L0, STEPS = [1, 40, 1, 300, 2], [2000, 700, 90, 1300, 5000], 4


class Steps:
    """A mixed batch whose q, lengths and pages change from step to step, as a stream's work before the call."""

    def __init__(self, seed):
        self.b = Batch(DenseShape(D=128, HQ=16, HK=4, d_rope=64), T, [n + STEPS for n in L0], seed=seed)
        self.b.fill()
        g = torch.Generator().manual_seed(seed + 1)
        self.q = [randn(g, *self.b.q.shape, dtype=BF) for _ in range(STEPS)]
        self.len = [torch.tensor([0] + [n + i for n in L0], dtype=torch.int32, device=DEV)[:self.b.n_slots] for i in range(STEPS)]
        # the pages of request 0 and of request 3 in another order at every step
        self.table = []
        for i in range(STEPS):
            t = self.b.lb.block_table.clone()
            for r in (0, 3):
                s, n = self.b.slots_l[r], L0[r] // 128
                t[s, :n] = t[s, torch.randperm(n, generator=g).to(DEV)]
            self.table.append(t)
        assert self.b.slots_l == [1, 2, 3, 4, 5]
        need = C.csla_kv_workspace_size(self.b.lb.cfg(), self.b.B, self.b.N, self.b.max_new, self.b.max_len)
        self.ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
        self.qbuf, self.out = torch.zeros_like(self.b.q), torch.zeros((self.b.N, 16, 128), dtype=BF, device=DEV)
        self.b.q = self.qbuf

    def change(self, i):
        self.qbuf.copy_(self.q[i])
        self.b.lb.len.copy_(self.len[i])
        self.b.lb.block_table.copy_(self.table[i])

    def alone(self):
        """Every step with nothing else in flight."""
        want = []
        for i in range(STEPS):
            self.change(i)
            torch.cuda.synchronize()
            self.out.fill_(7.0)
            torch.cuda.synchronize()
            want.append(self.b.attend(out=self.out, ws=self.ws).clone())
            torch.cuda.synchronize()
        self.out.fill_(7.0)
        return want


def test_inputs_that_change_right_before_each_call():
    s = Steps(80)
    want = s.alone()
    # the last step against the formulas (its pages as they are now)
    s.b.table, s.b.L = s.b.lb.block_table.cpu(), [n + STEPS - 1 for n in L0]
    s.b.check_attend(want[-1])
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            got = []
            for _ in range(5):
                for i in range(STEPS):
                    s.change(i)
                    got.append(s.b.attend(out=s.out, ws=s.ws).clone())
                    s.out.fill_(7.0)       # and right behind it: the call is done with its output
            torch.cuda.synchronize()
        for j, o in enumerate(got):
            assert torch.equal(o, want[j % STEPS]), j
    no_device_error()


def test_a_graph_whose_inputs_change_between_and_inside_replays():
    s = Steps(82)
    want = s.alone()
    copies = [torch.zeros_like(s.out) for _ in range(STEPS)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(STEPS):
            s.change(i)
            s.b.attend(out=s.out, ws=s.ws)
            copies[i].copy_(s.out)
    for k in range(5):
        g.replay()
        s.out.fill_(7.0)
        torch.cuda.synchronize()
        for i in range(STEPS):
            assert torch.equal(copies[i], want[i]), (k, i)
            copies[i].zero_()
    # new queries in the buffers that the graph reads
    for i in range(STEPS):
        s.q[i].neg_()
    g.replay()
    got = [c.clone() for c in copies]
    want = s.alone()
    for i in range(STEPS):
        assert torch.equal(got[i], want[i]), i
    no_device_error()


def test_a_threads_first_call_inside_a_capture():
    """A thread that never made a second stream captures a mixed call: the same bits."""
    s = Steps(84)
    want = s.alone()
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            with torch.cuda.device(0):
                st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=st):
                    s.change(2)
                    s.b.attend(out=s.out, ws=s.ws)
                g.replay()
                torch.cuda.synchronize()
        except Exception as e:   # shown by the test's thread
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not errors, errors
    assert torch.equal(s.out, want[2])
    no_device_error()


def test_a_call_beside_a_capture_that_has_not_ended():
    """After a captured mixed call its thread's second stream is part of the capture: an eager call on another stream
    meanwhile is answered without it, and the capture is not disturbed."""
    s, o = Steps(86), Steps(88)
    want, other = s.alone(), o.alone()
    o.change(1)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.change(1)
        s.b.attend(out=s.out, ws=s.ws)
        o.b.attend(out=o.out, ws=o.ws, stream=st.cuda_stream)
        s.b.attend(out=s.out, ws=s.ws)
    torch.cuda.synchronize()
    assert torch.equal(o.out, other[1])
    for _ in range(2):
        s.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.out, want[1])
    no_device_error()
