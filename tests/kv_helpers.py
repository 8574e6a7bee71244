"""Dense paged layers on the GPU: pools whose unused rows hold NaN, scattered pages, and the calls around them."""
import torch

from compressed_sparse_long_append_b200 import csla as C
from compressed_sparse_long_append_b200.layer import DenseBuffers, DenseShape
from kv_reference import PAGE, append_rows, attend_request, with_output_step

DEV = "cuda"
DT = {torch.float32: C.CSLA_F32, torch.bfloat16: C.CSLA_BF16}


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, dtype=torch.float32).to(DEV).to(dtype)


class Batch:
    """A ragged batch on one dense layer: T[b] new tokens, L[b] context (new tokens included)."""

    def __init__(self, shape: DenseShape, T, L, seed=0, q_dtype=torch.bfloat16, norm=True, sink=True, extra_rows=0,
                 spare_pages=2, slot_order=None, uniform=False, pad=0):
        self.shape, self.T, self.L = shape, list(T), list(L)
        g = torch.Generator().manual_seed(seed)
        self.g = g
        B = len(T)
        self.B, self.n_slots = B, B + 1
        self.slots_l = slot_order or [(b + 1) % self.n_slots for b in range(B)]
        need = [-(-n // PAGE) for n in L]
        n_pages, stride = sum(need) + spare_pages, max(need + [1]) + 1
        perm = torch.randperm(n_pages, generator=g).tolist()
        self.lb = DenseBuffers(shape, self.n_slots, n_pages, stride, DEV)
        self.table = torch.full((self.n_slots, stride), -1, dtype=torch.int32)
        lens = torch.zeros(self.n_slots, dtype=torch.int32)
        for b, s in enumerate(self.slots_l):
            for i in range(need[b]):
                self.table[s, i] = perm.pop()
            lens[s] = L[b]
        self.lb.block_table.copy_(self.table)
        self.lb.len.copy_(lens)
        self.lb.k.fill_(float("nan"))
        self.lb.v.fill_(float("nan"))
        self.slots = torch.tensor(self.slots_l, dtype=torch.int32, device=DEV)
        st = [0]
        for t in T:
            st.append(st[-1] + t)
        self.start_l = st
        self.start = None if uniform else torch.tensor(st, dtype=torch.int32, device=DEV)
        self.N = st[-1] + extra_rows
        self.max_new, self.max_len = max(max(T), 1), max(max(L), 1)
        D, HQ, HK = shape.D, shape.HQ, shape.HK
        # q, k and v as slices of one fused projection (pad: further columns)
        x = randn(g, self.N, (HQ + 2 * HK) * D + pad, dtype=q_dtype)
        self.q, self.k_new, self.v_new = x[:, :HQ * D], x[:, HQ * D:(HQ + HK) * D], x[:, (HQ + HK) * D:(HQ + 2 * HK) * D]
        if pad == 0 and HQ > 1:
            self.q = self.q.contiguous()
        self.q_dtype = q_dtype
        self.gamma_q = 1.0 + 0.2 * randn(g, D) if norm else None
        self.gamma_k = 1.0 + 0.2 * randn(g, D) if norm else None
        self.sink = randn(g, HQ) if sink else None

    def fill(self, lo=None):
        """Random K and V at positions lo[b]..L[b]-1 of every request (NaN stays elsewhere)."""
        for b, s in enumerate(self.slots_l):
            a = 0 if lo is None else lo[b]
            p = torch.arange(a, self.L[b])
            page = self.table[s, p // PAGE].long().to(DEV)
            at = (p % PAGE).to(DEV)
            for pool in (self.lb.k, self.lb.v):
                pool[page, :, at] = randn(self.g, len(p), self.shape.HK, self.shape.D, dtype=torch.bfloat16)

    def rows(self, b, pool, lo=0):
        """Cache rows 0..L-1 of request b as float64 [L, HK, D] (zeros below lo: not read by the reference either)."""
        p = torch.arange(self.L[b])
        page = self.table[self.slots_l[b], p // PAGE].long()
        page = torch.where(page < 0, 0, page).to(DEV)
        return pool[page, :, (p % PAGE).to(DEV)].double()

    def append(self, stream=None):
        C.csla_kv_append(self.lb.cfg(), self.lb.cache(), self.slots, self.B, self.start, self.N, self.k_new,
                         self.k_new.stride(0), self.v_new, self.v_new.stride(0), DT[self.q_dtype], self.gamma_k, stream)

    def attend(self, out_dtype=torch.bfloat16, out=None, ws=None, stream=None):
        s = self.shape
        if out is None:
            out = torch.full((self.N, s.HQ, s.D), 7.0, dtype=out_dtype, device=DEV)
        need = C.csla_kv_workspace_size(self.lb.cfg(), self.B, self.N, self.max_new, self.max_len)
        if ws is None:   # what the call leaves unwritten must not matter: NaN everywhere
            ws = torch.full((max(need // 4, 4),), float("nan"), dtype=torch.float32, device=DEV)
        C.csla_kv_attend(self.lb.cfg(), self.lb.cache(), self.slots, self.B, self.start, self.N, self.max_new,
                         self.max_len, self.q, DT[self.q_dtype], self.q.stride(0), self.sink, self.gamma_q, out,
                         DT[out.dtype], ws, need, stream)
        return out

    @property
    def halves(self):
        return self.shape.rope_pairs == C.CSLA_ROPE_HALVES

    def check_attend(self, out, skip=()):
        s = self.shape
        q = self.q.reshape(self.N, s.HQ, s.D)
        for b in range(self.B):
            rows = slice(self.start_l[b], self.start_l[b + 1])
            if b in skip or self.T[b] == 0:
                assert bool((out[rows] == 7.0).all()), b
                continue
            o, tol = attend_request(q[rows], self.rows(b, self.lb.k), self.rows(b, self.lb.v),
                                    self.L[b] - self.T[b], s, self.halves, self.sink, self.gamma_q)
            tol = with_output_step(o, tol, out.dtype)
            err = (out[rows].double() - o).abs()
            assert bool(torch.isfinite(out[rows]).all()), b
            worst = float((err / tol.clamp(min=1e-30)).max())
            assert bool((err <= tol).all()), (b, self.T[b], self.L[b], worst)
        assert bool((out[self.start_l[-1]:] == 7.0).all())   # rows behind the last request

    def expected_append(self):
        """Pools after the append: expected K (float64) with its tolerance, V bits, and which rows are written."""
        s = self.shape
        k, tol = self.lb.k.double(), torch.zeros_like(self.lb.k, dtype=torch.float64)
        v, hit = self.lb.v.clone(), torch.zeros(self.lb.k.shape[:3], dtype=torch.bool, device=DEV)
        for b in range(self.B):
            rows = slice(self.start_l[b], self.start_l[b + 1])
            p = torch.arange(self.L[b] - self.T[b], self.L[b])
            page = self.table[self.slots_l[b], p // PAGE].long().to(DEV)
            at, p = (p % PAGE).to(DEV), p.to(DEV)
            kn = self.k_new[rows].reshape(-1, s.HK, s.D)
            y, t = append_rows(kn, p, s, self.halves, self.gamma_k)
            k[page, :, at], tol[page, :, at] = y, t
            v[page, :, at] = self.v_new[rows].reshape(-1, s.HK, s.D).to(torch.bfloat16)
            hit[page, :, at] = True
        return k, tol, v, hit


def no_device_error():
    rc, bits = C.csla_device_error()
    assert rc == C.CSLA_OK, "device error bits 0x%x" % bits
