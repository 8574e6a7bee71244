"""What the binding of the dense layer's calls accepts and refuses, without a GPU: on host tensors a call that is right in all but
the device is refused for the device, and for nothing else."""
import pytest
import torch

from compressed_sparse_long_append_b200 import csla as C
from compressed_sparse_long_append_b200.layer import DenseShape

N, B, HQ, HK, D = 6, 2, 4, 2, 64
F32, BF = torch.float32, torch.bfloat16
CFG = DenseShape(D=D, HQ=HQ, HK=HK).cfg()
KV = C.csla_kv_cache(1 << 40, 1 << 40, 1 << 40, 1 << 40, 8, 16, 4)
ADDR = 1 << 40


def _append(**kw):
    a = dict(slots=ADDR, B=B, q_start=ADDR, N=N, k=ADDR, ks=HK * D, v=ADDR, vs=HK * D, dt=C.CSLA_BF16, gamma=None)
    a.update(kw)
    return C.csla_kv_append(CFG, KV, a["slots"], a["B"], a["q_start"], a["N"], a["k"], a["ks"], a["v"], a["vs"], a["dt"],
                            a["gamma"], stream=1)


def _attend(**kw):
    a = dict(slots=ADDR, q_start=ADDR, q=ADDR, qs=HQ * D, sink=None, gamma=None, out=ADDR, odt=C.CSLA_BF16, ws=ADDR, wsb=1 << 30)
    a.update(kw)
    return C.csla_kv_attend(CFG, KV, a["slots"], B, a["q_start"], N, 4, 100, a["q"], C.CSLA_BF16, a["qs"], a["sink"], a["gamma"],
                            a["out"], a["odt"], a["ws"], a["wsb"], stream=1)


def _rows(heads, dtype=BF, n=N):
    return torch.zeros((n, heads, D), dtype=dtype)


FUSED = torch.zeros((N, (HQ + 2 * HK) * D), dtype=BF)
WIDE = FUSED.shape[1]


@pytest.mark.parametrize("call,kw", [
    (_attend, dict(q=_rows(HQ))), (_attend, dict(q=_rows(HQ).view(N, HQ * D))), (_attend, dict(q=_rows(HQ).view(2, 3, HQ, D))),
    (_attend, dict(q=FUSED[:, :HQ * D], qs=WIDE)), (_attend, dict(q=FUSED, qs=WIDE)),
    (_attend, dict(q=FUSED[:, :HQ * D].view(N, HQ, D), qs=WIDE)), (_attend, dict(q=FUSED.view(2, 3, WIDE)[:, :, :HQ * D], qs=WIDE)),
    (_attend, dict(q=_rows(HQ, n=2 * N)[::2], qs=2 * HQ * D)), (_attend, dict(q=_rows(HQ, n=N + 3))),
    (_attend, dict(q=torch.zeros(N * HQ * D, dtype=BF))),
    (_attend, dict(out=_rows(HQ))), (_attend, dict(out=_rows(HQ, F32), odt=C.CSLA_F32)), (_attend, dict(out=_rows(HQ, n=N + 1))),
    (_attend, dict(sink=torch.zeros(HQ))), (_attend, dict(gamma=torch.zeros(D))),
    (_attend, dict(slots=torch.zeros(B, dtype=torch.int32))), (_attend, dict(q_start=torch.zeros(B + 1, dtype=torch.int32))),
    (_append, dict(k=_rows(HK))), (_append, dict(v=FUSED[:, -HK * D:], vs=WIDE)), (_append, dict(gamma=torch.zeros(D))),
    (_append, dict(k=_rows(HK, F32), v=_rows(HK, F32), dt=C.CSLA_F32)),
    (_append, dict(slots=torch.zeros(B, dtype=torch.int32))), (_append, dict(q_start=torch.zeros(B + 1, dtype=torch.int32)))])
def test_right_but_for_the_device(call, kw):
    with pytest.raises(ValueError, match="is on cpu, not on the current device"):
        call(**kw)


@pytest.mark.parametrize("call,kw", [
    (_attend, dict(q=_rows(HQ, F32))), (_append, dict(k=_rows(HK, F32))), (_append, dict(v=_rows(HK, torch.float16))),
    (_attend, dict(q=torch.zeros((N, D, HQ), dtype=BF).transpose(1, 2))),        # dims outside heads
    (_attend, dict(q=torch.zeros((HQ, N, D), dtype=BF).transpose(0, 1), qs=D)),  # heads outside tokens
    (_attend, dict(q=torch.zeros((N, HQ, 2 * D), dtype=BF)[:, :, :D], qs=2 * HQ * D)),   # heads with gaps
    (_attend, dict(q=torch.zeros((N, HQ, 2 * D), dtype=BF)[:, :, ::2], qs=2 * HQ * D)),  # dims with gaps
    (_attend, dict(q=FUSED[:, :HQ * D], qs=HQ * D)), (_attend, dict(q=_rows(HQ, n=2 * N)[::2])),   # not the stride given
    (_attend, dict(q=_rows(HQ, n=N - 1))), (_attend, dict(q=FUSED[:-1, :HQ * D], qs=WIDE)),        # too few rows
    (_attend, dict(q=FUSED[:, :HQ * D - 64], qs=WIDE)),                                          # too few heads
    (_append, dict(k=_rows(HK, n=N - 1))), (_append, dict(v=torch.zeros((N, D, HK), dtype=BF).transpose(1, 2))),
    (_attend, dict(out=_rows(HQ, F32))), (_attend, dict(out=_rows(HQ, n=N - 1))), (_attend, dict(out=FUSED[:, :HQ * D])),
    (_attend, dict(sink=torch.zeros(HQ, dtype=BF))), (_attend, dict(sink=torch.zeros(HQ - 1))),
    (_attend, dict(sink=torch.zeros(2 * HQ)[::2])), (_attend, dict(gamma=torch.zeros(D, dtype=BF))),
    (_attend, dict(gamma=torch.zeros(D - 1))), (_append, dict(gamma=torch.zeros(D, dtype=BF))),
    (_append, dict(gamma=torch.zeros(D, dtype=torch.float64))),
    (_attend, dict(slots=torch.zeros(B, dtype=torch.int64))), (_attend, dict(slots=torch.zeros(B - 1, dtype=torch.int32))),
    (_attend, dict(slots=torch.zeros(2 * B, dtype=torch.int32)[::2])),
    (_attend, dict(q_start=torch.zeros(B, dtype=torch.int32).cumsum(0))), (_attend, dict(q_start=torch.zeros(B, dtype=torch.int32))),
    (_append, dict(slots=torch.zeros(B, dtype=torch.int64))), (_append, dict(q_start=torch.zeros(B + 1, dtype=torch.int64))),
    (_append, dict(q_start=torch.zeros(B, dtype=torch.int32)))])
def test_refused_for_type_or_layout(call, kw):
    with pytest.raises(ValueError) as e:
        call(**kw)
    assert "current device" not in str(e.value)


def test_workspaces():
    for ws in (torch.zeros(63, dtype=torch.uint8), torch.zeros((8, 16), dtype=torch.uint8)[:, :8], torch.zeros(16)):
        with pytest.raises(ValueError, match="fewer than 64 bytes"):
            _attend(ws=ws, wsb=64)   # too small, with gaps, on the host


def test_addresses_and_missing_structs_go_to_the_library():
    with pytest.raises(C.CslaError):
        _append(k=ADDR + 2)
    with pytest.raises(C.CslaError):
        C.csla_kv_append(None, KV, ADDR, B, ADDR, N, ADDR, HK * D, ADDR, HK * D, C.CSLA_BF16, None, 1)
    with pytest.raises(C.CslaError):
        _append(dt=7)


def test_the_stream_without_torchs_private_names(monkeypatch):
    class Stream:
        cuda_stream = 123

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    assert C._stream(None) == 123
    assert C._stream(7) == 7 and C._stream(Stream) == 123
    C._kv_here()
    assert C._kv_stream(None, 0) == 123 and C._kv_stream(7, 0) == 7
    monkeypatch.delattr(torch._C, "_cuda_getDevice")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert C._kv_here() == 3 and C._kv_stream(None, 3) == 123 and C._stream(None) == 123
