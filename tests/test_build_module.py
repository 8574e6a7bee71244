"""The build module's arguments, without compiling."""
import importlib.util
import os

from conftest import ROOT


def test_build_takes_its_arguments(monkeypatch, capsys):
    spec = importlib.util.spec_from_file_location("csla_build", os.path.join(ROOT, "compressed_sparse_long_append_b200", "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    ran = []
    monkeypatch.setattr(m.subprocess, "run", lambda cmd, check: ran.append(cmd))
    monkeypatch.setattr(m.os, "replace", lambda a, b: None)
    assert m.build(True, False, ["-Xptxas", "-v"]) == m.LIB
    assert len(ran) == len(m.sources()) + 1 and capsys.readouterr().out == ""
    assert all(("-Xptxas" in c) == ("-c" in c) for c in ran)
    # whole programs: the units that move registers between their warps
    alone = [c for c in ran if "-DCSLA_UNIT_ALONE" in c]
    assert [os.path.basename(c[-1]) for c in alone] == sorted(m.ALONE) and all("-rdc=true" not in c for c in alone)
    assert m.build(force=True, verbose=True) == m.LIB
    assert capsys.readouterr().out.count(m.NVCC) == len(m.sources()) + 1
    monkeypatch.setattr(m, "_stale", lambda: False)
    del ran[:]
    assert m.build(verbose=True) == m.LIB and not ran
