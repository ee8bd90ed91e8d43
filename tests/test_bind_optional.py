"""The native fast path of the Python binding (_bind.so) is a convenience: the
library loads without it, and one that was built for another torch or Python
is neither used nor kept by a build."""
import os
import shutil
import subprocess
import sys
import warnings

import pytest

import linear_attention_lm_gen_b200 as jet
from linear_attention_lm_gen_b200 import build as jbuild

CODE = """
import warnings
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import linear_attention_lm_gen_b200 as jet
    jet.load_library()
assert jet.__file__.startswith({where!r}), jet.__file__
assert jet._bind is None
assert any("_bind" in str(w.message) and issubclass(w.category, RuntimeWarning) for w in seen), seen
assert jet.jet_gdn_prefill_workspace_size(1, 100, 2, 96, 128) > 0
assert jet.jet_cache_compact_workspace_size(10) > 0
print("loaded")
"""


@pytest.mark.parametrize("broken", ["missing", "garbage", "no module"])
def test_the_library_loads_without_it(tmp_path, broken):
    jbuild.build()
    pkg = tmp_path / "linear_attention_lm_gen_b200"
    shutil.copytree(jbuild.PKG, pkg, ignore=shutil.ignore_patterns("__pycache__", "csrc", "_bind.so", "libjet.so"))
    os.symlink(jbuild.LIB, pkg / "libjet.so")
    if broken == "garbage":
        (pkg / "_bind.so").write_bytes(b"not a shared object")
    elif broken == "no module":                  # a shared object without the module's entry
        os.symlink(jbuild.LIB, pkg / "_bind.so")
    r = subprocess.run([sys.executable, "-c", CODE.format(where=str(tmp_path))], cwd=tmp_path, capture_output=True,
                       text=True, env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0 and "loaded" in r.stdout, r.stderr


def test_one_for_another_torch_or_python_is_not_used(monkeypatch):
    jbuild.build()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert jet._load_bind().abi == jbuild.bind_abi()
    monkeypatch.setattr(jbuild, "bind_abi", lambda: "torch 9.9 cpython-399")
    with pytest.warns(RuntimeWarning, match="_bind"):
        assert jet._load_bind() is None


def test_a_build_replaces_one_for_another_torch_or_python(monkeypatch, tmp_path):
    out = tmp_path / "_bind.so"
    monkeypatch.setattr(jbuild, "BIND", str(out))
    runs = []

    def compiler(cmd, check):
        runs.append(cmd)
        with open(str(out) + ".tmp", "wb") as f:
            f.write(b"x")
    monkeypatch.setattr(jbuild.subprocess, "run", compiler)
    for _ in range(2):
        jbuild.build_bind()
    assert len(runs) == 1                        # up to date the second time
    monkeypatch.setattr(jbuild, "bind_abi", lambda: "torch 9.9 cpython-399")
    for _ in range(2):
        jbuild.build_bind()
    assert len(runs) == 2 and any("torch 9.9 cpython-399" in x for x in runs[1])


@pytest.mark.gpu
def test_calls_without_it_are_the_same(monkeypatch):
    import torch
    from test_gpu_attn_binding import Case
    jbuild.build()
    jet.load_library()
    assert jet._bind is not None
    c = Case(jet)

    def calls():
        pool = torch.arange(80, device="cuda", dtype=torch.float32).view(10, 8)
        jet.jet_cache_copy([pool], [1, 1], [5, 6])
        out, live, ws = torch.empty_like(c.b.table), torch.empty(1, device="cuda", dtype=torch.int32), torch.empty(
            jet.jet_cache_compact_workspace_size(10), device="cuda", dtype=torch.uint8)
        table = torch.tensor([[9, 2, -1], [7, 2, 0]], device="cuda", dtype=torch.int32)
        out = torch.empty_like(table)
        jet.jet_cache_compact([pool], table, torch.tensor([20, 33], device="cuda", dtype=torch.int32), 16, out, live, ws)
        return [c.append().clone(), c.paged().clone(), pool, out, live]
    native = calls()
    monkeypatch.setattr(jet, "_bind", None)
    for a, b in zip(native, calls()):
        assert torch.equal(a, b)
    with pytest.raises(jet.JetError):
        c.paged(window=-1)
    assert jet.jet_device_error() == 0
