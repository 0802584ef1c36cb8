"""The library and the Python module over some of its calls are built apart (CPU only): a module that
cannot be built costs its own calls alone, and one built for another torch is not loaded."""
import os
import subprocess
import sys

import pytest

from mixture_experts_forward_moe_gb300 import build

BROKEN_MODULE = """
import os, sys, tempfile
from mixture_experts_forward_moe_gb300 import build
build.build()
build.CALLS = os.path.join(tempfile.mkdtemp(), "gb300moe_calls.so")  # not there
def broken(nvcc):
    raise RuntimeError("no host compiler")
build._compile_calls = broken
def unwanted(*a):
    raise AssertionError("the library is built again")
build._compile = unwanted
from mixture_experts_forward_moe_gb300 import binding as B
assert B.workspace_size(B.make_problem(8, 64, 8, 64, 2)) > 0
import torch
x = torch.zeros(2, 16, dtype=torch.bfloat16)
try:
    B.moe_linear(x, x)
except RuntimeError as e:
    assert "no host compiler" in str(e), e
else:
    raise AssertionError("moe_linear without its module")
print("fine")
"""


def test_a_module_that_cannot_be_built_costs_its_own_calls_alone():
    r = subprocess.run([sys.executable, "-c", BROKEN_MODULE], cwd=build.ROOT, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]


def test_a_module_for_another_torch_is_built_again(tmp_path, monkeypatch):
    import torch
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "gb300moe_calls.so"))
    assert not build.calls_up_to_date()
    with open(build.CALLS, "w"):
        pass
    assert not build.calls_up_to_date()  # not known what for
    with open(build.CALLS + ".built_for", "w") as f:
        f.write(build._calls_built_for())
    assert build.calls_up_to_date()
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert not build.calls_up_to_date()


def test_a_source_newer_than_its_target_is_built_again(tmp_path, monkeypatch):
    for name, fresh in (("LIB", build.library_up_to_date), ("CALLS", build.calls_up_to_date)):
        target = str(tmp_path / name)
        monkeypatch.setattr(build, name, target)
        for path, text in ((target, ""), (target + ".built_for", build._calls_built_for())):
            with open(path, "w") as f:
                f.write(text)
        assert fresh()
        os.utime(target, (1, 1))
        assert not fresh()


def test_the_library_is_in_place_before_the_module_fails(monkeypatch):
    done = []
    monkeypatch.setattr(build, "up_to_date", lambda: False)
    monkeypatch.setattr(build, "calls_up_to_date", lambda: False)
    monkeypatch.setattr(build, "build_library", lambda *a: done.append("library"))

    def broken(nvcc):
        raise RuntimeError("no host compiler")

    monkeypatch.setattr(build, "_compile_calls", broken)
    with pytest.raises(RuntimeError, match="no host compiler"):
        build.build()
    assert done == ["library"]
