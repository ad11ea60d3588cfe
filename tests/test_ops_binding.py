"""The binding of the operators around the attention, without a GPU."""
import importlib.util
import os
import subprocess
import sys
import sysconfig
import types

import pytest

import exact_io_aware_26_gb300 as fa
from exact_io_aware_26_gb300 import _builder, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_call_whose_plan_was_dropped_is_made_all_the_same(monkeypatch):
    """Another thread may register the plan that empties the table, or change the library,
    between a call's registration and its run: the call is registered again, never lost."""
    made = []

    class Dropping:
        def run(self, op, tensors, scalars):
            if len(made) < 3:
                return None
            return ("done",)

        def register(self, *a):
            made.append(a)

    monkeypatch.setattr(ops, "_launch", Dropping())
    device = types.SimpleNamespace(index=0)
    monkeypatch.setattr(ops, "load", lambda: types.SimpleNamespace(fa_kv4_append=ops.ctypes.CFUNCTYPE(None)(lambda: None)))
    got = ops._call(ops._APPEND, (None,), (), None, lambda *a: (device, [], [], [], None))
    assert got == ("done",) and len(made) == 3


@pytest.mark.parametrize("make", [
    lambda n: fa.FaPlanParams(4, n, 16, 10, 4, 4), lambda n: fa.FaPlanParams(4, 4, n, 10, 4, 4),
    lambda n: fa.FaPlanParams(R=4, T=4, page_size=16, num_pages=n, table_width=4, table_stride=4),
    lambda n: fa.FaKv4AttnParams(R=2, T=2, Hq=4, dtype=fa.FA_BF16, max_q_len=1, window=n, table_width=5, scale=0.1, table_stride=5),
    lambda n: fa.FaKv4AttnParams(2, 2, 4, fa.FA_BF16, n), lambda n: fa.FaKv4Cache(n, 64, 2, 64, 10240),
    lambda n: fa.FaKv4Rows(n, fa.FA_BF16), lambda n: fa.FaQkParams(B=1, N=n, Hq=1, Hk=1, d=64),
])
def test_numbers_that_a_c_int_does_not_hold_are_refused(make):
    """They would be cut to their low 32 bits, and the call made with another number."""
    make(2 ** 31 - 1)
    for n in (2 ** 31, 2 ** 32 + 1, 2 ** 32 + 16, -2 ** 31 - 1):
        with pytest.raises(ValueError, match=str(n)):
            make(n)


@pytest.mark.parametrize("absent", [["exact_io_aware_26_gb300._launch"], ["exact_io_aware_26_gb300._launch", "torch"]])
def test_the_attention_needs_the_library_alone(absent):
    """Neither the extension of the operators nor torch is needed to load libfa.so and to call
    a function that takes no tensor."""
    fa.build()
    code = f"""
import sys
sys.modules.update(dict.fromkeys({absent!r}))  # importing one of them raises ImportError
import exact_io_aware_26_gb300 as fa
fa.load()
p = fa.FaParams(B=1, H=1, N=128, d=64, dtype=fa.FA_BF16, scale=0.125)
assert fa.check_params(p) == fa.FA_OK
fa.use_library(fa.use_library(fa.LIB_PATH))
assert fa.load().fa_kv4_block_bytes(64) == 1280
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_an_operator_without_the_extension_says_what_to_do():
    code = """
import sys
sys.modules["exact_io_aware_26_gb300._launch"] = None
import torch
import exact_io_aware_26_gb300 as fa
i = torch.zeros(2, dtype=torch.int32)
try:
    fa.paged_plan(i, i, i[None], i, i, 16, 2)
except ImportError as e:
    assert "build()" in str(e)
else:
    raise SystemExit("no error")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_the_extension_is_built_again_for_another_python_or_torch(tmp_path, monkeypatch):
    """Its file is newer than its source, but it was linked against other libraries."""
    import torch
    torch_spec = importlib.util.find_spec("torch")
    monkeypatch.setattr(_builder, "LAUNCH", str(tmp_path / "_launch.so"))
    monkeypatch.setattr(_builder, "BUILD", str(tmp_path))
    built = []

    def run(cmd, **kw):
        built.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(_builder.subprocess, "run", run)
    _builder.build_launch()
    _builder.build_launch()
    assert len(built) == 1
    config_var = sysconfig.get_config_var
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda n: "cpython-399-none" if n == "SOABI" else config_var(n))
        _builder.build_launch()
        _builder.build_launch()
    assert len(built) == 2
    _builder.build_launch()
    assert len(built) == 3
    # a torch package with the files of this one, of another version
    other = tmp_path / "torch"
    other.mkdir()
    (other / "version.py").write_text("__version__ = '99.0'\n")
    spec = types.SimpleNamespace(submodule_search_locations=[str(other)], origin=str(other / "__init__.py"))
    with monkeypatch.context() as m:
        m.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else torch_spec)
        _builder.build_launch()
    assert len(built) == 4


def test_the_library_is_in_place_when_the_extension_fails(tmp_path, monkeypatch):
    """A compiler or a torch that the extension cannot be built with costs its operators only."""
    monkeypatch.setattr(_builder, "LIB", str(tmp_path / "libfa.so"))
    monkeypatch.setattr(_builder, "BUILD", str(tmp_path))
    monkeypatch.setattr(_builder, "_compile", lambda src, extra, build_dir: src)
    monkeypatch.setattr(_builder.subprocess, "run",
                        lambda cmd, **kw: (open(cmd[cmd.index("-o") + 1], "w").close(), subprocess.CompletedProcess(cmd, 0, "", ""))[1])

    def fails(force=False):
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(_builder, "build_launch", fails)
    with pytest.raises(RuntimeError, match=r"g\+\+ failed"):
        _builder.build(force=True)
    assert os.path.exists(tmp_path / "libfa.so")
