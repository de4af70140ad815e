"""What the Python package needs to be imported, built and used: a torch without CUDA, a
machine without the Python headers, a binding without its compiled part (no compute call
runs here)."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

import two_tier_sparse_gb300 as dsa
from two_tier_sparse_gb300 import build as dsa_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dsa_build.build()
    dsa.load()


def host_calls_are_refused():
    """Host tensors to every call that the compiled part takes: the binding's own answer."""
    i = dict(dtype=torch.int32)
    x, slots = torch.zeros((2, 512), dtype=torch.bfloat16), torch.zeros(2, **i)
    cache, ws = torch.zeros((4, 512), dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    pool, plan = dsa.PagePool.empty(2, 64, 2, 4, device="cpu"), dsa.StepPlan.empty(2, 2, device="cpu")
    cfg = dsa.config()
    for call in (lambda: dsa.norm_rope(None, dsa.HeadSet([dsa.Heads(x)])),
                 lambda: dsa.kv_write(cfg, x, slots, cache, ws),
                 lambda: dsa.kv_read(cfg, cache, slots, x, ws),
                 lambda: dsa.plan_step(cfg, slots, slots, pool, plan, ws)):
        with pytest.raises(ValueError, match="not the current CUDA device"):
            call()


def test_the_package_works_with_a_torch_without_cuda():
    """A torch built without CUDA lacks these functions; the package imports, and its host side
    (configurations, workspace sizes, handles, refusals) works."""
    code = textwrap.dedent("""
        import torch
        for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
            if hasattr(torch._C, name):
                delattr(torch._C, name)
        import two_tier_sparse_gb300 as dsa
        assert dsa.workspace_size(dsa.config(), 4, 4096) > 0
        from test_binding_parts import host_calls_are_refused
        host_calls_are_refused()
        print("fine")
    """)
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    p = subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True, text=True)
    assert p.returncode == 0 and p.stdout.strip() == "fine", p.stderr[-2000:]


def test_a_missing_compiled_part_leaves_the_calls_to_the_binding(monkeypatch, tmp_path):
    """The four calls are complete without it: they reach their own checks (and the library)."""
    monkeypatch.setattr(dsa, "_calls", None)
    monkeypatch.setattr(dsa, "LIB_PATH", str(tmp_path / "libdsa.so"))  # (loaded already)
    host_calls_are_refused()


@pytest.mark.parametrize("missing", ["headers", "compiler"])
def test_the_library_builds_without_what_the_compiled_part_needs(monkeypatch, tmp_path, missing, capsys):
    """No Python headers, or no C compiler: the library is built all the same, the compiled part
    is left out (said on stderr), and one that no longer fits its source does not stay."""
    if missing == "headers":
        monkeypatch.setattr(dsa_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    else:
        monkeypatch.setenv("PATH", str(tmp_path))
    old = tmp_path / "old.so"
    old.write_bytes(b"old")
    os.utime(old, (0, 0))
    monkeypatch.setattr(dsa_build, "CALLS", str(old))
    assert dsa_build.build() == dsa_build.LIB
    assert not old.exists()
    assert "calls.c" in capsys.readouterr().err
    dsa_build.build()  # and again, with none there


def test_the_compiled_part_is_of_this_interpreter(monkeypatch, tmp_path):
    """Its file name holds the interpreter's tag, so one that another Python built is not loaded."""
    import importlib.machinery
    if dsa_build.build_calls() is None:
        pytest.skip("no Python headers here")
    tag = importlib.machinery.EXTENSION_SUFFIXES[0]
    assert "cpython" in tag and os.path.basename(dsa_build.CALLS) == "_calls" + tag
    assert os.path.exists(dsa_build.CALLS)
    for name in ("_calls.so", "_calls.cpython-300-riscv64-linux-gnu.so"):
        (tmp_path / name).write_bytes(b"another interpreter's")
    monkeypatch.setattr(dsa, "_calls", None)
    monkeypatch.setattr(dsa, "LIB_PATH", str(tmp_path / "libdsa.so"))
    host_calls_are_refused()
