"""The C library needs neither torch nor the binding's native checks: it is linked before them, and its calls work without them."""
import os
import subprocess
import sys
import types

import pytest

import speculative_verify_attention_gb300 as package
from speculative_verify_attention_gb300 import binding
from speculative_verify_attention_gb300 import build as parts


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Compilers that write empty files, in a folder of their own; `fail` names what does not compile."""
    for name in ("LIB_PATH", "CALLS_PATH"):
        monkeypatch.setattr(parts, name, str(tmp_path / os.path.basename(getattr(parts, name))))
    monkeypatch.setattr(parts, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(parts, "_nvcc", lambda: "nvcc")
    seen = types.SimpleNamespace(fail=None, made=[])

    def run(cmd, **kwargs):
        out = cmd[cmd.index("-o") + 1]
        bad = seen.fail and any(str(a).endswith(seen.fail) for a in cmd)
        if not bad:
            open(out, "w").close()
            seen.made.append(out)
        return subprocess.CompletedProcess(cmd, 1 if bad else 0, "", "no such header" if bad else "")

    monkeypatch.setattr(parts.subprocess, "run", run)
    return seen


def test_the_c_library_is_there_when_the_checks_do_not_compile(compilers):
    compilers.fail = "calls.cpp"
    with pytest.raises(RuntimeError, match="calls.cpp"):
        parts.build(force=True)
    assert os.path.exists(parts.LIB_PATH) and not os.path.exists(parts.CALLS_PATH)
    compilers.fail = None
    assert parts.needs_build() and parts.build() == parts.LIB_PATH and os.path.exists(parts.CALLS_PATH)
    assert not parts.needs_build()


def test_without_torch_the_c_library_is_all_that_is_built(compilers, monkeypatch):
    find = parts.importlib.util.find_spec
    monkeypatch.setattr(parts.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert parts.build(force=True) == parts.LIB_PATH and os.path.exists(parts.LIB_PATH)
    assert not any("calls" in os.path.basename(made) for made in compilers.made)
    assert not parts.needs_build()


def test_the_library_loads_without_the_checks(monkeypatch):
    parts.build()
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_calls", None)
    monkeypatch.delattr(package, "_calls", raising=False)
    monkeypatch.setitem(sys.modules, package.__name__ + "._calls", None)     # its import fails
    assert binding.load_library().kvq8_status_str(0) == b"ok"
    assert binding.beam_select_workspace_bytes(4, 1000, 2, 5) > 0
    with pytest.raises(ImportError):
        binding._native()
    monkeypatch.setattr(parts, "CALLS_PATH", parts.CALLS_PATH + ".none")
    with pytest.raises(RuntimeError, match="is missing"):
        binding._native()
