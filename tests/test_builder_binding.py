"""Where the Python binding of the 8-bit row operators cannot be built, the library is built all the same: a torch without CUDA,
a Python without its headers, no torch. Runs without a GPU."""
import importlib.machinery
import os
import sysconfig

import pytest

from weight_only_quantized_wq4_gb300 import builder


def torch_at(monkeypatch, root, files):
    """importlib finds torch at `root`, whose lib/ holds `files`."""
    os.makedirs(os.path.join(root, "lib"))
    os.makedirs(os.path.join(root, "include"))
    for f in files:
        open(os.path.join(root, "lib", f), "w").close()
    open(os.path.join(root, "version.py"), "w").close()
    spec = importlib.machinery.ModuleSpec("torch", None, is_package=True)
    spec.submodule_search_locations = [str(root)]
    monkeypatch.setattr(builder.importlib.util, "find_spec", lambda name: spec if name == "torch" else None)


CPU_LIBS = ["libtorch_python.so", "libtorch_cpu.so", "libc10.so"]


def built(monkeypatch, tmp_path):
    """What _build_binding runs, with a compiler that only takes note."""
    ran = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done
    monkeypatch.setattr(builder.subprocess, "run", run)
    monkeypatch.setattr(builder, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setattr(builder, "BUILD", str(tmp_path / "build"))
    builder._build_binding(builder._binding_stamp())
    return ran


def test_torch_without_cuda(monkeypatch, tmp_path):
    torch_at(monkeypatch, tmp_path / "torch", CPU_LIBS)
    assert builder._binding_command() is None
    assert built(monkeypatch, tmp_path) == []


def test_torch_with_cuda(monkeypatch, tmp_path):
    torch_at(monkeypatch, tmp_path / "torch", CPU_LIBS + ["libc10_cuda.so"])
    ran = built(monkeypatch, tmp_path)
    assert len(ran) == 1 and "-lc10_cuda" in ran[0] and os.path.exists(tmp_path / "binding.so")


def test_python_without_headers(monkeypatch, tmp_path):
    torch_at(monkeypatch, tmp_path / "torch", CPU_LIBS + ["libc10_cuda.so"])
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a: {"include": str(tmp_path / "nowhere")})
    assert builder._binding_command() is None
    assert built(monkeypatch, tmp_path) == []


def test_no_torch(monkeypatch, tmp_path):
    monkeypatch.setattr(builder.importlib.util, "find_spec", lambda name: None)
    assert builder._binding_command() is None
    assert built(monkeypatch, tmp_path) == []


def test_a_failing_compiler_is_reported(monkeypatch, tmp_path):
    torch_at(monkeypatch, tmp_path / "torch", CPU_LIBS + ["libc10_cuda.so"])

    class Failed:
        returncode, stdout, stderr = 1, "", "wrong"
    monkeypatch.setattr(builder.subprocess, "run", lambda cmd, **kw: Failed)
    monkeypatch.setattr(builder, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(builder, "BINDING", str(tmp_path / "binding.so"))
    with pytest.raises(RuntimeError, match="wrong"):
        builder._build_binding("stamp")
