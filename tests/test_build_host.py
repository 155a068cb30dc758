"""What build() makes and when it makes it again (no GPU; compilers are not run)."""
import os
import subprocess

import pytest

from w4afp8_mixture_experts_gb300 import build as b


@pytest.fixture
def place(monkeypatch, tmp_path):
    """build() in a folder of its own, with compilers that only create their output; .ran lists the outputs made."""
    class Place:
        ran = []
        torch = (str(tmp_path / "torch"), 1, "2.0")

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        Place.ran.append(os.path.basename(out))
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def library(srcs, out, deps, extra=(), jobs=None):
        os.makedirs(os.path.dirname(out), exist_ok=True)
        if not os.path.exists(out):
            run(["nvcc", "-o", out])
        return out

    Place.ran = []
    Place.headers = tmp_path / "torch" / "include" / "torch" / "csrc" / "autograd"
    Place.headers.mkdir(parents=True)
    (Place.headers / "python_variable.h").write_text("")
    lib = str(tmp_path / "_lib")
    monkeypatch.setattr(b, "LIBDIR", lib)
    monkeypatch.setattr(b, "LIB", os.path.join(lib, "libw4a8moe.so"))
    monkeypatch.setattr(b, "EXT", os.path.join(lib, "w4a8_torch_ops.so"))
    monkeypatch.setattr(b, "_torch_paths", lambda: Place.torch)
    monkeypatch.setattr(b, "build_shared", library)
    monkeypatch.setattr(b, "nvcc_path", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(b.subprocess, "run", run)
    return Place


ALL = ["libw4a8moe.so", "torch_ops.o", "w4a8_torch_ops.so"]


def test_the_extension_is_made_again_for_another_torch(place, tmp_path):
    b.build()
    assert sorted(place.ran) == ALL
    place.ran.clear()
    b.build()
    assert place.ran == []
    place.torch = (place.torch[0], 1, "2.1")  # an upgrade in place
    b.build()
    assert place.ran == ["torch_ops.o", "w4a8_torch_ops.so"]
    place.ran.clear()
    place.torch = (place.torch[0], 0, "2.1")  # another C++ ABI
    b.build()
    assert place.ran == ["torch_ops.o", "w4a8_torch_ops.so"]


def test_the_library_needs_no_torch_headers(place):
    b.build()
    place.ran.clear()
    os.remove(b.LIB)
    os.remove(place.headers / "python_variable.h")
    with pytest.warns(UserWarning, match="headers are missing"):
        assert b.build() == b.LIB
    assert place.ran == ["libw4a8moe.so"]
    assert not os.path.exists(b.EXT)  # of a torch that is no longer there


def test_calls_without_the_extension_raise(place, monkeypatch):
    import w4afp8_mixture_experts_gb300._binding as binding
    monkeypatch.setattr(binding, "EXT", b.EXT)
    monkeypatch.setattr(binding, "_ops", None)
    monkeypatch.setattr(binding, "load", lambda: None)
    with pytest.raises(RuntimeError, match="missing"):
        binding.block_norm(None)
