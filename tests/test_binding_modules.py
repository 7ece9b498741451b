"""The library does not need the binding's native module: calls that do not use
it load, and the library builds, where the module is missing or does not fit."""
import ctypes

import pytest
import torch

from tensor_gemm_reduction_amd import build, tpfuse as tp


@pytest.fixture
def fresh(monkeypatch):
    """The binding as after an import."""
    monkeypatch.setattr(tp, "_lib", None)
    monkeypatch.setattr(tp, "_args", None)


@pytest.mark.parametrize("content", [None, b"not a library"])
def test_library_loads_without_the_native_module(fresh, monkeypatch, tmp_path, content):
    path = tmp_path / "_args.so"
    if content is not None:
        path.write_bytes(content)
    monkeypatch.setattr(tp, "ARGS_PATH", str(path))
    assert isinstance(tp.load(), ctypes.CDLL)
    assert tp.workspace_size(tp.OP_MATMUL_ALLREDUCE, 2, 8, 8, 8, sched="fold") > 0
    x, w = torch.zeros(4, 64).bfloat16(), torch.zeros(64, 8).bfloat16()
    with pytest.raises(ValueError, match="not on a GPU"):
        tp.matmul_allreduce([x], [w])
    with pytest.raises(RuntimeError, match="_args.so.*build it with"):
        tp.stash_pack([x])


def test_missing_library_is_named(fresh, monkeypatch, tmp_path):
    monkeypatch.setattr(tp, "LIB_PATH", str(tmp_path / "libtpfuse.so"))
    with pytest.raises(RuntimeError, match="libtpfuse.so is missing"):
        tp.load()


def no_headers(out):
    raise ImportError("no torch here")


@pytest.mark.parametrize("command", [lambda out: ["false"], lambda out: ["/nonexistent/compiler"], no_headers])
def test_library_builds_without_the_native_module(monkeypatch, tmp_path, command):
    src, obj = tmp_path / "empty.cpp", tmp_path / "empty.o"
    src.write_text("extern \"C\" int nothing() { return 7; }\n")
    monkeypatch.setattr(build, "LIBDIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "ARGS", str(tmp_path / "_args.so"))
    monkeypatch.setattr(build, "_compile_jobs", lambda cc: [("empty.cpp", str(obj),
                                                             ["g++", "-fPIC", "-c", str(src), "-o", str(obj)])])
    monkeypatch.setattr(build, "_args_command", command)
    with pytest.raises(RuntimeError, match="_args"):
        build.build()
    assert ctypes.CDLL(str(tmp_path / "lib.so")).nothing() == 7
    assert not (tmp_path / "_args.so").exists()


def test_a_source_that_fails_leaves_the_old_library(monkeypatch, tmp_path):
    lib = tmp_path / "lib.so"
    lib.write_bytes(b"old")
    monkeypatch.setattr(build, "LIBDIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "ARGS", str(tmp_path / "_args.so"))
    monkeypatch.setattr(build, "_compile_jobs", lambda cc: [("bad.cpp", str(tmp_path / "bad.o"), ["false"])])
    monkeypatch.setattr(build, "_args_command", lambda out: ["true"])
    with pytest.raises(RuntimeError, match="bad.cpp"):
        build.build()
    assert lib.read_bytes() == b"old"
