"""CPU-only: what the build makes where the host compiler or PyTorch is missing, and when it builds again.
The library's sources stand in as one small file."""
import os
import sys

import pytest

from learned_relative_gqa_b200 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "one.cu").write_text("extern \"C\" int one() { return 1; }\n")
    (csrc / "serving_ext.cpp").write_text("int module() { return 1; }\n")
    for name, value in dict(ROOT=tmp_path, CSRC=csrc, INCLUDE=csrc, LIB_PATH=tmp_path / "lib.so",
                            EXT_SOURCE=csrc / "serving_ext.cpp", EXT_PATH=tmp_path / "_serving.so").items():
        monkeypatch.setattr(B, name, str(value))
    monkeypatch.setattr(B, "SOURCES", ["one.cu"])
    return tmp_path


def test_library_is_built_without_pytorch(tree, monkeypatch, capfd):
    """The C ABI needs nvcc alone: without PyTorch the module is left out, with a word, and nothing is due again."""
    monkeypatch.setitem(sys.modules, "torch", None)
    assert B.build(out_path=B.LIB_PATH) == B.LIB_PATH
    assert os.path.exists(B.LIB_PATH) and not os.path.exists(B.EXT_PATH)
    assert "_serving.so" in capfd.readouterr().err
    t = os.path.getmtime(B.LIB_PATH)
    B.build(out_path=B.LIB_PATH)
    assert os.path.getmtime(B.LIB_PATH) == t


def test_library_is_built_without_a_host_compiler_for_the_module(tree, monkeypatch, capfd):
    which = B.shutil.which
    monkeypatch.setattr(B.shutil, "which", lambda name, *a, **k: None if name == "g++" else which(name, *a, **k))
    B.build(out_path=B.LIB_PATH)
    assert os.path.exists(B.LIB_PATH) and not os.path.exists(B.EXT_PATH)
    assert "g++" in capfd.readouterr().err


def test_a_module_that_does_not_compile_leaves_the_library_built(tree, capfd):
    with open(B.EXT_SOURCE, "w") as f:
        f.write("this is no source\n")
    with open(B.EXT_PATH, "w") as f:
        f.write("an older module, which may not fit the new library")
    os.utime(B.EXT_PATH, (0, 0))
    with pytest.raises(RuntimeError, match="serving_ext.cpp"):
        B.build(out_path=B.LIB_PATH)
    assert os.path.exists(B.LIB_PATH) and not os.path.exists(B.EXT_PATH)


def test_a_source_that_does_not_compile_is_named(tree, capfd):
    with open(os.path.join(B.CSRC, "one.cu"), "w") as f:
        f.write("this is no source\n")
    with pytest.raises(RuntimeError, match="one.cu"):
        B.build(out_path=B.LIB_PATH)
    assert not os.path.exists(B.LIB_PATH) and not os.path.exists(B.EXT_PATH)


def test_module_is_due_again_for_another_pytorch(tree, monkeypatch, capfd):
    """A module built against another PyTorch or interpreter is built again, and the library is not."""
    import torch
    with open(B.EXT_SOURCE, "w") as f:
        f.write('extern "C" const char* const built_for;\nconst char* const built_for = "serving module for " INKLING_BUILT_FOR;\n')
    B.build(out_path=B.LIB_PATH)
    lib, ext = os.path.getmtime(B.LIB_PATH), os.path.getmtime(B.EXT_PATH)
    B.build(out_path=B.LIB_PATH)
    assert os.path.getmtime(B.EXT_PATH) == ext
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert B.ext_stale()
    B.build(out_path=B.LIB_PATH)
    assert not B.ext_stale()
    assert os.path.getmtime(B.EXT_PATH) > ext and os.path.getmtime(B.LIB_PATH) == lib


def test_module_of_another_pytorch_is_not_used(monkeypatch):
    """The calls say so, rather than run against tensors of another layout."""
    from learned_relative_gqa_b200 import binding
    B.build()
    binding._serving()
    monkeypatch.setattr(binding, "_bound", None)
    monkeypatch.setattr(binding._ext, "built_for", "another", raising=True)
    with pytest.raises(RuntimeError, match="another"):
        binding._serving()
