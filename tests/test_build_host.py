"""What a build leaves behind where the extension for PyTorch cannot be made.  No GPU; nvcc on a file of one line."""
import os
import sys

import pytest

from depthwise_convolution_gb300 import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    for name in ("LIB", "OPS"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "_sources", lambda: [str(src)])
    return tmp_path


def test_without_pytorch_the_c_library_is_built_alone(small, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    assert build.needs_build()
    build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.OPS)
    assert not build.needs_build()


def test_an_extension_that_does_not_compile_leaves_nothing(small, monkeypatch):
    monkeypatch.setattr(build, "_compile_ops", lambda: ("torch_ops.cpp", [], 1, "no such header"))
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert not os.path.exists(build.LIB) and not os.path.exists(build.OPS)
