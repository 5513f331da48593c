"""The extension behind the 8-bit operators' Python calls is theirs alone: without it
the library builds, loads and makes handles, and those calls say what is missing."""
import os
import sys

import pytest
import torch

from dense_gemm_tmem_gb300 import binding as B
from dense_gemm_tmem_gb300 import build
from dense_gemm_tmem_gb300.gemm import Gemm


@pytest.fixture
def no_compiler(monkeypatch, tmp_path):
    """No extension has been built, and the host compiler is missing."""
    B.load()
    monkeypatch.setattr(build, "NATIVE", str(tmp_path / "_dgemm_native.so"))
    monkeypatch.setattr(B, "_native", None)
    monkeypatch.setenv("CXX", str(tmp_path / "no-such-compiler"))


def test_the_library_does_not_need_the_extension(no_compiler):
    with pytest.warns(UserWarning, match="8-bit"):
        assert build.build() == build.LIB
    assert B.load(build_if_missing=False) is not None
    with pytest.raises((OSError, RuntimeError)):
        B.native()


def test_a_handle_does_not_need_the_extension(no_compiler, monkeypatch):
    monkeypatch.setattr(B, "gemm_create", lambda device: 1)
    monkeypatch.setattr(B, "gemm_destroy", lambda handle: 0)
    g = Gemm(torch.device("cuda", 0))
    with pytest.raises((OSError, RuntimeError)):
        g.fp8_quantize(torch.zeros(1, 1))
    g.handle = None


def test_one_extension_for_each_python_and_torch():
    name = os.path.basename(build.NATIVE)
    assert sys.implementation.cache_tag in name and torch.__version__ in name
    assert os.path.exists(build.NATIVE) or not build.native_up_to_date()
