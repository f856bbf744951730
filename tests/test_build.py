"""Building: the library needs nvcc alone, the native binding is built beside it where it can be."""
import os
import shutil

import pytest

from nvfp4_quantized_moe_topk_gb300 import build as B


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of one small translation unit in a folder of its own."""
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libmoe_nvfp4.so"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "moe_binding.so"))
    monkeypatch.setattr(B, "sources", lambda: [os.path.join(B.CSRC, "combine.cu")])
    return tmp_path


@pytest.mark.parametrize("why", ["no torch", "no compiler", "the compiler fails"])
def test_the_library_is_built_where_the_binding_cannot_be(elsewhere, monkeypatch, why):
    (elsewhere / "moe_binding.so").write_text("of an earlier build")
    os.utime(elsewhere / "moe_binding.so", (1, 1))

    def fail(*_):
        if why == "no compiler":
            raise FileNotFoundError("g++")
        raise RuntimeError(why)

    monkeypatch.setattr(B, "_torch_dir" if why == "no torch" else "_compile_binding", fail)
    with pytest.warns(UserWarning, match="binding|operators around the layer"):
        assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)
    # the library is not compiled again, the binding is tried again
    before = os.path.getmtime(B.LIB)
    with pytest.warns(UserWarning):
        B.build()
    assert os.path.getmtime(B.LIB) == before and not B.up_to_date()


def test_a_failing_library_is_an_error(elsewhere, monkeypatch):
    monkeypatch.setattr(B, "FLAGS", [*B.FLAGS, "--no-such-flag"])
    monkeypatch.setattr(B, "_compile_binding", lambda: "")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        B.build()
    assert not os.path.exists(B.LIB)


def test_torch_missing_says_so(monkeypatch):
    import importlib.util

    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None)
    with pytest.raises(RuntimeError, match="torch is not installed"):
        B._torch_dir()
