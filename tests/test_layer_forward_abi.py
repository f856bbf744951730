"""The whole-layer call without a GPU: the argument struct's layout and the refusals of a missing handle."""
import os
import shutil
import subprocess

import pytest

from nvfp4_quantized_moe_topk_gb300 import api
from nvfp4_quantized_moe_topk_gb300 import build as B


def test_struct_layout_matches_the_header(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_nvfp4.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu", sizeof(moe_layer_args), offsetof(moe_layer_args, router_dtype),'
                   ' offsetof(moe_layer_args, x), offsetof(moe_layer_args, logits));\nreturn 0; }\n')
    exe = tmp_path / "layout"
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([gcc, "-std=c99", f"-I{inc}", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [80, 8, 16, 72]


def test_no_handle_is_refused():
    B.build()
    lib = api.load()
    assert lib.moe_nvfp4_layer_forward(None, None, None) == 1
    assert lib.moe_nvfp4_layer_forward(None, b"\0" * 80, None) == 1


def test_tensors_and_layer_are_checked_before_the_library_is_called():
    import torch

    layer = api.MoeLayer.__new__(api.MoeLayer)
    layer._h, layer.hidden, layer.n_experts, layer.top_k = None, 64, 9, 3
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(api.MoeError, match="closed"):
        layer.layer_forward(t, t, t, shared_experts=1)
    native = api._binding()
    for bad in (-1, 3, 9):
        with pytest.raises(api.MoeError, match="shared_experts"):
            native.layer_forward(4096, 64, 9, 3, t, t, t, None, None, bad, None, None, None, None)
    with pytest.raises(api.MoeError, match="CUDA"):
        native.layer_forward(4096, 64, 9, 3, t, t, t, None, None, 1, None, None, None, None)
