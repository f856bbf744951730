"""The projections without a GPU: struct layouts, workspace sizes and the refusals that come before any CUDA call (no
accepted call is made here: the addresses are not memory)."""
import ctypes
import os
import shutil
import struct
import subprocess

import pytest

from nvfp4_quantized_moe_topk_gb300 import api
from nvfp4_quantized_moe_topk_gb300 import build as B

ARGS = struct.Struct("@8if4xPPPqPqPqPq")
GRADS = struct.Struct("@3i4xPqPqPP")
A = 4096  # an aligned address that is never looked at
GOOD = dict(n=4, inp=64, out_=32, act=0, bt=1, rt=0, zt=0, ot=0, scale=1.0, w=6 * A, bias=A, x=7 * A, xst=0, res=A, rst=0,
            z=A, zst=0, out=2 * A, ost=0)
GRAD = dict(dyt=0, dxt=0, dwt=1, dy=A, dyst=0, dx=3 * A, dxst=0, dw=4 * A, db=5 * A)


def args(**kw):
    return ARGS.pack(*dict(GOOD, **kw).values())


def grads(**kw):
    return GRADS.pack(*dict(GRAD, **kw).values())


@pytest.fixture(scope="module")
def lib():
    B.build()
    return api.load()


def test_struct_layouts_match_the_header(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_nvfp4.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu %zu %zu %zu", sizeof(moe_linear_args), sizeof(moe_linear_grads),'
                   ' offsetof(moe_linear_args, residual_scale), offsetof(moe_linear_args, weight),'
                   ' offsetof(moe_linear_args, x), offsetof(moe_linear_args, out), offsetof(moe_linear_grads, d_weight));\n'
                   'return 0; }\n')
    exe = tmp_path / "layout"
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([gcc, "-std=c99", f"-I{inc}", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ARGS.size, GRADS.size, 32, 40, 56, 104, 48]


BAD = [(1, dict(n=-1)), (1, dict(inp=0)), (1, dict(out_=-8)), (2, dict(inp=60)), (2, dict(out_=12)),
       (2, dict(inp=(1 << 24) + 8)), (1, dict(act=4)), (1, dict(act=-1)), (1, dict(zt=2)), (1, dict(x=A + 8)),
       (1, dict(xst=56)), (1, dict(xst=68)), (1, dict(w=A + 2)), (1, dict(z=A + 4)), (1, dict(zst=24))]


@pytest.mark.parametrize("want,kw", BAD + [
    (1, dict(bt=3)), (1, dict(rt=-1)), (1, dict(ot=2)), (1, dict(x=0)), (1, dict(w=0)), (1, dict(out=0)),
    (1, dict(out=A + 8)), (1, dict(bias=A + 2)), (1, dict(bias=A + 1, bt=0)), (1, dict(res=A + 2)), (1, dict(rst=31)),
    (1, dict(out=7 * A)), (1, dict(out=6 * A)), (1, dict(z=7 * A)),
    (1, dict(out=A, ot=1, z=0)), (1, dict(out=A, ost=64, z=0)), (1, dict(out=A, res=0))])
def test_refusals(lib, want, kw):
    assert lib.moe_linear(args(**kw), None) == want


@pytest.mark.parametrize("want,kw,gk", [(w, kw, {}) for w, kw in BAD] + [
    (1, {}, dict(dyt=2)), (1, {}, dict(dxt=-1)), (1, {}, dict(dwt=9)), (1, {}, dict(dy=0)), (1, {}, dict(dy=A + 2)),
    (1, {}, dict(dxst=8)), (1, {}, dict(dw=A + 4)), (1, {}, dict(db=A + 2)), (1, dict(act=2, z=0), {}),
    (1, dict(x=0), {}), (1, dict(w=0), {}), (1, {}, dict(dx=A)), (1, {}, dict(dx=7 * A)), (1, {}, dict(dw=6 * A)),
    (1, {}, dict(db=A))])
def test_backward_refusals(lib, want, kw, gk):
    assert lib.moe_linear_backward(args(**kw), grads(**gk), 8 * A, 1 << 40, None) == want


def test_the_kept_argument_is_not_the_residual(lib):
    """The residual is read after z has been written, part by part."""
    assert lib.moe_linear(args(z=16 * A, res=16 * A), None) == 1


def test_null_empty_and_workspace(lib):
    need = lib.moe_linear_workspace_bytes(4, 64, 32)
    assert need > 0 and lib.moe_linear_workspace_bytes(-1, 64, 32) == 0 and lib.moe_linear_workspace_bytes(1, 0, 8) == 0
    assert lib.moe_linear(None, None) == 1
    assert lib.moe_linear(args(n=0, x=0, w=0, out=0, res=0, z=0), None) == 0
    assert lib.moe_linear_backward(None, grads(), A, need, None) == 1
    assert lib.moe_linear_backward(args(), None, A, need, None) == 1
    assert lib.moe_linear_backward(args(), grads(), 8 * A + 8, need, None) == 1
    assert lib.moe_linear_backward(args(), grads(), 8 * A, need - 1, None) == 3
    assert lib.moe_linear_backward(args(), grads(), None, 0, None) == 3
    assert lib.moe_linear_backward(args(n=0), grads(dw=0, db=0), None, 0, None) == 0
    assert lib.moe_linear_get_device_error(ctypes.POINTER(ctypes.c_int32)()) == 1


def test_tensors_are_checked_before_the_library_is_called():
    import torch

    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(api.MoeError) as e:
        api.linear(t, t, t)
    assert e.value.status == 1 and "CUDA" in str(e.value)
    for bad in ("tanh", None, 1):
        with pytest.raises(api.MoeError):
            api.linear(t, t, t, activation=bad)
    with pytest.raises(api.MoeError):
        api.linear(None, t, t)
    with pytest.raises(api.MoeError):
        api.linear_backward(t, None, t)
