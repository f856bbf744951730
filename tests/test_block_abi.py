"""The operators around the layer, without a GPU: struct layouts, workspace sizes and the refusals that come before any
CUDA call (no accepted call is made here: the addresses are not memory)."""
import os
import shutil
import struct
import subprocess

import pytest

from nvfp4_quantized_moe_topk_gb300 import api
from nvfp4_quantized_moe_topk_gb300 import build as B

# the argument structs of the header, packed
NORM_ARGS = struct.Struct("@7i4f4xPqPqPqPPPqPqPP")
NORM_GRADS = struct.Struct("@PqPqPqPqPqPP")
ROUTER_ARGS = struct.Struct("@4if4xPPPPPPP")
LORA_ARGS = struct.Struct("@7i4xPPPPPPqPqPq")
A = 4096  # an aligned address that is never looked at


@pytest.fixture(scope="module")
def lib():
    B.build()
    return api.load()


def test_struct_layouts_match_the_header(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    fields = {
        "moe_block_norm_args": ["n", "weight_offset", "residual", "branch", "gate", "post_weight", "pre_weight",
                                "residual_out", "x_out", "rstd_post", "rstd_pre"],
        "moe_block_norm_grads": ["d_residual_out", "d_x", "d_residual", "d_branch", "d_gate", "d_post_weight",
                                 "d_pre_weight"],
        "moe_router_args": ["n", "n_seqs", "coef", "logits", "bias", "topk_ids", "token_mask", "seq_offsets", "counts",
                            "tokens"],
        "moe_lora_args": ["n", "out_dtype", "a", "b", "scale", "ranks", "adapter_ids", "x", "y", "out"]}
    src = tmp_path / "layout.c"
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe_nvfp4.h"', "int main(void) {"]
    for s, names in fields.items():
        lines.append(f'printf("%zu", sizeof({s}));')
        lines += [f'printf(" %zu", offsetof({s}, {f}));' for f in names]
        lines.append('printf("\\n");')
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([gcc, "-std=c99", f"-I{inc}", str(src), "-o", str(exe)], check=True)
    got = [[int(v) for v in l.split()] for l in subprocess.run([str(exe)], capture_output=True,
                                                               text=True).stdout.splitlines()]
    assert [g[0] for g in got] == [NORM_ARGS.size, NORM_GRADS.size, ROUTER_ARGS.size,
                                   LORA_ARGS.size]
    assert got[0][1:] == [0, 40, 48, 64, 80, 96, 104, 112, 128, 144, 152]
    assert got[1][1:] == [0, 16, 32, 48, 64, 80, 88]
    assert got[2][1:] == [0, 12, 16, 24, 32, 40, 48, 56, 64, 72]
    assert got[3][1:] == [0, 24, 32, 40, 48, 56, 64, 72, 88, 104]


NORM = dict(n=4, hidden=64, res=0, act=0, par=0, kind=0, sig=0, eps=1e-6, rs=1.0, bs=1.0, off=0.0, residual=A, rst=0,
            branch=A, bst=0, gate=0, gst=0, post=A, pre=A, out=A, ost=0, x=A, xst=0, rp=A, ru=A)
GRAD = dict(dro=A, drost=0, dx=A, dxst=0, dr=A, drst=0, db=A, dbst=0, dg=0, dgst=0, dpost=A, dpre=A)
ROUTER = dict(n=4, E=16, k=2, S=1, coef=0.1, logits=A, bias=A, ids=A, mask=0, seq=0, counts=A, tokens=A)
LORA = dict(n=4, inp=64, out_=64, L=2, R=16, yd=0, od=0, a=A, b=A, scale=A, ranks=A, ids=A, x=A, xst=0, y=A, yst=0,
            out=A + 65536, ost=0)


def norm(**kw):
    return NORM_ARGS.pack(*dict(NORM, **kw).values())


def grad(**kw):
    return NORM_GRADS.pack(*dict(GRAD, **kw).values())


def router(**kw):
    return ROUTER_ARGS.pack(*dict(ROUTER, **kw).values())


def lora(**kw):
    return LORA_ARGS.pack(*dict(LORA, **kw).values())


@pytest.mark.parametrize("want,kw", [
    (1, dict(n=-1)), (1, dict(hidden=0)), (2, dict(hidden=60)), (2, dict(hidden=8200)), (1, dict(res=2)),
    (1, dict(act=-1)), (1, dict(par=5)), (1, dict(kind=4, gate=A)), (1, dict(kind=0, sig=1)), (1, dict(kind=1, sig=2)),
    (1, dict(kind=1, gate=0)), (1, dict(kind=0, gate=A)), (1, dict(eps=0.0)), (1, dict(eps=float("nan"))),
    (1, dict(residual=0)), (1, dict(residual=A + 2)), (1, dict(rst=63)), (1, dict(rst=68)), (1, dict(branch=A + 8)),
    (1, dict(branch=0)), (1, dict(branch=0, post=0, rp=A)), (1, dict(pre=0)), (1, dict(x=0)),
    (1, dict(pre=0, x=0, ru=0, out=0)), (1, dict(pre=0, x=0)), (1, dict(post=0)), (1, dict(post=A + 4)),
    (1, dict(rp=A + 2)), (1, dict(kind=3, gate=A, gst=60)), (1, dict(kind=2, gate=A + 2)), (1, dict(ost=-64))])
def test_norm_refusals(lib, want, kw):
    assert lib.moe_block_norm(norm(**kw), None) == want


def test_norm_null_and_empty(lib):
    assert lib.moe_block_norm(None, None) == 1
    assert lib.moe_block_norm(norm(n=0, residual=0, branch=0, out=0, x=0), None) == 0
    assert lib.moe_block_norm_workspace_bytes(-1, 64) == 0
    assert lib.moe_block_norm_workspace_bytes(10 ** 6, 4096) >= 2 * 4096 * 4


@pytest.mark.parametrize("want,kw,gk", [
    (1, dict(hidden=0), {}), (1, {}, dict(dro=A + 2)), (1, {}, dict(dxst=10)), (1, {}, dict(dg=A)),
    (1, dict(kind=3, gate=A), dict(dg=A + 4)), (1, dict(post=0, rp=0), {}), (1, dict(pre=0), {}),
    (1, dict(branch=0, post=0, rp=0), dict(dpost=0)), (1, dict(rp=0), {}), (1, dict(ru=0), {}), (1, dict(out=0), {}),
    (1, {}, dict(dpost=A + 1))])
def test_norm_backward_refusals(lib, want, kw, gk):
    assert lib.moe_block_norm_backward(norm(**kw), grad(**gk), A, 1 << 30, None) == want


def test_norm_backward_workspace(lib):
    need = lib.moe_block_norm_workspace_bytes(4, 64)
    assert lib.moe_block_norm_backward(None, grad(), A, need, None) == 1
    assert lib.moe_block_norm_backward(norm(), None, A, need, None) == 1
    assert lib.moe_block_norm_backward(norm(), grad(), A + 8, need, None) == 1
    assert lib.moe_block_norm_backward(norm(), grad(), A, need - 1, None) == 3
    assert lib.moe_block_norm_backward(norm(), grad(), None, 0, None) == 3


@pytest.mark.parametrize("want,kw", [
    (1, dict(n=-1)), (1, dict(E=0)), (1, dict(k=0)), (1, dict(S=0)), (2, dict(E=1025)), (2, dict(k=33, E=64)),
    (1, dict(S=2)), (1, dict(logits=0)), (1, dict(ids=0)), (1, dict(logits=A + 2)), (1, dict(seq=A + 1)),
    (1, dict(counts=0)), (1, dict(tokens=0)), (1, dict(tokens=A + 2))])
def test_router_refusals(lib, want, kw):
    assert lib.moe_balance_loss(router(**kw), A, A, A, 1 << 40, None) == want


def test_router_other_refusals(lib):
    need = lib.moe_router_workspace_bytes(4, 16, 1)
    assert need > 0 and lib.moe_router_workspace_bytes(4, 16, 0) == 0
    assert lib.moe_balance_loss(None, A, A, A, need, None) == 1
    assert lib.moe_balance_loss(router(), None, A, A, need, None) == 1
    assert lib.moe_balance_loss(router(), A, A + 1, A, need, None) == 1
    assert lib.moe_balance_loss(router(), A, A, A, need - 1, None) == 3
    assert lib.moe_balance_loss(router(), A, A, None, 0, None) == 3
    assert lib.moe_router_backward(None, A, A, A, A, A, A, need, None) == 1
    assert lib.moe_router_backward(router(), A, None, A, A, A, A, need, None) == 1
    assert lib.moe_router_backward(router(), A, A, A, None, A, A, need, None) == 1
    assert lib.moe_router_backward(router(counts=0), A, A, A, A, A, A, need, None) == 1
    assert lib.moe_router_backward(router(), A, A, A + 2, A, A, A, need, None) == 1
    assert lib.moe_router_backward(router(), A, A, A, A, A, A, need - 1, None) == 3
    assert lib.moe_router_backward(router(n=0), None, None, None, None, None, A, 1 << 20, None) == 0


@pytest.mark.parametrize("want,kw", [
    (1, dict(n=-1)), (1, dict(inp=0)), (1, dict(out_=-8)), (1, dict(L=0)), (1, dict(R=0)), (2, dict(inp=60)),
    (2, dict(inp=(1 << 24) + 8)), (2, dict(out_=(1 << 24) + 8)), (2, dict(out_=4)), (2, dict(R=12)), (2, dict(R=136)), (2, dict(L=1025)), (1, dict(yd=2)), (1, dict(od=-1)),
    (1, dict(a=0)), (1, dict(b=0)), (1, dict(ids=0)), (1, dict(x=0)), (1, dict(out=0)), (1, dict(a=A + 8)),
    (1, dict(scale=A + 2)), (1, dict(xst=56)), (1, dict(xst=68)), (1, dict(out=A, od=1)), (1, dict(out=A, ost=72))])
def test_lora_refusals(lib, want, kw):
    assert lib.moe_lora_apply(lora(**kw), A, 1 << 40, None) == want


def test_lora_null_and_empty(lib):
    assert lib.moe_lora_apply(None, A, 1 << 30, None) == 1
    assert lib.moe_lora_apply(lora(n=0, x=0, out=0, ids=0, a=0, b=0), None, 0, None) == 0
    assert lib.moe_lora_workspace_bytes(-1, 2) == 0


def test_tensors_are_checked_before_the_library_is_called():
    """On the CPU every tensor is on the wrong device: refused, with the framework's error."""
    import torch

    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(api.MoeError) as e:
        api.block_norm(t, pre_weight=t[0], x_out=t)
    assert e.value.status == api.MOE_OK + 1 and "CUDA" in str(e.value)
