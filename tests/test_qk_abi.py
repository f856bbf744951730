"""The queries' and keys' norms with rotation, without a GPU: struct layout, workspace size and the refusals that come
before any CUDA call (no accepted call is made here: the addresses are not memory)."""
import os
import shutil
import struct
import subprocess

import pytest

from nvfp4_quantized_moe_topk_gb300 import api
from nvfp4_quantized_moe_topk_gb300 import build as B

ARGS = struct.Struct("@14i3f4xPPPPPqPqPqPq")
GRADS = struct.Struct("@PqPqPqPqPP")
A = 4096  # an aligned address that is never looked at

GOOD = dict(n=4, qh=3, kh=1, D=64, rot=32, axes=1, pi=0, si=0, s0=0, s1=0, s2=0, s3=0, dt=0, pdt=0, eps=1e-6, off=0.0,
            scale=1.0, pos=A, freq=A, qw=A, kw=A, q=A, qst=0, k=A, kst=0, qo=A, qost=0, ko=A, kost=0)
GRAD = dict(dqo=A, dqost=0, dko=A, dkost=0, dq=A, dqst=0, dk=A, dkst=0, dqw=A, dkw=A)


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
                   'printf("%zu %zu %zu %zu %zu %zu %zu", sizeof(moe_qk_args), sizeof(moe_qk_grads),'
                   ' offsetof(moe_qk_args, sections), offsetof(moe_qk_args, eps), offsetof(moe_qk_args, positions),'
                   ' offsetof(moe_qk_args, q), offsetof(moe_qk_grads, d_q_weight));\nreturn 0; }\n')
    exe = tmp_path / "layout"
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([gcc, "-std=c99", f"-I{inc}", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ARGS.size, GRADS.size, 32, 56, 72, 104, 64]


BAD = [(1, dict(n=-1)), (1, dict(qh=0, kh=0)), (1, dict(qh=-1)), (1, dict(D=0)), (2, dict(D=60)), (2, dict(D=264)),
       (1, dict(rot=-16)), (1, dict(rot=80)), (2, dict(rot=24)), (1, dict(axes=0)), (1, dict(axes=5)),
       (1, dict(axes=2, s0=8, s1=7)), (1, dict(axes=2, s0=17, s1=-1)), (1, dict(dt=2)), (1, dict(pdt=-1)),
       (1, dict(pi=2)), (1, dict(si=-1)), (1, dict(eps=0.0)), (1, dict(eps=float("nan"))), (1, dict(pos=0)),
       (1, dict(freq=0)), (1, dict(pos=A + 2)), (1, dict(freq=A + 1)), (2, dict(qh=65537)), (1, dict(qw=A + 2)),
       (1, dict(kh=0)), (1, dict(q=A + 8)), (1, dict(kst=63)), (1, dict(kst=68)), (1, dict(qst=-192))]


@pytest.mark.parametrize("want,kw", BAD + [(1, dict(q=0)), (1, dict(ko=0)), (1, dict(qst=200))])
def test_refusals(lib, want, kw):
    assert lib.moe_qk_norm_rope(args(**kw), None) == want


@pytest.mark.parametrize("want,kw,gk", [(w, kw, {}) for w, kw in BAD] + [
    (1, {}, dict(dqw=A + 2)), (1, {}, dict(dqo=0)), (1, dict(kw=0), {}), (1, dict(k=0), {}), (1, {}, dict(dqst=200)),
    (1, {}, dict(dkost=60)), (1, {}, dict(dk=A + 4))])
def test_backward_refusals(lib, want, kw, gk):
    need = lib.moe_qk_workspace_bytes(4, 3, 1, 64)
    assert lib.moe_qk_norm_rope_backward(args(**kw), grads(**gk), A, need, None) == want


def test_null_empty_and_workspace(lib):
    need = lib.moe_qk_workspace_bytes(4, 3, 1, 64)
    assert need > 0 and lib.moe_qk_workspace_bytes(-1, 3, 1, 64) == 0 and lib.moe_qk_workspace_bytes(4, 3, 1, 512) == 0
    assert lib.moe_qk_norm_rope(None, None) == 1
    assert lib.moe_qk_norm_rope(args(n=0, q=0, k=0, qo=0, ko=0, pos=0), None) == 0
    assert lib.moe_qk_norm_rope_backward(None, grads(), A, need, None) == 1
    assert lib.moe_qk_norm_rope_backward(args(), None, A, need, None) == 1
    assert lib.moe_qk_norm_rope_backward(args(), grads(), A + 8, need, None) == 1
    assert lib.moe_qk_norm_rope_backward(args(), grads(), A, need - 1, None) == 3
    assert lib.moe_qk_norm_rope_backward(args(), grads(), None, 0, None) == 3
    # nothing to compute: nothing is enqueued
    nothing = dict(dqo=0, dko=0, dq=0, dk=0, dqw=0, dkw=0)
    assert lib.moe_qk_norm_rope_backward(args(), grads(**nothing), None, 0, None) == 0
    assert lib.moe_qk_norm_rope_backward(args(n=0), grads(dqw=0, dkw=0), None, 0, None) == 0


def test_tensors_are_checked_before_the_library_is_called():
    import torch

    t = torch.zeros(4, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(api.MoeError) as e:
        api.qk_norm_rope(t, None, t, None)
    assert e.value.status == 1 and "CUDA" in str(e.value)
    for bad in (None, t[0], 5):
        with pytest.raises(api.MoeError):
            api.qk_norm_rope(bad, None, t, None)
    with pytest.raises(api.MoeError):
        api.qk_norm_rope_backward(None, None, None, None, None, None)
