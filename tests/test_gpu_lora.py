"""GPU parity of the adapters (moe_lora_apply) with the definition in 64 bits.

Tolerance, for token t and output o, with V[i] = sum_c |a[i][c] x[c]| and v[i] the exact first product:
  first product: bf16 products are exact; sums of at most 4096 terms over partial sums of at most 512 and a tree, each
    addition within 2^-23 (the matrix instructions may truncate): at most 40 effective roundings of V, 5e-6 V;
  v on its way to the second product: 16 bits of mantissa for a bf16 out (2^-16 |v|), 24 for an fp32 out;
  second product: at most 128 terms, 16 2^-23 = 2e-6 of its absolute terms; scale, y and the sum: 4 2^-24 of theirs.
In all  |err| <= scale sum_i |b[o][i]| (5e-6 V[i] + (2^-16 or 0) |v[i]| + 3e-6 |v[i]|) + 3e-7 (|y| + |out|), and half a
unit in the last place (2^-8 |out|) for a bf16 out."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    api.load(build_if_missing=True)
    return torch.device("cuda:0")


class Case:
    def __init__(self, dev, ids, inp, out, L, R, y="bf16", o="bf16", ranks=None, scale=True, seed=0):
        import torch

        t = {"bf16": torch.bfloat16, "fp32": torch.float32, None: torch.bfloat16}
        g = torch.Generator(device=dev).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        self.n, self.inp, self.o, self.L, self.R = len(ids), inp, out, L, R
        self.ids = torch.tensor(ids, dtype=torch.int32, device=dev)
        self.x = r(self.n, inp).bfloat16()
        self.a = (r(L, R, inp) / inp ** 0.5).bfloat16()
        self.b = (r(L, out, R) / R ** 0.5).bfloat16()
        self.scale = torch.rand(L, generator=g, device=dev) + 0.5 if scale else None
        self.ranks = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device=dev)
        self.y = None if y is None else r(self.n, out).to(t[y])
        self.out_type = t[o]

    def run(self, out=None, workspace=None, stream=None):
        import torch

        from nvfp4_quantized_moe_topk_gb300 import api

        out = torch.full((self.n, self.o), 9.0, dtype=self.out_type, device=self.x.device) if out is None else out
        assert api.lora_apply(self.x, self.ids, self.a, self.b, self.y, out, scale=self.scale, ranks=self.ranks,
                              workspace=workspace, stream=stream) is out
        return out

    def check(self, out):
        import torch

        n, o = self.n, self.o
        want = torch.zeros(n, o, dtype=torch.float64, device=out.device)
        tol = torch.zeros_like(want)
        y = want.clone() if self.y is None else self.y.double()
        split = 2.0 ** -16 if out.dtype == torch.bfloat16 else 0.0
        for l in range(self.L):
            rows = (self.ids == l).nonzero()[:, 0]
            r = self.R if self.ranks is None else min(max(int(self.ranks[l]), 0), self.R)
            if not rows.numel() or r == 0:
                continue
            x, a, b = self.x[rows].double(), self.a[l, :r].double(), self.b[l, :, :r].double()
            s = 1.0 if self.scale is None else float(self.scale[l])
            v, V = x @ a.T, x.abs() @ a.abs().T
            want[rows] = s * (v @ b.T)
            tol[rows] = abs(s) * ((5e-6 * V + (split + 3e-6) * v.abs()) @ b.abs().T)
        want = want + y
        tol = tol + 3e-7 * (y.abs() + want.abs()) + 1e-30
        if out.dtype == torch.bfloat16:
            tol = tol + want.abs() * 2.0 ** -8
        err = (out.double() - want).abs()
        assert bool((err <= tol).all()), (float((err / tol).max()), (err / tol).argmax())
        rest = (self.ids < 0) | (self.ids >= self.L)
        if bool(rest.any()):  # no adapter: y itself
            assert torch.equal(out[rest], y[rest].to(out.dtype))


def _ids(n, L, seed, run=1, none=0.2):
    import random

    r, ids = random.Random(seed), []
    while len(ids) < n:
        ids += [-1 if r.random() < none else r.randrange(L)] * r.randint(1, 2 * run - 1)
    return ids[:n]


@pytest.mark.parametrize("n,inp,out,L,R", [
    (1, 8, 8, 1, 8), (1, 2688, 1856, 8, 16), (2, 64, 64, 3, 8), (7, 1000, 504, 4, 24), (32, 2688, 1856, 16, 32),
    (33, 264, 4096, 40, 64), (65, 520, 72, 2, 128), (130, 4096, 256, 200, 16), (300, 256, 128, 5, 40),
    (1030, 384, 392, 7, 16), (4500, 136, 264, 3, 64)])
@pytest.mark.parametrize("y,o", [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32"), ("bf16", "fp32")])
def test_sizes_and_types(dev, n, inp, out, L, R, y, o):
    c = Case(dev, _ids(n, L, n, run=1 if n < 200 else 40), inp, out, L, R, y, o, seed=n)
    c.check(c.run())


@pytest.mark.parametrize("n,run", [(1, 1), (40, 1), (40, 6), (600, 1), (600, 100), (5000, 700)])
@pytest.mark.parametrize("R", [8, 16, 32, 64, 128])
def test_mixed_ranks(dev, n, run, R):
    """Ranks from 0 up to the bank's (odd ones too, and some outside that are clamped); what lies beyond them is NaN."""
    import torch

    L = 9
    ranks = [0, R, R // 2, 1, R - 1, 7, -3, R + 5, min(R, 13)]
    c = Case(dev, _ids(n, L, n + R, run), 328, 136, L, R, "fp32", "bf16", ranks, seed=R)
    for l in range(L):
        r = min(max(ranks[l], 0), R)
        c.a[l, r:] = float("nan")
        c.b[l, :, r:] = float("nan")
    c.check(c.run())


@pytest.mark.parametrize("n", [3, 64, 700, 5000])
def test_one_adapter_for_all_and_none_for_all(dev, n):
    import torch

    c = Case(dev, [2] * n, 264, 136, 4, 16, "fp32", "fp32")
    c.check(c.run())
    c.ids.fill_(-1)
    assert torch.equal(c.run(), c.y)


def test_ids_outside_the_bank(dev):
    c = Case(dev, [0, 5, -1, 3, 2 ** 31 - 1, -2 ** 31, 4, 2], 264, 136, 5, 16)
    c.check(c.run())


def test_without_y_scale_or_ranks_and_in_place(dev):
    import torch

    ids = _ids(50, 4, 1)
    c = Case(dev, ids, 264, 136, 4, 16, None, "fp32", scale=False)
    c.check(c.run())
    c = Case(dev, ids, 264, 136, 4, 16, "bf16", "bf16")
    want = c.run()
    kept = c.y.clone()
    assert torch.equal(c.run(out=c.y), want)
    c.y = kept
    c.check(want)


def test_row_strides(dev):
    """x, y and out are slices of wider matrices; what lies beside them is left alone."""
    import torch

    c = Case(dev, _ids(45, 4, 2), 264, 136, 4, 16)
    want = c.run()
    wide = torch.full((45, 600), 3.0, dtype=torch.bfloat16, device=dev)
    x, y, out = wide[:, 8:272], wide[:, 280:416], wide[:, 424:560]
    x.copy_(c.x)
    y.copy_(c.y)
    c.x, c.y = x, y
    assert torch.equal(c.run(out=out), want)
    for part in (wide[:, :8], wide[:, 272:280], wide[:, 416:424], wide[:, 560:]):
        assert bool((part == 3).all())


@pytest.mark.parametrize("n", [40, 5000])
def test_a_bad_token_stays_to_itself(dev, n):
    """NaN and infinity in one token's x reach that token's row alone (others of the same adapter are in its tile)."""
    import torch

    c = Case(dev, [1] * n, 264, 136, 2, 16)
    want = c.run()
    c.x[3, 7] = float("nan")
    c.x[n - 2, 9] = float("inf")
    got = c.run()
    rest = torch.ones(n, dtype=torch.bool, device=dev)
    rest[[3, n - 2]] = False
    assert torch.equal(got[rest], want[rest])
    assert bool(torch.isnan(got[3]).all()) and not bool(torch.isfinite(got[n - 2]).any())


@pytest.mark.parametrize("n", [20, 3000])
def test_repeated_calls_and_stale_workspaces(dev, n):
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    c = Case(dev, _ids(n, 6, 3, 5), 1000, 520, 6, 16)
    ws = api.lora_workspace(n, 6)
    want = c.run(workspace=ws)
    ws.fill_(0xFF)
    assert torch.equal(c.run(workspace=ws), want)
    ws.fill_(0x11)
    assert torch.equal(c.run(workspace=ws), want)
    # a token's result does not depend on the tokens beside it
    one = Case(dev, [int(c.ids[0])], 1000, 520, 6, 16)
    one.x, one.y, one.a, one.b, one.scale = c.x[:1].clone(), c.y[:1].clone(), c.a, c.b, c.scale
    one.check(one.run())


def test_on_another_stream(dev):
    import torch

    c = Case(dev, _ids(3000, 6, 4, 50), 264, 136, 6, 16)
    want = c.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        with torch.cuda.stream(s):
            got = c.run(stream=handle)
        s.synchronize()
        assert torch.equal(got, want)


def test_no_tokens(dev):
    c = Case(dev, [], 264, 136, 6, 16)
    assert c.run().shape == (0, 136)


def test_in_a_captured_graph(dev):
    """Captured once, replayed on new contents of the same buffers."""
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    for n in (16, 2000):
        c = Case(dev, _ids(n, 6, 5, 9), 264, 136, 6, 16)
        out = torch.empty(n, 136, dtype=torch.bfloat16, device=dev)
        ws = api.lora_workspace(n, 6)
        c.run(out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=out, workspace=ws)
        c.ids.copy_(torch.tensor(_ids(n, 6, 6, 2), dtype=torch.int32))
        c.x.normal_()
        g.replay()
        torch.cuda.synchronize()
        c.check(out)


def test_refusals(dev):
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    c = Case(dev, [0, 1, -1], 264, 136, 2, 16, ranks=[16, 8])
    out = c.run()
    ok = dict(x=c.x, adapter_ids=c.ids, a=c.a, b=c.b, y=c.y, out=out, scale=c.scale, ranks=c.ranks)
    api.lora_apply(**ok)
    for bad in (dict(x=c.x.float()), dict(x=c.x.cpu()), dict(x=c.x[:2]), dict(adapter_ids=c.ids.long()),
                dict(a=c.a[:, :, :8]), dict(a=c.a.float()), dict(b=c.b[:1]), dict(b=c.b.transpose(1, 2)),
                dict(y=c.y.half()), dict(y=c.y[:, :8]), dict(out=None), dict(out=c.x), dict(scale=c.scale.double()),
                dict(ranks=c.ranks[:1]), dict(out=out[:1].expand(3, 136)), dict(x=c.x.t().contiguous().t())):
        with pytest.raises(api.MoeError):
            api.lora_apply(**dict(ok, **bad))
    for inp, o, R in ((12, 16, 8), (16, 12, 8), (16, 16, 4), (16, 16, 136)):
        t = Case(dev, [0], inp, o, 1, R)
        with pytest.raises(api.MoeError) as e:
            t.run()
        assert e.value.status == 2, (inp, o, R)


# ------------------------------------------------------------------ batches that fill the GPU with tiles of 128 tokens

LONG = 12400  # 96 full tiles of 128 and more


@pytest.mark.parametrize("inp,out,R", [(8, 8, 8), (72, 136, 16), (264, 72, 24), (1000, 504, 64), (200, 264, 128),
                                       (64, 64, 40), (456, 1032, 32)])
@pytest.mark.parametrize("y,o", [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32"), ("bf16", "fp32")])
def test_long_sizes_and_types(dev, inp, out, R, y, o):
    from nvfp4_quantized_moe_topk_gb300 import api

    c = Case(dev, _ids(LONG, 5, inp, run=300), inp, out, 5, R, y, o, seed=R)
    c.check(c.run())
    assert api.lora_device_error() == 0


@pytest.mark.parametrize("run", [1, 90, 3000])
@pytest.mark.parametrize("R", [8, 16, 64, 128])
def test_long_mixed_ranks(dev, run, R):
    L = 9
    ranks = [0, R, R // 2, 1, R - 1, 7, -3, R + 5, min(R, 13)]
    c = Case(dev, _ids(LONG + 37, L, R, run), 328, 136, L, R, "fp32", "bf16", ranks, seed=R)
    for l in range(L):
        r = min(max(ranks[l], 0), R)
        c.a[l, r:] = float("nan")
        c.b[l, :, r:] = float("nan")
    c.check(c.run())


def test_long_one_adapter_none_and_many(dev):
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    c = Case(dev, [2] * LONG, 264, 136, 4, 16, "fp32", "fp32")
    c.check(c.run())
    c.ids.fill_(-1)
    assert torch.equal(c.run(), c.y)
    c = Case(dev, _ids(LONG, 700, 3, run=2), 136, 72, 700, 16)
    c.check(c.run())
    assert api.lora_device_error() == 0


def test_long_without_y_in_place_strides_and_bad_tokens(dev):
    import torch

    n = LONG
    ids = _ids(n, 4, 1, run=400)
    c = Case(dev, ids, 264, 136, 4, 32, None, "fp32", scale=False)
    c.check(c.run())
    c = Case(dev, ids, 264, 136, 4, 32)
    want = c.run()
    c.check(want)
    kept = c.y.clone()
    assert torch.equal(c.run(out=c.y), want)
    c.y = kept
    wide = torch.full((n, 600), 3.0, dtype=torch.bfloat16, device=dev)
    x, y, out = wide[:, 8:272], wide[:, 280:416], wide[:, 424:560]
    x.copy_(c.x)
    y.copy_(c.y)
    c.x, c.y = x, y
    assert torch.equal(c.run(out=out), want)
    for part in (wide[:, :8], wide[:, 272:280], wide[:, 416:424], wide[:, 560:]):
        assert bool((part == 3).all())
    c.ids.fill_(1)
    want = c.run()
    c.x[3, 7] = float("nan")
    c.x[n - 2, 9] = float("inf")
    got = c.run()
    rest = torch.ones(n, dtype=torch.bool, device=dev)
    rest[[3, n - 2]] = False
    assert torch.equal(got[rest], want[rest])
    assert bool(torch.isnan(got[3]).all()) and not bool(torch.isfinite(got[n - 2]).any())


def test_long_repeated_on_another_stream_and_in_a_graph(dev):
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    c = Case(dev, _ids(LONG, 6, 4, 50), 264, 136, 6, 16)
    ws = api.lora_workspace(LONG, 6)
    want = c.run(workspace=ws)
    ws.fill_(0xFF)
    assert torch.equal(c.run(workspace=ws), want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = c.run(stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    c.run(out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(out=out, workspace=ws)
    c.ids.copy_(torch.tensor(_ids(LONG, 6, 7, 20), dtype=torch.int32))
    c.x.normal_()
    g.replay()
    torch.cuda.synchronize()
    c.check(out)


# ------------------------------------------------------------------ tiles that a cluster shares

@pytest.mark.parametrize("n,L", [(520, 3), (1300, 5), (2600, 2), (4400, 16), (7000, 6)])
@pytest.mark.parametrize("inp,out", [(8, 1040), (328, 8), (2056, 520)])
@pytest.mark.parametrize("R", [8, 48, 64, 96, 128])
def test_clusters(dev, n, L, inp, out, R):
    """Few tiles of many tokens: CTAs of a cluster split both products, some of them with nothing to do in one."""
    from nvfp4_quantized_moe_topk_gb300 import api

    y, o = [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32"), ("bf16", "fp32")][(n // 20 + R // 8) % 4]
    ranks = [max(R - 3 * l, 0) for l in range(L)]
    c = Case(dev, _ids(n, L, n + R, run=150), inp, out, L, R, y, o, ranks, seed=R)
    for l in range(L):
        c.a[l, ranks[l]:] = float("nan")
        c.b[l, :, ranks[l]:] = float("nan")
    got = c.run()
    c.check(got)
    import torch

    assert torch.equal(c.run(), got)
    assert api.lora_device_error() == 0


@pytest.mark.parametrize("n", [128, 129, 256, 257, 2048, 2049])
@pytest.mark.parametrize("L,run", [(1, 300), (1024, 1), (1024, 40), (255, 3), (256, 3)])
def test_grouping(dev, n, L, run):
    """Both sides of each way to group the tokens, few and many adapters, in runs and in random order."""
    c = Case(dev, _ids(n, L, n + L, run), 72, 40, L, 8, "fp32", "fp32")
    c.check(c.run())
