"""The whole layer from the tokens on, against the definition in 64 bits and against the calls it is made of.

Tolerances.  The up products are off by a sum's error (H / 16 + 16 steps of 2^-22 of sum |W x|, the logits too), a by
that through its slope and by one rounding to bf16 (2^-8 of it; silu's own 2^-20); both pass through |W_down|, whose sum
adds (I / 16 + 16) 2^-22 of sum |W a|.  The weighted sum of k + S rows and the residual adds 2^-20 of its terms, and dst is
rounded once: 2^-8."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from nvfp4_quantized_moe_topk_gb300 import api  # noqa: E402

DEV, D = "cuda", torch.float64
E2M1 = [0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6]


class Layer:
    def __init__(self, H=256, I=128, E=16, k=4, S=1, gated=False, router="bf16", most=256, seed=3, single=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.randn = randn = lambda *s: torch.randn(*s, generator=g, device=DEV)
        rint = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV, dtype=torch.uint8)  # noqa: E731
        self.H, self.I, self.E, self.k, self.S, self.gated = H, I, E, k, S, gated
        self.w = {}
        for name, r, c in (("up", I, H), ("down", H, I)) + ((("gate", I, H),) if gated else ()):
            self.w[name + "_codes"] = rint(0, 256, E + S, r, c // 2)
            self.w[name + "_scales"] = rint(0x30, 0x40, E + S, r, c // 16)
            self.w[name + "_global"] = (torch.rand(E + S, generator=g, device=DEV) * 0.2 + 0.2) / c ** 0.5
        self.router = (randn(E, H) / H ** 0.5).to(torch.bfloat16 if router == "bf16" else torch.float32)
        self.bias = randn(E) * 0.5
        self.layer = api.MoeLayer(H, I, E + S, k + S, most, *[self.w[n] for n in (
            "up_codes", "up_scales", "down_codes", "down_scales", "up_global", "down_global")], single_max_tokens=single,
            **{n: v for n, v in self.w.items() if n.startswith("gate")})

    def matrix(self, name, e):
        codes, scales = self.w[name + "_codes"][e].long(), self.w[name + "_scales"][e].view(torch.float8_e4m3fn).to(D)
        v = torch.tensor(E2M1, dtype=D, device=DEV)[torch.stack([codes % 16, codes // 16], -1)].flatten(-2)
        return v * scales.repeat_interleave(16, -1) * float(self.w[name + "_global"][e])

    def call(self, x, residual=None, bias=True, dst=None, **kw):
        n = x.shape[0]
        dst = torch.full((n, self.H), 9.0, dtype=torch.bfloat16, device=DEV) if dst is None else dst
        ids = torch.empty(n, self.k, dtype=torch.int32, device=DEV)
        weights, logits = torch.empty(n, self.k, device=DEV), torch.empty(n, self.E, device=DEV)
        self.layer.layer_forward(x, self.router, dst, residual, self.bias if bias else None, shared_experts=self.S,
                                 topk_ids=ids, topk_weights=weights, logits=logits, **kw)
        return dst, ids, weights, logits

    def check(self, n, residual=True, bias=True):
        x = self.randn(n, self.H).to(torch.bfloat16)
        res = self.randn(n, self.H).to(torch.bfloat16) if residual else None
        dst, ids, weights, logits = self.call(x, res, bias)
        # logits, and the picks of them
        xd, r = x.to(D), self.router.to(D)
        steps = lambda c: (c / 16 + 16) * 2.0 ** -22  # noqa: E731
        assert bool(((logits.to(D) - xd @ r.t()).abs() <= steps(self.H) * (xd.abs() @ r.abs().t())).all())
        want_ids, want_w = torch.empty_like(ids), torch.empty_like(weights)
        api.router_topk(logits, self.bias if bias else None, want_ids, want_w)
        assert torch.equal(ids, want_ids) and torch.equal(weights, want_w)
        out = torch.zeros(n, self.H, dtype=D, device=DEV) if res is None else res.to(D)
        size = torch.zeros_like(out)
        for e in range(self.E + self.S):
            if e < self.E:
                by = ((ids == e) * weights.to(D)).sum(1, keepdim=True)
                rows = (ids == e).any(1)
            else:
                by, rows = torch.ones(n, 1, dtype=D, device=DEV), torch.ones(n, dtype=torch.bool, device=DEV)
            if not bool(rows.any()):
                continue
            x1, by = xd[rows], by[rows]
            up, down = self.matrix("up", e), self.matrix("down", e)
            h, dh = x1 @ up.t(), steps(self.H) * (x1.abs() @ up.abs().t())
            if self.gated:
                gate = self.matrix("gate", e)
                q, dq = x1 @ gate.t(), steps(self.H) * (x1.abs() @ gate.abs().t())
                s = q * torch.sigmoid(q)
                a, da = s * h, s.abs() * dh + 1.1 * dq * (h.abs() + dh) + 2.0 ** -20 * (s * h).abs()
            else:
                a = h.clamp(min=0).square()
                da = (2 * h.abs() + dh) * dh
            da = da + 2.0 ** -8 * (a.abs() + da)
            out[rows] += by * (a @ down.t())
            size[rows] += by * (da @ down.abs().t() + steps(self.I) * (a.abs() @ down.abs().t()))
        bound = size + 2.0 ** -20 * (out.abs() + size)
        assert bool(((dst.to(D) - out).abs() <= bound + 2.0 ** -8 * (out.abs() + bound)).all())
        assert self.layer.device_error() == 0


@pytest.mark.parametrize("n", [1, 2, 8, 9, 33, 64, 65, 200])
@pytest.mark.parametrize("kw", [dict(), dict(S=2, gated=True, router="fp32"), dict(S=0, E=13, k=6)])
def test_layer(n, kw):
    layer = Layer(**kw)
    layer.check(n, residual=n % 2 == 0, bias=n % 3 != 0)
    layer.check(n, residual=n % 2 == 1)  # again with the same handle


@pytest.mark.parametrize("kw,n", [(dict(H=2688, I=1856, E=128, k=6), 1), (dict(H=2688, I=1856, E=128, k=6, S=2, gated=True), 32),
                                  (dict(E=3, k=1, S=3), 64), (dict(H=4096, I=64, E=300, k=8, S=1), 17),
                                  (dict(H=64, I=64, E=1000, k=3, S=1), 40), (dict(H=64, I=64, E=1000, k=30, S=2), 33),
                                  (dict(H=2688, I=1856, E=128, k=6, S=2, gated=True), 1), (dict(H=1024, I=192, E=64, k=6), 8),
                                  (dict(H=64, I=64, E=1000, k=30, S=2), 8), (dict(H=4096, I=64, E=300, k=8, S=2, gated=True), 5),
                                  (dict(single=-1), 5), (dict(single=8), 9), (dict(E=40, router="fp32"), 130),
                                  (dict(H=64, I=64, E=768, k=12, S=1), 70)])
def test_sizes(kw, n):
    Layer(**kw).check(n)


@pytest.mark.parametrize("n", [100, 200])
def test_without_shared_experts_it_is_the_forward(n):
    """The same picks through moe_nvfp4_forward onto the same residual: the same bits where one launch does not take the
    batch (a smaller one sums in another order)."""
    layer = Layer(S=0)
    x, res = layer.randn(n, 256).to(torch.bfloat16), layer.randn(n, 256).to(torch.bfloat16)
    dst, ids, weights, _ = layer.call(x, res)
    want = res.clone()
    layer.layer.forward(x, ids, weights, want)
    assert torch.equal(dst, want)


@pytest.mark.parametrize("n", [1, 7, 20, 100])
def test_residuals(n):
    """In place, x itself, and none: as with buffers of their own."""
    layer = Layer(S=1)
    x, res = layer.randn(n, 256).to(torch.bfloat16), layer.randn(n, 256).to(torch.bfloat16)
    want = layer.call(x, res)[0]
    assert torch.equal(layer.call(x, dst=res, residual=res)[0], want)
    assert torch.equal(layer.call(x, x)[0], layer.call(x, x.clone())[0])
    assert torch.equal(layer.call(x)[0], layer.call(x, torch.zeros_like(x))[0])


@pytest.mark.parametrize("n", [3, 30, 80])
def test_ties_take_the_lower_expert(n):
    """Logits that are small whole numbers, exact in any order of summation: many ties."""
    layer = Layer(S=1, E=24, k=5)
    x = torch.randint(-1, 2, (n, 256), device=DEV).to(torch.bfloat16)
    layer.router = torch.randint(-1, 2, (24, 256), device=DEV).to(torch.bfloat16)
    layer.router[10:] = layer.router[:14].clone()
    _, ids, _, logits = layer.call(x, bias=False)
    exact = x.double() @ layer.router.double().t()
    assert torch.equal(logits.double(), exact)
    assert torch.equal(ids.long(), torch.sort(exact, dim=1, descending=True, stable=True).indices[:, :5])


@pytest.mark.parametrize("n", [1, 24, 90])
def test_same_bits_streams_graphs_and_calls_between(n):
    layer = Layer(S=2)
    x = layer.randn(n, 256).to(torch.bfloat16)
    first = layer.call(x)
    ids, w = torch.zeros(n, 6, dtype=torch.int32, device=DEV), torch.ones(n, 6, device=DEV)
    ids += torch.arange(6, dtype=torch.int32, device=DEV)
    layer.layer.forward(x, ids, w, torch.zeros_like(x))  # another forward of the handle
    for a, b in zip(first, layer.call(x)):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = layer.call(x)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again[0], first[0])
    graph = torch.cuda.CUDAGraph()
    dst = torch.empty_like(x)
    with torch.cuda.graph(graph):
        layer.layer.layer_forward(x, layer.router, dst, None, layer.bias, shared_experts=2)
    x.mul_(-1.0)
    for _ in range(3):
        graph.replay()
    want = layer.call(x)[0]
    assert torch.equal(dst, want)


def test_no_tokens_and_refusals():
    layer = Layer(S=1, most=32)
    x = layer.randn(4, 256).to(torch.bfloat16)
    layer.call(x[:0])
    dst = torch.empty_like(x)
    m, r = layer.layer, layer.router
    bad = [lambda: m.layer_forward(x.float(), r, dst, shared_experts=1), lambda: m.layer_forward(x, r, dst),
           lambda: m.layer_forward(x, r[:8], dst, shared_experts=1), lambda: m.layer_forward(x, r, x, shared_experts=1),
           lambda: m.layer_forward(x, r.half(), dst, shared_experts=1), lambda: m.layer_forward(x, r, dst[:3], shared_experts=1),
           lambda: m.layer_forward(x, r, dst, shared_experts=5), lambda: m.layer_forward(x, r, dst, shared_experts=-1),
           lambda: m.layer_forward(x, r, dst, x[:3], shared_experts=1),
           lambda: m.layer_forward(x, r, dst, router_bias=layer.bias[:3], shared_experts=1),
           lambda: m.layer_forward(x, r, dst, shared_experts=1, topk_ids=torch.empty(4, 5, dtype=torch.int32, device=DEV)),
           lambda: m.layer_forward(x, r, dst, shared_experts=1, logits=torch.empty(4, 17, device=DEV)),
           lambda: m.layer_forward(x[:, :128], r, dst, shared_experts=1), lambda: m.layer_forward(x, None, dst, shared_experts=1)]
    for call in bad:
        with pytest.raises(api.MoeError):
            call()
    big = layer.randn(33, 256).to(torch.bfloat16)
    with pytest.raises(api.MoeError) as e:
        m.layer_forward(big, r, torch.empty_like(big), shared_experts=1)
    assert e.value.status == 3
    m.close()
    with pytest.raises(api.MoeError):
        m.layer_forward(x, r, dst, shared_experts=1)
    torch.cuda.synchronize()


@pytest.mark.parametrize("n,kw", [(9, dict(S=0)), (33, dict(S=1)), (64, dict(S=2, gated=True)), (64, dict(S=1, E=5, k=3)),
                                  (64, dict(S=3, E=990, k=7, H=64, I=64)), (40, dict(S=0, E=700, k=12, H=64, I=64))])
def test_experts_that_many_tokens_pick(n, kw):
    """A bias that sends most tokens to a few experts: experts of more than 8 tokens beside experts of one."""
    layer = Layer(**kw)
    layer.bias[: layer.k - 1] += 4.0
    layer.check(n)
    first = layer.call(layer.randn(n, layer.H).to(torch.bfloat16))
    assert int(torch.bincount(first[1].view(-1).long()).max()) > 8


def test_a_few_tokens_leave_no_packed_rows():
    """One token packs no rows, so there are none to look at; a call that packs some brings them back."""
    b = Layer()
    x = b.randn(40, b.H).to(torch.bfloat16)
    b.call(x)
    counts = torch.zeros(b.E + b.S, dtype=torch.int32, device=DEV)
    b.call(x[:1])
    for read in (b.layer.debug_routing, b.layer.debug_intermediates):
        with pytest.raises(api.MoeError, match="UNSUPPORTED"):
            read()
    b.call(x)
    b.layer.debug_routing(counts)
    assert int(counts.sum()) > 0
