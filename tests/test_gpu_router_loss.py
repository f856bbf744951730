"""GPU parity of the router's balance loss and backward pass with their definitions in 64 bits.

Tolerances.  Counts are exact.  A probability's relative error is that of expf (2 units in the last place, 2.4e-7), of
its argument's rounding (|z - max| 2^-24, under 40 2^-24 = 2.4e-6 for the logits drawn here) and of a sum of at most 32
terms and a tree (37 2^-24): 5e-6 in all (PROB).  Sums over tokens add positive terms in at most 3 (a warp's tokens here)
+ 8 (warps) + 304 (blocks) additions: 315 2^-24 = 1.9e-5 more for prob_sums, the same again for the loss's sum over
experts (4 + 5 + 8 additions) and sequences.  Gradients are held to PROB times the sum of the absolute values of their
terms, three times over (g, its mean, the product), their column sums to that and 1.9e-5."""
import pytest

pytestmark = pytest.mark.gpu
PROB = 5e-6
SUMS = 1.9e-5


@pytest.fixture(scope="module")
def dev():
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    api.load(build_if_missing=True)
    return torch.device("cuda:0")


class Batch:
    def __init__(self, dev, n, E, k, ends=None, masked=0.0, sigma=1.0, seed=0):
        import torch

        g = torch.Generator(device=dev).manual_seed(seed)
        self.n, self.E, self.k, self.coef = n, E, k, 0.02
        self.logits = torch.randn(n, E, generator=g, device=dev)
        self.bias = sigma * torch.randn(E, generator=g, device=dev) if sigma else None
        z = self.logits if self.bias is None else self.logits + self.bias
        self.ids = z.topk(k, dim=1).indices.to(torch.int32)
        self.weights = torch.softmax(z.gather(1, self.ids.long()), 1)
        self.d_weights = torch.randn(n, k, generator=g, device=dev) / max(n, 1)
        self.d_loss = torch.tensor([1.7], device=dev)
        self.mask = torch.rand(n, generator=g, device=dev) >= masked if masked else None
        self.ends = ends
        self.S = 1 if ends is None else len(ends) - 1
        self.offsets = None if ends is None else torch.tensor(ends, dtype=torch.int32, device=dev)

    def reference(self):
        """(loss, prob_sums, counts, tokens, d_logits, scale of d_logits) in 64 bits, by a loop over the sequences."""
        import torch

        dev, E = self.logits.device, self.E
        z = (self.logits if self.bias is None else self.logits + self.bias).double()
        kept = torch.ones(self.n, dtype=torch.bool, device=dev) if self.mask is None else self.mask.bool()
        dead = (z == -float("inf")).all(1)
        p = torch.softmax(torch.where((dead | ~kept)[:, None], 0.0, z), 1)
        p = torch.where((dead | ~kept)[:, None], 0.0, p)
        ends = [0, self.n] if self.ends is None else self.ends
        N = int(kept.sum())
        counts = torch.zeros(self.S, E, dtype=torch.int64, device=dev)
        sums = torch.zeros(self.S, E, dtype=torch.float64, device=dev)
        grow = torch.zeros(self.n, E, dtype=torch.float64, device=dev)
        tokens, loss = [], 0.0
        for s in range(self.S):
            a, b = ends[s], ends[s + 1]
            m = kept[a:b]
            ids = self.ids[a:b][m].reshape(-1).long()
            ids = ids[(ids >= 0) & (ids < E)]
            counts[s] = torch.bincount(ids, minlength=E)
            sums[s] = p[a:b].sum(0)
            Ns = int(m.sum())
            tokens.append(Ns)
            if Ns:
                loss = loss + self.coef * E / (N * self.k) * (counts[s] * sums[s]).sum() / Ns
                grow[a:b] = m[:, None] * (float(self.d_loss) * self.coef * E / (N * self.k * Ns)) * counts[s][None]
        mean = (grow * p).sum(1, keepdim=True)
        d, scale = p * (grow - mean), p * (grow + mean)
        w, dw = self.weights.double(), self.d_weights.double()
        ok = (self.ids >= 0) & (self.ids < E)
        at = torch.where(ok, self.ids, 0).long()
        dz = w * (dw - (w * dw).sum(1, keepdim=True))
        Sz = w * (dw.abs() + (w * dw).abs().sum(1, keepdim=True))
        d = d.scatter_add(1, at, torch.where(ok, dz, 0.0))
        scale = scale.scatter_add(1, at, torch.where(ok, Sz, 0.0))
        return float(loss), sums, counts, tokens + [N], d, scale

    def loss(self, stream=None, workspace=None):
        import torch

        from nvfp4_quantized_moe_topk_gb300 import api

        dev = self.logits.device
        loss = torch.full((1,), 9.0, device=dev)
        counts = torch.full((self.S, self.E), 9, dtype=torch.int32, device=dev)
        sums = torch.full((self.S, self.E), 9.0, device=dev)
        tokens = torch.full((self.S + 1,), 9, dtype=torch.int32, device=dev)
        assert api.balance_loss(self.logits, self.bias, self.ids, loss, counts, sums, tokens, coef=self.coef,
                                mask=self.mask, seq_offsets=self.offsets, stream=stream, workspace=workspace) is loss
        return loss, counts, sums, tokens

    def backward(self, counts, tokens, weights=True, bias=True, stream=None, workspace=None):
        import torch

        from nvfp4_quantized_moe_topk_gb300 import api

        dev = self.logits.device
        d = torch.full((self.n, self.E), 9.0, device=dev)
        db = torch.full((self.E,), 9.0, device=dev) if bias else None
        api.router_backward(self.logits, self.bias, self.ids, self.weights if weights else None,
                            self.d_weights if weights else None, counts, tokens, d, db, d_loss=self.d_loss,
                            coef=self.coef, mask=self.mask, seq_offsets=self.offsets, stream=stream,
                            workspace=workspace)
        return d, db


def _check(b):
    import torch

    loss, counts, sums, tokens = b.loss()
    rloss, rsums, rcounts, rtokens, rd, scale = b.reference()
    assert torch.equal(counts.long(), rcounts)
    assert tokens.tolist() == rtokens
    assert bool(((sums - rsums).abs() <= (PROB + SUMS) * rsums).all())
    assert abs(float(loss) - rloss) <= (PROB + 2 * SUMS) * rloss
    d, db = b.backward(counts, tokens)
    assert bool(((d - rd).abs() <= 3 * PROB * scale).all()), float(((d - rd).abs() / scale.clamp(min=1e-30)).max())
    assert bool(((db - rd.sum(0)).abs() <= (3 * PROB + SUMS) * scale.sum(0) + 1e-30).all())
    return loss, counts, sums, tokens, d, db


@pytest.mark.parametrize("n,E,k,ends", [
    (1, 1, 1, None), (1, 128, 6, None), (33, 40, 3, None), (5, 8, 2, [0, 1, 2, 3, 4, 5]), (64, 37, 4, None),
    (700, 128, 6, [0, 3, 650, 700]), (130, 256, 8, [0, 0, 130]), (100, 1024, 32, [0, 50, 50, 50, 99, 100]),
    (4000, 512, 8, [0, 1000, 1001, 1001, 2500, 4000]), (9, 33, 33 - 1, None), (3000, 65, 1, None), (257, 130, 5, None)])
@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("sigma", [0.0, 2.0])
def test_sizes(dev, n, E, k, ends, masked, sigma):
    _check(Batch(dev, n, E, k, ends, masked, sigma, seed=n + E))


def test_many_short_sequences(dev):
    """Three tokens each: most blocks meet several sequences."""
    _check(Batch(dev, 3000, 64, 4, list(range(0, 3001, 3)), 0.2))


@pytest.mark.parametrize("n,ends", [
    (1, [0] * 40 + [1] * 24), (3, [0, 1, 1, 2, 3]), (16, list(range(17))), (33, sorted(list(range(34)) + [5, 5, 9, 33])),
    (64, [0, 10, 20, 20, 50, 64]), (96, [0, 0, 96]), (97, [0, 40, 97]), (300, list(range(301)))])
def test_few_tokens_of_several_sequences(dev, n, ends):
    _check(Batch(dev, n, 72, 3, ends, 0.1, seed=n))


def test_sequences_wholly_masked_and_all_masked(dev):
    import torch

    b = Batch(dev, 90, 128, 6, [0, 30, 60, 90], 0.1)
    b.mask[30:60] = False
    _check(b)
    b.mask[:] = False
    loss, counts, sums, tokens, d, db = _check(b)
    assert float(loss) == 0 and int(counts.sum()) == 0 and float(sums.sum()) == 0 and tokens.tolist() == [0] * 4
    d, db = b.backward(counts, tokens, weights=False)
    assert bool((d == 0).all()) and bool((db == 0).all())


def test_logits_of_masked_tokens_are_not_looked_at(dev):
    import torch

    b = Batch(dev, 200, 128, 6, None, 0.3)
    clean = b.loss()
    cd, cdb = b.backward(clean[1], clean[3], weights=False)
    b.logits[~b.mask] = float("nan")
    b.logits[int((~b.mask).nonzero()[0])] = float("inf")
    got = b.loss()
    assert all(torch.equal(p, q) for p, q in zip(got, clean))
    d, db = b.backward(got[1], got[3], weights=False)
    assert torch.equal(d, cd) and torch.equal(db, cdb)


def test_masked_bytes_other_than_one(dev):
    """Any byte but 0 takes part."""
    import torch

    b = Batch(dev, 50, 16, 2, None, 0.5)
    want = b.loss()
    b.mask = b.mask.to(torch.uint8) * 200
    assert all(torch.equal(p, q) for p, q in zip(b.loss(), want))


def test_minus_infinity(dev):
    """Experts turned off by a logit or bias of -inf have probability and gradient 0; a row of nothing else has none."""
    import torch

    b = Batch(dev, 60, 40, 3, None, 0.0, 1.0)
    b.bias[7] = -float("inf")
    b.logits[:, 11] = -float("inf")
    z = b.logits + b.bias
    b.ids = z.topk(3, dim=1).indices.to(torch.int32)
    b.weights = torch.softmax(z.gather(1, b.ids.long()), 1)
    b.logits[5] = -float("inf")
    loss, counts, sums, tokens, d, db = _check(b)
    assert float(sums[0, 7]) == 0 and float(sums[0, 11]) == 0 and bool((d[:, [7, 11]] == 0).all())
    d, _ = b.backward(counts, tokens, weights=False)
    assert bool((d[5] == 0).all()) and bool(torch.isfinite(d).all())


def test_bad_and_repeated_ids(dev):
    """Ids outside the experts count nowhere and get no gradient; a repeated one adds up."""
    b = Batch(dev, 80, 128, 6, [0, 40, 80], 0.1)
    b.ids[::3, 1] = -1
    b.ids[1::3, 2] = 128
    b.ids[::5, 3] = b.ids[::5, 4]
    b.ids[7, :] = 2 ** 31 - 1
    b.ids[8, :] = -2 ** 31
    _check(b)


def test_terms_on_their_own(dev):
    import torch

    b = Batch(dev, 300, 128, 6, None, 0.2)
    _, counts, _, tokens = b.loss()
    both, db = b.backward(counts, tokens)
    only_loss, _ = b.backward(counts, tokens, weights=False)
    only_weights, dw_bias = b.backward(None, None)
    assert bool((both - (only_loss + only_weights)).abs().max() <= 1e-6 * both.abs().max())
    assert torch.equal(b.backward(counts, tokens, bias=False)[0], both)
    # without a loss term the picks alone have a gradient
    picked = torch.zeros(300, 128, dtype=torch.bool, device=dev).scatter_(1, b.ids.long(), True)
    assert bool((only_weights[~picked] == 0).all())


def test_no_tokens(dev):
    b = Batch(dev, 0, 64, 4)
    loss, counts, sums, tokens = b.loss()
    assert float(loss) == 0 and int(counts.sum()) == 0 and float(sums.sum()) == 0 and tokens.tolist() == [0, 0]
    _, db = b.backward(counts, tokens)
    assert bool((db == 0).all())


def test_repeated_calls_and_stale_workspaces(dev):
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    b = Batch(dev, 5000, 128, 8, [0, 1700, 1701, 5000], 0.1, 2.0)
    ws = api.router_workspace(5000, 128, 3)
    want = b.loss(workspace=ws)
    want_b = b.backward(want[1], want[3], workspace=ws)
    ws.fill_(0xFF)
    assert all(torch.equal(p, q) for p, q in zip(b.loss(workspace=ws), want))
    ws.fill_(0x7F)
    assert all(torch.equal(p, q) for p, q in zip(b.backward(want[1], want[3], workspace=ws), want_b))


def test_on_another_stream(dev):
    import torch

    b = Batch(dev, 900, 128, 6, [0, 400, 900], 0.1)
    want = b.loss()
    want_b = b.backward(want[1], want[3])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        with torch.cuda.stream(s):
            got = b.loss(stream=handle)
            got_b = b.backward(got[1], got[3], stream=handle)
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got + got_b, want + want_b))


def test_backward_against_differences(dev):
    """<d_logits, direction> against a central difference of d_loss * loss + <weights, d_weights> in 64 bits, the counts
    held (they are piecewise constant).  Error of the difference h^2 ~ 1e-8 relative, of the gradient 1.5e-5 of its
    terms."""
    import torch

    b = Batch(dev, 40, 24, 4, [0, 11, 40], 0.2)
    _, counts, _, tokens = b.loss()
    d, db = b.backward(counts, tokens)
    g = torch.Generator(device=dev).manual_seed(4)
    v = torch.randn(40, 24, generator=g, device=dev, dtype=torch.float64)
    v[:, 3] += 1.0

    def value(h):
        z = (b.logits + b.bias).double() + h * v
        p = torch.softmax(z, 1)
        w = torch.softmax(z.gather(1, b.ids.long()), 1)
        total = (w * b.d_weights.double()).sum()
        for s, (lo, hi) in enumerate(((0, 11), (11, 40))):
            m = b.mask[lo:hi]
            P = p[lo:hi][m].sum(0)
            total = total + float(b.d_loss) * b.coef * 24 / (int(tokens[2]) * 4 * int(tokens[s])) * (counts[s] * P).sum()
        return float(total)

    h = 1e-4
    diff = (value(h) - value(-h)) / (2 * h)
    terms = d.double() * v
    assert abs(float(terms.sum()) - diff) <= 1e-4 * float(terms.abs().sum())
    assert bool((db - d.sum(0)).abs().max() <= 1e-5 * d.abs().sum(0).max())


def test_refusals(dev):
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    b = Batch(dev, 8, 16, 2, [0, 3, 8], 0.2)
    loss, counts, sums, tokens = b.loss()
    ok = dict(logits=b.logits, bias=b.bias, topk_ids=b.ids, loss=loss, counts=counts, prob_sums=sums, tokens=tokens,
              coef=0.1, mask=b.mask, seq_offsets=b.offsets)
    api.balance_loss(**ok)
    for bad in (dict(logits=b.logits.bfloat16()), dict(logits=b.logits.cpu()), dict(logits=b.logits.t()),
                dict(bias=b.bias[:5]), dict(topk_ids=b.ids.long()), dict(counts=counts[:1]), dict(loss=None),
                dict(tokens=tokens[:2]), dict(prob_sums=sums.double()), dict(mask=b.mask[:4]),
                dict(seq_offsets=b.offsets[:1]), dict(seq_offsets=None), dict(counts=None)):
        with pytest.raises(api.MoeError):
            api.balance_loss(**dict(ok, **bad))
    with pytest.raises(api.MoeError) as e:
        api.balance_loss(**dict(ok, workspace=torch.empty(16, dtype=torch.uint8, device=dev)))
    assert e.value.status == 3
    for E, k in ((1025, 2), (64, 33)):
        big = Batch(dev, 2, 2000, 40)
        with pytest.raises(api.MoeError) as e:
            api.balance_loss(big.logits[:, :E].contiguous(), None, big.ids[:, :k].contiguous(), loss,
                             torch.empty(1, E, dtype=torch.int32, device=dev), torch.empty(1, E, device=dev),
                             tokens[:2].contiguous(), coef=0.1)
        assert e.value.status == 2
    d = torch.empty(8, 16, device=dev)
    with pytest.raises(api.MoeError):
        api.router_backward(b.logits, b.bias, b.ids, b.weights, None, counts, tokens, d, coef=0.1, mask=b.mask,
                            seq_offsets=b.offsets)
    with pytest.raises(api.MoeError):
        api.router_backward(b.logits, b.bias, b.ids, None, None, counts, None, d, coef=0.1, seq_offsets=b.offsets)
