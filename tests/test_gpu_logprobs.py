"""dflash_token_logprobs against a plain 64-bit implementation."""
import math

import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests.prompt_ref import FILL, Workspace, dims, ptr

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


class Scores:
    def __init__(self, logits, k=5, T=1.0, tokens=None, offset=0):
        M, V = logits.shape
        self.M, self.V, self.k, self.T = M, V, k, T
        self.buf = torch.full((M * V + 8,), NAN, device="cuda")
        self.logits = self.buf[offset:offset + M * V].view(M, V)
        self.logits.copy_(logits)
        g = torch.Generator().manual_seed(M + V)
        self.tokens = (torch.randint(0, V, (M,), generator=g) if tokens is None else torch.tensor(tokens)).int().cuda()
        f = lambda *s: torch.full(s, FILL, device="cuda")
        self.logprob, self.entropy, self.top = f(M), f(M), f(M, max(k, 1))
        self.ids = torch.full((M, max(k, 1)), -7, dtype=torch.int32, device="cuda")
        a = self.a = D.dflash_token_logprobs_args()
        a.dims = dims(vocab=V)
        a.n_rows, a.logits, a.temperature, a.topk = M, ptr(self.logits), T, k
        a.tokens, a.logprob, a.entropy = ptr(self.tokens), ptr(self.logprob), ptr(self.entropy)
        a.top_ids, a.top_logprobs = ptr(self.ids), ptr(self.top)
        self.ws = Workspace(D.DFLASH_OP_TOKEN_LOGPROBS, a)

    def run(self):
        D.dflash_token_logprobs(self.a, self.ws.ptr, self.ws.bytes)

    def check(self, status=D.DFLASH_OK):
        """Log probabilities: y = (x - max) / T with two roundings and 1/T's, 2^-22
        |y|; ln z: an error of z's terms of 2^-22 (the exponential) + 2^-22 y (its
        argument, over terms that weigh e^y: |y| e^y < 0.4) and of its sum of
        at most 2^10 partial sums in a row, 2^-14 at the very worst; here 2^-18
        for sums whose errors do not all agree, and the result's own rounding.
        Entropy: the same for sum y e^y / z <= ln V, and for ln z."""
        torch.cuda.synchronize()
        assert self.ws.status() == status
        x = self.logits.double()
        lp = torch.log_softmax(x / self.T, -1)
        good = torch.isfinite(lp).any(-1) & ~torch.isnan(lp).any(-1)
        ent = -torch.where(lp == -INF, 0.0, lp.exp() * lp).sum(-1)
        y = (x - x.amax(-1, keepdim=True)) / self.T
        lnv = math.log(self.V) + 1
        tok = self.tokens.long()
        has = (tok >= 0) & (tok < self.V)
        want = lp.gather(1, tok.clamp(0, self.V - 1)[:, None])[:, 0]
        at = y.gather(1, tok.clamp(0, self.V - 1)[:, None])[:, 0]
        self._close(self.logprob, want, 2.0 ** -22 * at.abs() + 2.0 ** -18, has & good)
        assert bool((self.logprob[~has] == FILL).all()), "a row without a token was written"
        assert bool(torch.isnan(self.logprob[has & ~good]).all())
        self._close(self.entropy, ent, 2.0 ** -18 * (1 + lnv), good)
        assert bool(torch.isnan(self.entropy[~good]).all())
        if self.k == 0:
            assert bool((self.ids == -7).all()) and bool((self.top == FILL).all())
            return
        order = torch.sort(self.logits, dim=-1, descending=True, stable=True).indices[:, :self.k]
        assert torch.equal(self.ids[good].long(), order[good])
        best = lp.gather(1, order)
        self._close(self.top, best, 2.0 ** -22 * y.gather(1, order).abs() + 2.0 ** -18, good)
        assert bool((self.ids[~good] == -1).all()) and bool(torch.isnan(self.top[~good]).all())

    @staticmethod
    def _close(got, ref, tol, rows):
        got, ref = got[rows].double(), ref[rows]
        tol = torch.broadcast_to(torch.as_tensor(tol, device="cuda"), (len(rows),) + ref.shape[1:])[rows] \
            if not torch.is_tensor(tol) else tol[rows]
        inf = torch.isinf(ref)
        assert torch.equal(got[inf], ref[inf])
        err = (got - ref).abs()[~inf] - tol[~inf] - 2.0 ** -24 * ref.abs()[~inf]
        assert err.numel() == 0 or float(err.max()) <= 0, float(err.max())


def rand(M, V, seed=0, amp=3.0):
    return torch.randn(M, V, generator=torch.Generator().manual_seed(seed)) * amp


@pytest.mark.parametrize("M,V", [(1, 1), (3, 2), (5, 40), (33, 1021), (2, 4097), (300, 32000), (1, 151936), (9, 151937),
                                 (160, 50001), (700, 130)])
@pytest.mark.parametrize("k", [0, 1, 5, 32])
def test_rows(M, V, k):
    p = Scores(rand(M, V, V + k), min(k, V), T=0.8)
    p.run()
    p.check()


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("V", [5, 1022, 20003])
def test_alignment(offset, V):
    """Rows that begin anywhere; what lies beside a row is NaN or another row's."""
    p = Scores(rand(7, V), 5, offset=offset)
    p.run()
    p.check()


@pytest.mark.parametrize("T", [1e-3, 0.5, 1.0, 7.0, 1e4])
def test_temperatures(T):
    p = Scores(rand(5, 5000, 3), 20, T=T)
    p.run()
    p.check()


@pytest.mark.parametrize("V", [1000, 70000])
@pytest.mark.parametrize("kind", ["ascending", "descending", "equal", "zeros of both signs", "few values", "one large"])
def test_orders_and_ties(V, kind):
    """Equal logits go by their index; sorted rows make every element a candidate."""
    x = {"ascending": torch.arange(V).float() * 0.01, "descending": -torch.arange(V).float() * 0.01,
         "equal": torch.full((V,), 2.5), "zeros of both signs": torch.where(torch.arange(V) % 3 == 0, -0.0, 0.0),
         "few values": torch.randint(0, 4, (V,), generator=torch.Generator().manual_seed(1)).float(),
         "one large": torch.where(torch.arange(V) == V - 2, 90.0, 0.0)}[kind]
    for k in (1, 20, 32):
        p = Scores(x.expand(3, V).contiguous(), k)
        p.run()
        p.check()


@pytest.mark.parametrize("V", [300, 152000])
@pytest.mark.parametrize("left", [1, 3, 31, 100])
def test_masked_vocabularies(V, left):
    """Rows where few tokens are allowed, fewer than alternatives asked for."""
    x = torch.full((4, V), -INF)
    g = torch.Generator().manual_seed(left)
    for m in range(4):
        at = torch.randperm(V, generator=g)[:left]
        x[m, at] = torch.randn(left, generator=g)
    p = Scores(x, 32)
    p.run()
    p.check()


@pytest.mark.parametrize("V", [100, 40000])
def test_extreme_logits(V):
    x = rand(4, V, 5)
    x[0, 17] = 3e38
    x[1] = -3e38
    x[2] *= 1e30
    x[3] = -3.4028234663852886e38
    p = Scores(x, 8, T=1.0)
    p.run()
    p.check()


@pytest.mark.parametrize("V", [100, 40000])
def test_rows_that_are_no_distribution(V):
    x = rand(6, V, 6)
    x[1, V - 1] = NAN
    x[2, 3] = INF
    x[4] = -INF
    p = Scores(x, 8)
    p.run()
    p.check(status=D.DFLASH_ERR_NUMERIC)


@pytest.mark.parametrize("V", [5, 33, 40000])
def test_rows_of_nan_of_either_sign(V):
    """All of a row NaN, or all but one element: every alternative says so."""
    x = rand(4, V, 7)
    x[0] = -NAN
    x[1] = NAN
    x[2] = torch.copysign(torch.full((V,), NAN), torch.tensor(-1.0))
    x[2, 1] = 1.0
    p = Scores(x, 5)
    p.run()
    p.check(status=D.DFLASH_ERR_NUMERIC)


def test_tokens():
    p = Scores(rand(5, 1000), 3, tokens=[0, 999, -1, 5, -1])
    p.run()
    p.check()
    for bad in (1000, -2, 2 ** 31 - 1):
        p = Scores(rand(3, 1000), 3, tokens=[1, bad, 2])
        p.run()
        p.check(status=D.DFLASH_ERR_INVALID_ARG)


def test_outputs_are_optional():
    x = rand(4, 3000)
    full = Scores(x, 4)
    full.run()
    for drop in (("tokens", "logprob"), ("entropy",), ("tokens", "logprob", "entropy"), ()):
        p = Scores(x, 4)
        for f in drop:
            setattr(p.a, f, 0)
        if not drop:
            p.a.topk, p.a.top_ids, p.a.top_logprobs = 0, 0, 0
        p.run()
        torch.cuda.synchronize()
        assert "entropy" in drop or torch.equal(p.entropy, full.entropy)
        assert "logprob" in drop or torch.equal(p.logprob, full.logprob)
        assert not drop or (torch.equal(p.ids, full.ids) and torch.equal(p.top, full.top))


def test_past_2_to_31_elements():
    """More than 2^31 logits in a call."""
    M, V = 15000, 151936
    x = torch.zeros(M, V, device="cuda")
    x[M - 1, V - 1] = 20.0
    p = Scores(x[:1], 2, tokens=[0])
    a, keep = p.a, [torch.full((M,), FILL, device="cuda"), torch.zeros(M, 2, dtype=torch.int32, device="cuda"),
                    torch.zeros(M, 2, device="cuda")]
    a.n_rows, a.logits, a.tokens, a.logprob = M, ptr(x), 0, 0
    a.entropy, a.top_ids, a.top_logprobs = (ptr(t) for t in keep)
    p.run()
    torch.cuda.synchronize()
    assert p.ws.status() == D.DFLASH_OK
    assert (keep[1][:-1].cpu() == torch.tensor([0, 1], dtype=torch.int32)).all()
    assert keep[1][-1].tolist() == [V - 1, 0]
    assert float((keep[0][:-1].double() - math.log(V)).abs().max()) < 1e-4


def test_repeats_and_replays():
    p = Scores(rand(6, 151936, 9), 20)
    p.run()
    torch.cuda.synchronize()
    first = [x.clone() for x in (p.logprob, p.entropy, p.ids, p.top)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (p.logprob, p.entropy, p.ids, p.top)))
    p.logits.copy_(rand(6, 151936, 10))
    g.replay()
    p.check()


@pytest.mark.parametrize("M,V", [(1, 50), (3, 1021), (1, 151936), (40, 151936), (200, 32000), (400, 5000)])
@pytest.mark.parametrize("shift", [6.0, 14.0, 30.0, 60.0])
def test_nearly_certain_tokens(M, V, shift):
    """The most likely token's log probability is small, and right to its last
    bits all the same: ln(1 + r), r the others' weights, each off by 2 (|y| + 4)
    2^-24 for its argument and 2^-22 for the exponential; their sums add a
    rounding a term, at most V / 1024 + 64 in a row in halves of a thread's
    elements, warps and clusters; 2^-22 for the logarithm."""
    g = torch.Generator().manual_seed(V + M)
    x = torch.randn(M, V, generator=g)
    at = torch.randint(0, V, (M,), generator=g)
    x[torch.arange(M), at] += shift + math.log(V)
    p = Scores(x.cuda(), k=1, tokens=at.tolist())
    p.run()
    p.check()
    # (not by log_softmax, which rounds 1 + r at 2^-53: 2e-16 where ln(1 + r) is 5e-14)
    rel = p.logits.double() - p.logits.double().amax(-1, keepdim=True)
    lp = -torch.log1p(rel.exp().scatter(1, at.cuda()[:, None], 0.0).sum(-1))
    y = 2 * (shift + math.log(V) + 12) * 1.45
    tol = lp.abs() * (2 * (y + 4) * 2.0 ** -24 + 2.0 ** -21 + (V / 1024 + 64) * 2.0 ** -24) + 2.0 ** -126
    for got in (p.logprob, p.top[:, 0]):
        assert bool(((got.double() - lp).abs() <= tol).all()), float(((got.double() - lp).abs() / tol).max())


@pytest.mark.parametrize("n", [1, 2, 3])
def test_equal_largest_logits_of_any_size(n):
    """One, two or three tokens share the row, the rest has no weight."""
    for big in (0.0, 80.0, -3.4028234663852886e38):
        x = torch.full((4, 3000), -INF, device="cuda")
        for r in range(4):
            x[r, [7 + r, 1500, 2999][:n]] = big
        p = Scores(x, k=3, tokens=[7, 8, 9, 10])
        p.run()
        p.check()
        assert torch.equal(p.logprob.cpu(), torch.full((4,), -math.log(n)))
