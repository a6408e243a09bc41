"""dflash_tree_attention held to fp32-like weights: cancelling values, so that
the output's own rounding does not cover the weights' errors."""
import numpy as np
import pytest
import torch

from tests import tree_ref as R
from tests.test_gpu_tree_attn import FILL, PAD, TYPES, Tree, trees

pytestmark = pytest.mark.gpu


def rel_bound(p, s, i):
    """Row i's bound, per query head: the relative error of a weight p_j / sum, plus what
    the sum over p_j v_j adds to it (against sum_j p_j |v_j|):
      score        fp32 sums of d products of each operand's one or two parts:
                   at most 4 d additions and 8 roundings of scaling and
                   argument, each 2^-23 of sum |q k| scale (truncation counted);
                   with an 8-bit cache also queries' and tree keys' elements
                   held to 2^-10 of a scale that takes their largest to 224 at
                   least;
      exponential  2^-22, twice (weight and sum);
      split        hi + lo of a weight in bf16: 2^-8 of 2^-8;
      sums         n weights, 2 n products: 2^-23 each;
      rescalings   eight roundings of 2^-23: 2^-20."""
    n, grp, sc = p.lens[s] + p.rows, p.nq // p.nkv, p.scale or p.d ** -0.5
    see = sorted(R.sees(p.parents[s])[i])
    q = p.q[s * p.rows + i].double().view(p.nq, p.d).abs()
    kb = p.kb[s * p.rows:(s + 1) * p.rows].double().abs()[see]  # [visible][nkv][d]
    k = torch.cat([p.ctx["k"][s].double().abs(), kb.transpose(0, 1)], 1).repeat_interleave(grp, 0)
    eps = (4 * p.d + 8) * 2.0 ** -23 * torch.einsum("hd,hnd->hn", q, k).amax(-1) * sc
    if p.cache == "e4m3" and p.dtype == "bf16":
        dl = 2.0 ** -10 / 224
        kt = kb.transpose(0, 1).repeat_interleave(grp, 0)
        eps = eps + dl * sc * (q.amax(-1) * k.sum(-1).amax(-1) + kt.amax((1, 2)) * q.sum(-1))
    rel = torch.expm1(2 * eps) + 2 * 2.0 ** -22 + 2.0 ** -16 + 3 * n * 2.0 ** -23 + 2.0 ** -20
    return rel.numpy()[:, None]


def check(p, skip=()):
    torch.cuda.synchronize()
    assert p.ws.status() == 0
    got = p.out.cpu().double().view(p.S, p.rows, p.nq, p.d).numpy()
    sc = p.scale or p.d ** -0.5
    rnd = 2.0 ** -8 if p.dtype == "bf16" else 2.0 ** -24
    for s in range(p.S):
        sl = slice(s * p.rows, (s + 1) * p.rows)
        out, mag, _ = R.attention(p.q[sl].double().view(p.rows, p.nq, p.d).numpy(), p.ctx["k"][s].double().numpy(),
                                  p.ctx["v"][s].double().numpy(), p.kb[sl].double().numpy(), p.vb[sl].double().numpy(),
                                  p.parents[s], sc)
        for i in range(p.rows):
            if (s, i) in skip:
                continue
            if np.isnan(out[i]).all():
                assert (got[s, i] == FILL).all(), (s, i, "a padding row was written")
                continue
            tol = (rnd * np.abs(out[i]) + rel_bound(p, s, i) * mag[i]) * (1 + rnd)
            err = np.abs(got[s, i] - out[i])
            assert (err <= tol).all(), (s, i, float((err / tol).max()))


def cancel(p):
    """Slots 2 j + 1 of every context repeat 2 j with one dimension of the key
    negated (another, near weight) and the value negated; small tree values."""
    for x, dims in (("k", [5]), ("v", list(range(p.d)))):
        t = p.dev[x]
        for s, n in enumerate(p.lens):
            m = n // 2 * 2
            a = t[s, :, 0:m:2].clone()
            if t.dtype == torch.uint8:
                a[..., dims] ^= 128
                p.dev[x + "e"][s, :, 1:m:2] = p.dev[x + "e"][s, :, 0:m:2]
            else:
                a[..., dims] = -a[..., dims]
            t[s, :, 1:m:2] = a
            b = p.ctx[x][s][:, 0:m:2].clone()
            b[..., dims] = -b[..., dims]
            p.ctx[x][s][:, 1:m:2] = b
    p.vb = (p.vb.float() * 2.0 ** -6).to(p.dt)
    p.vb_d.copy_(p.vb)


CACHES = ["bf16", "e4m3"]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nkv,rows", [(8, 2, 5), (16, 2, 17), (7, 1, 40), (4, 4, 33)])
def test_weights_keep_their_digits(cache, d, nq, nkv, rows):
    p = Tree([2, 6, 20, 44, 0], trees(d + nq, [rows, 1, rows, max(1, rows - 2), 3], rows), nq, nkv, d, "bf16", cache,
             q_amp=0.1, seed=rows)
    cancel(p)
    p.run()
    check(p)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("nq,rows", [(4, 9), (16, 33)])
def test_weights_keep_their_digits_over_many_chunks(cache, nq, rows):
    """Contexts cut into pieces of several CTAs, joined from their partials."""
    p = Tree([130, 1400, 260], trees(nq, [rows] * 3, rows), nq, 2, 128, "bf16", cache, q_amp=0.1, seed=rows)
    cancel(p)
    p.run()
    check(p)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("nq,rows", [(4, 9), (16, 33)])
def test_scores_that_move_the_reference(cache, nq, rows):
    """Scores of a few hundred, growing along the context: the reference of the
    weights moves, and with it what is already summed."""
    p = Tree([400, 261], trees(nq + 1, [rows] * 2, rows), nq, 2, 64, "bf16", cache, q_amp=4.0, scale=0.5, seed=rows)
    p.run()
    check(p)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("nq,rows", [(4, 9), (16, 33)])
def test_values_of_very_different_size(dtype, cache, nq, rows):
    """Rows of V between 2^-25 and 2^25 times the others', those of the tree
    too: every row counts by its weight times its own size."""
    p = Tree([0, 3, 200, 390], trees(nq, [rows] * 4, rows), nq, 2, 64, dtype, cache, q_amp=3.0, seed=rows)
    g = torch.Generator().manual_seed(rows)
    for s, n in enumerate(p.lens):
        t = torch.randint(-25, 26, (2, n), generator=g)
        p.ctx["v"][s] = p.ctx["v"][s].double() * torch.exp2(t.double())[..., None]
        if cache == "e4m3":
            p.dev["ve"][s, :, :n] = (p.dev["ve"][s, :, :n].int() + t.cuda()).to(torch.uint8)
        else:
            p.dev["v"][s, :, :n] *= torch.exp2(t.float()).cuda()[..., None].to(p.dt)
    t = torch.randint(-25, 26, (len(p.vb), 2, 1), generator=g)
    p.vb = (p.vb.float() * torch.exp2(t.float())).to(p.dt)
    p.vb_d.copy_(p.vb)
    p.run()
    check(p)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("big", [1e30, -1e30, 3e4])
@pytest.mark.parametrize("nq", [4, 64])
def test_large_finite_rows_reach_their_descendants_only(dtype, cache, big, nq):
    """Padding rows and rows of other branches may hold any finite number."""
    par = [-1, 0, 0, 1, 2, 2, PAD]
    p = Tree([130, 0], [par, par], nq, 2, 128, dtype, cache)
    for s in (0, 1):
        for i in (2, 6):  # seen by 2, 4, 5; padding
            for t in (p.kb, p.kb_d):
                t[s * 7 + i] = big
            for t in (p.vb, p.vb_d):
                t[s * 7 + i, :, 3:70] = big
    p.run()
    check(p, skip=[(s, i) for s in (0, 1) for i in (2, 4, 5)])
    for s in (0, 1):  # the values alone: their descendants too
        for t in (p.kb, p.kb_d):
            t[s * 7 + 2] = 0.25
    p.run()
    check(p)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("nq,rows", [(4, 9), (64, 9)])
@pytest.mark.parametrize("q,k", [(0.0, 0.0), (1e-20, 0.0), (1e-25, 1e-25), (0.0, 1.0), (1.0, 0.0), (2.0 ** -126, 2.0 ** -126)])
def test_zero_and_tiny_queries_and_keys(dtype, cache, nq, rows, q, k):
    """A head whose queries are (next to) zero weighs what it sees alike, and
    no hidden or padding row changes that."""
    p = Tree([0, 1, 140], trees(nq, [rows, 2, 5], rows), nq, 2, 64, dtype, cache)
    for t in (p.q, p.q_d):
        t.view(-1, nq, 64)[:, 1] *= q
    for t in (p.kb, p.kb_d):
        t *= k
    p.run()
    check(p)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("nq,rows", [(4, 9), (16, 33), (16, 128)])
def test_large_values_under_large_scores(dtype, cache, nq, rows):
    """Every score near 50 ln 2, values near 2^85: weights against the
    reference 0 would leave fp32's range, the output is far inside it."""
    p = Tree([0, 0], trees(nq, [rows] * 2, rows), nq, 2, 64, dtype, cache, seed=rows)
    for t in (p.q, p.q_d, p.kb, p.kb_d):
        t.copy_(t.abs() * 0.5 + 0.5)
    for t in (p.vb, p.vb_d):
        t *= 2.0 ** 85
    p.scale = p.a.scale = float(np.float32(50 * np.log(2) / (0.9 * 0.9 * 64)))
    p.run()
    check(p)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq,nkv", [(16, 8), (56, 8), (64, 1)])
def test_many_short_items_per_cta(cache, nq, nkv):
    """More items than CTAs, most of them a chunk or two: every buffer of a
    CTA's run is used many times over.  Twice, with the same bits."""
    rng = np.random.default_rng(nq)
    lens = [int(x) for x in rng.choice([0, 0, 1, 30, 128, 129, 300], 320)]
    p = Tree(lens, trees(nq, [int(x) for x in rng.integers(1, 4, 320)], 3), nq, nkv, 64, "bf16", cache, seed=nq)
    p.run()
    check(p)
    first = p.out.clone()
    p.out.fill_(FILL)
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(first, p.out)


def paged_values(c):
    """Values that tell slots apart: slot j of a chunk holds 2^chunk in column j, keys 0, so that
    every column of the output is the sum of what the chunks' slots hold."""
    S, rows, nq, nkv, d = c["S"], c["rows"], c["nq"], c["nkv"], c["d"]
    p = Tree(c["lens"], [list(range(-1, rows - 1))] * S, nq, nkv, d, "bf16", "e4m3", page=128, cap=384, chain=True)
    eye = torch.eye(128, d)
    p.dev["k"].zero_()
    p.dev["ve"].fill_(127)
    for s in range(S):
        for ch in range(3):
            p.dev["v"][p.pages[s, ch]] = (eye * 2.0 ** ch).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    for t in (p.kb, p.kb_d, p.vb, p.vb_d):
        t.zero_()
    return p


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,rows", [(32, 64), (32, 8)])
def test_every_chunk_brings_its_own_values(d, nq, rows):
    """A chunk's values stay until they have been read, however soon the next
    ones come (again and again, with a cache that lies in L2)."""
    rng = np.random.default_rng(d + rows)
    lens = [int(x) for x in rng.choice([0, 1, 128, 129, 256, 257, 300, 384], 33)]
    p = paged_values(dict(S=33, rows=rows, nq=nq, nkv=8, d=d, lens=lens))
    want = torch.zeros(33, rows, d, dtype=torch.float64)
    for s, n in enumerate(lens):
        for j in range(n):
            if j % 128 < d:
                want[s, :, j % 128] += 2.0 ** (j // 128)
        want[s] /= torch.arange(n + 1, n + rows + 1)[:, None]
    want = want[:, :, None].expand(33, rows, nq, d)
    # equal weights: at most 2^-8 of the value in the output's rounding, 2^-16 and the sum's 512 2^-23 before
    tol = want * (2.0 ** -8 + 2.0 ** -16 + 512 * 2.0 ** -23) * (1 + 2.0 ** -8)
    want, tol = want.cuda(), tol.cuda()
    for _ in range(300):
        p.out.zero_()
        p.run()
        assert bool(((p.out.view(33, rows, nq, d).double() - want).abs() <= tol).all())
    assert p.ws.status() == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq,nkv,rows", [(32, 4, 5), (7, 1, 5), (32, 8, 33), (16, 2, 100)])
def test_same_bits_beside_any_other_rows(cache, nq, nkv, rows):
    """Tiles that are filled in part: the bits of a row depend neither on what
    shared memory held nor on what the padding rows beside it hold."""
    lens = [0, 5, 128, 201, 300, 142] * 4
    n = max(1, rows - 2)
    p = Tree(lens, trees(rows, [n] * 24, rows), nq, nkv, 128, "bf16", cache, seed=rows)
    p.run()
    check(p)
    first = p.out.clone()
    other = Tree(lens, trees(rows, [rows] * 24, rows), nq, nkv, 128, "bf16", cache, seed=rows + 1, q_amp=50.0)
    pad = torch.zeros(24, rows, dtype=torch.bool)
    pad[:, n:] = True
    pad = pad.view(-1).cuda()
    for fill in (None, 1e30, float("nan"), float("inf"), 1e-30):
        other.run()  # (leaves other scales and scores behind)
        if fill is not None:
            for t in (p.q_d, p.kb_d, p.vb_d):
                t[pad] = fill
        p.out.fill_(FILL)
        p.run()
        torch.cuda.synchronize()
        assert torch.equal(first, p.out), (fill, torch.nonzero((first != p.out).any(1)).flatten().tolist())
    assert p.ws.status() == 0
