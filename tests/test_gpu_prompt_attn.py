"""dflash_prompt_attention against a plain 64-bit implementation."""
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests.prompt_ref import FILL, Prompt, attend, half_step, weight_error

pytestmark = pytest.mark.gpu

DTYPES = ["f32", "bf16"]
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nkv", [(4, 4), (8, 2), (7, 1), (16, 2), (10, 2), (3, 1)])
def test_ragged(dtype, d, nq, nkv):
    """Lengths around the borders of tiles and chunks, empty sequences among them."""
    p = Prompt([1, 2, 0, 31, 32, 33, 64, 0, 65, 127, 128, 129, 200, 257, 0], nq, nkv, d, dtype, seed=nq + d)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [0, 128, 256])
@pytest.mark.parametrize("nq,nkv,d", [(8, 2, 128), (4, 4, 64), (14, 2, 128)])
def test_context(dtype, page, nq, nkv, d):
    """Rows behind a cached context; slots behind it and unused pages hold NaN."""
    ctx = [0, 1, 127, 128, 129, 300, 511, 640, 3, 77]
    p = Prompt([5, 1, 64, 130, 1, 33, 2, 100, 0, 300], nq, nkv, d, dtype, ctx=ctx, page=page, seed=page + d)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ctx", [None, 333])
def test_single_tokens(dtype, ctx):
    """One token a sequence, as in decoding."""
    p = Prompt([1] * 40, 8, 2, 128, dtype, ctx=None if ctx is None else [(i * 37) % ctx for i in range(40)])
    p.run()
    p.check()


@pytest.mark.parametrize("dtype,lens", [("bf16", [5000]), ("bf16", [1, 1500, 40, 2500, 7]), ("f32", [700, 900]),
                                        ("bf16", [128, 256, 384, 512])])
def test_long(dtype, lens):
    p = Prompt(lens, 8, 2, 128, dtype, seed=len(lens))
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_context_few_rows(dtype):
    """Work split over a long context and joined."""
    p = Prompt([1, 3], 8, 1, 64, dtype, ctx=[9000, 20001], page=128)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_no_sequence(dtype, d):
    """Rows before the first and behind the last sequence hold NaN, and their outputs stay."""
    p = Prompt([3, 70, 129], 8, 2, d, dtype, ctx=[0, 130, 64], lead=5, tail=77)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("nq,nkv", [(4, 4), (8, 2)])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_values_that_later_rows_hold(dtype, nq, nkv, bad):
    """A NaN or infinite value reaches the rows that see it and no other."""
    p = Prompt([200, 64, 300], nq, nkv, 64, dtype, seed=5)
    for row, g, e in ((150, 0, 3), (199, nkv - 1, 60), (200 + 10, 0, 0), (264 + 128, 0, 17), (264 + 299, nkv - 1, 1)):
        p.vb[row, g, e] = bad
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_keys_that_later_rows_hold(dtype):
    """A NaN key or an infinite one spoils the rows that see it and no other."""
    p = Prompt([200, 300], 8, 2, 64, dtype, seed=6)
    p.kb[150, 0, 3] = NAN
    p.kb[200 + 130, 1, :] = INF
    p.run()
    torch.cuda.synchronize()
    fine = torch.isfinite(p.out)
    assert fine[:150].all() and fine[150:200, 4:].all() and not fine[150:200, :4].any()
    assert fine[200:330].all() and fine[330:, :4].all() and not fine[330:, 4:].any()
    clean = Prompt([200, 300], 8, 2, 64, dtype, seed=6)
    clean.run()
    torch.cuda.synchronize()
    assert torch.equal(clean.out[fine], p.out[fine])


@pytest.mark.parametrize("dtype", DTYPES)
def test_infinite_value_in_the_context(dtype):
    p = Prompt([40], 8, 2, 128, dtype, ctx=[300])
    p.vc[0, 1, 299, 7] = INF
    p.vc[0, 0, 5, 8] = NAN
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("amp,scale", [(40.0, 0.0), (1.0, 3.0), (1e-4, 0.0), (0.0, 0.0)])
def test_scores_of_any_size(dtype, amp, scale):
    p = Prompt([100, 257, 3], 8, 2, 128, dtype, ctx=[140, 0, 60], q_amp=amp, scale=scale, seed=8)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [-300.0, 300.0, 60.0])
def test_all_scores_far_from_zero(dtype, shift):
    """Scores that share a large part, of either sign: the reference leaves 0."""
    p = Prompt([100, 200], 4, 2, 64, dtype, ctx=[150, 0], seed=9)
    p.q[:, :, 0] = 8 * shift / 8
    p.kb[:, :, 0] = 8.0
    p.kc[0, :, :150, 0] = 8.0
    p.run()
    p.check()


@pytest.mark.parametrize("growth", [1.0, -1.0])
def test_scores_that_grow_along_the_keys(growth):
    """Each chunk outgrows the one before (or vanishes beside it)."""
    p = Prompt([900], 4, 4, 64, "bf16", seed=10)
    p.q[:, :, 0] = 16.0
    p.kb[:, :, 0] = growth * torch.arange(900, device="cuda").bfloat16()[:, None] / 4
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_cancelling_values(dtype):
    """Values that cancel: an output far smaller than its terms."""
    p = Prompt([256, 200], 8, 2, 64, dtype, q_amp=0.05, seed=11)
    sign = torch.where(torch.arange(456, device="cuda") % 2 == 0, 1.0, -1.0)
    p.vb.copy_((p.vb.float() * 1e-3 + 50 * sign[:, None, None]).to(p.dt))
    p.run()
    p.check()


def test_values_of_any_size():
    p = Prompt([300, 150], 8, 2, 128, "bf16", ctx=[200, 0], seed=12)
    size = torch.randint(-60, 60, p.vb.shape, generator=torch.Generator().manual_seed(12)).float()
    p.vb *= torch.exp2(size).cuda().bfloat16()
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S", [700])
def test_many_short_sequences(dtype, S):
    lens = [(7 * i) % 5 for i in range(S)]
    p = Prompt(lens, 4, 2, 64, dtype, ctx=[(11 * i) % 40 for i in range(S)], seed=13)
    p.run()
    p.check()


@pytest.mark.parametrize("nq,nkv", [(128, 1), (100, 1), (48, 1)])
def test_wide_groups(nq, nkv):
    for dtype in DTYPES:
        p = Prompt([3, 140], nq, nkv, 64, dtype, ctx=[130, 0], seed=14)
        p.run()
        p.check()


def test_pages_past_2_to_31_elements():
    """A page pool of more than 2^32 bytes, with sequences on its last pages."""
    pool, nkv, d = 17000, 8, 128
    p = Prompt([70, 5], 16, nkv, d, "bf16", ctx=[300, 129], page=128, spare=pool, seed=15)
    assert p.kc.numel() > 2 ** 31
    last = torch.arange(p.pool - p.pages.numel(), p.pool, device="cuda", dtype=torch.int32).flip(0).view_as(p.pages)
    for x in (p.kc, p.vc):
        x[last.long()] = x[p.pages.long()].clone()
    p.pages.copy_(last)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("start", [[-3, 40, 90, 150], [0, 40, 90, 151], [0, 120, 20, 150], [0, 150, 0, 150],
                                   [0, 2 ** 31 - 1, -2 ** 31, 5], [160, 170, 180, 190]])
def test_bad_starts_are_reported(dtype, start):
    """Nothing is written, and nothing read out of bounds."""
    p = Prompt([40, 50, 60], 8, 2, 64, dtype, ctx=[10, 20, 30], seed=16)
    p.row_start.copy_(torch.tensor(start, dtype=torch.int32))
    p.run()
    torch.cuda.synchronize()
    assert p.ws.status() == D.DFLASH_ERR_INVALID_ARG
    assert (p.out == FILL).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("base", [-1, 31, 2 ** 31 - 1])
def test_bad_contexts_are_reported(dtype, base):
    """The other sequences are as they would be."""
    p = Prompt([40, 50, 60], 8, 2, 64, dtype, ctx=[10, 20, 30], seed=16)
    p.base[1] = base
    p.run()
    p.check(status=D.DFLASH_ERR_INVALID_ARG, seqs=[0, 2])


@pytest.mark.parametrize("dtype", DTYPES)
def test_unmapped_page_is_reported(dtype):
    p = Prompt([40, 50], 8, 2, 64, dtype, ctx=[200, 300], page=128, seed=18)
    p.pages[1, 1] = p.pool
    p.kc[0], p.vc[0] = 1.0, 1.0  # (page 0 is read instead)
    p.run()
    p.check(status=D.DFLASH_ERR_INVALID_ARG, seqs=[0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_rows_at_all(dtype):
    """Every sequence empty: nothing is written."""
    p = Prompt([0, 0, 0], 8, 2, 64, dtype, ctx=[5, 0, 9], tail=4)
    p.run()
    p.check()
    assert (p.out == FILL).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_repeats_and_replays(dtype):
    """The same bits again, and from a captured graph that two problems share a workspace in."""
    p = Prompt([300, 70, 1], 8, 2, 128, dtype, ctx=[100, 0, 513], seed=19)
    p.run()
    torch.cuda.synchronize()
    first = p.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for _ in range(3):
        p.out.fill_(FILL)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, p.out)
    p.q.copy_(torch.randn(p.q.shape, device="cuda").to(p.dt))
    p.row_start.copy_(torch.tensor([0, 200, 370, 371], dtype=torch.int32))
    p.start, p.lens = [0, 200, 370, 371], [200, 170, 1]
    g.replay()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_two_streams(dtype):
    ps = [Prompt([300 + 7 * i, 70], 8, 2, 128, dtype, seed=20 + i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(5):
        for p, st in zip(ps, streams):
            p.run(st)
    for p in ps:
        p.check()


def test_expired_waits_are_reported():
    """With its K/V copies switched off the call gives up within its limit,
    reports it, and the next one on the same workspace is exact."""
    p = Prompt([300, 70, 1], 8, 2, 128, "bf16", ctx=[100, 0, 513], seed=21)
    D.dflash_workspace_control(p.ws.ptr, p.ws.bytes, wait_limit_ns=2_000_000, stall_kv_loads=True)
    p.run()
    torch.cuda.synchronize()
    assert p.ws.status() == D.DFLASH_ERR_TIMEOUT
    D.dflash_workspace_control(p.ws.ptr, p.ws.bytes)
    p.out.fill_(FILL)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_problems_that_share_a_workspace(dtype):
    """Two captured calls of different lengths in turn on one workspace."""
    ps = [Prompt([400, 3], 8, 2, 64, dtype, seed=22), Prompt([5, 129, 700, 0, 64], 8, 2, 64, dtype, ctx=[0, 7, 300, 9, 128],
                                                             seed=23)]
    big = max(ps, key=lambda p: p.ws.bytes)
    graphs = []
    for p in ps:
        p.ws = big.ws
        p.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run()
        graphs.append(g)
    for p in ps:
        p.out.fill_(FILL)
    for g in graphs * 3:
        g.replay()
    for p in ps:
        p.check()


def test_rows_past_2_to_31_elements():
    """More than 2^31 elements of queries and outputs."""
    p = Prompt([140] * 999 + [300], 128, 8, 128, "bf16", seed=24)
    assert p.q.numel() > 2 ** 31
    p.run()
    p.check(seqs=[0, 1, 500, 998, 999])


@pytest.mark.parametrize("d", [64, 128])
def test_a_very_long_prompt(d):
    """70000 rows: the last ones against the reference."""
    n, few = 70001, 40
    p = Prompt([n], 4, 1, d, "bf16", seed=25)
    p.run()
    torch.cuda.synchronize()
    assert p.ws.status() == D.DFLASH_OK
    out, mag, big = attend(p.q[-few:].double(), p.kb.double(), p.vb.double(), n - few, d ** -0.5)
    tol = half_step(p.dt) * out.abs() + weight_error(d, n, big, p.dt)[..., None] * mag
    assert bool(((p.out[-few:].double() - out).abs() <= tol * (1 + half_step(p.dt))).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ctx", [0, 300, 5000])
def test_rows_whose_scores_are_all_minus_infinity(dtype, ctx):
    """The softmax of nothing but -inf is NaN, in whole items and joined ones;
    the other rows are as they are without."""
    p, clean = (Prompt([90], 4, 2, 64, dtype, ctx=[ctx], seed=26) for _ in range(2))
    for x in (p, clean):
        x.kb[:, 0, 5] = 1.0
        x.kc[0, 0, :, 5] = 1.0
        x.run()
    assert p.out.isfinite().all()
    p.q[60:70, 1, 5] = -INF
    p.run()
    torch.cuda.synchronize()
    assert p.ws.status() == D.DFLASH_OK
    spoiled = torch.zeros(90, 4, dtype=torch.bool, device="cuda")
    spoiled[60:70, 1] = True
    assert bool(p.out[spoiled].isnan().all()) and torch.equal(p.out[~spoiled], clean.out[~spoiled])


FEW = [  # at most a tile's tokens per sequence on average: lens, contexts
    ([1], [0]),
    ([1], [1]),
    ([1] * 40, [37 * i for i in range(40)]),
    ([1, 0, 2, 0, 0, 5, 1], [128, 9, 0, 640, 1, 127, 4000]),
    ([3] * 9 + [90], [1000, 0, 0, 129, 1, 256, 2, 0, 77, 300]),
    ([16, 1, 1, 1, 1, 1, 1, 1], [0, 5000, 0, 0, 0, 700, 0, 0]),
    ([7], [9000]),
]


@pytest.mark.parametrize("nq,nkv,d", [(32, 8, 128), (8, 1, 64), (4, 4, 128), (14, 2, 64)])
@pytest.mark.parametrize("page", [0, 128])
@pytest.mark.parametrize("lens,ctx", FEW)
def test_few_rows_a_sequence(lens, ctx, page, nq, nkv, d):
    """Items of a single tile, whose chunks the streams share out."""
    p = Prompt(lens, nq, nkv, d, "bf16", ctx=ctx, page=page, seed=27)
    p.run()
    p.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_few_rows_with_values_that_later_rows_hold(bad, d):
    p = Prompt([16, 1, 9, 2, 100, 3, 1, 1, 1, 1], 4, 1, d, "bf16", ctx=[0, 300, 128, 0, 250, 7, 0, 900, 2, 0], seed=28)
    for row, e in ((9, 3), (15, 0), (20, 17), (28 + 60, 5), (28 + 99, 1), (130, 40)):
        p.vb[row, 0, e] = bad
    p.vc[4, 0, 249, 9] = bad
    p.vc[7, 0, 3, 9] = bad
    p.run()
    p.check()


def test_few_rows_captured_and_replayed():
    """The same bits from every replay."""
    p = Prompt([1] * 30 + [20], 8, 2, 128, "bf16", ctx=[200 * i for i in range(31)], seed=29)
    p.run()
    torch.cuda.synchronize()
    first = p.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for _ in range(5):
        p.out.fill_(FILL)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.out, first)
    assert p.ws.status() == D.DFLASH_OK


def test_few_rows_expired_waits_are_reported():
    p = Prompt([1, 1, 20], 8, 2, 128, "bf16", ctx=[100, 0, 1513], seed=30)
    D.dflash_workspace_control(p.ws.ptr, p.ws.bytes, wait_limit_ns=2_000_000, stall_kv_loads=True)
    p.run()
    torch.cuda.synchronize()
    assert p.ws.status() == D.DFLASH_ERR_TIMEOUT
    D.dflash_workspace_control(p.ws.ptr, p.ws.bytes)
    p.out.fill_(FILL)
    p.run()
    p.check()


@pytest.mark.parametrize("nq,nkv,d", [(32, 8, 128), (8, 1, 64), (14, 2, 128)])
@pytest.mark.parametrize("lens,ctx", [([200], [9000]), ([100, 0, 70], [5000, 77, 12000])])
def test_items_that_many_ctas_share(lens, ctx, nq, nkv, d):
    """Two tiles an item, joined by a kernel of their own; rows of no sequence stay."""
    p = Prompt(lens, nq, nkv, d, "bf16", ctx=ctx, lead=3, tail=50, seed=31)
    p.vb[3 + 60, 0, 5] = NAN
    p.run()
    p.check()
    first = p.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for _ in range(3):
        p.out.fill_(FILL)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first.isnan(), p.out.isnan()) and torch.equal(first.nan_to_num(), p.out.nan_to_num())
