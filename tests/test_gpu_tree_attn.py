"""dflash_tree_attention against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests import tree_ref as R

pytestmark = pytest.mark.gpu

PAD = D.DFLASH_TREE_PAD
FILL = 3.0  # what outputs hold before a call


class Tree:
    """One tree attention problem on the device."""

    def __init__(self, lens, parents, nq, nkv, d, dtype="bf16", cache=None, page=0, cap=None, chain=False, scale=0.0,
                 seed=0, garbage=True, q_amp=1.0):
        g = torch.Generator().manual_seed(seed)
        cache = cache or dtype
        S, rows = len(lens), len(parents[0])
        self.S, self.rows, self.nq, self.nkv, self.d, self.dtype, self.cache = S, rows, nq, nkv, d, dtype, cache
        self.lens, self.parents, self.scale = lens, [list(range(-1, rows - 1))] * S if chain else parents, scale
        unit = page or 1
        cap = cap or -(-max(max(lens), 1) // unit) * unit
        dt = self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        rnd = lambda *s: torch.randn(*s, generator=g)
        self.q = (rnd(S * rows, nq * d) * q_amp).to(dt)
        self.kb, self.vb = rnd(S * rows, nkv, d).to(dt), rnd(S * rows, nkv, d).to(dt)
        # contexts [S][nkv][n][d] as the cache holds them, and the cache around them
        self.pages, self.pool = None, 0
        if page:
            self.pool = S * (cap // page) + 3
            self.pages = torch.randperm(self.pool, generator=g)[:S * (cap // page)].view(S, -1).int()
            shape = (self.pool, nkv, page, d)
        else:
            shape = (S, nkv, cap, d)
        self.page, self.cap = page, cap
        self.ctx, self.dev = {}, {}
        for x in "kv":
            full = rnd(*shape) * (torch.rand(shape[:-1] + (1,), generator=g) * 3 + 0.25)
            if cache == "e4m3":
                e = (torch.ceil(torch.log2(full.abs().amax(-1) / 448)) + 127).to(torch.uint8)
                c = (full * torch.exp2(127 - e.float()).unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
                val = torch.from_numpy(R.value_rows(c.numpy(), e.numpy()))
            else:
                c, e = full.to(dt), None
                val = c.double()
            self.ctx[x] = [self._rows(val, s, lens[s]).clone() for s in range(S)]
            if garbage:  # slots no sequence reaches hold NaN
                used = torch.zeros(shape[:-1], dtype=torch.bool)
                for s in range(S):
                    for a in range(lens[s]):
                        i, o = (int(self.pages[s, a // page]), a % page) if page else (s, a)
                        used[i, :, o] = True
                if cache == "e4m3":
                    c[~used] = 127
                    e[~used] = 255
                else:
                    c[~used] = float("nan")
            self.dev[x] = c.cuda()
            self.dev[x + "e"] = None if e is None else e.cuda()
        self.out = torch.full((S * rows, nq * d), FILL, dtype=dt, device="cuda")
        self.base = torch.tensor(lens, dtype=torch.int32).cuda()
        self.parent = None if chain else torch.tensor(parents, dtype=torch.int32).cuda()
        self.q_d, self.kb_d, self.vb_d = self.q.cuda(), self.kb.cuda(), self.vb.cuda()
        self.pages_d = None if self.pages is None else self.pages.cuda()
        a = self.a = D.dflash_tree_attention_args()
        a.dims = R.dims(nq, nkv, d, dtype)
        a.n_seqs, a.rows, a.max_pos, a.scale = S, rows, cap, scale
        a.base_pos, a.parent = R.ptr(self.base), R.ptr(self.parent)
        a.q, a.kb, a.vb, a.out = R.ptr(self.q_d), R.ptr(self.kb_d), R.ptr(self.vb_d), R.ptr(self.out)
        a.kv = R.kv_desc(cap, self.dev["k"], self.dev["v"], self.dev["ke"], self.dev["ve"], self.pages_d, page, self.pool)
        self.ws = R.Workspace(D.DFLASH_OP_TREE_ATTENTION, a)

    def _rows(self, full, s, n):
        if not self.page:
            return full[s, :, :n]
        ids = self.pages[s, :-(-n // self.page)].long()
        return full[ids].transpose(0, 1).flatten(1, 2)[:, :n]

    def run(self):
        D.dflash_tree_attention(self.a, self.ws.ptr, self.ws.bytes)

    def check(self, status=D.DFLASH_OK, skip=(), seqs=None):
        """Bounds, per element: the output's rounding (half a step), and the
        weights' errors against A = sum_j p_j |v_j|: twice the score error
        (fp32 sums of d products: (d + 4) 2^-24 of sum |q k| scale), 2^-20 for
        the exponential and the products' scales, n 2^-24 for the sum of n
        weights, and the rounding of the weights in the tensor-core product
        (2^-8 bf16; 2^-11 fp16 with an 8-bit cache; none in fp32)."""
        torch.cuda.synchronize()
        assert self.ws.status() == status
        got = self.out.cpu().double().view(self.S, self.rows, self.nq, self.d).numpy()
        sc = self.scale or 1 / np.sqrt(self.d)
        rnd_out = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -24
        rnd_p = 0.0 if self.dtype == "f32" else 2.0 ** -8
        worst = 0.0
        for s in range(self.S) if seqs is None else seqs:
            sl = slice(s * self.rows, (s + 1) * self.rows)
            out, mag, big = R.attention(self.q[sl].double().view(self.rows, self.nq, self.d).numpy(),
                                        self.ctx["k"][s].double().numpy(), self.ctx["v"][s].double().numpy(),
                                        self.kb[sl].double().numpy(), self.vb[sl].double().numpy(), self.parents[s], sc)
            for i in range(self.rows):
                if (s, i) in skip:
                    continue
                if np.isnan(out[i]).all():
                    assert (got[s, i] == FILL).all(), (s, i, "a padding row was written")
                    continue
                n = self.lens[s] + self.rows
                rel = np.expm1(2 * (self.d + 4) * 2.0 ** -24 * big) + 2.0 ** -20 + n * 2.0 ** -24 + rnd_p
                tol = (rnd_out * np.abs(out[i]) + rel * mag[i]) * (1 + rnd_out)
                err = np.abs(got[s, i] - out[i])
                assert (err <= tol).all(), (s, i, float((err - tol).max()), float((err / tol).max()))
                worst = max(worst, float((err / tol).max()))
        return worst


def trees(seed, ns, rows=None, levels=16):
    rng = np.random.default_rng(seed)
    rows = rows or max(ns)
    return [R.random_tree(rng, n, levels, rows) for n in ns]


TYPES = [("f32", "f32"), ("f32", "e4m3"), ("bf16", "bf16"), ("bf16", "e4m3")]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nkv", [(4, 4), (8, 2), (7, 1), (16, 2)])
def test_ragged_trees(dtype, cache, d, nq, nkv):
    """Odd contexts around chunk borders, ragged trees with padding rows."""
    p = Tree([0, 1, 127, 128, 129, 300], trees(d + nq, [1, 5, 13, 17, 9, 12], 17), nq, nkv, d, dtype, cache)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("rows", [1, 2, 31, 32, 33, 64, 65, 127, 128])
def test_tree_sizes(dtype, cache, rows):
    p = Tree([70, 261], trees(rows, [rows, rows]), 8, 2, 128, dtype, cache, seed=rows)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("page", [128, 256])
def test_paged(dtype, cache, page):
    p = Tree([5, 600, 255, 256], trees(page, [9, 20, 1, 16], 20), 8, 2, 128, dtype, cache, page=page, cap=768)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_chain_without_parents(dtype, cache):
    p = Tree([200, 3], [[0] * 40] * 2, 4, 1, 64, dtype, cache, chain=True)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_long_context(dtype, cache):
    p = Tree([5003], trees(4, [6]), 4, 2, 128, dtype, cache)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_many_sequences_of_many_lengths(dtype, cache):
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 900, 23)] + [2500, 1]
    p = Tree(lens, trees(5, [int(x) for x in rng.integers(1, 25, 25)], 24), 8, 2, 64, dtype, cache)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("nq,nkv,rows", [(32, 4, 64), (16, 1, 128), (32, 8, 64)])
def test_many_query_rows_per_kv_head(dtype, cache, nq, nkv, rows):
    p = Tree([400, 33], trees(rows, [rows, rows - 3], rows), nq, nkv, 128, dtype, cache)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_large_scores_and_scale(dtype, cache):
    """Scores of a few hundred: one key takes (nearly) all the weight."""
    p = Tree([150, 260], trees(9, [7, 7]), 4, 2, 128, dtype, cache, scale=0.7, q_amp=4.0)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_several_roots_and_bad_parents(dtype, cache):
    parents = [[-1, -1, 1, 0, PAD, 4, -1, 6], [-1, 0, 2, 1, 99, -7, 0, 5]]
    p = Tree([40, 41], parents, 4, 2, 64, dtype, cache)
    p.run()
    p.check(D.DFLASH_ERR_INVALID_ARG)  # row 2 of sequence 1 is its own parent, 99 and -7 are no rows
    p.parents = [[-1] * 8] * 2
    p.parent[:] = -1
    p.run()
    p.check()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_hidden_rows_may_hold_anything(dtype, cache, bad):
    """A node's keys and values reach its descendants only."""
    par = [-1, 0, 0, 1, 2, 2, PAD]
    p = Tree([130, 0], [par, par], 4, 2, 128, dtype, cache)
    for s in (0, 1):  # rows 2 (seen by 2, 4, 5) and 6 (padding)
        for i in (2, 6):
            p.kb_d[s * 7 + i] = bad
            p.vb_d[s * 7 + i, :, 3:70] = bad
    p.run()
    p.check(skip=[(s, i) for s in (0, 1) for i in (2, 4, 5)])
    assert torch.isnan(p.out.view(2, 7, 4, 128)[:, 6].float()).sum() == 0


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_visible_bad_values_are_not_hidden(dtype, cache, bad):
    par = [-1, 0, 0, 1]
    p = Tree([100], [par], 4, 2, 64, dtype, cache)
    p.vb_d[1, 1, 5] = bad  # node 1, KV head 1: seen by rows 1 and 3 of heads 2, 3
    p.run()
    torch.cuda.synchronize()
    o = p.out.float().view(4, 4, 64)
    hit = ~torch.isfinite(o)
    want = torch.zeros_like(hit)
    want[1, 2:, 5] = want[3, 2:, 5] = True
    assert torch.equal(hit, want)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_unmapped_page(dtype, cache):
    p = Tree([300, 200], trees(2, [5, 5]), 4, 2, 128, dtype, cache, page=128)
    p.pages_d[0, 1] = p.pool + 5
    p.run()
    p.check(D.DFLASH_ERR_INVALID_ARG, seqs=[1])
    p.pages_d[0, 1] = p.pages[0, 1]
    p.run()
    p.check()


def test_f32_bits_do_not_depend_on_the_batch():
    lens = [100, 700, 3]
    par = trees(7, [9, 14, 5], 14)
    p = Tree(lens, par, 8, 2, 64, "f32", cap=1024)
    p.run()
    torch.cuda.synchronize()
    for s in range(3):
        one = Tree(lens, par, 8, 2, 64, "f32", cap=1024)
        a = one.a
        a.n_seqs = 1
        off = s * 14
        a.base_pos, a.parent = one.base.data_ptr() + 4 * s, one.parent.data_ptr() + 4 * off
        a.q, a.out = one.q_d[off:].data_ptr(), one.out[off:].data_ptr()
        a.kb, a.vb = one.kb_d[off:].data_ptr(), one.vb_d[off:].data_ptr()
        a.kv.k, a.kv.v = one.dev["k"][s].data_ptr(), one.dev["v"][s].data_ptr()
        one.run()
        torch.cuda.synchronize()
        assert torch.equal(one.out[off:off + 14], p.out[off:off + 14])


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_same_bits_every_time_and_in_a_graph(dtype, cache):
    p = Tree([700, 90, 1300], trees(3, [20, 9, 31], 31), 8, 2, 128, dtype, cache)
    p.run()
    p.check()
    first = p.out.clone()
    for _ in range(3):
        p.out.fill_(FILL)
        p.run()
        torch.cuda.synchronize()
        assert torch.equal(first, p.out)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        p.run()
    p.out.fill_(FILL)
    # the lengths are device data: a replay follows them
    p.base.copy_(torch.tensor([699, 90, 1200], dtype=torch.int32))
    p.ctx = {x: [c[0][:, :699], c[1], c[2][:, :1200]] for x, c in p.ctx.items()}
    p.lens = [699, 90, 1200]
    g.replay()
    p.check()


def test_two_calls_at_once_on_two_streams():
    """Each with its own workspace."""
    ps = [Tree([900, 40 + i], trees(i, [12, 12]), 8, 2, 128, "bf16", seed=i) for i in range(2)]
    torch.cuda.synchronize()
    sts = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for p, st in zip(ps, sts):
            with torch.cuda.stream(st):
                p.run()
    for p in ps:
        p.check()
