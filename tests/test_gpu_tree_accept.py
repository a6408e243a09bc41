"""dflash_tree_accept and dflash_tree_build against plain implementations."""
import numpy as np
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests import tree_ref as R

pytestmark = pytest.mark.gpu


class Accept:
    def __init__(self, S, rows, V, levels=6, drawn=True, T=0.8, seed=0, parents=None, dup=False, chain=False,
                 close=1.0, u=None):
        rng = self.rng = np.random.default_rng(seed)
        self.S, self.rows, self.V, self.levels, self.T = S, rows, V, levels, T
        self.parents = [list(range(-1, rows - 1))] * S if chain else parents or \
            [R.random_tree(rng, rows, levels) for _ in range(S)]
        self.draft = (rng.standard_normal((S, levels, V)) * 2).astype(np.float32) if drawn else None
        base = self.draft if drawn else (rng.standard_normal((S, levels, V)) * 2).astype(np.float32)
        self.target = np.zeros((S, rows, V), dtype=np.float32)
        self.tokens = np.zeros((S, rows), dtype=np.int32)
        for s in range(S):
            depth, kids = [0] * rows, [0] * rows
            order = [np.argsort(-(base[s, j] / T + rng.gumbel(size=V))) for j in range(levels)]
            for i in range(rows):
                p = self.parents[s][i]
                if i and 0 <= p < i:
                    depth[i] = depth[p] + 1
                    self.tokens[s, i] = order[min(depth[i], levels) - 1][0 if dup else kids[p] % V]
                    kids[p] += 1
                self.target[s, i] = base[s, min(depth[i], levels - 1)] + close * rng.standard_normal(V)
        self.u = rng.random((S, rows)).astype(np.float32) if u is None else np.full((S, rows), u, dtype=np.float32)
        self.noise = rng.exponential(size=(S, V)).astype(np.float32).clip(1e-30)
        self.base = rng.integers(0, 1000, S).astype(np.int32)
        self.chain = chain
        self.put()

    def put(self):
        d = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
        self.dev = dict(parent=None if self.chain else d(np.array(self.parents, dtype=np.int32)), tokens=d(self.tokens),
                        target_logits=d(self.target), draft_logits=d(self.draft), u=d(self.u), noise=d(self.noise),
                        base_pos=d(self.base))
        i32 = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")
        self.o = dict(accept_len=i32(self.S), path=i32(self.S, self.rows), out_tokens=i32(self.S, self.rows),
                      next_anchor=i32(self.S), commit_base=i32(self.S), commit_count=i32(self.S))
        a = self.a = D.dflash_tree_accept_args()
        a.dims = R.dims(vocab=self.V)
        a.n_seqs, a.rows, a.levels, a.temperature = self.S, self.rows, self.levels if self.draft is not None else 0, self.T
        for k, t in {**self.dev, **self.o}.items():
            setattr(a, k, R.ptr(t))
        a.update_base_pos = 1
        self.ws = R.Workspace(D.DFLASH_OP_TREE_ACCEPT, a)

    def run(self):
        D.dflash_tree_accept(self.a, self.ws.ptr, self.ws.bytes)

    def want(self, s):
        return R.accept(self.parents[s], self.tokens[s], self.target[s], None if self.draft is None else self.draft[s],
                        self.u[s], self.noise[s], self.T, self.levels)

    def check(self, status=D.DFLASH_OK, seqs=None, unsure=0):
        """Every decision equal to the 64-bit walk's.  A walk with a decision
        closer to its border than 1e-5 (fp32 weights and their sums: a few
        2^-24 each, times 1 / Z of the residuals) proves nothing; at most
        `unsure` of them may differ."""
        torch.cuda.synchronize()
        assert self.ws.status() == status
        o = {k: t.cpu().numpy() for k, t in self.o.items()}
        ks = []
        for s in range(self.S) if seqs is None else seqs:
            (k, path, out, last), gap = self.want(s)
            ks.append(k)
            got = (o["accept_len"][s], list(o["path"][s]), list(o["out_tokens"][s]), o["next_anchor"][s])
            if gap < 1e-5 and got != (k, path, out, last):
                unsure -= 1
                assert unsure >= 0, (s, gap)
                continue
            assert got == (k, path, out, last), (s, gap, got, (k, path, out, last))
            assert o["commit_base"][s] == self.base[s] and o["commit_count"][s] == k + 1
            assert int(self.dev["base_pos"][s]) == self.base[s] + k + 1
        return ks


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V", [1, 2, 5, 31, 1000, 1021, 4096, 20001])
@pytest.mark.parametrize("rows", [1, 2, 13, 40])
def test_random_trees(drawn, V, rows):
    p = Accept(5, rows, V, drawn=drawn, seed=V + rows)
    p.run()
    p.check()


@pytest.mark.parametrize("drawn", [True, False])
def test_full_vocabulary(drawn):
    p = Accept(3, 20, 151936, drawn=drawn, T=1.0, seed=4, close=0.4)
    p.run()
    p.check(unsure=1)


@pytest.mark.parametrize("S", [1, 9, 40, 200])
def test_batches(S):
    p = Accept(S, 12, 3001, seed=S)
    p.run()
    ks = p.check(unsure=S // 100)
    if S >= 40:
        assert 0 in ks and max(ks) >= 2  # the walks reach several depths


@pytest.mark.parametrize("drawn", [True, False])
def test_widest_and_deepest_trees(drawn):
    p = Accept(2, 128, 500, drawn=drawn, parents=[[-1] + [0] * 127] * 2, u=0.999, seed=1)
    p.run()
    p.check()
    p = Accept(2, 128, 500, levels=127, drawn=drawn, chain=True, u=1e-7, seed=2)
    p.run()
    ks = p.check()
    assert max(ks) > 20


@pytest.mark.parametrize("drawn", [True, False])
def test_same_token_twice_among_siblings(drawn):
    p = Accept(6, 9, 50, drawn=drawn, dup=True, parents=[[-1] + [0] * 8] * 6, u=0.9, seed=3)
    p.run()
    p.check()


@pytest.mark.parametrize("drawn", [True, False])
def test_masked_vocabulary(drawn):
    """-inf logits (also at a candidate), one token left, sharp rows."""
    p = Accept(4, 8, 300, drawn=drawn, seed=5)
    p.target[0, :, 10:] = -np.inf
    p.target[1, :, :] = -np.inf
    p.target[1, :, 7] = 1.0
    p.target[2, :, :] *= 40
    for i in range(8):
        p.target[3, i, p.tokens[3]] = -np.inf
    p.put()
    p.run()
    p.check()


def test_draft_equal_to_target_accepts_everything():
    p = Accept(3, 5, 700, levels=5, chain=True, close=0.0, seed=6)
    for s in range(3):
        for i in range(5):
            p.target[s, i] = p.draft[s, min(i, 4)]
    p.u[:] = 0.99
    p.put()
    p.run()
    torch.cuda.synchronize()
    assert p.o["accept_len"].tolist() == [4, 4, 4]


def test_nothing_accepted_and_everything_accepted():
    p = Accept(2, 6, 64, chain=True, drawn=False, levels=6, seed=7)
    p.u[0], p.u[1] = 1.0 - 2 ** -24, 0.0
    p.put()
    p.run()
    ks = p.check()
    assert ks == [0, 5]


def test_token_out_of_range():
    par = [[-1, 0, 0, 0]] * 2
    p = Accept(2, 4, 90, parents=par, drawn=False, seed=8, u=0.0)
    p.tokens[0, 1], p.tokens[1, 2] = 90, -5
    p.put()
    p.run()
    ks = p.check(D.DFLASH_ERR_INVALID_ARG)
    assert ks == [1, 1]


def test_children_below_the_last_draft_row():
    p = Accept(2, 6, 90, levels=2, chain=True, u=0.0, seed=9)
    p.run()
    assert p.check(D.DFLASH_ERR_INVALID_ARG) == [2, 2]


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("drawn", [True, False])
def test_bad_logit(bad, drawn):
    p = Accept(3, 6, 400, drawn=drawn, seed=10)
    p.target[1, 0, 33] = bad
    p.put()
    p.run()
    p.check(D.DFLASH_ERR_NUMERIC, seqs=[0, 2])
    assert 0 <= int(p.o["next_anchor"][1]) < 400


def test_without_optional_outputs():
    p = Accept(2, 7, 200, seed=11)
    for k in ("next_anchor", "commit_base", "commit_count", "base_pos"):
        setattr(p.a, k, 0)
    p.a.update_base_pos = 0
    p.run()
    torch.cuda.synchronize()
    for s in range(2):
        (k, path, out, _), _ = p.want(s)
        assert int(p.o["accept_len"][s]) == k and p.o["path"][s].tolist() == path
        assert p.o["out_tokens"][s].tolist() == out
    assert p.o["next_anchor"].tolist() == [77, 77]


def test_captured_and_replayed():
    p = Accept(4, 16, 5000, seed=12)
    p.a.update_base_pos = 0
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        p.run()
    p.u = p.rng.random((4, 16)).astype(np.float32)
    p.dev["u"].copy_(torch.from_numpy(p.u))
    g.replay()
    torch.cuda.synchronize()
    p.a.update_base_pos = 1
    p.dev["base_pos"] += torch.tensor([p.want(s)[0][0] + 1 for s in range(4)], dtype=torch.int32).cuda()
    p.check()


def greedy(parent, tokens, am):
    node, path, toks = 0, [0], []
    while True:
        nxt = [j for j in range(node + 1, len(parent)) if parent[j] == node and tokens[j] == am[node]]
        if not nxt:
            break
        node = nxt[0]
        path.append(node)
        toks.append(int(tokens[node]))
    n = len(parent)
    k = len(toks)
    return k, path + [-1] * (n - k - 1), toks + [int(am[node])] + [-1] * (n - k - 1)


@pytest.mark.parametrize("rows", [1, 7, 32, 33, 64, 128])
@pytest.mark.parametrize("chain", [False, True])
def test_greedy_walk(rows, chain):
    rng = np.random.default_rng(rows)
    S, V = 20, 3
    par = [list(range(-1, rows - 1)) if chain else R.random_tree(rng, max(1, rows - s % 4), 40, rows) for s in range(S)]
    tok = rng.integers(0, V, (S, rows)).astype(np.int32)
    am = rng.integers(0, V, (S, rows)).astype(np.int32)
    dev = [torch.tensor(np.array(x), dtype=torch.int32).cuda() for x in (par, tok, am)]
    a = D.dflash_tree_accept_args()
    a.dims = R.dims(vocab=V)
    a.n_seqs, a.rows, a.temperature = S, rows, 0.0
    a.parent, a.tokens, a.target_argmax = 0 if chain else R.ptr(dev[0]), R.ptr(dev[1]), R.ptr(dev[2])
    out = [torch.full((S,), 9, dtype=torch.int32, device="cuda") for _ in range(2)] + \
        [torch.full((S, rows), 9, dtype=torch.int32, device="cuda") for _ in range(2)]
    a.accept_len, a.next_anchor, a.path, a.out_tokens = (R.ptr(t) for t in out)
    ws = R.Workspace(D.DFLASH_OP_TREE_ACCEPT, a)
    D.dflash_tree_accept(a, ws.ptr, ws.bytes)
    torch.cuda.synchronize()
    assert ws.status() == D.DFLASH_OK
    for s in range(S):
        k, path, toks = greedy(par[s], tok[s], am[s])
        assert (int(out[0][s]), out[2][s].tolist(), out[3][s].tolist()) == (k, path, toks), s
        assert int(out[1][s]) == toks[k]


def test_build():
    S, levels, topk = 3, 4, 5
    parent = [-1, 0, 0, 1, 3, 4, 5, D.DFLASH_TREE_PAD, 7, 2, 10, 1]
    rank = [0, 0, 4, 1, 2, 3, 0, 0, 0, 5, 0, -1]
    rng = np.random.default_rng(0)
    cand = rng.integers(0, 1000, (S, levels, topk)).astype(np.int32)
    dev = [torch.tensor(np.array(x), dtype=torch.int32).cuda() for x in (parent, rank, cand, [7, 8, 9], [100, 0, 5])]
    rows = len(parent)
    out = [torch.full((S, rows), -77, dtype=torch.int32, device="cuda") for _ in range(3)]
    a = D.dflash_tree_build_args(S, rows, levels, topk, *(R.ptr(t) for t in dev + out))
    ws = R.Workspace(D.DFLASH_OP_TREE_BUILD, a)
    D.dflash_tree_build(a, ws.ptr, ws.bytes)
    torch.cuda.synchronize()
    # row 6 is deeper than the levels, 9's and 11's ranks are out of range, 10 is its own parent
    assert ws.status() == D.DFLASH_ERR_INVALID_ARG
    depth = [0, 1, 1, 2, 3, 4, None, None, None, None, None, None]
    for s in range(S):
        for i in range(rows):
            dp = depth[i]
            assert int(out[0][s, i]) == (parent[i] if dp is not None else D.DFLASH_TREE_PAD), i
            assert int(out[1][s, i]) == (cand[s, dp - 1, rank[i]] if dp else 7 + s)
            assert int(out[2][s, i]) == [100, 0, 5][s] + (dp or 0)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V", [1536, 1537, 2048, 10240, 10241, 25000])
def test_slices_of_several_batches(drawn, V):
    """More sequences than a device holds clusters of: a CTA per sequence walks
    the whole row, in one batch of its registers or several; candidates sit on
    both sides of the batches' borders."""
    S = 81
    p = Accept(S, 9, V, levels=4, drawn=drawn, seed=V)
    for s, x in enumerate((0, V - 1, min(10239, V - 1), min(10240, V - 1), min(20480, V - 1))):
        p.tokens[s, 1] = x
        p.target[s, :, x] += 6.0
    p.put()
    p.run()
    p.check(seqs=[0, 1, 2, 3, 4, 40, 79, 80], unsure=1)
