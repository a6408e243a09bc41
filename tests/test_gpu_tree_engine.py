"""Tree cycles end to end: the operators run together as the engine uses them
(candidates, tree, target forward over the tree, acceptance, commit, fusion),
8-bit target caches, captured cycles, and the layer's tree mode against its
causal one."""
import numpy as np
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from block_diffusion_speculative_step_gb300 import synth
from block_diffusion_speculative_step_gb300.engine import Engine
from tests import gpu_common as G
from tests import helpers as Hh
from tests import tree_ref as R
from tests.test_gpu_tree_attn import Tree, trees

pytestmark = pytest.mark.gpu


def small(dtype, topk=4, **kw):
    base = dict(dtype=dtype, H=256, nq=4, nkv=2, d=64, I=384, V=512, t_layers=3, d_layers=2, taps=(0, 1), block=6,
                topk=topk, rank=16 if topk else 0)
    base.update(kw)
    return Hh.small_workload(**base)


def template(seed, n, block, topk):
    """A random tree whose siblings take different candidates."""
    rng = np.random.default_rng(seed)
    parent, rank, depth, used = [-1], [0], [0], {0: set()}
    while len(parent) < n:
        p = int(rng.integers(len(parent)))
        if depth[p] == block - 1 or len(used[p]) == topk:
            continue
        used[p].add(len(used[p]))
        parent.append(p)
        rank.append(len(used[p]) - 1)
        depth.append(depth[p] + 1)
        used[len(parent) - 1] = set()
    return parent, rank


def engine(w, seed, S, cap=128, tree=None, **kw):
    eng = Engine(w, G.to_dev(synth.make_model(w, seed=seed, jitter=0.1, with_target=True)), S, cap, **kw)
    if tree:
        eng.set_tree(*tree)
    return eng


def prompts_of(w, S, n=20):
    return torch.stack([synth.make_tokens(10 + s, n, w.vocab) for s in range(S)]).cuda()


@pytest.mark.parametrize("S,topk,rows,page", [(1, 4, 1, 0), (1, 4, 13, 0), (3, 4, 33, 0), (2, 4, 24, 128), (2, 0, 6, 0)])
def test_tree_generate_is_greedy(S, topk, rows, page):
    """Greedy acceptance emits the target's own greedy tokens, whatever the tree."""
    w = small("f32", topk)
    n = 40
    prompts = prompts_of(w, S)
    greedy = engine(w, 3, S).greedy_generate(prompts, n)
    eng = engine(w, 3, S, tree=template(rows, rows, w.block, max(topk, 1)))
    if page:
        eng.page_caches(page, seed=1, spare_pages=2)
    out, acc = eng.tree_generate(prompts, n)
    assert eng.status() == D.DFLASH_OK
    np.testing.assert_array_equal(out.numpy(), greedy.numpy())
    assert (acc >= 0).all() and (acc <= w.block - 1).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [0, 128])
def test_committed_rows_of_an_8_bit_cache(dtype, page):
    """After a cycle the cache holds exactly the accepted path's keys and
    values, quantised; the slots behind them are as they were."""
    w = small(dtype)
    S, N = 2, 17
    eng = engine(w, 5, S, 256, tree=template(2, N, w.block, 4), kv8=True)
    eng.prefill(prompts_of(w, S))
    if page:
        eng.page_caches(page, seed=2, spare_pages=1)

    def snapshot(xs):  # [S][nkv][cap] codes or exponents
        if not page:
            return [x.cpu() for x in xs]
        table, ps, mp, _ = eng.paging["t"]
        return [torch.cat([x[table[:, j].long()] for j in range(mp)], 2).cpu() for x in xs]

    sides = (("k", eng.caches.tk, eng.caches.tke, eng.tkb), ("v", eng.caches.tv, eng.caches.tve, eng.tvb))
    for _ in range(3):
        base = eng.base_pos.cpu()
        before = [(snapshot(c), snapshot(e)) for _, c, e, _ in sides]
        eng.tree_cycle()
        assert eng.status() == D.DFLASH_OK
        k, path = eng.accept_len.cpu(), eng.t_path.cpu()
        assert torch.equal(eng.base_pos.cpu(), base + k + 1)
        for (name, c, e, rows), (c0, e0) in zip(sides, before):
            c1, e1 = snapshot(c), snapshot(e)
            for j in range(w.target.layers):
                src = rows[j][:S * N].cpu().double().view(S, N, w.target.n_kv, -1).numpy()
                for s in range(S):
                    for i in range(int(k[s]) + 1):
                        for g in range(w.target.n_kv):
                            codes, ex = R.quantise_row(src[s, int(path[s, i]), g])
                            p = int(base[s]) + i
                            got = c1[j][s, g, p].numpy()
                            assert int(e1[j][s, g, p]) == ex, (name, j, s, i, g)
                            np.testing.assert_array_equal(R.E4M3[got], R.E4M3[codes])
                            c0[j][s, g, p], e0[j][s, g, p] = c1[j][s, g, p], e1[j][s, g, p]
                assert torch.equal(c0[j], c1[j]) and torch.equal(e0[j], e1[j])


def test_8_bit_cache_runs_the_chain_paths():
    """With 8-bit target caches the chain cycle and plain decoding run on tree
    forwards too; decoding one token at a time equals decoding by cycles that
    accept nothing, for both read the same quantised rows."""
    w = small("f32")
    n = 16
    prompts = prompts_of(w, 2)
    greedy = engine(w, 3, 2, kv8=True).greedy_generate(prompts, n)
    eng = engine(w, 3, 2, tree=([-1], [0]), kv8=True)
    out, acc = eng.tree_generate(prompts, n)
    assert eng.status() == D.DFLASH_OK and int(acc.abs().max()) == 0
    np.testing.assert_array_equal(out.numpy(), greedy.numpy())
    eng = engine(w, 3, 2, kv8=True)
    eng.speculative_generate(prompts, n)
    assert eng.status() == D.DFLASH_OK


def test_sampled_tree_cycle_follows_the_walk():
    """T > 0: the emitted tokens are those of the 64-bit walk over the cycle's own logits."""
    w = small("f32")
    S, N, T = 3, 21, 0.7
    eng = engine(w, 6, S, tree=template(4, N, w.block, 4))
    eng.prefill(prompts_of(w, S))
    g = torch.Generator().manual_seed(0)
    for _ in range(3):
        u = torch.rand(S, N, generator=g)
        noise = torch.empty(S, w.vocab).exponential_(generator=g)
        u_d, noise_d = u.cuda(), noise.cuda()
        eng.tree_cycle(T, u_d, noise_d)
        assert eng.status() == D.DFLASH_OK
        for s in range(S):
            (k, path, toks, _), gap = R.accept(eng.t_parent[s].tolist(), eng.t_tokens[s].tolist(),
                                               eng.t_logits.view(S, N, -1)[s].cpu().double().numpy(), None,
                                               u[s].double().numpy(), noise[s].double().numpy(), T, 0)
            if gap < 1e-5:  # a decision within the fp32 error of its border
                continue
            assert int(eng.accept_len[s]) == k
            assert eng.t_path[s].tolist() == list(path) and eng.t_out[s].tolist() == list(toks)


@pytest.mark.parametrize("kv8", [False, True])
def test_captured_cycles(kv8):
    """A cycle captured into a graph and replayed gives the eager cycles'
    tokens; an eager cycle of another engine runs in between."""
    w = small("bf16")
    S, N = 2, 17
    tree = template(3, N, w.block, 4)
    prompts = prompts_of(w, S)
    ref, eng, other = (engine(w, 7, S, tree=tree, kv8=kv8) for _ in range(3))
    for e in (ref, eng, other):
        e.prefill(prompts)
    want = []
    for _ in range(4):
        ref.tree_cycle()
        want.append((ref.accept_len.clone(), ref.t_out.clone(), ref.base_pos.clone()))
    state = [x.clone() for x in (eng.anchor, eng.base_pos)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eng.tree_cycle()  # warm-up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eng.tree_cycle()
    eng.prefill(prompts)  # the warm-up's rows are written again by the same cycles
    assert all(torch.equal(a, b) for a, b in zip(state, (eng.anchor, eng.base_pos)))
    for a, t, p in want:
        graph.replay()
        other.tree_cycle()
        torch.cuda.synchronize()
        assert torch.equal(eng.accept_len, a) and torch.equal(eng.t_out, t) and torch.equal(eng.base_pos, p)
    assert eng.status() == D.DFLASH_OK and other.status() == D.DFLASH_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 6, 64])
def test_layer_tree_chain_is_causal(dtype, rows):
    """A chain in tree mode sees what the same rows see in causal mode.  The
    projections are the same kernels (queries, keys, values equal bit by bit);
    each attention output is within its own bound of the exact one: half a
    step of the output, and of the weights (2^-8 of the largest |v| in bf16,
    the fp32 sums of at most 512 terms otherwise)."""
    w = small(dtype, H=256, nq=8, nkv=2, d=128)
    S, cap = 2, 512
    base = [0, 300]
    eng = engine(w, 8, S, cap, tree=([-1] * rows, [0] * rows))
    g = torch.Generator().manual_seed(1)
    t = w.target
    for c in (eng.caches.tk[0], eng.caches.tv[0]):
        c.copy_(torch.randn(c.shape, generator=g).to(c.dtype))
    h0 = torch.randn(S * rows, t.hidden, generator=g).cuda()
    eng.base_pos.copy_(torch.tensor(base, dtype=torch.int32))
    pos = (eng.base_pos[:, None] + torch.arange(rows, dtype=torch.int32, device="cuda")).view(-1)
    got = {}
    for mode in ("tree", "causal"):
        h = h0.clone()
        a = (eng.tree_layer_args(0, rows, h, pos) if mode == "tree" else eng.target_layer_args(0, rows, h))
        q, o = (torch.zeros(S * rows, t.n_q * t.head_dim, dtype=eng.dt, device="cuda") for _ in range(2))
        a.out_q, a.out_attn = q.data_ptr(), o.data_ptr()
        need = D.dflash_workspace_bytes(D.DFLASH_OP_LAYER, a)
        if need > eng.ws_bytes:
            eng._new_workspace(int(need))
        D.dflash_decoder_layer_forward(a, eng.ws_ptr, eng.ws_bytes)
        assert eng.status() == D.DFLASH_OK
        got[mode] = q, o.double().cpu(), h.double().cpu()
    assert torch.equal(got["tree"][0], got["causal"][0])
    vmax = 0.0
    for name, c, rows_d in (("k", eng.caches.tk[0], eng.tkb[0]), ("v", eng.caches.tv[0], eng.tvb[0])):
        new = rows_d[:S * rows].view(S, rows, t.n_kv, t.head_dim)
        for s in range(S):
            assert torch.equal(c[s, :, base[s]:base[s] + rows], new[s].transpose(0, 1)), name
        vmax = max(vmax, float(c.double().abs().max()), float(new.double().abs().max()))
    o1, o2 = got["tree"][1], got["causal"][1]
    step = 2.0 ** -8 if dtype == "bf16" else 512 * 2.0 ** -24 * 4
    assert ((o1 - o2).abs() <= 2 * step * (o2.abs() + vmax)).all()


@pytest.mark.parametrize("dtype,cache,nq,rows", [("bf16", "bf16", 4, 17), ("bf16", "bf16", 16, 33), ("bf16", "e4m3", 4, 17),
                                                ("bf16", "e4m3", 16, 33)])
def test_expired_waits_are_reported(dtype, cache, nq, rows):
    """With the copies of keys and values switched off every wait gives up
    within its limit, the call reports it, and the next one is right."""
    p = Tree([40, 700, 0], trees(1, [rows] * 3, rows), nq, 4, 128, dtype, cache)
    D.dflash_workspace_control(p.ws.ptr, p.ws.bytes, wait_limit_ns=2_000_000, stall_kv_loads=True)
    p.run()
    torch.cuda.synchronize()
    assert p.ws.status() == D.DFLASH_ERR_TIMEOUT
    D.dflash_workspace_control(p.ws.ptr, p.ws.bytes)
    p.run()
    p.check()


def test_two_calls_at_once():
    """Two calls with workspaces of their own on two streams."""
    ps = [Tree([500, 90], trees(i, [33, 20], 33), 8, 2, 128, "bf16", c) for i, c in enumerate(("bf16", "e4m3"))]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(8):
        for p, st in zip(ps, streams):
            with torch.cuda.stream(st):
                p.run()
    for p in ps:
        p.check()


@pytest.mark.parametrize("cache,cap", [("bf16", 2_200_064), ("e4m3", 4_400_128)])
def test_offsets_past_32_bits(cache, cap):
    """A cache whose last heads lie more than 2^32 bytes in: the attention over
    it, and rows written to its last slots and read back."""
    nkv, d, n = 8, 128, 200
    p = Tree([n], trees(3, [9], 9), 16, nkv, d, "bf16", cache, cap=256)
    big = {}
    for x in ("k", "v", "ke", "ve"):
        small_x = p.dev[x]
        if small_x is None:
            big[x] = None
            continue
        big[x] = torch.zeros((1, nkv, cap) + small_x.shape[3:], dtype=small_x.dtype, device="cuda")
        big[x][:, :, :256] = small_x
    assert big["k"].numel() * big["k"].element_size() > 1 << 32
    p.a.kv = R.kv_desc(cap, big["k"], big["v"], big["ke"], big["ve"])
    p.run()
    p.check()
    rows = 3
    base = torch.tensor([cap - rows], dtype=torch.int32, device="cuda")
    src = [torch.randn(rows, nkv, d, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in range(2)]
    out = [torch.zeros_like(x) for x in src]
    kv = (D.dflash_kv * 1)(p.a.kv)
    arrays = [R.host_array([x]) for x in (*src, *out)]
    w, r = D.dflash_kv_write_args(), D.dflash_kv_read_args()
    for a in (w, r):
        a.dims, a.n_layers, a.n_seqs, a.rows = p.a.dims, 1, 1, rows
        a.base_pos, a.kv_layers = R.ptr(base), D.C.cast(kv, D.C.c_void_p)
    w.kb, w.vb, r.k_out, r.v_out = (D.C.cast(x, D.C.c_void_p) for x in arrays)
    ws = R.Workspace(D.DFLASH_OP_KV_WRITE, w)
    D.dflash_kv_write(w, ws.ptr, ws.bytes)
    D.dflash_kv_read(r, ws.ptr, ws.bytes)
    torch.cuda.synchronize()
    assert ws.status() == D.DFLASH_OK
    for x, y, c, e in zip(src, out, (big["k"], big["v"]), (big["ke"], big["ve"])):
        if e is None:
            assert torch.equal(x, y) and torch.equal(c[0, :, cap - rows:], x.transpose(0, 1))
            continue
        for i in range(rows):
            for g in range(nkv):
                codes, ex = R.quantise_row(x[i, g].double().cpu().numpy())
                assert int(e[0, g, cap - rows + i]) == ex
                np.testing.assert_array_equal(R.E4M3[c[0, g, cap - rows + i].cpu().numpy()], R.E4M3[codes])
                np.testing.assert_array_equal(y[i, g].double().cpu().numpy(), R.E4M3[codes] * 2.0 ** (ex - 127))
