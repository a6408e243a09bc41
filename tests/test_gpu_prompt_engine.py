"""The prompt operators together, as the engine and the layer use them: packed
prompts against prompts of one length, scores against the model in 64 bits,
head norms through every mode of a target layer."""
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from block_diffusion_speculative_step_gb300 import synth
from block_diffusion_speculative_step_gb300.engine import Engine
from tests import gpu_common as G
from tests import helpers as Hh

pytestmark = pytest.mark.gpu


def small(dtype, **kw):
    base = dict(dtype=dtype, H=256, nq=4, nkv=2, d=64, I=384, V=512, t_layers=3, d_layers=2, taps=(0, 1), block=6,
                topk=4, rank=16)
    base.update(kw)
    return Hh.small_workload(**base)


def model(w, seed, norms):
    m = synth.make_model(w, seed=seed, jitter=0.1, with_target=True)
    if norms:
        synth.add_qk_norms(m, w)
    return m


def engine(w, seed, S, cap=256, norms=False, **kw):
    return Engine(w, G.to_dev(model(w, seed, norms)), S, cap, **kw)


def prompts_of(w, lens):
    return [synth.make_tokens(20 + s, n, w.vocab).cuda() for s, n in enumerate(lens)]


def target64(w, m, tokens):
    """The target's logits at every position of one prompt, in 64 bits from the
    weights (no rounding between): the plain decoder with head norms."""
    t, eps, n = w.target, w.rms_eps, tokens.numel()
    W = lambda x: x.double()
    norm = lambda x, g: x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * W(g)
    h = W(m["embed"])[tokens.long().cpu()]
    f = w.rope_theta ** (-2.0 * torch.arange(t.head_dim // 2, dtype=torch.float64) / t.head_dim)
    ang = torch.arange(n, dtype=torch.float64)[:, None, None] * f
    hidden = torch.ones(n, n, dtype=torch.bool).triu(1)

    def turn(x):
        a, b = x.chunk(2, -1)
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)

    for L in m["target"]["layers"]:
        x = (norm(h, L["ln1"]) @ W(L["w_qkv"]).T).view(n, -1, t.head_dim)
        q, k, v = x.split([t.n_q, t.n_kv, t.n_kv], 1)
        if "q_norm" in L:
            q, k = norm(q, L["q_norm"]), norm(k, L["k_norm"])
        q, k = turn(q), turn(k).repeat_interleave(t.n_q // t.n_kv, 1)
        v = v.repeat_interleave(t.n_q // t.n_kv, 1)
        sc = torch.einsum("ihd,jhd->hij", q, k) / t.head_dim ** 0.5
        o = torch.einsum("hij,jhd->ihd", torch.softmax(sc.masked_fill(hidden, -float("inf")), -1), v)
        h = h + o.reshape(n, -1) @ W(L["w_o"]).T
        x = norm(h, L["ln2"]) @ W(L["w_gu"]).T
        gate, up = x.chunk(2, -1)
        h = h + (gate * torch.sigmoid(gate) * up) @ W(L["w_down"]).T
    return norm(h, m["target"]["final_norm"]) @ W(m["lm_head"]).T


@pytest.mark.parametrize("norms", [False, True])
@pytest.mark.parametrize("S", [1, 3])
def test_packed_equals_uniform(norms, S):
    """In fp32 prompts of one length give the same caches and the same tokens
    either way (the two attentions sum in their own orders: 1e-5 of the values'
    size of about 1 is 80 roundings of 2^-23)."""
    w = small("f32")
    prompts = prompts_of(w, [40] * S)
    a, b = engine(w, 3, S, norms=norms), engine(w, 3, S, norms=norms)
    a.prefill(torch.stack(prompts))
    b.prefill(prompts)
    assert a.status() == D.DFLASH_OK and b.status() == D.DFLASH_OK
    assert torch.equal(a.base_pos, b.base_pos) and torch.equal(a.anchor, b.anchor)
    for x, y in ((a.caches.tk, b.caches.tk), (a.caches.tv, b.caches.tv), (a.caches.dk, b.caches.dk),
                 (a.caches.dv, b.caches.dv)):
        for u, v in zip(x, y):
            assert float((u - v).abs().max()) < 1e-5 * max(1.0, float(u.abs().max()))


@pytest.mark.parametrize("norms", [False, True])
@pytest.mark.parametrize("kind", ["chain", "tree", "greedy"])
def test_generation_from_packed_prompts(norms, kind):
    """A sequence of a batch of different lengths goes on as it does alone."""
    w = small("f32")
    lens, n = [7, 64, 1, 33], 24
    prompts = prompts_of(w, lens)
    alone = [engine(w, 4, 1, norms=norms).greedy_generate(p[None], n)[0] for p in prompts]
    eng = engine(w, 4, len(lens), norms=norms)
    if kind == "tree":
        eng.set_tree([-1, 0, 0, 1, 1, 3], [0, 0, 1, 0, 1, 0])
        out, _ = eng.tree_generate(prompts, n)
    elif kind == "chain":
        out, _ = eng.speculative_generate(prompts, n)
    else:
        out = eng.greedy_generate(prompts, n)
    assert eng.status() == D.DFLASH_OK
    assert torch.equal(out, torch.stack(alone))


def test_window_rings():
    """Prompts longer than the draft's window: its ring holds the last positions."""
    w = small("f32", window=32)
    prompts = prompts_of(w, [200, 200])
    a, b = engine(w, 11, 2), engine(w, 11, 2)
    a.chunk = 32  # (rows at a time that a ring of 32 takes)
    a.prefill(torch.stack(prompts))
    b.prefill(prompts)
    assert a.status() == D.DFLASH_OK and b.status() == D.DFLASH_OK
    for x, y in zip(a.caches.dk + a.caches.dv, b.caches.dk + b.caches.dv):
        assert float((x - y).abs().max()) < 1e-5 * max(1.0, float(x.abs().max()))


@pytest.mark.parametrize("piece", [0, 7, 32])
@pytest.mark.parametrize("page", [0, 128])
def test_prompts_in_pieces(piece, page):
    w = small("f32")
    lens = [50, 3, 129, 32]
    prompts = prompts_of(w, lens)
    whole, eng = engine(w, 5, 4, norms=True), engine(w, 5, 4, norms=True)
    whole.prefill_packed(prompts)
    if page:
        eng.page_caches(page, seed=3, spare_pages=2)
    eng.prefill_packed(prompts, piece)
    assert eng.status() == D.DFLASH_OK
    assert torch.equal(whole.anchor, eng.anchor) and torch.equal(whole.base_pos, eng.base_pos)
    for kind in ("t", "d"):
        for x, y in zip(*(e.unpaged_caches()[kind] for e in (whole, eng))):
            for u, v in zip(x, y):
                for s, n in enumerate(lens):
                    assert float((u[s, :, :n] - v[s, :, :n]).abs().max()) < 1e-5 * max(1.0, float(u[s].abs().max()))


@pytest.mark.parametrize("dtype,kv8", [("f32", False), ("bf16", False), ("f32", True), ("bf16", True)])
@pytest.mark.parametrize("norms", [False, True])
def test_scores(dtype, kv8, norms):
    """Scores of whole prompts against the model in 64 bits.  fp32: errors of
    about 2^-24 times sums of a few hundred terms over three layers, 1e-4.
    bf16: the logits' own bound for bf16 networks, 2e-2 of a logit of size up
    to 2, doubled for the difference of a logit and the row's log sum."""
    w = small(dtype)
    lens, k = [40, 1, 75, 300], 5
    prompts = prompts_of(w, lens)
    m = model(w, 6, norms)
    eng = Engine(w, G.to_dev(m), 4, 512, kv8=kv8)
    got = eng.score(prompts, topk=k, T=0.9)
    assert eng.status() == D.DFLASH_OK
    tol = 1e-4 if dtype == "f32" else 2 * G.LOGIT_TOL["bf16"]
    for p, (lp, ent, ids, top) in zip(prompts, got):
        ref = torch.log_softmax(target64(w, m, p) / 0.9, -1)
        n = p.numel()
        assert lp.shape == (n - 1,) and ent.shape == (n,) and ids.shape == top.shape == (n, k)
        if n > 1:
            want = ref[:-1].gather(1, p.cpu().long()[1:, None])[:, 0]
            assert float((lp.cpu().double() - want).abs().max()) < tol
        assert float((ent.cpu().double() + (ref.exp() * ref).sum(-1)).abs().max()) < tol
        at = ref.gather(1, ids.cpu().long())
        assert float((top.cpu().double() - at).abs().max()) < tol
        best = torch.topk(ref, k, -1).values  # the alternatives are the best ones, but for near-ties
        assert float((best - at).abs().max()) < 2 * tol


def test_scores_in_pieces_and_generation_after():
    w = small("f32")
    prompts = prompts_of(w, [40, 300])
    a, b = engine(w, 7, 2, 512, norms=True), engine(w, 7, 2, 512, norms=True)
    x, y = a.score(prompts, topk=3), b.score(prompts, topk=3, piece=64)
    for u, v in zip(x, y):
        for i in (0, 1, 3):
            assert float((u[i] - v[i]).abs().max()) < 1e-4
    for _ in range(4):
        a.cycle()
        b.cycle()
    assert torch.equal(a.out_tokens, b.out_tokens) and torch.equal(a.base_pos, b.base_pos)
    assert a.status() == D.DFLASH_OK and b.status() == D.DFLASH_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_generation_from_packed_prompts_over_an_8_bit_cache(dtype):
    """A sequence goes on as it does alone: the rows of its prompt see each
    other unquantised either way.  (bf16: up to a near-tie, so only the caches.)"""
    w = small(dtype)
    lens, n = [40, 9, 130], 12
    prompts = prompts_of(w, lens)
    eng = engine(w, 12, 3, norms=True, kv8=True)
    out = eng.greedy_generate(prompts, n)
    assert eng.status() == D.DFLASH_OK
    for s, p in enumerate(prompts):
        one = engine(w, 12, 1, norms=True, kv8=True)
        alone = one.greedy_generate([p], n)[0]
        if dtype == "f32":
            assert torch.equal(out[s], alone)
            for x, y in zip(eng.caches.tk + eng.caches.tv, one.caches.tk + one.caches.tv):
                differ = (x[s, :, :lens[s]] != y[0, :, :lens[s]]).float().mean()
                assert float(differ) < 1e-3  # (codes on a rounding border)


@pytest.mark.parametrize("page", [0, 128])
def test_norms_in_causal_and_tree_layers(page):
    """The same chain through the causal mode and the tree mode, over the same cache."""
    w = small("f32")
    S, rows = 2, 9
    eng = engine(w, 8, S, norms=True)
    eng.prefill(prompts_of(w, [30, 17]))
    if page:
        eng.page_caches(page, seed=4)
    tok = torch.stack([synth.make_tokens(40 + s, rows, w.vocab) for s in range(S)]).cuda()
    pos = (eng.base_pos[:, None] + torch.arange(rows, device="cuda", dtype=torch.int32)).view(-1)
    eng._tree_buffers(rows)
    need = D.dflash_workspace_bytes(D.DFLASH_OP_LAYER, eng.tree_layer_args(0, rows, eng.h, pos))
    if need > eng.ws_bytes:
        eng._new_workspace(need)
    eng.tree_forward(rows, tok, pos)
    tree = eng.h[:S * rows].clone()
    eng.target_forward(rows, tok[:, 0].contiguous(), tok[:, 1:].contiguous())
    assert eng.status() == D.DFLASH_OK
    assert float((tree - eng.h[:S * rows]).abs().max()) < 1e-5 * max(1.0, float(tree.abs().max()))


def test_rows_of_no_sequence_in_a_layer():
    """Their residual stays finite, the others' is as without them."""
    for dtype in ("f32", "bf16"):
        w = small(dtype)
        eng = engine(w, 9, 2, norms=True)
        M, t = 60, w.target
        eng._prompt_buffers(M, 30)
        pos = torch.arange(M, dtype=torch.int32, device="cuda")
        h0 = torch.randn(M, t.hidden, device="cuda")
        out = []
        for start in ([0, 25, 60], [0, 25, 50], [5, 25, 50]):
            eng.ws[4096 + 131072:] = 0xFF  # (NaN in the scratch)
            h = h0.clone()
            st = torch.tensor(start, dtype=torch.int32, device="cuda")
            D.dflash_decoder_layer_forward(eng.prompt_layer_args(0, 2, M, h, st, pos), eng.ws_ptr, eng.ws_bytes)
            assert eng.status() == D.DFLASH_OK
            assert bool(torch.isfinite(h).all())
            out.append(h)
        assert torch.allclose(out[0][:50], out[1][:50], atol=1e-2 if dtype == "bf16" else 1e-5)
        assert torch.allclose(out[1][25:50], out[2][25:50], atol=1e-2 if dtype == "bf16" else 1e-5)


def test_positions_outside_the_table_are_reported():
    w = small("f32")
    for norms in (False, True):
        eng = engine(w, 9, 2, norms=norms)
        M = 20
        eng._prompt_buffers(M, 10)
        st = torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda")
        for bad in (-1, eng.rope_max):
            pos = torch.arange(M, dtype=torch.int32, device="cuda")
            pos[13] = bad
            h = torch.randn(M, w.target.hidden, device="cuda")
            eng.pkb[0].zero_()
            eng.pvb[0].zero_()
            D.dflash_decoder_layer_forward(eng.prompt_layer_args(0, 2, M, h, st, pos), eng.ws_ptr, eng.ws_bytes)
            assert eng.status() == D.DFLASH_ERR_INVALID_ARG


def test_layer_refusals():
    w = small("bf16")
    eng = engine(w, 9, 2, norms=True, kv8=True)
    eng._prompt_buffers(20, 10)
    x = torch.zeros(32, dtype=torch.int32, device="cuda")

    def refused(code, **kw):
        a = eng.prompt_layer_args(0, 2, 20, eng.ph, x, x)
        for k, v in kw.items():
            setattr(a, k, v)
        with pytest.raises(D.DFlashError) as e:
            D.dflash_decoder_layer_forward(a, eng.ws_ptr, eng.ws_bytes)
        assert e.value.code == code

    refused(D.DFLASH_ERR_UNSUPPORTED, base_pos=x.data_ptr())            # an 8-bit context
    refused(D.DFLASH_ERR_INVALID_ARG, prompt_start=0)
    refused(D.DFLASH_ERR_INVALID_ARG, tree_pos=0)
    refused(D.DFLASH_ERR_INVALID_ARG, n_seqs=0)
    refused(D.DFLASH_ERR_INVALID_ARG, rows=0)
    refused(D.DFLASH_ERR_INVALID_ARG, q_norm=eng.ph.data_ptr() + 4)
    a = engine(w, 9, 2, norms=True).target_layer_args(0, 4, eng.h)
    a.attn_mode = D.DFLASH_ATTN_BLOCK_BIDIR
    with pytest.raises(D.DFlashError) as e:
        D.dflash_decoder_layer_forward(a, eng.ws_ptr, eng.ws_bytes)
    assert e.value.code == D.DFLASH_ERR_UNSUPPORTED


def test_a_captured_prompt_layer():
    w = small("bf16")
    eng = engine(w, 10, 3, norms=True)
    M = 200
    eng._prompt_buffers(M, 100)
    st = torch.tensor([0, 70, 71, M], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in (70, 1, 129)]).cuda()
    h0 = torch.randn(M, w.target.hidden, device="cuda")
    h = h0.clone()
    call = lambda: D.dflash_decoder_layer_forward(eng.prompt_layer_args(0, 3, M, h, st, pos), eng.ws_ptr, eng.ws_bytes)
    call()
    torch.cuda.synchronize()
    want = h.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        h.copy_(h0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, want)
    assert eng.status() == D.DFLASH_OK


def test_captured_cycles_outlive_a_growing_workspace():
    """A cycle captured into a graph, then prompts that need a larger
    workspace: the graph's cycles are the eager ones."""
    w = small("bf16")
    short, long = prompts_of(w, [9, 4]), prompts_of(w, [700, 300])
    eng, ref = engine(w, 11, 2, 1024), engine(w, 11, 2, 1024)
    eng.prefill(short)
    eng.cycle()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        eng.cycle()
    before = eng.ws_ptr
    for e in (eng, ref):
        e.score(long, topk=2)
    assert eng.ws_ptr != before  # (or the case is none)
    junk = [torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(64)]  # whatever was freed
    for _ in range(4):
        g.replay()
        ref.cycle()
        assert torch.equal(eng.out_tokens, ref.out_tokens) and torch.equal(eng.base_pos, ref.base_pos)
    del junk
    assert eng.status() == D.DFLASH_OK and ref.status() == D.DFLASH_OK


def test_a_growing_workspace_keeps_the_status():
    w = small("f32")
    eng = engine(w, 12, 1, 1024)
    a = D.dflash_token_logprobs_args()
    x, t, o = torch.zeros(1, 8, device="cuda"), torch.tensor([8], dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda")
    a.dims.vocab, a.n_rows, a.temperature = 8, 1, 1.0
    a.logits, a.tokens, a.logprob = x.data_ptr(), t.data_ptr(), o.data_ptr()
    D.dflash_token_logprobs(a, eng.ws_ptr, eng.ws_bytes)  # a token outside the vocabulary
    before = eng.ws_ptr
    eng.prefill(prompts_of(w, [900]))
    eng._prompt_workspace(eng.ws_bytes + 1)
    assert eng.ws_ptr != before
    assert eng.status() == D.DFLASH_ERR_INVALID_ARG and eng.status() == D.DFLASH_OK


def test_prompts_as_they_come():
    """64-bit tokens, strided ones, tokens on the host; and a piece of no tokens."""
    w = small("f32")
    plain = prompts_of(w, [40, 7])
    wide = torch.zeros(40, 3, dtype=torch.int64, device="cuda")
    wide[:, 1] = plain[0]
    a, b = engine(w, 13, 2), engine(w, 13, 2)
    x, y = a.score(plain, topk=2), b.score([wide[:, 1], plain[1].long().cpu()], topk=2)
    for u, v in zip(x, y):
        assert all(torch.equal(i, j) for i, j in zip(u, v))
    assert torch.equal(a.anchor, b.anchor) and a.status() == b.status() == D.DFLASH_OK
    with pytest.raises(AssertionError):
        b.prefill_packed(plain, piece=-4)
