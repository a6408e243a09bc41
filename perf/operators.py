"""Tree-verification operators of the library: what they compute, on which
sizes they are measured, and the work they cannot do without.

Three operators of one serving path -- the target verifies a TREE of drafted
tokens instead of one chain:

  attn    softmax attention of the tree's nodes over the cached context and
          over their own ancestors (dflash_tree_attention);
  kv      the accepted path's keys and values written to the cache, quantised
          to 8 bits, and cache rows read back (dflash_kv_write, dflash_kv_read);
  accept  the walk down the tree that accepts drafted tokens against the
          target's probabilities from given random numbers (dflash_tree_accept).

`own` selects the library's kernels; otherwise run() computes the same from
elementary torch operations.
"""
from __future__ import annotations

import math
import random

import torch

own = False

PAD = -2        # parent of a row that holds no node
E4M3_MAX = 448.0
EXP_LIM = 60    # cache scales are 2^-60 .. 2^60
EXP_BIAS = 127

# --------------------------------------------------------------------- cases


def listed():
    q8 = dict(nq=32, nkv=8, d=128)         # the 8B-shaped target of the benchmark
    coder = dict(nq=32, nkv=4, d=128)      # the long-context shape of the benchmark
    return [
        # one user, a small tree over a 4k context: every verification step of interactive decoding (latency)
        dict(name="attn-b1-n16-4k-bf16", op="attn", S=1, rows=16, ctx_lo=4096, ctx_hi=4096, **q8, dtype="bf16",
             cache="bf16", page=0, pad=False),
        # the benchmark's ragged 32-sequence batch, 64-node trees
        dict(name="attn-b32-n64-8k-bf16", op="attn", S=32, rows=64, ctx_lo=1024, ctx_hi=8192, **q8, dtype="bf16",
             cache="bf16", page=0, pad=False),
        # the same batch on an 8-bit paged cache
        dict(name="attn-b32-n64-8k-e4m3", op="attn", S=32, rows=64, ctx_lo=1024, ctx_hi=8192, **q8, dtype="bf16",
             cache="e4m3", page=256, pad=False),
        # single-token decoding at the end of a 32k context, 8-bit cache
        dict(name="attn-b1-n1-32k-e4m3", op="attn", S=1, rows=1, ctx_lo=32767, ctx_hi=32767, **coder, dtype="bf16",
             cache="e4m3", page=0, pad=False),
        # ragged trees of up to 37 nodes (rows behind a tree's last node stay as they were), odd contexts, paged
        dict(name="attn-b5-n37-ragged-bf16", op="attn", S=5, rows=37, ctx_lo=1, ctx_hi=2047, **q8, dtype="bf16",
             cache="bf16", page=128, pad=True),
        # the full-precision verification of the tiny lossless configuration
        dict(name="attn-b3-n13-f32", op="attn", S=3, rows=13, ctx_lo=0, ctx_hi=131, nq=4, nkv=4, d=64, dtype="f32",
             cache="f32", page=0, pad=False),
        # a prompt's keys and values entering the 8-bit cache, then handed on in full width
        dict(name="kv-prefill-4k-bf16", op="kv", S=1, rows=4096, layers=1, base_hi=0, nkv=8, d=128, dtype="bf16",
             page=0, path=False),
        # the accepted paths of 32 sequences committed to all 36 layers' paged caches after one cycle
        dict(name="kv-commit-b32-36l-bf16", op="kv", S=32, rows=16, layers=36, base_hi=1000, nkv=8, d=128,
             dtype="bf16", page=128, path=True),
        # the same of one small fp32 model: the smallest call
        dict(name="kv-commit-b3-f32", op="kv", S=3, rows=8, layers=4, base_hi=77, nkv=4, d=64, dtype="f32", page=0,
             path=True),
        # candidates drawn from the draft's own distribution (its logits are known), one user
        dict(name="accept-b1-n16-drawn", op="accept", S=1, rows=16, vocab=151936, levels=15, drawn=True, T=0.8),
        # 64-node trees over the draft's best candidates, 32 sequences
        dict(name="accept-b32-n64-best", op="accept", S=32, rows=64, vocab=151936, levels=15, drawn=False, T=1.0),
        # a short vocabulary of odd size, drawn candidates
        dict(name="accept-b7-n33-v1021", op="accept", S=7, rows=33, vocab=1021, levels=9, drawn=True, T=0.6),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng: random.Random):
    op = rng.choice(["attn", "attn", "kv", "accept"])
    if op == "attn":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        S = _log_int(rng, 1, 32)
        rows = _log_int(rng, 1, 128)
        nq, nkv = rng.choice([(32, 8), (32, 4), (8, 8), (12, 4), (4, 2), (8, 1)])
        d = rng.choice([64, 128])
        # scores of one pass: at most half of the largest listed case's (a sixteenth in full precision)
        budget = 32 * 64 * 32 * 4608 // (2 if dtype == "bf16" else 16)
        hi = min(32768, max(2, budget // (S * rows * nq)))
        hi = _log_int(rng, 2, hi)
        return dict(op="attn", S=S, rows=rows, ctx_lo=rng.choice([0, 1, hi // 2, hi]), ctx_hi=hi, nq=nq, nkv=nkv, d=d,
                    dtype=dtype, cache=rng.choice([dtype, "e4m3"]), page=rng.choice([0, 128, 256]),
                    pad=rng.random() < 0.5)
    if op == "kv":
        S = _log_int(rng, 1, 32)
        layers = _log_int(rng, 1, 40)
        rows = _log_int(rng, 1, max(1, min(4096, 32 * 16 * 36 // (S * layers))))
        return dict(op="kv", S=S, rows=rows, layers=layers, base_hi=rng.choice([0, 5, 130, 1000]),
                    nkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "f32"]),
                    page=rng.choice([0, 128, 256]), path=rng.random() < 0.6)
    vocab = _log_int(rng, 40, 151936)
    rows = _log_int(rng, 1, 64)
    S = _log_int(rng, 1, max(1, min(32, 32 * 64 * 151936 // (4 * rows * vocab))))
    return dict(op="accept", S=S, rows=rows, vocab=vocab, levels=rng.randint(1, 15), drawn=rng.random() < 0.5,
                T=rng.choice([0.5, 0.7, 1.0, 1.3]))


# -------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _trees(r, S, rows, levels, pad):
    """Random trees in topological order: parent and rank among the siblings of each node, and the node counts."""
    parent, rank, counts = [], [], []
    for _ in range(S):
        n = r.randint(1, rows) if pad else rows
        p, k, depth, kids = [-1], [0], [0], [0]
        for i in range(1, n):
            ok = [j for j in range(i) if depth[j] < levels and kids[j] < 8]
            # half of the nodes lengthen the newest branch, the others widen the tree near its root
            j = ok[-1] if r.random() < 0.5 else r.choice(ok[:max(1, len(ok) // 2)])
            p.append(j)
            k.append(kids[j])
            kids[j] += 1
            kids.append(0)
            depth.append(depth[j] + 1)
        parent.append(p + [PAD] * (rows - n))
        rank.append(k + [0] * (rows - n))
        counts.append(n)
    return parent, rank, counts


def _pages(r, S, cap, page):
    """A shuffled page table [S][cap / page] and the pool's size (one page spare)."""
    per = cap // page
    ids = list(range(S * per + 1))
    r.shuffle(ids)
    return [ids[s * per:(s + 1) * per] for s in range(S)], S * per + 1


def _pow2(e):
    """2^e in 32 bits, for -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _row_exponent(x):
    """The cache scale's exponent of each row: the smallest e with max|x| <= 448 * 2^e."""
    m, k = torch.frexp(x.abs().amax(-1))
    e = k - 9 + (m > 0.875).to(k.dtype)
    return torch.where(m == 0, torch.full_like(e, -EXP_LIM), e).clamp(-EXP_LIM, EXP_LIM)


def _quantise(x):
    """Rows of x -> (e4m3 codes, biased exponents)."""
    x = x.float()
    e = _row_exponent(x)
    y = (x * _pow2(-e).unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn), (e + EXP_BIAS).to(torch.uint8)


def _values(codes, ex):
    return codes.float() * _pow2(ex.int() - EXP_BIAS).unsqueeze(-1)


def _prepare_attn(c, seed):
    g, r = _gen(seed), random.Random(seed)
    S, rows, nq, nkv, d, dt = c["S"], c["rows"], c["nq"], c["nkv"], c["d"], _dt(c["dtype"])
    lens = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(S)]
    parent, _, counts = _trees(r, S, rows, 16, c["pad"])
    unit = c["page"] or 1
    cap = -(-max(max(lens), 1) // unit) * unit
    if c["page"]:
        pages, pool = _pages(r, S, cap, c["page"])
        shape = (pool, nkv, c["page"], d)
    else:
        pages, shape = None, (S, nkv, cap, d)
    n = lambda *s, std=1.0: torch.empty(s, device="cuda").normal_(0.0, std, generator=g)
    st = dict(case=c, lens=lens, counts=counts, parent=_i32(parent), base=_i32(lens), cap=cap,
              q=n(S * rows, nq * d, std=1.5).to(dt), kb=n(S, rows, nkv, d).to(dt), vb=n(S, rows, nkv, d).to(dt),
              out=torch.zeros(S * rows, nq * d, dtype=dt, device="cuda"),
              pages=None if pages is None else _i32(pages), pool=shape[0] if pages else 0)
    for x in "kv":
        t = n(*shape)
        t *= torch.empty(shape[:-1] + (1,), device="cuda").uniform_(0.5, 2.0, generator=g)
        if c["cache"] == "e4m3":
            st[x + "c"], st[x + "e"] = _quantise(t)
        else:
            st[x + "c"], st[x + "e"] = t.to(dt), None
    return st


def _prepare_kv(c, seed):
    g, r = _gen(seed), random.Random(seed)
    S, rows, L, nkv, d, dt = c["S"], c["rows"], c["layers"], c["nkv"], c["d"], _dt(c["dtype"])
    base = [r.randint(0, c["base_hi"]) for _ in range(S)]
    valid = [r.randint(1, rows) if c["path"] else rows for _ in range(S)]
    index = [sorted(r.sample(range(rows), v)) + [-1] * (rows - v) for v in valid] if c["path"] else None
    unit = c["page"] or 1
    cap = -(-(max(base) + rows) // unit) * unit
    if c["page"]:
        pages, pool = _pages(r, S, cap, c["page"])
        shape = (L, pool, nkv, c["page"], d)
    else:
        pages, pool, shape = None, 0, (L, S, nkv, cap, d)
    st = dict(case=c, base_l=base, valid_l=valid, index_l=index, cap=cap, base=_i32(base), valid=_i32(valid),
              index=None if index is None else _i32(index), pages=None if pages is None else _i32(pages), pool=pool)
    for x in "kv":
        t = torch.empty((L, S, rows, nkv, d), device="cuda").normal_(0.0, 1.0, generator=g)
        t *= torch.empty((L, S, rows, nkv, 1), device="cuda").uniform_(0.25, 4.0, generator=g)
        st[x + "b"] = t.to(dt)
        st[x + "o"] = torch.zeros((L, S, rows, nkv, d), dtype=dt, device="cuda")
        st[x + "c"] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        st[x + "e"] = torch.full(shape[:-1], EXP_BIAS, dtype=torch.uint8, device="cuda")
    # each written slot's (page or sequence, offset), for the plain form
    s_of, i_of, src, at, off = [], [], [], [], []
    for s in range(S):
        for i in range(valid[s]):
            slot = base[s] + i
            s_of.append(s)
            i_of.append(i)
            src.append(index[s][i] if index else i)
            at.append(pages[s][slot // c["page"]] if pages else s)
            off.append(slot % c["page"] if pages else slot)
    st["map"] = [torch.tensor(x, device="cuda") for x in (s_of, i_of, src, at, off)]
    return st


def _prepare_accept(c, seed):
    g, r = _gen(seed), random.Random(seed)
    S, rows, V, levels, T = c["S"], c["rows"], c["vocab"], c["levels"], c["T"]
    parent, rank, counts = _trees(r, S, rows, levels, False)
    n = lambda *s, std=1.0: torch.empty(s, device="cuda").normal_(0.0, std, generator=g)
    draft = n(S, levels, V, std=2.0)
    # a language model's head: a few tokens carry most of the mass, in falling shares
    K = min(V, 12)
    first = torch.randint(0, V, (S, levels, 1), device="cuda", generator=g)
    step = torch.randint(1, V // K + 1, (S, levels, 1), device="cuda", generator=g)
    top = (first + step * torch.arange(K, device="cuda")) % V
    lift = math.log(V) * T + 2.0 / T + 2.5 * T - torch.arange(K, device="cuda") * 1.2 * T
    draft.scatter_(2, top, lift.expand(S, levels, K).contiguous())
    if c["drawn"]:  # without replacement, best first: the Gumbel-top-k order of each level's distribution
        noise = torch.empty_like(draft).exponential_(generator=g).clamp_(min=1e-30)
        cand = torch.topk(draft / T - torch.log(noise), min(8, V), dim=-1).indices
    else:
        cand = torch.topk(draft, min(8, V), dim=-1).indices
    depth = [[0] * rows for _ in range(S)]
    for s in range(S):
        for i in range(1, rows):
            depth[s][i] = depth[s][parent[s][i]] + 1
    dep, rnk = torch.tensor(depth, device="cuda"), torch.tensor(rank, device="cuda")
    seq = torch.arange(S, device="cuda")[:, None]
    tokens = torch.where(dep > 0, cand[seq, (dep - 1).clamp(min=0), rnk], torch.zeros_like(dep)).int()
    target = torch.empty(S, rows, V, device="cuda")
    for s in range(S):  # the target after node i agrees with the draft's next level up to noise
        target[s] = draft[s][dep[s].clamp(max=levels - 1)] + n(rows, V, std=0.4)
    st = dict(case=c, parent=_i32(parent), tokens=tokens, target=target, draft=draft if c["drawn"] else None,
              u=torch.rand(S, rows, device="cuda", generator=g),
              noise=torch.empty(S, V, device="cuda").exponential_(generator=g).clamp_(min=1e-30),
              base=_i32([r.randint(0, 4096) for _ in range(S)]))
    for k in ("accept_len", "next"):
        st[k] = torch.zeros(S, dtype=torch.int32, device="cuda")
    for k in ("path", "out"):
        st[k] = torch.zeros(S, rows, dtype=torch.int32, device="cuda")
    return st


def prepare(case, seed):
    st = {"attn": _prepare_attn, "kv": _prepare_kv, "accept": _prepare_accept}[case["op"]](case, seed)
    if own:
        {"attn": _handle_attn, "kv": _handle_kv, "accept": _handle_accept}[case["op"]](st)
    return st


# ------------------------------------------------- the library's calls


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _dims(D, c, nq=None, vocab=8):
    return D.dflash_dims(8, nq or c.get("nq", c.get("nkv", 1)), c.get("nkv", 1), c.get("d", 64), 8, vocab, 1e4, 1e-6,
                         D.DFLASH_BF16 if c.get("dtype") == "bf16" else D.DFLASH_F32)


def _workspace(D, st, op, args):
    st["ws_bytes"] = D.dflash_workspace_bytes(op, args)
    st["ws"] = torch.zeros(st["ws_bytes"] + 256, dtype=torch.uint8, device="cuda")
    st["ws_ptr"] = (st["ws"].data_ptr() + 255) & ~255
    D.dflash_workspace_init(st["ws_ptr"], st["ws_bytes"])


def _kv_desc(D, st, k, v, ke, ve):
    kv = D.dflash_kv(_ptr(k), _ptr(v), st["cap"], 0)
    if st["pages"] is not None:
        page = st["case"]["page"]
        kv.pages, kv.page_size, kv.max_pages, kv.pool_pages = _ptr(st["pages"]), page, st["cap"] // page, st["pool"]
    kv.k_exp, kv.v_exp = _ptr(ke), _ptr(ve)
    return kv


def _handle_attn(st):
    from block_diffusion_speculative_step_gb300 import dflash as D
    c = st["case"]
    a = D.dflash_tree_attention_args()
    a.dims = _dims(D, c)
    a.n_seqs, a.rows, a.max_pos = c["S"], c["rows"], st["cap"]
    a.base_pos, a.parent = _ptr(st["base"]), _ptr(st["parent"])
    a.q, a.kb, a.vb, a.out = _ptr(st["q"]), _ptr(st["kb"]), _ptr(st["vb"]), _ptr(st["out"])
    a.kv = _kv_desc(D, st, st["kc"], st["vc"], st["ke"], st["ve"])
    _workspace(D, st, D.DFLASH_OP_TREE_ATTENTION, a)
    st["D"], st["args"] = D, a


def _handle_kv(st):
    import ctypes as C

    from block_diffusion_speculative_step_gb300 import dflash as D
    c, L = st["case"], st["case"]["layers"]
    ptrs = lambda t: (C.c_void_p * L)(*[t[j].data_ptr() for j in range(L)])
    st["arrays"] = [ptrs(st["kb"]), ptrs(st["vb"]), ptrs(st["ko"]), ptrs(st["vo"]),
                    (D.dflash_kv * L)(*[_kv_desc(D, st, st["kc"][j], st["vc"][j], st["ke"][j], st["ve"][j])
                                        for j in range(L)])]
    kb, vb, ko, vo, kvs = [C.addressof(x) for x in st["arrays"]]
    w, r = D.dflash_kv_write_args(), D.dflash_kv_read_args()
    for a in (w, r):
        a.dims, a.n_layers, a.kv_layers = _dims(D, c), L, kvs
        a.n_seqs, a.rows, a.base_pos, a.valid = c["S"], c["rows"], _ptr(st["base"]), _ptr(st["valid"])
    w.kb, w.vb, w.row_index = kb, vb, _ptr(st["index"])
    r.k_out, r.v_out = ko, vo
    _workspace(D, st, D.DFLASH_OP_KV_WRITE, w)
    st["D"], st["args"] = D, (w, r)


def _handle_accept(st):
    from block_diffusion_speculative_step_gb300 import dflash as D
    c = st["case"]
    a = D.dflash_tree_accept_args()
    a.dims = _dims(D, c, nq=1, vocab=c["vocab"])
    a.n_seqs, a.rows, a.levels, a.temperature = c["S"], c["rows"], c["levels"], c["T"]
    a.parent, a.tokens = _ptr(st["parent"]), _ptr(st["tokens"])
    a.target_logits, a.draft_logits = _ptr(st["target"]), _ptr(st["draft"])
    a.u, a.noise, a.base_pos = _ptr(st["u"]), _ptr(st["noise"]), _ptr(st["base"])
    a.accept_len, a.path, a.out_tokens, a.next_anchor = (_ptr(st[k]) for k in ("accept_len", "path", "out", "next"))
    _workspace(D, st, D.DFLASH_OP_TREE_ACCEPT, a)
    st["D"], st["args"] = D, a


def _run_own(st):
    D, a, ws = st["D"], st["args"], (st["ws_ptr"], st["ws_bytes"])
    op = st["case"]["op"]
    if op == "attn":
        D.dflash_tree_attention(a, *ws)
        return st["out"]
    if op == "kv":
        D.dflash_kv_write(a[0], *ws)
        D.dflash_kv_read(a[1], *ws)
        return [st["ko"], st["vo"]]
    D.dflash_tree_accept(a, *ws)
    return [st["accept_len"], st["path"], st["out"], st["next"]]


# ------------------------------------------------------------ the plain form


def _ancestors(parent):
    """[rows][rows] truth values: row i sees row j (its ancestors and itself)."""
    n = parent.shape[0]
    see = torch.eye(n, dtype=torch.bool, device=parent.device)
    hop = torch.zeros(n, n, dtype=torch.float32, device=parent.device)
    idx = torch.arange(n, device=parent.device)
    hop[idx, parent.clamp(min=0)] = (parent >= 0).float()
    reach = hop
    for _ in range(max(1, (n - 1).bit_length())):
        reach = ((reach + reach @ reach) > 0).float()
    return see | (reach > 0)


def _context(st, x, s, n):
    """The first n cached rows of sequence s: [nkv][n][d], in 32 bits."""
    c, t, e = st["case"], st[x + "c"], st[x + "e"]
    if c["page"]:
        ids = st["pages"][s, :-(-n // c["page"])].long()
        pick = lambda y: y[ids].transpose(0, 1).flatten(1, 2)[:, :n]
    else:
        pick = lambda y: y[s, :, :n]
    return _values(pick(t), pick(e)) if e is not None else pick(t).float()


def _plain_attn(st):
    c, out = st["case"], st["out"]
    S, rows, nq, nkv, d = c["S"], c["rows"], c["nq"], c["nkv"], c["d"]
    q = st["q"].float().view(S, rows, nkv, nq // nkv, d)
    o = out.view(S, rows, nkv, nq // nkv, d)
    for s in range(S):
        n = st["lens"][s]
        k = torch.cat([_context(st, "k", s, n), st["kb"][s].float().transpose(0, 1)], 1)
        v = torch.cat([_context(st, "v", s, n), st["vb"][s].float().transpose(0, 1)], 1)
        see = _ancestors(st["parent"][s])
        sc = torch.matmul(q[s].permute(1, 2, 0, 3).reshape(nkv, -1, d), k.transpose(1, 2)) / math.sqrt(d)
        sc = sc.view(nkv, nq // nkv, rows, -1)
        sc[..., n:] = sc[..., n:].masked_fill(~see, -math.inf)
        p = torch.exp(sc - sc.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        r = torch.matmul(p.view(nkv, -1, p.shape[-1]), v).view(nkv, nq // nkv, rows, d).permute(2, 0, 1, 3)
        m = st["counts"][s]
        o[s, :m] = r[:m].to(out.dtype)
    return out


def _plain_kv(st):
    s, i, src, at, off = st["map"]
    for x in "kv":
        codes, ex = _quantise(st[x + "b"][:, s, src])  # [layers][slots][nkv][d]
        st[x + "c"][:, at, :, off] = codes.view(torch.uint8).transpose(0, 1)
        st[x + "e"][:, at, :, off] = ex.transpose(0, 1)
    for x in "kv":
        codes, ex = st[x + "c"][:, at, :, off].view(torch.float8_e4m3fn), st[x + "e"][:, at, :, off]
        st[x + "o"][:, s, i] = _values(codes, ex).to(st[x + "o"].dtype).transpose(0, 1)
    return [st["ko"], st["vo"]]


def _plain_accept(st):
    c = st["case"]
    S, rows, V, T = c["S"], c["rows"], c["vocab"], c["T"]
    seq = torch.arange(S, device="cuda")
    parent, tokens = st["parent"].long(), st["tokens"].long()

    def weights(l):  # exp(l / T) against the row's maximum, and their sum in 64 bits
        e = torch.exp((l - l.amax(-1, keepdim=True)) / T)
        return e, e.sum(-1, dtype=torch.float64)

    cur = torch.zeros(S, dtype=torch.long, device="cuda")
    k = torch.zeros(S, dtype=torch.long, device="cuda")
    path = torch.full((S, rows), -1, dtype=torch.int32, device="cuda")
    out = torch.full((S, rows), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    p, z = weights(st["target"][:, 0])
    if st["draft"] is not None:
        q, y = weights(st["draft"][:, 0])
    for i in range(1, rows):
        test = parent[:, i] == cur
        x = tokens[:, i]
        px = p[seq, x].double() / z
        qx = q[seq, x].double() / y if st["draft"] is not None else torch.ones_like(px)
        ok = test & (st["u"][:, i].double() * qx < px)
        no = test & ~ok
        # a rejected candidate: the target keeps what the proposal did not cover
        if st["draft"] is not None:
            res = (p.double() / z[:, None] - q.double() / y[:, None]).clamp(min=0)
            rs = res.sum(-1)
            use = (no & (rs > 0))[:, None]
            p = torch.where(use, res, p.double())
            z = torch.where(use[:, 0], rs, z)
            q = q.clone()
            q[seq, x] = torch.where(no, torch.zeros_like(q[seq, x]), q[seq, x])
            y = torch.where(no, q.sum(-1, dtype=torch.float64), y)
        else:
            p = p.clone()
            p[seq, x] = torch.where(no, torch.zeros_like(p[seq, x]), p[seq, x])
            z = torch.where(no, p.sum(-1, dtype=torch.float64), z)
        # an accepted one: the walk goes on below it
        out[seq, k] = torch.where(ok, x.int(), out[seq, k])
        k = k + ok.long()
        cur = torch.where(ok, torch.full_like(cur, i), cur)
        path[seq, k] = torch.where(ok, cur.int(), path[seq, k])
        pn, zn = weights(st["target"][seq, cur])
        p = torch.where(ok[:, None], pn.to(p.dtype), p)
        z = torch.where(ok, zn, z)
        if st["draft"] is not None:
            qn, yn = weights(st["draft"][seq, k.clamp(max=c["levels"] - 1)])
            q = torch.where(ok[:, None], qn, q)
            y = torch.where(ok, yn, y)
    last = torch.argmax(p.double() / st["noise"].double(), -1).int()
    out[seq, k] = last
    return [k.int(), path, out, last]


def run(st):
    if own:
        return _run_own(st)
    return {"attn": _plain_attn, "kv": _plain_kv, "accept": _plain_accept}[st["case"]["op"]](st)


# ------------------------------------------------- the definition in 64 bits


def _exact_attn(st):
    c = st["case"]
    S, rows, nq, nkv, d = c["S"], c["rows"], c["nq"], c["nkv"], c["d"]
    out = torch.zeros(S, rows, nq, d, dtype=torch.float64, device="cuda")
    q = st["q"].double().view(S, rows, nq, d)
    parent = st["parent"].tolist()

    def row64(x, s, n):
        t, e = st[x + "c"], st[x + "e"]
        parts, scales = [], []
        step = c["page"] or max(n, 1)
        for a in range(0, n, step):
            b = min(n, a + step)
            at = int(st["pages"][s, a // step]) if c["page"] else s
            parts.append(t[at, :, :b - a].double())
            if e is not None:
                scales.append(torch.pow(2.0, e[at, :, :b - a].double() - EXP_BIAS))
        parts = [p * w[..., None] for p, w in zip(parts, scales)] if scales else parts
        return torch.cat(parts + [st[x + "b"][s].double().transpose(0, 1)], 1)

    for s in range(S):
        n = st["lens"][s]
        hide = torch.ones(rows, n + rows, dtype=torch.bool)
        hide[:, :n] = False
        for i in range(rows):
            j = i
            while j >= 0:
                hide[i, n + j] = False
                j = parent[s][j]
        hide = hide.cuda()
        k, v = row64("k", s, n), row64("v", s, n)
        for h in range(nq):
            g = h // (nq // nkv)
            sc = (q[s, :, h] @ k[g].T) / d ** 0.5
            out[s, :, h] = torch.softmax(sc.masked_fill(hide, -math.inf), -1) @ v[g]
        out[s, st["counts"][s]:] = 0
    return out.view(S * rows, nq * d)


def _exact_kv(st):
    c = st["case"]
    two_to = lambda e: ((e.long() + 1023) << 52).view(torch.float64)  # exact, so that ties stay ties
    res = []
    for x in "kv":
        src = st[x + "b"].double()
        out = torch.zeros_like(src)
        for s in range(c["S"]):
            for i in range(st["valid_l"][s]) if c["path"] else [slice(0, st["valid_l"][s])]:
                y = src[:, s, st["index_l"][s][i] if c["path"] else i]
                # (1e-9: log2 may land just above the whole number that a power of two has)
                e = torch.ceil(torch.log2(y.abs().amax(-1, keepdim=True) / E4M3_MAX) - 1e-9).clamp(-EXP_LIM, EXP_LIM)
                y = y * two_to(-e)
                ulp = two_to(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
                out[:, s, i] = torch.round(y / ulp) * ulp * two_to(e)
        res.append(out)
    return res


def _exact_accept(st):
    c = st["case"]
    S, rows, T = c["S"], c["rows"], c["T"]
    parent, tokens, u = st["parent"].tolist(), st["tokens"].tolist(), st["u"].double().tolist()
    lens, paths, outs, lasts = [], [], [], []
    for s in range(S):
        node, path, toks = 0, [0], []
        while True:
            p = torch.softmax(st["target"][s, node].double() / T, -1)
            q = torch.softmax(st["draft"][s, len(toks)].double() / T, -1) if st["draft"] is not None and \
                len(toks) < c["levels"] else None
            went = None
            for i in [j for j in range(rows) if j > 0 and parent[s][j] == node]:
                x = tokens[s][i]
                if u[s][i] * (float(q[x]) if q is not None else 1.0) < float(p[x]):
                    went = i
                    break
                if q is not None:
                    left = torch.clamp(p - q, min=0)
                    if float(left.sum()) > 0:
                        p = left / left.sum()
                    q[x] = 0
                    if float(q.sum()) > 0:
                        q = q / q.sum()
                else:
                    p[x] = 0
                    if float(p.sum()) > 0:
                        p = p / p.sum()
            if went is None:
                break
            node = went
            path.append(node)
            toks.append(tokens[s][node])
        lasts.append(int(torch.argmax(p / st["noise"][s].double())))
        lens.append(len(toks))
        paths.append(path + [-1] * (rows - len(path)))
        outs.append(toks + [lasts[-1]] + [-1] * (rows - len(toks) - 1))
    return [_i32(lens), _i32(paths), _i32(outs), _i32(lasts)]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"attn": _exact_attn, "kv": _exact_kv, "accept": _exact_accept}[case["op"]](st)


# ---------------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] == "attn":
        es = 2 if c["dtype"] == "bf16" else 4
        ctx = (c["ctx_lo"] + c["ctx_hi"]) / 2 * c["S"]
        nodes = (c["rows"] + 1) / 2 if c["pad"] else c["rows"]
        slot = 2 * c["nkv"] * (c["d"] + 1 if c["cache"] == "e4m3" else c["d"] * es)
        tree = c["S"] * nodes * c["d"] * es * (2 * c["nkv"] + 2 * c["nq"])
        keys = ctx / c["S"] + min(nodes, 8)  # the context and the ancestors of a node
        return {"bytes": ctx * slot + tree, "flops": 4.0 * c["S"] * nodes * c["nq"] * keys * c["d"]}
    if c["op"] == "kv":
        es = 2 if c["dtype"] == "bf16" else 4
        n = (c["rows"] + 1) / 2 if c["path"] else c["rows"]
        vecs = 2.0 * c["layers"] * c["S"] * c["nkv"] * n
        # the source read, codes and exponent written, read back, the values written
        return {"bytes": vecs * (2 * c["d"] * es + 2 * (c["d"] + 1)), "flops": vecs * c["d"] * 4}
    # the rows of logits that the walk visits: about five accepted tokens where the tree is that deep
    rows = min(6, c["rows"], c["levels"] + 1)
    row = c["vocab"] * 4.0
    return {"bytes": c["S"] * row * (rows * (2 if c["drawn"] else 1) + 1), "flops": c["S"] * c["vocab"] * rows * 8.0}
