"""The prompt's operators of the library: what they compute, on which sizes
they are measured, and the work they cannot do without.

Three operators of one serving path -- prompts of different lengths, packed
one behind the other, enter the target and are scored:

  attn    causal attention of packed prompts, or of their next pieces over
          what the cache holds of them (dflash_prompt_attention);
  qk      RMS norms of every query and key head and the position rotation in
          one pass over the projection's output, keys and values to the cache
          or token-major (dflash_qk_norm_rope);
  scores  the log probabilities of given tokens, the entropy and the best
          alternatives of every row of logits (dflash_token_logprobs).

`own` selects the library's kernels; otherwise run() computes the same from
elementary torch operations.
"""
from __future__ import annotations

import math
import random

import torch

own = False

THETA = 1e6
EPS = 1e-6

# --------------------------------------------------------------------- cases


def listed():
    q8 = dict(nq=32, nkv=8, d=128)         # the 8B-shaped target of the benchmark
    coder = dict(nq=32, nkv=4, d=128)      # the long-context shape of the benchmark
    return [
        # one long prompt, whole
        dict(name="attn-b1-8k-bf16", op="attn", S=1, lo=8192, hi=8192, ctx_lo=0, ctx_hi=0, **q8, dtype="bf16", page=0),
        # a serving batch: 16 prompts of 64 to 4096 tokens in one call
        dict(name="attn-b16-ragged-bf16", op="attn", S=16, lo=64, hi=4096, ctx_lo=0, ctx_hi=0, **q8, dtype="bf16",
             page=0),
        # the last 512 tokens of a 32k prompt taken in pieces, over a paged cache
        dict(name="attn-b1-n512-32k-bf16", op="attn", S=1, lo=512, hi=512, ctx_lo=32256, ctx_hi=32256, **coder,
             dtype="bf16", page=256),
        # a few short follow-ups of odd lengths over short cached turns: the smallest call (latency)
        dict(name="attn-b7-short-bf16", op="attn", S=7, lo=1, hi=33, ctx_lo=0, ctx_hi=131, nq=8, nkv=2, d=64,
             dtype="bf16", page=128),
        # the prompts of the tiny lossless configuration, in full precision
        dict(name="attn-b3-n64-f32", op="attn", S=3, lo=64, hi=64, ctx_lo=0, ctx_hi=0, nq=4, nkv=4, d=64, dtype="f32",
             page=0),
        # one token of one user: every layer of every decoding step (latency)
        dict(name="qk-b1-n1-bf16", op="qk", S=1, rows=1, base_hi=4000, **q8, dtype="bf16", src="f32", norm=True,
             cache=True, page=0, gap=0),
        # 32 sequences' verification blocks, into a paged cache
        dict(name="qk-b32-n16-bf16", op="qk", S=32, rows=16, base_hi=1900, **q8, dtype="bf16", src="f32", norm=True,
             cache=True, page=128, gap=0),
        # a packed prompt of 8k tokens, token-major
        dict(name="qk-8k-bf16", op="qk", S=8192, rows=1, base_hi=8191, **q8, dtype="bf16", src="f32", norm=True,
             cache=False, page=0, gap=0),
        # one decoded token's scores with five alternatives (latency)
        dict(name="scores-1-v151936", op="scores", M=1, vocab=151936, k=5, T=1.0),
        # a prompt's scores, as an evaluation asks for them
        dict(name="scores-512-v151936", op="scores", M=512, vocab=151936, k=20, T=1.0),
        # a short vocabulary of odd size
        dict(name="scores-33-v1021", op="scores", M=33, vocab=1021, k=8, T=0.7),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng: random.Random):
    op = rng.choice(["attn", "attn", "qk", "scores"])
    if op == "attn":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        S = _log_int(rng, 1, 32)
        nq, nkv = rng.choice([(32, 8), (32, 4), (8, 8), (12, 4), (14, 2), (4, 4), (8, 1)])
        d = rng.choice([64, 128])
        # pairs of one pass: at most half of the largest listed case's (a thirty-second in full precision)
        budget = 32 * 8192 * 8192 // (4 if dtype == "bf16" else 64)
        hi = _log_int(rng, 1, max(2, min(8192, int(math.sqrt(2 * budget / (S * nq))))))
        left = max(1, budget // (S * nq * hi) - hi // 2)
        ctx = rng.choice([0, 0, 1, _log_int(rng, 1, min(32768, left))])
        return dict(op="attn", S=S, lo=rng.choice([0, 1, hi]), hi=hi, ctx_lo=rng.choice([0, ctx]), ctx_hi=ctx, nq=nq,
                    nkv=nkv, d=d, dtype=dtype, page=rng.choice([0, 128, 256]))
    if op == "qk":
        S = _log_int(rng, 1, 64)
        rows = _log_int(rng, 1, max(1, 8192 // (2 * S)))
        nq, nkv = rng.choice([(32, 8), (32, 4), (8, 8), (12, 4), (14, 2), (4, 4), (8, 1)])
        return dict(op="qk", S=S, rows=rows, base_hi=rng.choice([0, 5, 130, 1000]), nq=nq, nkv=nkv,
                    d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    src=rng.choice(["bf16", "f32"]), norm=rng.random() < 0.8, cache=rng.random() < 0.5,
                    page=rng.choice([0, 128, 256]), gap=rng.choice([0, 0, 64]))
    vocab = _log_int(rng, 40, 151936)
    M = _log_int(rng, 1, max(1, min(1024, 512 * 151936 // (2 * vocab))))
    return dict(op="scores", M=M, vocab=vocab, k=rng.choice([0, 1, 5, 20, 32]), T=rng.choice([0.5, 0.7, 1.0, 1.3]))


# -------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _lengths(c):
    """A case's prompt and context lengths: part of the case, as the work is."""
    r = random.Random("%d %d %d %d %d" % (c["S"], c["lo"], c["hi"], c["ctx_lo"], c["ctx_hi"]))
    rows = [r.randint(c["lo"], c["hi"]) for _ in range(c["S"])]
    rows[-1] = max(rows[-1], 1)
    return rows, [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["S"])]


def _pages(r, S, cap, page):
    """A shuffled page table [S][cap / page] and the pool's size (one page spare)."""
    per = cap // page
    ids = list(range(S * per + 1))
    r.shuffle(ids)
    return [ids[s * per:(s + 1) * per] for s in range(S)], S * per + 1


def _prepare_attn(c, seed):
    g, r = _gen(seed), random.Random(seed)
    S, nq, nkv, d, dt = c["S"], c["nq"], c["nkv"], c["d"], _dt(c["dtype"])
    lens, ctx = _lengths(c)
    start = [0]
    for n in lens:
        start.append(start[-1] + n)
    M = start[-1]
    n = lambda *s, std=1.0: torch.empty(s, device="cuda").normal_(0.0, std, generator=g)
    st = dict(case=c, lens=lens, ctx=ctx, start=start, row_start=_i32(start), base=_i32(ctx), cap=0, pages=None, pool=0,
              q=n(M, nq * d, std=1.5).to(dt), kb=n(M, nkv, d).to(dt), vb=n(M, nkv, d).to(dt),
              out=torch.zeros(M, nq * d, dtype=dt, device="cuda"), kc=None, vc=None)
    if c["ctx_hi"] > 0:
        unit = c["page"] or 1
        st["cap"] = -(-max(max(ctx), 1) // unit) * unit
        shape = (S, nkv, st["cap"], d)
        if c["page"]:
            pages, st["pool"] = _pages(r, S, st["cap"], c["page"])
            st["pages"] = _i32(pages)
            shape = (st["pool"], nkv, c["page"], d)
        st["kc"], st["vc"] = n(*shape).to(dt), n(*shape).to(dt)
    return st


def _prepare_qk(c, seed):
    g, r = _gen(seed), random.Random(seed)
    S, rows, nq, nkv, d, dt = c["S"], c["rows"], c["nq"], c["nkv"], c["d"], _dt(c["dtype"])
    M, width = S * rows, (nq + 2 * nkv) * d
    base = [r.randint(0, c["base_hi"]) for _ in range(S)]
    n = lambda *s, std=1.0: torch.empty(s, device="cuda").normal_(0.0, std, generator=g)
    qkv = n(M, width + c["gap"])  # a projection's rows, of different sizes, perhaps part of a wider buffer
    qkv *= torch.empty(M, 1, device="cuda").uniform_(0.2, 5.0, generator=g)
    z = lambda *s: torch.zeros(s, dtype=dt, device="cuda")
    st = dict(case=c, base=_i32(base), max_pos=c["base_hi"] + rows, qkv=qkv.to(_dt(c["src"])), q=z(M, nq * d),
              qn=(1 + n(d, std=0.1)).to(dt) if c["norm"] else None, kn=(1 + n(d, std=0.1)).to(dt) if c["norm"] else None,
              cap=0, pages=None, pool=0)
    if c["cache"]:
        unit = c["page"] or 1
        st["cap"] = -(-st["max_pos"] // unit) * unit
        shape = (S, nkv, st["cap"], d)
        if c["page"]:
            pages, st["pool"] = _pages(r, S, st["cap"], c["page"])
            st["pages"] = _i32(pages)
            shape = (st["pool"], nkv, c["page"], d)
        st["k"], st["v"] = z(*shape), z(*shape)
    else:
        st["k"], st["v"] = z(M, nkv, d), z(M, nkv, d)
    return st


def _prepare_scores(c, seed):
    g = _gen(seed)
    M, V, k = c["M"], c["vocab"], c["k"]
    logits = torch.empty(M, V, device="cuda").normal_(0.0, 2.0, generator=g)
    # a language model's head: a few tokens carry most of the mass, in falling shares
    K = min(V, 12)
    first = torch.randint(0, V, (M, 1), device="cuda", generator=g)
    step = torch.randint(1, V // K + 1, (M, 1), device="cuda", generator=g)
    top = (first + step * torch.arange(K, device="cuda")) % V
    lift = torch.empty(M, 1, device="cuda").uniform_(4.0, 16.0, generator=g) - torch.arange(K, device="cuda") * 0.9
    logits.scatter_add_(1, top, lift.contiguous())
    # most given tokens are likely ones
    likely = top.gather(1, torch.randint(0, K, (M, 1), device="cuda", generator=g))[:, 0]
    anyone = torch.randint(0, V, (M,), device="cuda", generator=g)
    tokens = torch.where(torch.rand(M, device="cuda", generator=g) < 0.8, likely, anyone).int()
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
    return dict(case=c, logits=logits, tokens=tokens, logprob=z(M), entropy=z(M), ids=z(M, max(k, 1), dt=torch.int32),
                top=z(M, max(k, 1)))


def prepare(case, seed):
    st = {"attn": _prepare_attn, "qk": _prepare_qk, "scores": _prepare_scores}[case["op"]](case, seed)
    if own:
        {"attn": _handle_attn, "qk": _handle_qk, "scores": _handle_scores}[case["op"]](st)
    return st


# ------------------------------------------------- the library's calls


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _dims(D, c):
    return D.dflash_dims(8, c.get("nq", 1), c.get("nkv", 1), c.get("d", 64), 8, c.get("vocab", 8), THETA, EPS,
                         D.DFLASH_BF16 if c.get("dtype") == "bf16" else D.DFLASH_F32)


def _workspace(D, st, op, args):
    st["ws_bytes"] = D.dflash_workspace_bytes(op, args)
    st["ws"] = torch.zeros(st["ws_bytes"] + 256, dtype=torch.uint8, device="cuda")
    st["ws_ptr"] = (st["ws"].data_ptr() + 255) & ~255
    D.dflash_workspace_init(st["ws_ptr"], st["ws_bytes"])


def _kv_desc(D, st, k, v):
    kv = D.dflash_kv(_ptr(k), _ptr(v), st["cap"], 0)
    if st["pages"] is not None:
        page = st["case"]["page"]
        kv.pages, kv.page_size, kv.max_pages, kv.pool_pages = _ptr(st["pages"]), page, st["cap"] // page, st["pool"]
    return kv


def _handle_attn(st):
    from block_diffusion_speculative_step_gb300 import dflash as D
    a = D.dflash_prompt_attention_args()
    a.dims = _dims(D, st["case"])
    a.n_seqs, a.n_rows = st["case"]["S"], st["start"][-1]
    a.row_start = _ptr(st["row_start"])
    a.q, a.kb, a.vb, a.out = _ptr(st["q"]), _ptr(st["kb"]), _ptr(st["vb"]), _ptr(st["out"])
    if st["kc"] is not None:
        a.base_pos, a.max_pos = _ptr(st["base"]), st["cap"]
        a.kv = _kv_desc(D, st, st["kc"], st["vc"])
    _workspace(D, st, D.DFLASH_OP_PROMPT_ATTENTION, a)
    st["call"], st["args"] = D.dflash_prompt_attention, a


def _handle_qk(st):
    from block_diffusion_speculative_step_gb300 import dflash as D
    c = st["case"]
    st["rope"] = torch.zeros(st["max_pos"], c["d"] // 2, 2, device="cuda")
    D.dflash_rope_table(THETA, c["d"], st["max_pos"], st["rope"].data_ptr())
    a = D.dflash_qk_norm_rope_args()
    a.dims = _dims(D, c)
    a.n_seqs, a.rows, a.base_pos = c["S"], c["rows"], _ptr(st["base"])
    a.qkv, a.qkv_stride = _ptr(st["qkv"]), st["qkv"].shape[1]
    a.qkv_dtype = D.DFLASH_BF16 if c["src"] == "bf16" else D.DFLASH_F32
    a.q_norm, a.k_norm = _ptr(st["qn"]), _ptr(st["kn"])
    a.rope_cs, a.rope_max_pos = _ptr(st["rope"]), st["max_pos"]
    a.q = _ptr(st["q"])
    if c["cache"]:
        a.kv = _kv_desc(D, st, st["k"], st["v"])
    else:
        a.kb, a.vb = _ptr(st["k"]), _ptr(st["v"])
    _workspace(D, st, D.DFLASH_OP_QK_NORM_ROPE, a)
    st["call"], st["args"] = D.dflash_qk_norm_rope, a


def _handle_scores(st):
    from block_diffusion_speculative_step_gb300 import dflash as D
    c = st["case"]
    a = D.dflash_token_logprobs_args()
    a.dims = _dims(D, c)
    a.n_rows, a.logits, a.temperature, a.topk = c["M"], _ptr(st["logits"]), c["T"], c["k"]
    a.tokens, a.logprob, a.entropy = _ptr(st["tokens"]), _ptr(st["logprob"]), _ptr(st["entropy"])
    a.top_ids, a.top_logprobs = _ptr(st["ids"]), _ptr(st["top"])
    _workspace(D, st, D.DFLASH_OP_TOKEN_LOGPROBS, a)
    st["call"], st["args"] = D.dflash_token_logprobs, a


def _outputs(st):
    return {"attn": ["out"], "qk": ["q", "k", "v"], "scores": ["logprob", "entropy", "ids", "top"]}[st["case"]["op"]]


def _run_own(st):
    st["call"](st["args"], st["ws_ptr"], st["ws_bytes"])
    return [st[k] for k in _outputs(st)]


# ------------------------------------------------------------ the plain form


def _context(st, x, s, n):
    """The first n cached rows of sequence s: [nkv][n][d], in 32 bits."""
    t = st[x + "c"]
    if st["pages"] is None:
        return t[s, :, :n].float()
    ids = st["pages"][s, :-(-n // st["case"]["page"])].long()
    return t[ids].transpose(0, 1).flatten(1, 2)[:, :n].float()


def _plain_attn(st):
    c, out = st["case"], st["out"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    for s in range(c["S"]):
        n, p, r = st["lens"][s], st["ctx"][s], slice(st["start"][s], st["start"][s + 1])
        if n == 0:
            continue
        q = st["q"][r].float().view(n, nkv, nq // nkv, d).permute(1, 2, 0, 3)
        k, v = st["kb"][r].float().transpose(0, 1), st["vb"][r].float().transpose(0, 1)
        if p:
            k, v = torch.cat([_context(st, "k", s, p), k], 1), torch.cat([_context(st, "v", s, p), v], 1)
        sc = torch.matmul(q.reshape(nkv, -1, d), k.transpose(1, 2)).view(nkv, nq // nkv, n, p + n)
        sc *= 1.0 / math.sqrt(d)
        row = torch.arange(n, device="cuda")
        sc[..., p:].masked_fill_(row[None, :] > row[:, None], -math.inf)
        sc -= sc.amax(-1, keepdim=True)
        sc.exp_()
        w = torch.matmul(sc.view(nkv, -1, p + n), v).view(nkv, nq // nkv, n, d)
        out[r] = (w / sc.sum(-1, keepdim=True)).permute(2, 0, 1, 3).reshape(n, nq * d).to(out.dtype)
    return [out]


def _plain_qk(st):
    c = st["case"]
    S, rows, nq, nkv, d, dt = c["S"], c["rows"], c["nq"], c["nkv"], c["d"], _dt(c["dtype"])
    pos = (st["base"].long()[:, None] + torch.arange(rows, device="cuda")).view(-1)
    ang = pos.double()[:, None] * THETA ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def turned(x, gain):
        if gain is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.float()
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(dt)

    x = st["qkv"].float()
    cut = [0, nq * d, (nq + nkv) * d, (nq + 2 * nkv) * d]
    q, k, v = (x[:, a:b].reshape(S * rows, -1, d) for a, b in zip(cut, cut[1:]))
    st["q"].copy_(turned(q, st["qn"]).reshape(S * rows, -1))
    k, v = turned(k, st["kn"]), v.to(dt)
    if not c["cache"]:
        st["k"].copy_(k)
        st["v"].copy_(v)
    else:
        seq, at = torch.arange(S, device="cuda").repeat_interleave(rows), pos
        if st["pages"] is not None:
            seq, at = st["pages"][seq, pos // c["page"]].long(), pos % c["page"]
        st["k"][seq, :, at] = k
        st["v"][seq, :, at] = v
    return [st["q"], st["k"], st["v"]]


def _plain_scores(st):
    c = st["case"]
    x = st["logits"] / c["T"]
    y = x - x.amax(-1, keepdim=True)
    e = y.exp()
    z = e.sum(-1, dtype=torch.float64)
    st["logprob"].copy_(y.gather(1, st["tokens"].long()[:, None])[:, 0] - z.log())
    st["entropy"].copy_(z.log() - (e * y).sum(-1, dtype=torch.float64) / z)
    if c["k"]:
        ids = torch.sort(st["logits"], dim=-1, descending=True, stable=True).indices[:, :c["k"]]
        st["ids"].copy_(ids)
        st["top"].copy_(y.gather(1, ids) - z.log()[:, None])
    return [st[k] for k in _outputs(st)]


def run(st):
    if own:
        return _run_own(st)
    return {"attn": _plain_attn, "qk": _plain_qk, "scores": _plain_scores}[st["case"]["op"]](st)


# ------------------------------------------------- the definition in 64 bits


def _exact_attn(st):
    c = st["case"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    out = torch.zeros(st["start"][-1], nq, d, dtype=torch.float64, device="cuda")

    def rows64(x, s, g, p, a, b):
        own_rows = st[x + "b"][a:b, g].double()
        if not p:
            return own_rows
        t, step = st[x + "c"], c["page"] or p
        at = (lambda i: int(st["pages"][s, i])) if c["page"] else (lambda i: s)
        return torch.cat([t[at(i), g, :min(step, p - i * step)].double() for i in range(-(-p // step))] + [own_rows])

    for s in range(c["S"]):
        a, b, p = st["start"][s], st["start"][s + 1], st["ctx"][s]
        hidden = torch.ones(b - a, p + b - a, dtype=torch.bool, device="cuda").triu(p + 1)
        for g in range(nkv):
            k, v = rows64("k", s, g, p, a, b), rows64("v", s, g, p, a, b)
            for h in range(g * (nq // nkv), (g + 1) * (nq // nkv)):
                sc = st["q"][a:b, h * d:(h + 1) * d].double() @ k.T / d ** 0.5
                out[a:b, h] = torch.softmax(sc.masked_fill(hidden, -math.inf), -1) @ v
    return [out.view(-1, nq * d)]


def _exact_qk(st):
    c = st["case"]
    S, rows, nq, nkv, d = c["S"], c["rows"], c["nq"], c["nkv"], c["d"]
    pos = (st["base"].double()[:, None] + torch.arange(rows, device="cuda")).view(-1)
    w = torch.exp(torch.arange(d // 2, device="cuda", dtype=torch.float64) * (-2.0 * math.log(THETA) / d))
    turn = torch.polar(torch.ones_like(pos)[:, None, None], pos[:, None, None] * w)
    x = st["qkv"][:, :(nq + 2 * nkv) * d].double().view(S * rows, nq + 2 * nkv, d)

    def head(y, gain):
        if gain is not None:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / d + EPS) * gain.double()
        y = torch.complex(y[..., :d // 2].contiguous(), y[..., d // 2:].contiguous()) * turn
        return torch.cat([y.real, y.imag], -1)

    q, k, v = head(x[:, :nq], st["qn"]), head(x[:, nq:nq + nkv], st["kn"]), x[:, nq + nkv:]
    if c["cache"]:
        place = []
        for y in (k, v):
            t = torch.zeros(st["k"].shape, dtype=torch.float64, device="cuda")
            for s, base in enumerate(st["base"].tolist()):
                table = st["pages"][s].tolist() if st["pages"] is not None else None
                for i in range(rows):
                    n = base + i
                    if table is None:
                        t[s, :, n] = y[s * rows + i]
                    else:
                        t[table[n // c["page"]], :, n % c["page"]] = y[s * rows + i]
            place.append(t)
        k, v = place
    return [q.reshape(S * rows, nq * d), k, v]


def _exact_scores(st):
    c = st["case"]
    logits = st["logits"].double()
    p = torch.log_softmax(logits / c["T"], -1)
    lp = torch.gather(p, 1, st["tokens"].long()[:, None])[:, 0]
    ent = -(p.exp() * p).sum(-1)
    ids, top = st["ids"].clone(), torch.zeros_like(st["top"], dtype=torch.float64)
    left = logits.clone()
    row = torch.arange(c["M"], device="cuda")
    for j in range(c["k"]):
        best = left.amax(-1, keepdim=True)
        at = torch.where(left == best, torch.arange(c["vocab"], device="cuda"), c["vocab"]).amin(-1)
        ids[:, j] = at.int()
        top[:, j] = p[row, at]
        left[row, at] = -math.inf
    return [lp, ent, ids, top]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"attn": _exact_attn, "qk": _exact_qk, "scores": _exact_scores}[case["op"]](st)


# ---------------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] == "attn":
        es = 2 if c["dtype"] == "bf16" else 4
        lens, ctx = _lengths(c)
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(lens, ctx))  # (row, key it sees)
        # queries, the rows' keys and values and the seen context read, the output written
        vecs = sum(lens) * (2 * c["nq"] + 2 * c["nkv"]) + sum(p for n, p in zip(lens, ctx) if n) * 2 * c["nkv"]
        return {"bytes": float(vecs * c["d"] * es), "flops": 4.0 * pairs * c["nq"] * c["d"]}
    if c["op"] == "qk":
        es, ss = (2 if x == "bf16" else 4 for x in (c["dtype"], c["src"]))
        heads = c["S"] * c["rows"] * (c["nq"] + 2 * c["nkv"])
        return {"bytes": float(heads * c["d"] * (es + ss)), "flops": 10.0 * heads * c["d"]}
    return {"bytes": c["M"] * (c["vocab"] * 4.0 + c["k"] * 8 + 12), "flops": 6.0 * c["M"] * c["vocab"]}
