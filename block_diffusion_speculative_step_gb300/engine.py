"""Device buffers and the call sequence of one DFlash cycle on the C ABI.

A cycle ("DFlash ..." guide, section 4) is, all on one CUDA stream and with
no host synchronisation:

  draft_block(anchor, base_pos)            -> drafts        (draft model, block-bidirectional)
  embed([anchor, drafts]); target layers   -> h, tap feats  (causal verification forward)
  verify_accept(h, drafts)                 -> accept_len, out_tokens; anchor := bonus,
                                              commit = (base_pos, k + 1), base_pos += k + 1
  fuse_context(feats, commit)              -> draft context K/V of the committed positions

A tree cycle (tree_cycle) verifies several candidates a position instead of
one: the draft's candidates become a tree of rows, the target runs over the
tree, the walk down the tree accepts a path, and only that path's keys and
values are committed to the target cache.

Torch here only allocates device memory, provides the stream and puts rows in
order (tokens of a tree forward, the accepted rows' tap features); every
other step of a cycle runs in libdflash kernels.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import torch

from . import dflash as D
from . import synth


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def dims_of(w: synth.Workload, s: synth.Shape) -> D.dflash_dims:
    return D.dflash_dims(s.hidden, s.n_q, s.n_kv, s.head_dim, s.inter, w.vocab, w.rope_theta, w.rms_eps,
                         D.DFLASH_BF16 if w.dtype == "bf16" else D.DFLASH_F32)


def layer_weights(L: dict) -> D.dflash_layer_weights:
    return D.dflash_layer_weights(_ptr(L["w_qkv"]), _ptr(L["w_o"]), _ptr(L["w_gu"]), _ptr(L["w_down"]),
                                  _ptr(L["ln1"]), _ptr(L["ln2"]))


@dataclass
class Caches:
    tk: list  # target K per layer [S][nkv][cap][d]
    tv: list
    dk: list  # draft context K per layer [S][nkv][dcap][d]
    dv: list
    tke: list  # 8-bit target caches: scale exponents [S][nkv][cap]
    tve: list


class Engine:
    """One target + draft pair resident on the GPU, n_seqs sequences.

    kv8: the target's caches hold 8-bit e4m3 rows with a power-of-two scale
    per (slot, KV head), half the bytes of bf16.  Target forwards then run as
    tree forwards (a chain where no tree is given) whose keys and values are
    committed by dflash_kv_write.  The rows of one forward see each other
    unquantised, later ones see them quantised: over an 8-bit cache tree cycles,
    chain cycles and one-token decoding may part within the quantisation."""

    def __init__(self, w: synth.Workload, model: dict, n_seqs: int, cap: int, device="cuda",
                 prefill_chunk: int = 256, fuse_rows: int = 0, kv8: bool = False):
        self.w = w
        self.m = model
        self.S = n_seqs
        self.B = w.block
        self.cap = cap
        self.dev = torch.device(device)
        self.dt = synth.torch_dtype(w)
        self.chunk = min(prefill_chunk, D.DFLASH_MAX_TREE) if kv8 else prefill_chunk
        self.kv8 = kv8
        self.F = len(w.taps)
        tdims = w.target
        self.ddims = dims_of(w, w.draft)
        self.tdims = dims_of(w, tdims) if "target" in model else None
        self.has_target = "target" in model
        H = w.draft.hidden
        S, B = n_seqs, self.B
        z = lambda *shape, dt=None: torch.zeros(shape, dtype=dt or self.dt, device=self.dev)
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=self.dev)
        # caches
        dcap = w.window if w.window > 0 else cap
        self.dcap = dcap
        n_tl = tdims.layers if self.has_target else 0
        tdt = torch.uint8 if kv8 else self.dt
        self.caches = Caches(
            tk=[z(S, tdims.n_kv, cap, tdims.head_dim, dt=tdt) for _ in range(n_tl)],
            tv=[z(S, tdims.n_kv, cap, tdims.head_dim, dt=tdt) for _ in range(n_tl)],
            dk=[z(S, w.draft.n_kv, dcap, w.draft.head_dim) for _ in range(w.draft.layers)],
            dv=[z(S, w.draft.n_kv, dcap, w.draft.head_dim) for _ in range(w.draft.layers)],
            tke=[z(S, tdims.n_kv, cap, dt=tdt) for _ in range(n_tl if kv8 else 0)],
            tve=[z(S, tdims.n_kv, cap, dt=tdt) for _ in range(n_tl if kv8 else 0)])
        # RoPE tables (positions up to cap)
        self.rope_max = cap + B
        self.rope_t = z(self.rope_max, tdims.head_dim // 2, 2, dt=torch.float32) if self.has_target else None
        self.rope_d = z(self.rope_max, w.draft.head_dim // 2, 2, dt=torch.float32)
        # cycle state
        self.anchor = i32(S)
        self.base_pos = i32(S)
        self.drafts = i32(S, max(B - 1, 1))
        self.argmax = i32(S, B)
        self.margin = z(S, B, dt=torch.float32)
        self.accept_len = i32(S)
        self.out_tokens = i32(S, B)
        self.commit_base = i32(S)
        self.commit_count = i32(S)
        self.h = z(S * max(B, prefill_chunk), H, dt=torch.float32)
        self.feats = z(S * max(B, prefill_chunk), self.F, H)
        self.ones = torch.ones(S, dtype=torch.int32, device=self.dev)
        self.ws = None
        self.paging = {}  # "t" / "d" -> (page table, page size, max pages, pool pages) once paged
        # DFlash 2 draft convolutions: on when the workload has them (the
        # weights sit in the draft layers as conv_w1 / conv_w2)
        self.conv_rank = w.conv_rank
        self.tree = None  # (parent, rank) of the tree template, once set_tree was called
        self.tree_rows = 0
        if kv8 and self.has_target:
            self._tree_buffers(max(B, self.chunk))
        self.ws_bytes = 0
        self._size_workspace(fuse_rows)
        st = torch.cuda.current_stream()
        if self.has_target:
            D.dflash_rope_table(w.rope_theta, tdims.head_dim, self.rope_max, self.rope_t.data_ptr(), st)
        D.dflash_rope_table(w.rope_theta, w.draft.head_dim, self.rope_max, self.rope_d.data_ptr(), st)

    # ------------------------------------------------------------ arg builders

    def target_layer_args(self, li: int, rows: int, h, tap=None, tap_offset=0, base_pos=None):
        t = self.w.target
        a = D.dflash_layer_args()
        a.dims = self.tdims
        a.w = layer_weights(self.m["target"]["layers"][li])
        a.n_seqs, a.rows = self.S, rows
        a.base_pos = _ptr(self.base_pos if base_pos is None else base_pos)
        a.h = _ptr(h)
        a.kv = self._kv("t", li)
        a.attn_mode = D.DFLASH_ATTN_CAUSAL
        a.max_pos = self.cap
        a.rope_cs = _ptr(self.rope_t)
        a.rope_max_pos = self.rope_max
        if tap is not None:
            a.tap = _ptr(tap)
            a.tap_stride = self.F * t.hidden
            a.tap_offset = tap_offset
        return a

    def fuse_args(self, rows: int, feats, base_pos, valid):
        d = self.w.draft
        a = D.dflash_fuse_args()
        a.dims = self.ddims
        a.n_taps = self.F
        a.w_fc = _ptr(self.m["fc"])
        a.fc_norm = _ptr(self.m["fc_norm"])
        a.n_layers = d.layers
        for j in range(d.layers):
            a.w_qkv_layers[j] = _ptr(self.m["draft"]["layers"][j]["w_qkv"])
            a.kv_layers[j] = self._kv("d", j)
        a.feats = _ptr(feats)
        a.n_seqs, a.rows = self.S, rows
        a.base_pos = _ptr(base_pos)
        a.valid = _ptr(valid)
        a.rope_cs = _ptr(self.rope_d)
        a.rope_max_pos = self.rope_max
        return a

    def _kv(self, kind: str, j: int):
        """The dflash_kv of target ("t") or draft-context ("d") cache layer j."""
        if kind == "t":
            k, v, cap, win = self.caches.tk[j], self.caches.tv[j], self.cap, 0
        else:
            k, v, cap, win = self.caches.dk[j], self.caches.dv[j], self.dcap, self.w.window
        kv = D.dflash_kv(_ptr(k), _ptr(v), cap, win)
        if kind == "t" and self.kv8:
            kv.k_exp, kv.v_exp = _ptr(self.caches.tke[j]), _ptr(self.caches.tve[j])
        if kind in self.paging:
            table, ps, mp, pool = self.paging[kind]
            kv.pages, kv.page_size, kv.max_pages, kv.pool_pages = _ptr(table), ps, mp, pool
        return kv

    def page_caches(self, page_size: int = 128, seed: int = 0, spare_pages: int = 0):
        """Move the target and draft-context caches into page pools
        [pool][n_kv][page_size][head_dim] whose pages are handed out in a
        seeded random order (page table [S][max_pages], one table per cache
        kind shared by its layers), copying the current contents; the calls
        then address the caches through the page tables.  spare_pages adds
        unmapped pages to each pool."""
        g = torch.Generator().manual_seed(seed)
        for kind, ks, vs, cap in (("t", self.caches.tk, self.caches.tv, self.cap),
                                  ("d", self.caches.dk, self.caches.dv, self.dcap)):
            if not ks:
                continue
            assert cap % page_size == 0, "capacity must be a multiple of the page size"
            mp = cap // page_size
            S, nkv, _, d = ks[0].shape
            pool = S * mp + spare_pages
            table = torch.randperm(pool, generator=g)[:S * mp].view(S, mp).to(torch.int32)
            idx = table.view(-1).long().to(self.dev)
            for lst in (ks, vs):
                for j, c in enumerate(lst):
                    pages = c.view(S, nkv, mp, page_size, d).permute(0, 2, 1, 3, 4).reshape(S * mp, nkv, page_size, d)
                    p = torch.zeros(pool, nkv, page_size, d, dtype=c.dtype, device=self.dev)
                    p[idx] = pages
                    lst[j] = p
            for lst in (self.caches.tke, self.caches.tve) if kind == "t" else ():
                for j, c in enumerate(lst):
                    pages = c.view(S, nkv, mp, page_size).permute(0, 2, 1, 3).reshape(S * mp, nkv, page_size)
                    p = torch.zeros(pool, nkv, page_size, dtype=c.dtype, device=self.dev)
                    p[idx] = pages
                    lst[j] = p
            self.paging[kind] = (table.to(self.dev), page_size, mp, pool)

    def unpaged_caches(self):
        """The caches' contents in the contiguous layout [S][n_kv][cap][d]
        (copies when paged; the codes of 8-bit ones)."""
        out = {}
        for kind, ks, vs, cap in (("t", self.caches.tk, self.caches.tv, self.cap),
                                  ("d", self.caches.dk, self.caches.dv, self.dcap)):
            if kind not in self.paging:
                out[kind] = ([c.clone() for c in ks], [c.clone() for c in vs])
                continue
            table, ps, mp, pool = self.paging[kind]
            idx = table.view(-1).long()
            S = table.shape[0]
            conv = lambda p: p[idx].view(S, mp, p.shape[1], ps, p.shape[3]).permute(0, 2, 1, 3, 4).reshape(
                S, p.shape[1], mp * ps, p.shape[3])
            out[kind] = ([conv(p) for p in ks], [conv(p) for p in vs])
        return out

    def draft_args(self, logits=None, rounds: int = 1, conv_rank: int | None = None):
        d = self.w.draft
        a = D.dflash_draft_args()
        a.dims = self.ddims
        a.n_layers = d.layers
        for j in range(d.layers):
            a.layers[j] = layer_weights(self.m["draft"]["layers"][j])
            a.kv_layers[j] = self._kv("d", j)
        a.final_norm = _ptr(self.m["draft"]["final_norm"])
        a.embed = _ptr(self.m["embed"])
        a.lm_head = _ptr(self.m["lm_head"])
        a.n_seqs, a.block = self.S, self.B
        a.anchor = _ptr(self.anchor)
        a.base_pos = _ptr(self.base_pos)
        a.mask_token = self.w.mask_id
        a.max_pos = self.cap
        a.rope_cs = _ptr(self.rope_d)
        a.rope_max_pos = self.rope_max
        a.drafts = _ptr(self.drafts)
        a.logits = _ptr(logits)
        if self.w.path_topk:
            a.path_topk, a.path_rank = self.w.path_topk, self.w.path_rank
            a.path_u, a.path_v = _ptr(self.m["path_u"]), _ptr(self.m["path_v"])
        a.denoise_rounds = rounds
        r = self.conv_rank if conv_rank is None else conv_rank
        if r:
            a.conv_rank = r
            for j in range(d.layers):
                L = self.m["draft"]["layers"][j]
                a.conv_w1[j], a.conv_w2[j] = _ptr(L["conv_w1"]), _ptr(L["conv_w2"])
        return a

    def verify_args(self, block: int, h, drafts=None, logits=None, update=True):
        a = D.dflash_verify_args()
        a.dims = self.tdims
        a.h = _ptr(h)
        a.final_norm = _ptr(self.m["target"]["final_norm"])
        a.lm_head = _ptr(self.m["lm_head"])
        a.n_seqs, a.block = self.S, block
        a.drafts = _ptr(drafts)
        a.argmax = _ptr(self.argmax)
        a.margin = _ptr(self.margin)
        a.accept_len = _ptr(self.accept_len)
        a.out_tokens = _ptr(self.out_tokens)
        if update:
            a.next_anchor = _ptr(self.anchor)
            a.base_pos = _ptr(self.base_pos)
            a.commit_base = _ptr(self.commit_base)
            a.commit_count = _ptr(self.commit_count)
        a.logits = _ptr(logits)
        return a

    def embed_args(self, dims, rows: int, h, first, rest=None, fill=0):
        a = D.dflash_embed_args()
        a.dims = dims
        a.embed = _ptr(self.m["embed"])
        a.n_seqs, a.rows = self.S, rows
        a.first = _ptr(first)
        a.rest = _ptr(rest)
        a.fill_token = fill
        a.h = _ptr(h)
        return a

    # ------------------------------------------------------------- tree calls

    def _tree_buffers(self, rows: int):
        """Buffers of target forwards over up to `rows` tree rows a sequence."""
        if rows <= self.tree_rows:
            return
        t, S = self.w.target, self.S
        self.tree_rows = rows
        new = lambda *shape, dt=torch.int32: torch.zeros(shape, dtype=dt, device=self.dev)
        self.tkb = [new(S * rows, t.n_kv, t.head_dim, dt=self.dt) for _ in range(t.layers)]
        self.tvb = [new(S * rows, t.n_kv, t.head_dim, dt=self.dt) for _ in range(t.layers)]
        self.steps = torch.arange(rows, dtype=torch.int32, device=self.dev)

    def tree_layer_args(self, li: int, rows: int, h, pos, parent=None, tap=None, tap_offset=0, base_pos=None):
        a = self.target_layer_args(li, rows, h, tap, tap_offset, base_pos)
        a.attn_mode = D.DFLASH_ATTN_TREE
        a.max_pos = self.cap + rows  # (the rows take no slots: the context may fill the cache)
        a.tree_parent, a.tree_pos = _ptr(parent), _ptr(pos)
        a.out_kb, a.out_vb = _ptr(self.tkb[li]), _ptr(self.tvb[li])
        return a

    def kv_write_args(self, j0: int, n: int, rows: int, base_pos, valid=None, row_index=None):
        """Commits rows of the target's layers [j0, j0 + n), n <= DFLASH_KV_MAX_LAYERS."""
        a = D.dflash_kv_write_args()
        a.dims = self.tdims
        a.n_layers = n
        kb = (C.c_void_p * n)(*[_ptr(x) for x in self.tkb[j0:j0 + n]])
        vb = (C.c_void_p * n)(*[_ptr(x) for x in self.tvb[j0:j0 + n]])
        kv = (D.dflash_kv * n)(*[self._kv("t", j) for j in range(j0, j0 + n)])
        a._keep = (kb, vb, kv)  # host arrays, read during the call
        a.kb, a.vb, a.kv_layers = (C.cast(x, C.c_void_p) for x in a._keep)
        a.n_seqs, a.rows = self.S, rows
        a.base_pos, a.valid, a.row_index = _ptr(base_pos), _ptr(valid), _ptr(row_index)
        return a

    def tree_forward(self, rows: int, tokens, pos, parent=None, taps=True, base_pos=None):
        """Embed tokens [S][rows] and run every target layer over them as a
        tree (parent [S][rows]; None: a chain) at the positions pos [S*rows];
        the caches are read only.  Keys and values go to self.tkb / self.tvb,
        tap features to self.feats."""
        self._tree_buffers(rows)
        e = self.embed_args(self.tdims, 1, self.h, tokens)
        e.n_seqs = self.S * rows
        D.dflash_embed(e, self.ws_ptr, self.ws_bytes)
        for li in range(self.w.target.layers):
            tapped = taps and li in self.w.taps
            off = self.w.taps.index(li) * self.w.target.hidden if tapped else 0
            D.dflash_decoder_layer_forward(
                self.tree_layer_args(li, rows, self.h, pos, parent, self.feats if tapped else None, off, base_pos),
                self.ws_ptr, self.ws_bytes)

    def tree_commit(self, rows: int, base_pos, valid=None, row_index=None):
        """Write the last tree forward's rows (row_index [S][rows]: those, in
        that order) to the target caches from position base_pos on."""
        L = self.w.target.layers
        for j in range(0, L, D.DFLASH_KV_MAX_LAYERS):
            n = min(D.DFLASH_KV_MAX_LAYERS, L - j)
            D.dflash_kv_write(self.kv_write_args(j, n, rows, base_pos, valid, row_index), self.ws_ptr, self.ws_bytes)

    def set_tree(self, parent, rank):
        """The template of tree_cycle: node i >= 1 hangs below node parent[i]
        and takes candidate rank[i] of its position (0: the best); parent[0]
        = -1 is the anchor.  Candidates beyond the first need the workload's
        path selector, which lists path_topk of them.  May replace the buffers
        and the workspace: cycles captured before are to be captured again."""
        n = len(parent)
        assert n == len(rank) and 1 <= n <= D.DFLASH_MAX_TREE and parent[0] == -1
        S = self.S
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=self.dev)
        self.tree = tuple(torch.tensor(x, dtype=torch.int32, device=self.dev) for x in (parent, rank))
        self.t_parent, self.t_tokens, self.t_pos = i32(S, n), i32(S, n), i32(S * n)
        self.t_path, self.t_out, self.t_argmax = i32(S, n), i32(S, n), i32(S, n)
        self.t_zero = i32(S, n)
        self.t_dummy = i32(S), i32(S, n)
        if self.w.path_topk:
            self.t_cand = i32(S, self.B - 1, self.w.path_topk)
        self._tree_buffers(n)
        if self.h.shape[0] < S * n:
            self.h = torch.zeros(S * n, self.h.shape[1], dtype=torch.float32, device=self.dev)
            self.feats = torch.zeros(S * n, *self.feats.shape[1:], dtype=self.dt, device=self.dev)
        need = max(self.ws_bytes,
                   D.dflash_workspace_bytes(D.DFLASH_OP_LAYER, self.tree_layer_args(0, n, self.h, self.t_pos,
                                                                                    self.t_parent)),
                   D.dflash_workspace_bytes(D.DFLASH_OP_FUSE, self.fuse_args(n, self.feats, self.base_pos, None)),
                   D.dflash_workspace_bytes(D.DFLASH_OP_VERIFY, self.tree_verify_args(0, min(S, self._verify_seqs()))))
        if need > self.ws_bytes:
            self._new_workspace(int(need))

    def _verify_seqs(self) -> int:
        """Sequences per verification call, which takes 1024 rows at most."""
        return max(1, 1024 // self.tree[0].numel())

    def tree_verify_args(self, s0: int, n: int, logits=None):
        """The target's argmax (and logits) at the tree rows of sequences [s0, s0 + n)."""
        N = self.tree[0].numel()
        a = self.verify_args(N, self.h[s0 * N:], self.t_zero[s0:], None if logits is None else logits[s0 * N:],
                             update=False)
        a.n_seqs = n
        a.argmax, a.margin = _ptr(self.t_argmax[s0:]), 0
        a.accept_len, a.out_tokens = _ptr(self.t_dummy[0]), _ptr(self.t_dummy[1])  # (of a chain: not used)
        return a

    def tree_cycle(self, T: float = 0.0, u=None, noise=None):
        """One draft-and-verify cycle over the tree set by set_tree.  T = 0
        accepts the target's greedy tokens; T > 0 the draft's candidates by
        the random numbers u [S][rows] in [0, 1) and noise [S][V] (draws of
        an Exp(1) distribution), which leaves every token distributed as the
        target's softmax at temperature T."""
        parent, rank = self.tree
        S, N, V = self.S, parent.numel(), self.w.vocab
        a = self.draft_args()
        cand, topk = self.drafts, 1
        if self.w.path_topk:
            cand, topk = self.t_cand, self.w.path_topk
            a.path_cand_out = _ptr(cand)
        D.dflash_draft_block(a, self.ws_ptr, self.ws_bytes)
        b = D.dflash_tree_build_args()
        b.n_seqs, b.rows, b.levels, b.topk = S, N, self.B - 1, topk
        b.parent, b.rank, b.cand = _ptr(parent), _ptr(rank), _ptr(cand)
        b.anchor, b.base_pos = _ptr(self.anchor), _ptr(self.base_pos)
        b.parent_out, b.tokens_out, b.pos_out = _ptr(self.t_parent), _ptr(self.t_tokens), _ptr(self.t_pos)
        D.dflash_tree_build(b, self.ws_ptr, self.ws_bytes)
        self.tree_forward(N, self.t_tokens, self.t_pos, self.t_parent)
        if T > 0 and (getattr(self, "t_logits", None) is None or self.t_logits.shape[0] < S * N):
            self.t_logits = torch.zeros(S * N, V, dtype=torch.float32, device=self.dev)
        step = self._verify_seqs()
        for s0 in range(0, S, step):
            D.dflash_verify_accept(self.tree_verify_args(s0, min(step, S - s0), self.t_logits if T > 0 else None),
                                   self.ws_ptr, self.ws_bytes)
        c = D.dflash_tree_accept_args()
        c.dims = self.tdims
        c.n_seqs, c.rows, c.temperature = S, N, T
        c.parent, c.tokens = _ptr(self.t_parent), _ptr(self.t_tokens)
        if T > 0:
            c.target_logits, c.u, c.noise = _ptr(self.t_logits), _ptr(u), _ptr(noise)
        else:
            c.target_argmax = _ptr(self.t_argmax)
        c.base_pos, c.update_base_pos = _ptr(self.base_pos), 1
        c.accept_len, c.path, c.out_tokens = _ptr(self.accept_len), _ptr(self.t_path), _ptr(self.t_out)
        c.next_anchor = _ptr(self.anchor)
        c.commit_base, c.commit_count = _ptr(self.commit_base), _ptr(self.commit_count)
        D.dflash_tree_accept(c, self.ws_ptr, self.ws_bytes)
        self.tree_commit(N, self.commit_base, self.commit_count, self.t_path)
        # the accepted rows' features, in order (rows past the path: not injected)
        rows = min(N, self.B)
        f = self.feats[:S * N].view(S, N, -1)
        idx = self.t_path[:, :rows].clamp(min=0).long()[:, :, None].expand(S, rows, f.shape[2])
        self.fuse_with(f.gather(1, idx).view(S * rows, *self.feats.shape[1:]), rows, self.commit_base, self.commit_count)

    def tree_generate(self, prompts: torch.Tensor, n_new: int):
        """Greedy generation by tree cycles: the tokens and, per cycle, the accepted counts."""
        self.prefill(prompts)
        outs = [[int(a)] for a in self.anchor.cpu()]
        accepts = []
        while min(len(o) for o in outs) < n_new:
            self.tree_cycle()
            k, toks = self.accept_len.cpu(), self.t_out.cpu()
            accepts.append(k.clone())
            for s in range(self.S):
                outs[s].extend(int(t) for t in toks[s, :int(k[s]) + 1])
        return torch.tensor([o[:n_new] for o in outs], dtype=torch.int32), torch.stack(accepts, 1)

    def _size_workspace(self, fuse_rows: int):
        need = D.dflash_workspace_bytes(D.DFLASH_OP_DRAFT, self.draft_args())
        rows_list = [self.B, 1, min(self.chunk, self.cap)]
        if fuse_rows:
            need = max(need, D.dflash_workspace_bytes(D.DFLASH_OP_FUSE, self.fuse_args(fuse_rows, self.feats,
                                                                                      self.base_pos, None)))
        for rows in rows_list:
            need = max(need, D.dflash_workspace_bytes(D.DFLASH_OP_FUSE, self.fuse_args(rows, self.feats,
                                                                                      self.base_pos, None)))
            if self.has_target:
                layer = (self.tree_layer_args(0, rows, self.h, self.h) if self.kv8 else
                         self.target_layer_args(0, rows, self.h))
                need = max(need, D.dflash_workspace_bytes(D.DFLASH_OP_LAYER, layer))
                need = max(need, D.dflash_workspace_bytes(D.DFLASH_OP_VERIFY, self.verify_args(rows, self.h)))
        self._new_workspace(int(need))

    def _new_workspace(self, n: int):
        self.ws_bytes = n
        self.ws = torch.zeros(self.ws_bytes + 256, dtype=torch.uint8, device=self.dev)
        self.ws_ptr = (self.ws.data_ptr() + 255) & ~255
        D.dflash_workspace_init(self.ws_ptr, self.ws_bytes)

    # -------------------------------------------------------------- the steps

    def status(self) -> int:
        return D.dflash_read_status(self.ws_ptr)

    def target_forward(self, rows: int, first, rest=None, taps=True, base_pos=None):
        """Embed the rows and run every target layer causally; keeps tap
        features (rows x F x H) in self.feats."""
        t = self.w.target
        if self.kv8:  # a chain, committed after the forward
            base = self.base_pos if base_pos is None else base_pos
            tokens = first.view(self.S, 1) if rows == 1 else torch.cat([first.view(self.S, 1), rest], 1)
            pos = (base[:, None] + self.steps[:rows]).view(-1)
            self.tree_forward(rows, tokens.contiguous(), pos, None, taps, base)
            self.tree_commit(rows, base)
            return
        D.dflash_embed(self.embed_args(self.tdims, rows, self.h, first, rest), self.ws_ptr, self.ws_bytes)
        for li in range(t.layers):
            tap = None
            off = 0
            if taps and li in self.w.taps:
                tap = self.feats
                off = self.w.taps.index(li) * t.hidden
            D.dflash_decoder_layer_forward(self.target_layer_args(li, rows, self.h, tap, off, base_pos), self.ws_ptr,
                                           self.ws_bytes)

    def draft(self, logits=None, rounds: int = 1, conv_rank: int | None = None):
        D.dflash_draft_block(self.draft_args(logits, rounds, conv_rank), self.ws_ptr, self.ws_bytes)

    def verify(self, block: int, drafts=None, logits=None):
        D.dflash_verify_accept(self.verify_args(block, self.h, drafts, logits), self.ws_ptr, self.ws_bytes)

    def fuse(self, rows: int, base_pos, valid):
        D.dflash_fuse_context(self.fuse_args(rows, self.feats, base_pos, valid), self.ws_ptr, self.ws_bytes)

    def fuse_with(self, feats, rows: int, base_pos, valid):
        """Inject caller-provided tap features feats [S*rows][F][H]."""
        D.dflash_fuse_context(self.fuse_args(rows, feats, base_pos, valid), self.ws_ptr, self.ws_bytes)

    def prefill(self, prompts: torch.Tensor):
        """prompts [S][L] int32 on the device.  Runs the target over the
        prompt (chunks of prefill_chunk rows, then the last token alone),
        injects every prompt position into the draft context, and sets
        anchor = the first greedy token, base_pos = L."""
        S, L = prompts.shape
        assert S == self.S and L + self.B <= self.cap
        c0 = 0
        while c0 < L - 1:
            rows = min(self.chunk, L - 1 - c0)
            self.base_pos.fill_(c0)
            tok = prompts[:, c0:c0 + rows].contiguous()
            self.target_forward(rows, tok[:, 0].contiguous(), tok[:, 1:].contiguous() if rows > 1 else None)
            self.fuse(rows, self.base_pos, None)
            c0 += rows
        self.base_pos.fill_(L - 1)
        self.target_forward(1, prompts[:, L - 1].contiguous())
        self.fuse(1, self.base_pos, None)
        self.verify(1)  # anchor := greedy token after the prompt, base_pos := L

    def cycle(self, planted_drafts=None):
        """One draft-and-verify cycle (see the module docstring)."""
        self.draft()
        if planted_drafts is not None:
            self.drafts.copy_(planted_drafts)
        self.target_forward(self.B, self.anchor, self.drafts)
        self.verify(self.B, self.drafts)
        self.fuse(self.B, self.commit_base, self.commit_count)

    def cycle_sampled(self, T: float, seed: int, cycle: int, top_k: int = 0, top_p: float = 1.0):
        """One cycle in sampling mode (speculative sampling at temperature T,
        optionally over the top_k / top_p filtered distributions): the
        draft's logits give drafts drawn from its distribution, the target's
        logits the acceptance tests and the final draw.  `cycle` numbers the
        random draws; give every cycle its own."""
        S, B, V = self.S, self.B, self.w.vocab
        if getattr(self, "dlogits", None) is None:
            self.dlogits = torch.zeros(S * (B - 1), V, dtype=torch.float32, device=self.dev)
            self.tlogits = torch.zeros(S * B, V, dtype=torch.float32, device=self.dev)
            self.dlse = torch.zeros(S, B - 1, dtype=torch.float32, device=self.dev)
        if self.w.path_topk:
            return self._cycle_sampled_path(T, seed, cycle, top_k, top_p)
        self.draft(self.dlogits)
        a = D.dflash_sample_drafts_args()
        a.dims = self.ddims
        a.n_seqs, a.block, a.temperature, a.cycle, a.seed = S, B, T, cycle, seed
        a.base_pos, a.draft_logits = _ptr(self.base_pos), _ptr(self.dlogits)
        a.drafts, a.draft_lse = _ptr(self.drafts), _ptr(self.dlse)
        a.top_k, a.top_p = top_k, top_p
        D.dflash_sample_drafts(a, self.ws_ptr, self.ws_bytes)
        self.target_forward(B, self.anchor, self.drafts)
        D.dflash_verify_accept(self.verify_args(B, self.h, self.drafts, self.tlogits, update=False), self.ws_ptr,
                               self.ws_bytes)
        b = D.dflash_sample_accept_args()
        b.dims = self.tdims
        b.n_seqs, b.block, b.temperature, b.cycle, b.seed = S, B, T, cycle, seed
        b.target_logits, b.draft_logits, b.draft_lse = _ptr(self.tlogits), _ptr(self.dlogits), _ptr(self.dlse)
        b.drafts, b.base_pos, b.update_base_pos = _ptr(self.drafts), _ptr(self.base_pos), 1
        b.accept_len, b.out_tokens, b.next_anchor = _ptr(self.accept_len), _ptr(self.out_tokens), _ptr(self.anchor)
        b.commit_base, b.commit_count = _ptr(self.commit_base), _ptr(self.commit_count)
        b.top_k, b.top_p = top_k, top_p
        D.dflash_sample_accept(b, self.ws_ptr, self.ws_bytes)
        self.fuse(B, self.commit_base, self.commit_count)

    def _cycle_sampled_path(self, T: float, seed: int, cycle: int, top_k: int, top_p: float):
        """Sampling mode with the DFlash 2 path selector: the drafts are the
        path walked by sampling over each row's candidates, and the
        acceptance runs against that walk's sparse proposal."""
        S, B, K = self.S, self.B, self.w.path_topk
        if getattr(self, "pcand", None) is None:
            self.pcand = torch.zeros(S, B - 1, K, dtype=torch.int32, device=self.dev)
            self.plogq = torch.zeros(S, B - 1, K, dtype=torch.float32, device=self.dev)
        a = self.draft_args()
        a.path_temperature, a.path_seed, a.path_cycle = T, seed, cycle
        a.path_cand_out, a.path_logq = _ptr(self.pcand), _ptr(self.plogq)
        D.dflash_draft_block(a, self.ws_ptr, self.ws_bytes)
        self.target_forward(B, self.anchor, self.drafts)
        D.dflash_verify_accept(self.verify_args(B, self.h, self.drafts, self.tlogits, update=False), self.ws_ptr,
                               self.ws_bytes)
        b = D.dflash_sample_accept_args()
        b.dims = self.tdims
        b.n_seqs, b.block, b.temperature, b.cycle, b.seed = S, B, T, cycle, seed
        b.target_logits = _ptr(self.tlogits)
        b.draft_topk, b.draft_cand, b.draft_logq = K, _ptr(self.pcand), _ptr(self.plogq)
        b.drafts, b.base_pos, b.update_base_pos = _ptr(self.drafts), _ptr(self.base_pos), 1
        b.accept_len, b.out_tokens, b.next_anchor = _ptr(self.accept_len), _ptr(self.out_tokens), _ptr(self.anchor)
        b.commit_base, b.commit_count = _ptr(self.commit_base), _ptr(self.commit_count)
        b.top_k, b.top_p = top_k, top_p
        D.dflash_sample_accept(b, self.ws_ptr, self.ws_bytes)
        self.fuse(B, self.commit_base, self.commit_count)

    def greedy_step(self):
        """Plain autoregressive step: one target forward of the anchor."""
        self.target_forward(1, self.anchor, taps=False)
        self.verify(1)

    # ---------------------------------------------------------------- loops

    def greedy_generate(self, prompts: torch.Tensor, n_new: int):
        self.prefill(prompts)
        out = [self.anchor.clone()]
        while len(out) < n_new:
            self.greedy_step()
            out.append(self.anchor.clone())
        return torch.stack(out, 1).cpu()

    def speculative_generate(self, prompts: torch.Tensor, n_new: int):
        self.prefill(prompts)
        outs = [[int(a)] for a in self.anchor.cpu()]
        accepts = []
        while min(len(o) for o in outs) < n_new:
            self.cycle()
            k = self.accept_len.cpu()
            toks = self.out_tokens.cpu()
            accepts.append(k.clone())
            for s in range(self.S):
                outs[s].extend(int(t) for t in toks[s, :int(k[s]) + 1])
        return torch.tensor([o[:n_new] for o in outs], dtype=torch.int32), torch.stack(accepts, 1)
