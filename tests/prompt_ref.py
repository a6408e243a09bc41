"""Plain 64-bit implementations of the prompt operators and the set-up their
tests share.  Written from the definitions in include/dflash.h; no code of the
library is used for a value."""
from __future__ import annotations

import math

import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests.tree_ref import Workspace, dims, kv_desc, ptr  # noqa: F401

FILL = 3.0  # what outputs hold before a call


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# --------------------------------------------------------------- attention

def attend(q, k, v, first, scale):
    """Rows q [n][nq][d] over keys k, v [T][nkv][d]: row i sees keys 0 ..
    first + i.  Returns the outputs, sum_j p_j |v_j| and max_j sum |q k| scale.
    What a row does not see is left out, whatever it holds."""
    n, nq, d = q.shape
    T, nkv = k.shape[0], k.shape[1]
    out = torch.empty(n, nq, d, dtype=torch.float64, device=q.device)
    mag, big = torch.empty_like(out), torch.empty(n, nq, dtype=torch.float64, device=q.device)
    see = torch.arange(T, device=q.device)[None, :] <= first + torch.arange(n, device=q.device)[:, None]
    for h in range(nq):
        g = h // (nq // nkv)
        sc = torch.where(see, q[:, h] @ k[:, g].T * scale, -math.inf)
        p = torch.softmax(sc, -1)
        w, a = torch.where(see, p, 0.0), v[:, g]
        if bool(torch.isfinite(a).all()):
            out[:, h], mag[:, h] = w @ a, w @ a.abs()
        else:
            for i in range(n):
                m = int(first + i + 1)
                out[i, h], mag[i, h] = w[i, :m] @ a[:m], w[i, :m] @ a[:m].abs()
        big[:, h] = torch.where(see, q[:, h].abs() @ k[:, g].abs().T * scale, 0.0).amax(-1)
    return out, mag, big


def weight_error(d, n, big, dtype):
    """Relative error of a weight against the sum of the weights' sizes: twice
    the score's (an fp32 sum of d products, (d + 4) 2^-24 of sum |q k| scale),
    2^-20 for the exponential, 2 n 2^-24 for the two sums of n, and two bf16
    terms' 2^-16 where the products run in bf16."""
    return torch.expm1(2 * (d + 4) * 2.0 ** -24 * big) + 2.0 ** -20 + 2 * n * 2.0 ** -24 + \
        (2.0 ** -16 if dtype == torch.bfloat16 else 0.0)


class Prompt:
    """One packed attention problem on the device: sequence s has lens[s] rows
    over ctx[s] cached slots; `lead` and `tail` rows belong to no sequence."""

    def __init__(self, lens, nq=8, nkv=2, d=128, dtype="bf16", ctx=None, page=0, lead=0, tail=0, scale=0.0, seed=0,
                 q_amp=1.0, cap=None, spare=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.S, self.lens, self.ctx, self.nq, self.nkv, self.d, self.scale = len(lens), lens, ctx, nq, nkv, d, scale
        self.dt = dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dtype = dtype
        start = [lead]
        for n in lens:
            start.append(start[-1] + n)
        self.start, self.M = start, start[-1] + tail
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        M = self.M
        self.q, self.kb, self.vb = (rnd(M, nq, d) * q_amp).to(dt), rnd(M, nkv, d).to(dt), rnd(M, nkv, d).to(dt)
        for x in (self.q, self.kb, self.vb):  # rows of no sequence
            x[:lead] = float("nan")
            x[start[-1]:] = float("nan")
        self.pages, self.pool, self.page, self.kc, self.vc = None, 0, page, None, None
        self.cap = 0
        if ctx is not None:
            unit = page or 1
            self.cap = cap or -(-max(max(ctx), 1) // unit) * unit
            shape = (self.S, nkv, self.cap, d)
            if page:
                self.pool = self.S * (self.cap // page) + spare
                ids = torch.randperm(self.pool, generator=torch.Generator().manual_seed(seed))
                self.pages = ids[:self.S * (self.cap // page)].view(self.S, -1).int().cuda()
                shape = (self.pool, nkv, page, d)
            nan = lambda: torch.full(shape, float("nan"), dtype=dt, device="cuda")  # slots no sequence reaches
            self.kc, self.vc = nan(), nan()
            for s, n in enumerate(ctx):
                for x in (self.kc, self.vc):
                    rows = rnd(nkv, n, d).to(dt)
                    for a in range(0, n, page or max(n, 1)):
                        b = min(n, a + (page or n))
                        x[int(self.pages[s, a // page]) if page else s, :, :b - a] = rows[:, a:b]
        self.out = torch.full((M, nq, d), FILL, dtype=dt, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.row_start, self.base = i32(start), None if ctx is None else i32(ctx)
        a = self.a = D.dflash_prompt_attention_args()
        a.dims = dims(nq, nkv, d, dtype)
        a.n_seqs, a.n_rows, a.row_start, a.base_pos = self.S, M, ptr(self.row_start), ptr(self.base)
        a.q, a.kb, a.vb, a.out, a.scale = ptr(self.q), ptr(self.kb), ptr(self.vb), ptr(self.out), scale
        if ctx is not None:
            a.max_pos = self.cap
            a.kv = kv_desc(self.cap, self.kc, self.vc, None, None, self.pages, page, self.pool)
        self.ws = Workspace(D.DFLASH_OP_PROMPT_ATTENTION, a)

    def run(self, stream=None):
        D.dflash_prompt_attention(self.a, self.ws.ptr, self.ws.bytes, stream)

    def cached(self, x, s):
        """The cached rows of sequence s, [n][nkv][d]."""
        n, t = self.ctx[s], x
        if not self.page:
            return t[s, :, :n].transpose(0, 1)
        ids = self.pages[s, :-(-n // self.page)].long()
        return t[ids].transpose(0, 1).flatten(1, 2)[:, :n].transpose(0, 1)

    def check(self, status=D.DFLASH_OK, seqs=None):
        """Each element: half a step of the output, and weight_error times sum_j p_j |v_j|."""
        torch.cuda.synchronize()
        assert self.ws.status() == status
        worst = 0.0
        for s in range(self.S) if seqs is None else seqs:
            r = slice(self.start[s], self.start[s + 1])
            if self.lens[s] == 0:
                continue
            k, v, n = self.kb[r], self.vb[r], 0
            if self.ctx is not None:
                n = self.ctx[s]
                k, v = torch.cat([self.cached(self.kc, s), k]), torch.cat([self.cached(self.vc, s), v])
            out, mag, big = attend(self.q[r].double(), k.double(), v.double(), n, self.scale or self.d ** -0.5)
            got = self.out[r].double()
            fine = torch.isfinite(out)
            assert torch.equal(torch.isfinite(got), fine), s
            tol = half_step(self.dt) * out.abs() + weight_error(self.d, n + self.lens[s], big, self.dt)[..., None] * mag
            tol = tol * (1 + half_step(self.dt))
            err = torch.where(fine, (got - out).abs() / tol, 0.0)
            assert float(err.max()) <= 1.0, (s, float(err.max()), (err > 1).nonzero()[:4].tolist())
            worst = max(worst, float(err.max()))
        for rows in (self.out[:self.start[0]], self.out[self.start[-1]:]):
            assert bool((rows == FILL).all()), "a row of no sequence was written"
        return worst
