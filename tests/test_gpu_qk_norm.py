"""dflash_qk_norm_rope against a plain 64-bit implementation."""
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests.prompt_ref import FILL, Workspace, dims, half_step, kv_desc, ptr

pytestmark = pytest.mark.gpu

THETA, EPS = 1e4, 1e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Heads:
    """One problem: S sequences of `rows` rows from base on; cap > 0: keys and values go to a cache."""

    def __init__(self, base, rows, nq=8, nkv=2, d=128, dtype="bf16", src="f32", norm="qk", cap=0, page=0, gap=0, seed=0,
                 table=0, amp=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.S, self.rows, self.nq, self.nkv, self.d, self.dt = len(base), rows, nq, nkv, d, DT[dtype]
        self.base, self.M, self.cap, self.page = base, len(base) * rows, cap, page
        self.width = (nq + 2 * nkv) * d
        self.qkv = (rnd(self.M, self.width + gap) * amp).to(DT[src])
        self.qkv[:, self.width:] = float("nan")
        self.qn = (1 + 0.2 * rnd(d)).to(self.dt) if "q" in norm else None
        self.kn = (1 + 0.2 * rnd(d)).to(self.dt) if "k" in norm else None
        self.table = table or max(base) + rows
        self.rope = torch.zeros(self.table, d // 2, 2, device="cuda")
        D.dflash_rope_table(THETA, d, self.table, self.rope.data_ptr())
        full = lambda *s: torch.full(s, FILL, dtype=self.dt, device="cuda")
        self.q, self.pages, self.pool = full(self.M, nq, d), None, 0
        if cap:
            shape = (self.S, nkv, cap, d)
            if page:
                self.pool = self.S * (cap // page) + 2
                self.pages = torch.randperm(self.pool, generator=torch.Generator().manual_seed(seed))
                self.pages = self.pages[:self.S * (cap // page)].view(self.S, -1).int().cuda()
                shape = (self.pool, nkv, page, d)
            self.k, self.v = full(*shape), full(*shape)
        else:
            self.k, self.v = full(self.M, nkv, d), full(self.M, nkv, d)
        self.base_d = torch.tensor(base, dtype=torch.int32, device="cuda")
        a = self.a = D.dflash_qk_norm_rope_args()
        a.dims = dims(nq, nkv, d, dtype)
        a.dims.rms_eps = EPS
        a.n_seqs, a.rows, a.base_pos = self.S, rows, ptr(self.base_d)
        a.qkv, a.qkv_stride = ptr(self.qkv), self.width + gap if gap else 0
        a.qkv_dtype = D.DFLASH_BF16 if src == "bf16" else D.DFLASH_F32
        a.q_norm, a.k_norm = ptr(self.qn), ptr(self.kn)
        a.rope_cs, a.rope_max_pos, a.q = ptr(self.rope), self.table, ptr(self.q)
        if cap:
            a.kv = kv_desc(cap, self.k, self.v, None, None, self.pages, page, self.pool)
        else:
            a.kb, a.vb = ptr(self.k), ptr(self.v)
        self.ws = Workspace(D.DFLASH_OP_QK_NORM_ROPE, a)

    def run(self):
        D.dflash_qk_norm_rope(self.a, self.ws.ptr, self.ws.bytes)

    def expect(self):
        pos = (torch.tensor(self.base)[:, None] + torch.arange(self.rows)).view(-1).double().cuda()
        w = THETA ** (-2.0 * torch.arange(self.d // 2, dtype=torch.float64, device="cuda") / self.d)
        cos, sin = torch.cos(pos[:, None, None] * w), torch.sin(pos[:, None, None] * w)
        x = self.qkv[:, :self.width].double().view(self.M, -1, self.d)

        def head(y, gain):
            if gain is not None:
                y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * gain.double()
            a, b = y.chunk(2, -1)
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1), torch.cat([a.abs() + b.abs()] * 2, -1)

        return head(x[:, :self.nq], self.qn), head(x[:, self.nq:self.nq + self.nkv], self.kn), x[:, self.nq + self.nkv:]

    def place(self, x):
        """Token-major rows [M][nkv][d] as the cache holds them."""
        out = torch.full(self.k.shape, FILL, dtype=torch.float64, device="cuda")
        for m in range(self.M):
            s, n = m // self.rows, self.base[m // self.rows] + m % self.rows
            if self.page:
                out[int(self.pages[s, n // self.page]), :, n % self.page] = x[m]
            else:
                out[s, :, n] = x[m]
        return out

    def check(self, status=D.DFLASH_OK):
        """Half a step of the output, and of |a| + |b| for the pair (a, b): 2^-24
        each for the product and the sum, 2^-23 for the table's cos and sin and
        the two products of the norm, and (d / 2 + 8) 2^-24 for half the sum of
        squares of d terms, the mean, the square root's reciprocal."""
        torch.cuda.synchronize()
        assert self.ws.status() == status
        (q, qa), (k, ka), v = self.expect()
        rel = (4 + 2 + 2 + self.d / 2 + 8) * 2.0 ** -24
        if self.cap:
            k, v, ka = self.place(k), self.place(v), self.place(ka)
        for name, got, ref, tol in (("q", self.q, q, rel * qa), ("k", self.k, k, rel * ka), ("v", self.v, v, 0.0)):
            h = half_step(self.dt)
            err, tol = (got.double() - ref).abs(), (h * ref.abs() + tol) * (1 + h)
            assert bool((err <= tol).all()), (name, float((err - tol).max()), (err > tol).nonzero()[:4].tolist())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nkv", [(1, 1), (8, 2), (7, 1), (32, 4)])
def test_token_major(dtype, src, d, nq, nkv):
    p = Heads([0, 5, 4000, 77, 130], 1, nq, nkv, d, dtype, src, seed=nq)
    p.run()
    p.check()


@pytest.mark.parametrize("norm", ["", "q", "k", "qk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norms_are_optional(norm, dtype):
    p = Heads([3, 900], 33, norm=norm, dtype=dtype, gap=64)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [0, 128, 256])
@pytest.mark.parametrize("rows", [1, 16, 37])
def test_into_the_cache(dtype, page, rows):
    """Slots that no row has stay as they were."""
    p = Heads([0, 127, 128, 300, 250], rows, 8, 2, 64, dtype, cap=512, page=page, seed=rows)
    p.run()
    p.check()


@pytest.mark.parametrize("M", [1, 2, 63, 1021, 5000])
def test_row_counts(M):
    p = Heads([(i * 7) % 3000 for i in range(M)], 1, 12, 4, 128, seed=M)
    p.run()
    p.check()


@pytest.mark.parametrize("amp", [0.0, 1e-12, 1e-3, 1e4])
def test_sizes_of_values(amp):
    """All zeros (the epsilon alone), values below and above the epsilon."""
    p = Heads([10, 20], 5, amp=amp, dtype="f32")
    p.run()
    p.check()


def test_nan_stays_in_its_head():
    p = Heads([10, 20], 5, dtype="f32")
    p.qkv[3, 2 * 128 + 7] = float("nan")
    p.run()
    torch.cuda.synchronize()
    bad = torch.isnan(p.q).any(-1)
    assert bad[3, 2] and int(bad.sum()) == 1 and not torch.isnan(p.k).any() and not torch.isnan(p.v).any()


@pytest.mark.parametrize("cap", [0, 256])
def test_positions_outside_the_table(cap):
    p = Heads([10, 200, -2, 30], 4, cap=cap, table=202, dtype="f32")
    p.run()
    torch.cuda.synchronize()
    assert p.ws.status() == D.DFLASH_ERR_INVALID_ARG
    q = p.q.view(4, 4, -1)
    wrote = (q != FILL).any(-1).cpu().tolist()
    assert wrote == [[True] * 4, [True, True, False, False], [False, False, True, True], [True] * 4]
    if cap:
        slots = (p.k != FILL).any(-1).any(1).cpu()
        assert [int(x) for x in slots.sum(1)] == [4, 2, 2, 4]
        assert slots[2, :2].all() and slots[1, 200:202].all()


@pytest.mark.parametrize("page", [0, 128])
def test_slots_outside_the_cache(page):
    """Queries are written, keys and values beyond the capacity or on an unmapped page are not."""
    p = Heads([254, 10], 4, cap=256, page=page, dtype="f32")
    if page:
        p.pages[1, 0] = -1
    p.run()
    torch.cuda.synchronize()
    assert p.ws.status() == D.DFLASH_ERR_INVALID_ARG
    assert (p.q != FILL).any(-1).all()
    assert int((p.k != FILL).any(-1).any(1).sum()) == (2 if page else 6)
    assert int((p.v != FILL).any(-1).any(1).sum()) == (2 if page else 6)


def test_equals_the_projection_without_norms():
    """Without gains the rotation is the projections' own, bit for bit: their
    epilogue rounds each product and the sum on its own."""
    p = Heads([1234], 3, norm="", dtype="f32")
    p.run()
    torch.cuda.synchronize()
    cs = p.rope[1234:1237]
    a, b = p.qkv[:, :8 * 128].view(3, 8, 128).chunk(2, -1)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    ref = torch.cat([(a * c).sub(b * s), (b * c).add(a * s)], -1)
    assert torch.equal(p.q, ref)


def test_a_cache_past_2_to_31_elements():
    p = Heads([262143, 5], 1, 8, 8, 128, cap=1 << 21, table=262144)
    assert p.k.numel() > 2 ** 31
    p.run()
    torch.cuda.synchronize()
    assert p.ws.status() == D.DFLASH_OK
    (_, _), (k, ka), v = p.expect()
    for s, n in ((0, 262143), (1, 5)):
        assert torch.equal(p.v[s, :, n].double(), v[s].to(p.dt).double())
        assert bool(((p.k[s, :, n].double() - k[s]).abs() <= 2.0 ** -7 * ka[s]).all())


def test_replays():
    p = Heads([100, 30], 9, cap=256, page=128, table=256)
    g = torch.cuda.CUDAGraph()
    p.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        p.run()
    p.qkv.copy_(torch.randn(p.qkv.shape, device="cuda"))
    p.base = [7, 128]
    p.base_d.copy_(torch.tensor(p.base, dtype=torch.int32))
    for x in (p.k, p.v):
        x.fill_(FILL)
    g.replay()
    p.check()


def test_rows_past_2_to_31_elements():
    """A projection of more than 2^31 elements: its last rows as they are alone."""
    M, n = 150000, 3
    big = Heads([0] * n, 1, 96, 8, 128, src="bf16")
    qkv = torch.zeros(M, big.width, dtype=torch.bfloat16, device="cuda")
    assert qkv.numel() > 2 ** 31
    qkv[-n:] = big.qkv
    base = torch.zeros(M, dtype=torch.int32, device="cuda")
    q = torch.full((M, 96, 128), FILL, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.full((M, 8, 128), FILL, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    big.run()
    a = big.a
    a.n_seqs, a.qkv, a.base_pos, a.q, a.kb, a.vb = M, ptr(qkv), ptr(base), ptr(q), ptr(k), ptr(v)
    big.run()
    torch.cuda.synchronize()
    assert big.ws.status() == D.DFLASH_OK
    for got, want in ((q, big.q), (k, big.k), (v, big.v)):
        assert torch.equal(got[-n:], want) and not bool(got[:-n].any())
