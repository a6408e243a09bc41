"""dflash_kv_write / dflash_kv_read against a plain 64-bit implementation:
codes, exponents and read-back values are exact, everything else in the cache
stays as it was."""
import ctypes as C

import numpy as np
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests import tree_ref as R

pytestmark = pytest.mark.gpu


class Rows:
    """One write / read problem on the device with random cache contents."""

    def __init__(self, S, rows, nkv, d, dtype, cap, base, valid=None, index=None, layers=1, q8=True, page=0, window=0,
                 seed=0, amp=1.0):
        self.__dict__.update(locals())
        g = torch.Generator().manual_seed(seed)
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dt = dt
        rnd = lambda *s: (torch.randn(*s, generator=g) * amp).to(dt)
        self.kb = [rnd(S * rows, nkv, d).cuda() for _ in range(layers)]
        self.vb = [rnd(S * rows, nkv, d).cuda() for _ in range(layers)]
        self.pages, self.pool = None, 0
        if page:
            self.pool = S * (cap // page) + 2
            self.pages = torch.randperm(self.pool, generator=g)[:S * (cap // page)].view(S, -1).int().cuda()
            shape = (self.pool, nkv, page, d)
        else:
            shape = (S, nkv, cap, d)
        mk = (lambda: torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda()) if q8 else \
            (lambda: torch.randn(shape, generator=g).to(dt).cuda())
        self.kc, self.vc = [mk() for _ in range(layers)], [mk() for _ in range(layers)]
        mke = (lambda: torch.randint(0, 256, shape[:-1], generator=g, dtype=torch.uint8).cuda()) if q8 else lambda: None
        self.ke, self.ve = [mke() for _ in range(layers)], [mke() for _ in range(layers)]
        i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32).cuda()
        self.base_t, self.valid_t, self.index_t = i32(base), i32(valid), i32(index)
        self.ko = [torch.full((S * rows, nkv, d), 7.0, dtype=dt).cuda() for _ in range(layers)]
        self.vo = [torch.full((S * rows, nkv, d), 7.0, dtype=dt).cuda() for _ in range(layers)]
        self.kvs = (D.dflash_kv * layers)(*[
            R.kv_desc(cap, self.kc[j], self.vc[j], self.ke[j], self.ve[j], self.pages, page, self.pool, window)
            for j in range(layers)])
        self.arr = [R.host_array(x) for x in (self.kb, self.vb, self.ko, self.vo)]
        self.w, self.r = D.dflash_kv_write_args(), D.dflash_kv_read_args()
        for a in (self.w, self.r):
            a.dims, a.n_layers, a.kv_layers = R.dims(nkv, nkv, d, dtype), layers, C.addressof(self.kvs)
            a.n_seqs, a.rows, a.base_pos, a.valid = S, rows, R.ptr(self.base_t), R.ptr(self.valid_t)
        self.w.kb, self.w.vb, self.w.row_index = C.addressof(self.arr[0]), C.addressof(self.arr[1]), R.ptr(self.index_t)
        self.r.k_out, self.r.v_out = C.addressof(self.arr[2]), C.addressof(self.arr[3])
        self.ws = R.Workspace(D.DFLASH_OP_KV_WRITE, self.w)

    def write(self):
        D.dflash_kv_write(self.w, self.ws.ptr, self.ws.bytes)

    def read(self):
        D.dflash_kv_read(self.r, self.ws.ptr, self.ws.bytes)

    def at(self, s, slot):
        """(first index, slot index) of a slot in the cache tensors; None: not mapped."""
        if self.pages is None:
            return s, slot
        pg = int(self.pages[s, slot // self.page])
        return (pg, slot % self.page) if 0 <= pg < self.pool else None

    def expected(self):
        """The caches after the write, on the CPU."""
        kc, vc = [x.cpu().clone() for x in self.kc], [x.cpu().clone() for x in self.vc]
        ke, ve = ([None if x is None else x.cpu().clone() for x in y] for y in (self.ke, self.ve))
        for s in range(self.S):
            n = self.rows if self.valid is None else min(self.valid[s], self.rows)
            for i in range(n):
                src = i if self.index is None else self.index[s][i]
                slot = self.base[s] + i
                if self.window:
                    slot %= self.window
                if not 0 <= src < self.rows or not 0 <= slot < self.cap or self.at(s, slot) is None:
                    continue
                a, o = self.at(s, slot)
                for j in range(self.layers):
                    for cache, ex, b in ((kc, ke, self.kb), (vc, ve, self.vb)):
                        x = b[j].view(self.S, self.rows, self.nkv, self.d)[s, src].cpu()
                        for h in range(self.nkv):
                            if self.q8:
                                c, e = R.quantise_row(x[h].double().numpy())
                                cache[j][a, h, o] = torch.from_numpy(c)
                                ex[j][a, h, o] = e
                            else:
                                cache[j][a, h, o] = x[h]
        return kc, vc, ke, ve

    def check_write(self, status=D.DFLASH_OK):
        want = self.expected()
        self.write()
        torch.cuda.synchronize()
        assert self.ws.status() == status
        for got, ref in zip((self.kc, self.vc, self.ke, self.ve), want):
            for x, y in zip(got, ref):
                if x is not None:
                    x = x.cpu()
                    if self.q8 and x.dim() == 4:  # a zero of either sign, and either NaN, are the same value
                        x, y = torch.from_numpy(R.E4M3[x.numpy()]), torch.from_numpy(R.E4M3[y.numpy()])
                    assert torch.equal(torch.nan_to_num(x.double(), 1e9), torch.nan_to_num(y.double(), 1e9))

    def check_read(self, status=D.DFLASH_OK):
        self.read()
        torch.cuda.synchronize()
        assert self.ws.status() == status
        for cache, ex, out in ((self.kc, self.ke, self.ko), (self.vc, self.ve, self.vo)):
            for j in range(self.layers):
                want = torch.full((self.S, self.rows, self.nkv, self.d), 7.0, dtype=torch.float64)
                c = cache[j].cpu()
                val = torch.from_numpy(R.value_rows(c.numpy(), ex[j].cpu().numpy())) if self.q8 else c.double()
                for s in range(self.S):
                    n = self.rows if self.valid is None else min(self.valid[s], self.rows)
                    for i in range(n):
                        slot = self.base[s] + i
                        if self.window:
                            slot %= self.window
                        if 0 <= slot < self.cap and self.at(s, slot) is not None:
                            a, o = self.at(s, slot)
                            want[s, i] = val[a, :, o]
                want = want.to(self.dt).view(-1, self.nkv, self.d)
                assert torch.equal(torch.nan_to_num(out[j].cpu().float(), 1e9), torch.nan_to_num(want.float(), 1e9))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("page", [0, 128])
def test_write_then_read(dtype, d, q8, page):
    p = Rows(3, 9, 2, d, dtype, 256, [0, 121, 37], valid=[9, 8, 0], layers=3, q8=q8, page=page, seed=d + page)
    p.check_write()
    p.check_read()


@pytest.mark.parametrize("S,rows,nkv", [(1, 1, 1), (1, 1000, 8), (40, 1, 3), (2, 129, 5)])
def test_sizes(S, rows, nkv):
    p = Rows(S, rows, nkv, 64, "bf16", rows + 3, [i % 4 for i in range(S)], seed=rows)
    p.check_write()
    p.check_read()


def test_path_order_repeats_and_ragged_counts():
    index = [[0, 3, 4, 7, 7, 1, -1, 99], [5, 5, 5, 5, 5, 5, 5, 5]]
    p = Rows(2, 8, 4, 128, "bf16", 64, [10, 56], valid=[6, 8], index=index, layers=2)
    p.check_write()
    p.check_read()


def test_more_layers_than_a_model_has():
    p = Rows(1, 2, 1, 64, "f32", 4, [1], layers=64)
    p.check_write()
    p.check_read()


@pytest.mark.parametrize("amp", [0.0, 1e-30, 2.0 ** -60, 1e-3, 448.0, 1e20, 3e37])
def test_magnitudes(amp):
    """Zero rows, rows below the smallest and above the largest scale."""
    p = Rows(1, 4, 2, 128, "f32", 8, [0], amp=amp, seed=5)
    p.check_write()
    p.check_read()


def test_borders_of_the_scale():
    """Maxima at 448 * 2^k and one fp32 step either side, and exact ties."""
    p = Rows(1, 6, 1, 64, "f32", 8, [0])
    x = p.kb[0].view(6, 64)
    for i, mx in enumerate((448.0, np.nextafter(np.float32(448), np.float32(449)), 1.75, 224.0, 7.0 * 2 ** -20, 1.0)):
        x[i] = 0
        x[i, :32] = float(mx) * torch.arange(32).cuda() / 32
        x[i, 0] = -float(mx)
    x[3, 1:17] = torch.tensor([(8 + i) * 0.5 + 0.25 for i in range(16)]).cuda()  # halfway between codes
    p.check_write()


def test_nan_and_infinity():
    p = Rows(1, 3, 2, 64, "bf16", 4, [0])
    p.kb[0][0, 0, 5] = float("nan")
    p.kb[0][1, 1, 63] = float("-inf")
    p.vb[0][2, 0] = float("inf")
    p.check_write(D.DFLASH_ERR_NUMERIC)
    p.check_read()
    assert torch.isnan(p.ko[0][0, 0, 5]) and not torch.isnan(p.ko[0][0, 0, :5]).any()


def test_window_ring():
    """Of more rows than the ring holds the last ones stay."""
    p = Rows(2, 13, 2, 64, "bf16", 8, [3, 100], window=8, valid=[13, 5])
    p.check_write()
    p.valid, p.valid_t[:] = [8, 5], torch.tensor([8, 5], dtype=torch.int32).cuda()
    p.check_read()


def test_slots_and_pages_out_of_range():
    p = Rows(3, 4, 2, 64, "bf16", 256, [254, -2, 0], page=128)
    p.pages[2, 0] = p.pool  # not mapped
    p.check_write(D.DFLASH_ERR_INVALID_ARG)
    p.check_read(D.DFLASH_ERR_INVALID_ARG)
    assert bool((p.ko[0].view(3, 4, 2, 64)[2] == 7).all())


def test_captured_and_replayed_on_another_stream():
    p = Rows(2, 5, 2, 128, "bf16", 64, [0, 9])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        p.write()
        p.read()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            p.write()
            p.read()
    p.kb[0].mul_(-3)
    torch.cuda.synchronize()
    want = p.expected()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.kc[0].cpu(), want[0][0]) and torch.equal(p.ke[0].cpu(), want[2][0])
    p.check_read()
