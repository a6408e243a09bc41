"""Plain 64-bit implementations of the tree verification operators (CPU), and
the device-side set-up the GPU tests share.  Written from the definitions in
include/dflash.h; no code of the library is used for a value."""
from __future__ import annotations

import ctypes as C
import math

import numpy as np
import torch

from block_diffusion_speculative_step_gb300 import dflash as D

PAD = D.DFLASH_TREE_PAD


# ------------------------------------------------------------ 8-bit rows

def e4m3_values():
    """The value of every e4m3 code (NaN for 0x7f and 0xff)."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = math.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


E4M3 = e4m3_values()


def quantise_row(x):
    """One row -> (codes, biased exponent): the smallest e in [-60, 60] with
    max |x| <= 448 * 2^e over the finite elements, codes the nearest e4m3
    values of x * 2^-e (ties to the even code), NaN / inf -> the NaN code."""
    x = np.asarray(x, dtype=np.float64)
    fin = np.isfinite(x)
    mx = np.abs(x[fin]).max() if fin.any() else 0.0
    e = -60
    while e < 60 and mx > 448.0 * 2.0 ** e:
        e += 1
    y = np.clip(np.where(fin, x, 0.0) * 2.0 ** -e, -448.0, 448.0)
    mags = E4M3[:127]  # ascending non-negative values
    hi = np.searchsorted(mags, np.abs(y), side="left").clip(0, 126)
    lo = (hi - 1).clip(0)
    dl, dh = np.abs(y) - mags[lo], mags[hi] - np.abs(y)
    c = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(np.signbit(y), c | 128, c)
    return np.where(fin, c, 127).astype(np.uint8), e + 127


def value_rows(codes, ex):
    return E4M3[codes] * np.exp2(ex.astype(np.float64) - 127)[..., None]


# ------------------------------------------------------------------ trees

def random_tree(rng, n, levels=16, rows=None):
    """Parents of a random tree of n nodes, then padding up to `rows`."""
    p, depth = [-1], [0]
    for i in range(1, n):
        ok = [j for j in range(i) if depth[j] < levels]
        j = ok[-1] if rng.random() < 0.5 else ok[int(rng.integers(len(ok)))]
        p.append(j)
        depth.append(depth[j] + 1)
    return p + [PAD] * ((rows or n) - n)


def sees(parent):
    """see[i][j]: row i attends row j; None for a padding row."""
    out = []
    for i in range(len(parent)):
        row, j = set(), i
        while j >= 0:
            row.add(j)
            p = parent[j]
            if p < -1 or p >= j:
                row = None
                break
            j = p
        out.append(row)
    return out


def attention(q, k, v, kb, vb, parent, scale):
    """q [rows][nq][d], context k, v [nkv][n][d], tree kb, vb [rows][nkv][d],
    float64.  Returns out and A = sum_j p_j |v_j| (both [rows][nq][d], NaN in
    padding rows), and the largest sum_e |q_e k_e| * scale."""
    rows, nq, d = q.shape
    nkv, n = k.shape[0], k.shape[1]
    out = np.full((rows, nq, d), np.nan)
    mag = np.full((rows, nq, d), np.nan)
    big = 0.0
    for i, see in enumerate(sees(parent)):
        if see is None:
            continue
        idx = sorted(see)
        for h in range(nq):
            g = h // (nq // nkv)
            K = np.concatenate([k[g], kb[idx, g]])
            W = np.concatenate([v[g], vb[idx, g]])
            sc = K @ q[i, h] * scale
            big = max(big, float((np.abs(K) @ np.abs(q[i, h])).max()) * scale)
            p = np.exp(sc - sc.max())
            p /= p.sum()
            out[i, h] = p @ W
            mag[i, h] = p @ np.abs(W)
    return out, mag, big


# -------------------------------------------------------------- acceptance

def softmax(x, T):
    x = np.asarray(x, dtype=np.float64) / T
    e = np.exp(x - x.max())
    return e / e.sum()


def accept(parent, tokens, target, draft, u, noise, T, levels):
    """The walk of dflash_tree_accept for one sequence.  Also returns the
    smallest distance of any decision from its border, relative to the
    larger side (a decision closer than the fp32 error may go either way)."""
    node, path, toks, gap = 0, [0], [], math.inf
    while True:
        p = softmax(target[node], T)
        kids = [j for j in range(node + 1, len(parent)) if parent[j] == node]
        q = None
        if draft is not None:
            if len(toks) >= levels:
                kids = []
            else:
                q = softmax(draft[len(toks)], T)
        went = None
        for i in kids:
            x = tokens[i]
            if not 0 <= x < p.size:
                if q is not None:
                    left = np.maximum(p - q, 0)
                    p = left / left.sum() if left.sum() > 0 else p
                continue
            a, b = u[i] * (q[x] if q is not None else 1.0), p[x]
            if max(a, b) > 0:
                gap = min(gap, abs(a - b) / max(a, b))
            if a < b:
                went = i
                break
            if q is not None:
                left = np.maximum(p - q, 0)
                if left.sum() > 0:
                    p = left / left.sum()
                q = q.copy()
                q[x] = 0
                if q.sum() > 0:
                    q /= q.sum()
            else:
                p = p.copy()
                p[x] = 0
                if p.sum() > 0:
                    p /= p.sum()
        if went is None:
            break
        node = went
        path.append(node)
        toks.append(int(tokens[node]))
    r = p / np.asarray(noise, dtype=np.float64)
    last = int(np.argmax(r))
    if r.size > 1:
        two = np.partition(r, -2)[-2:]
        if two[1] > 0:
            gap = min(gap, (two[1] - two[0]) / two[1])
    N = len(parent)
    k = len(toks)
    return (k, path + [-1] * (N - len(path)), toks + [last] + [-1] * (N - k - 1), last), gap


# ------------------------------------------------------------- device side

def ptr(t):
    return 0 if t is None else t.data_ptr()


def dims(nq=1, nkv=1, d=64, dtype="bf16", vocab=8):
    return D.dflash_dims(8, nq, nkv, d, 8, vocab, 1e4, 1e-6, D.DFLASH_BF16 if dtype == "bf16" else D.DFLASH_F32)


class Workspace:
    def __init__(self, op, args):
        self.bytes = D.dflash_workspace_bytes(op, args)
        assert self.bytes > 0, D.dflash_last_error()
        self.buf = torch.full((self.bytes + 256 + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        self.ptr = (self.buf.data_ptr() + 255) & ~255
        D.dflash_workspace_init(self.ptr, self.bytes)
        self.end = self.ptr - self.buf.data_ptr() + self.bytes

    def status(self):
        st = D.dflash_read_status(self.ptr)
        assert bool((self.buf[self.end:] == 0xA5).all()), "written past the workspace's end"
        return st


def kv_desc(cap, k, v, ke=None, ve=None, pages=None, page=0, pool=0, window=0):
    kv = D.dflash_kv(ptr(k), ptr(v), cap, window)
    if pages is not None:
        kv.pages, kv.page_size, kv.max_pages, kv.pool_pages = ptr(pages), page, cap // page, pool
    kv.k_exp, kv.v_exp = ptr(ke), ptr(ve)
    return kv


def host_array(tensors):
    return (C.c_void_p * len(tensors))(*[ptr(t) for t in tensors])
