"""Tree verification and cache-row entry points without a GPU: struct layouts,
argument checks that fail before any launch, and workspace sizing."""
import ctypes as C
import os
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dflash.h")


@pytest.fixture(scope="module")
def D():
    from block_diffusion_speculative_step_gb300 import build
    build.build()
    import torch  # noqa: F401  (loads the shared CUDA runtime first, as in use)
    from block_diffusion_speculative_step_gb300 import dflash
    return dflash


def test_struct_layouts_match_c(D):
    structs = ["dflash_kv", "dflash_layer_args", "dflash_tree_attention_args", "dflash_tree_build_args",
               "dflash_tree_accept_args", "dflash_kv_write_args", "dflash_kv_read_args"]
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{HEADER}"', "int main(void) {"]
    for s in structs:
        lines.append(f'  printf("{s} %zu\\n", sizeof({s}));')
        for fname, _ in getattr(D, s)._fields_:
            lines.append(f'  printf("{s}.{fname} %zu\\n", offsetof({s}, {fname}));')
    for name in ("DFLASH_ATTN_TREE", "DFLASH_OP_TREE_ATTENTION", "DFLASH_OP_TREE_ACCEPT", "DFLASH_OP_KV_WRITE",
                 "DFLASH_OP_KV_READ", "DFLASH_OP_TREE_BUILD", "DFLASH_MAX_TREE", "DFLASH_TREE_PAD",
                 "DFLASH_KV_MAX_LAYERS"):
        lines.append(f'  printf("{name} %d\\n", (int){name});')
    lines.append("  return 0; }")
    with tempfile.TemporaryDirectory() as td:
        src, exe = os.path.join(td, "l.c"), os.path.join(td, "l")
        open(src, "w").write("\n".join(lines))
        subprocess.check_call(["gcc", "-o", exe, src])
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    ref = dict(l.rsplit(" ", 1) for l in out.splitlines())
    for s in structs:
        cls = getattr(D, s)
        assert C.sizeof(cls) == int(ref[s]), s
        for fname, _ in cls._fields_:
            assert getattr(cls, fname).offset == int(ref[f"{s}.{fname}"]), f"{s}.{fname}"
    for name, v in ref.items():
        if name.startswith("DFLASH_"):
            assert getattr(D, name) == int(v), name


def attn_args(D, **kw):
    a = D.dflash_tree_attention_args()
    a.dims = D.dflash_dims(256, 8, 2, 128, 512, 1000, 1e4, 1e-6, D.DFLASH_BF16)
    a.n_seqs, a.rows, a.max_pos = 2, 16, 512
    a.base_pos = a.q = a.kb = a.vb = a.out = 4096
    a.kv = D.dflash_kv(4096, 4096, 512, 0)
    for k, v in kw.items():
        setattr(a.kv if k in ("capacity", "window", "pages", "page_size", "max_pages", "pool_pages", "k_exp", "v_exp",
                              "k", "v") else a, k, v)
    return a


@pytest.mark.parametrize("change,word", [
    (dict(rows=0), "rows"), (dict(rows=129), "at most 128 rows"), (dict(n_seqs=0), "n_seqs"),
    (dict(max_pos=513), "max_pos"), (dict(max_pos=-1), "max_pos"), (dict(window=512), "window"),
    (dict(capacity=0), "capacity"), (dict(k_exp=4096), "k_exp"), (dict(scale=-1.0), "scale"),
    (dict(scale=float("nan")), "scale"), (dict(q=0), "NULL"), (dict(base_pos=0), "NULL"), (dict(out=4104), "aligned"),
    (dict(k=4104), "aligned"), (dict(v=0), "NULL"),
    (dict(pages=4096, page_size=100, max_pages=4, pool_pages=9), "page_size"),
    (dict(pages=4096, page_size=128, max_pages=3, pool_pages=9), "max_pages"),
    (dict(capacity=1 << 30, max_pos=16), "2^31"),
])
def test_tree_attention_refusals(D, change, word):
    a = attn_args(D, **change)
    assert D.lib().dflash_tree_attention(C.byref(a), C.c_void_p(256), 1 << 40, None) == D.DFLASH_ERR_INVALID_ARG
    assert word in D.dflash_last_error(), D.dflash_last_error()


def test_tree_attention_workspace(D):
    a = attn_args(D)
    need = D.dflash_workspace_bytes(D.DFLASH_OP_TREE_ATTENTION, a)
    assert need > 0
    assert D.lib().dflash_tree_attention(C.byref(a), C.c_void_p(256), need - 1, None) == D.DFLASH_ERR_WORKSPACE
    assert D.lib().dflash_tree_attention(C.byref(a), C.c_void_p(264), need, None) == D.DFLASH_ERR_INVALID_ARG
    assert D.lib().dflash_tree_attention(C.byref(a), None, need, None) == D.DFLASH_ERR_INVALID_ARG
    assert D.dflash_workspace_bytes(D.DFLASH_OP_TREE_ATTENTION, attn_args(D, rows=500)) == 0


def accept_args(D, **kw):
    a = D.dflash_tree_accept_args()
    a.dims = D.dflash_dims(8, 1, 1, 64, 8, 1000, 1e4, 1e-6, D.DFLASH_F32)
    a.n_seqs, a.rows, a.levels, a.temperature = 2, 16, 4, 1.0
    for k in ("tokens", "target_logits", "draft_logits", "u", "noise", "base_pos", "accept_len", "path", "out_tokens"):
        setattr(a, k, 4096)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,word", [
    (dict(rows=0), "rows"), (dict(rows=129), "rows"), (dict(n_seqs=-1), "n_seqs"), (dict(temperature=-0.5), "temperature"),
    (dict(temperature=float("inf")), "temperature"), (dict(temperature=1e-9), "temperature"), (dict(levels=-1), "levels"), (dict(levels=0), "levels"),
    (dict(tokens=0), "NULL"), (dict(path=0), "NULL"), (dict(noise=0), "noise"), (dict(u=0), "noise"),
    (dict(target_logits=0), "target_logits"), (dict(temperature=0.0), "target_argmax"),
    (dict(base_pos=0, update_base_pos=1), "base_pos"), (dict(base_pos=0, commit_base=4096), "base_pos"),
])
def test_tree_accept_refusals(D, change, word):
    a = accept_args(D, **change)
    assert D.lib().dflash_tree_accept(C.byref(a), C.c_void_p(256), 1 << 40, None) == D.DFLASH_ERR_INVALID_ARG
    assert word in D.dflash_last_error(), D.dflash_last_error()


def rows_args(D, read, n_layers=2, **kw):
    a = D.dflash_kv_read_args() if read else D.dflash_kv_write_args()
    a.dims = D.dflash_dims(256, 8, 2, 128, 512, 1000, 1e4, 1e-6, D.DFLASH_BF16)
    a.n_layers = n_layers
    ptrs = (C.c_void_p * 64)(*[4096] * 64)
    kvs = (D.dflash_kv * 64)(*[D.dflash_kv(4096, 4096, 512, 0) for _ in range(64)])
    for k, v in kw.pop("kv1", {}).items():
        setattr(kvs[1], k, v)
    if "src1" in kw:
        ptrs[1] = kw.pop("src1")
    a.kv_layers = C.addressof(kvs)
    for k in (("k_out", "v_out") if read else ("kb", "vb")):
        setattr(a, k, C.addressof(ptrs))
    a.n_seqs, a.rows, a.base_pos = 2, 16, 4096
    for k, v in kw.items():
        setattr(a, k, v)
    a.keep = (ptrs, kvs)
    return a


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("change,word", [
    (dict(n_layers=0), "n_layers"), (dict(n_layers=65), "n_layers"), (dict(rows=0), "rows"), (dict(n_seqs=0), "n_seqs"),
    (dict(kv_layers=0), "kv_layers"), (dict(base_pos=0), "NULL"), (dict(kv1=dict(capacity=256)), "geometry"),
    (dict(kv1=dict(k=0)), "layer 1"), (dict(kv1=dict(k_exp=4096)), "k_exp"),
    (dict(kv1=dict(k_exp=4096, v_exp=4096)), "geometry"), (dict(kv1=dict(window=7)), "window"),
    (dict(src1=0), "layer 1"), (dict(src1=4100), "aligned"), (dict(rows=1 << 28), "2^27"),
])
def test_cache_row_refusals(D, read, change, word):
    a = rows_args(D, read, **change)
    f = D.lib().dflash_kv_read if read else D.lib().dflash_kv_write
    assert f(C.byref(a), C.c_void_p(256), 1 << 40, None) == D.DFLASH_ERR_INVALID_ARG
    assert word in D.dflash_last_error(), D.dflash_last_error()


def test_null_args(D):
    for name in ("dflash_tree_attention", "dflash_tree_build", "dflash_tree_accept", "dflash_kv_write",
                 "dflash_kv_read"):
        assert getattr(D.lib(), name)(None, None, 0, None) == D.DFLASH_ERR_INVALID_ARG
        assert "NULL args" in D.dflash_last_error()


def layer_args(D, mode):
    a = D.dflash_layer_args()
    a.dims = D.dflash_dims(256, 4, 2, 64, 512, 1000, 1e4, 1e-6, D.DFLASH_BF16)
    a.w = D.dflash_layer_weights(*[4096] * 6)
    a.n_seqs, a.rows, a.attn_mode, a.max_pos, a.rope_max_pos = 2, 16, mode, 256, 512
    a.base_pos = a.h = a.rope_cs = 4096
    a.kv = D.dflash_kv(4096, 4096, 512, 0)
    return a


def test_layer_tree_mode_refusals(D):
    L = D.lib()
    a = layer_args(D, D.DFLASH_ATTN_TREE)
    assert L.dflash_decoder_layer_forward(C.byref(a), C.c_void_p(256), 1 << 40, None) == D.DFLASH_ERR_INVALID_ARG
    assert "tree_pos" in D.dflash_last_error()
    a.tree_pos, a.rows = 4096, 200
    assert L.dflash_decoder_layer_forward(C.byref(a), C.c_void_p(256), 1 << 40, None) == D.DFLASH_ERR_INVALID_ARG
    assert "128 rows" in D.dflash_last_error()
    assert D.dflash_workspace_bytes(D.DFLASH_OP_LAYER, layer_args(D, D.DFLASH_ATTN_TREE)) > 0
    # an 8-bit cache: refused outside the tree mode
    for mode in (D.DFLASH_ATTN_CAUSAL, D.DFLASH_ATTN_BLOCK_BIDIR):
        a = layer_args(D, mode)
        a.kv.k_exp = a.kv.v_exp = 4096
        assert L.dflash_decoder_layer_forward(C.byref(a), C.c_void_p(256), 1 << 40, None) == D.DFLASH_ERR_UNSUPPORTED
    f = D.dflash_fuse_args()
    f.dims = a.dims
    f.n_taps = f.n_layers = f.n_seqs = f.rows = 1
    f.w_fc = f.fc_norm = f.feats = f.base_pos = f.rope_cs = 4096
    f.w_qkv_layers[0] = 4096
    f.kv_layers[0] = a.kv
    assert L.dflash_fuse_context(C.byref(f), C.c_void_p(256), 1 << 40, None) == D.DFLASH_ERR_UNSUPPORTED
