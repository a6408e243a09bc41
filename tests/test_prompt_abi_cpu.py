"""Prompt entry points without a GPU: struct layouts, argument checks that fail
before any launch, and workspace sizing."""
import ctypes as C
import os
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dflash.h")
KV = ("capacity", "window", "pages", "page_size", "max_pages", "pool_pages", "k_exp", "v_exp", "k", "v")


@pytest.fixture(scope="module")
def D():
    from block_diffusion_speculative_step_gb300 import build
    build.build()
    import torch  # noqa: F401  (loads the shared CUDA runtime first, as in use)
    from block_diffusion_speculative_step_gb300 import dflash
    return dflash


def test_struct_layouts_match_c(D):
    structs = ["dflash_kv", "dflash_qk_norm_rope_args", "dflash_prompt_attention_args", "dflash_token_logprobs_args"]
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{HEADER}"', "int main(void) {"]
    for s in structs:
        lines.append(f'  printf("{s} %zu\\n", sizeof({s}));')
        for fname, _ in getattr(D, s)._fields_:
            lines.append(f'  printf("{s}.{fname} %zu\\n", offsetof({s}, {fname}));')
    for name in ("DFLASH_OP_QK_NORM_ROPE", "DFLASH_OP_PROMPT_ATTENTION", "DFLASH_OP_TOKEN_LOGPROBS", "DFLASH_NO_TOKEN",
                 "DFLASH_MAX_LOGPROBS"):
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


def _change(a, kw):
    for k, v in kw.items():
        setattr(a.kv if k in KV else a.dims if hasattr(a.dims, k) else a, k, v)
    return a


def _refuse(D, name, a, word, code=None):
    rc = getattr(D.lib(), name)(C.byref(a), C.c_void_p(256), 1 << 40, None)
    assert rc == (D.DFLASH_ERR_INVALID_ARG if code is None else code), rc
    assert word in D.dflash_last_error(), D.dflash_last_error()


def qk_args(D, **kw):
    a = D.dflash_qk_norm_rope_args()
    a.dims = D.dflash_dims(256, 8, 2, 128, 512, 1000, 1e4, 1e-6, D.DFLASH_BF16)
    a.n_seqs, a.rows, a.rope_max_pos, a.qkv_dtype = 2, 16, 512, D.DFLASH_F32
    a.base_pos = a.qkv = a.rope_cs = a.q = a.kb = a.vb = a.q_norm = a.k_norm = 4096
    a.kv = D.dflash_kv(4096, 4096, 512, 0)
    return _change(a, kw)


@pytest.mark.parametrize("change,word", [
    (dict(n_seqs=0), "n_seqs"), (dict(rows=0), "rows"), (dict(n_seqs=1 << 30), "too many"), (dict(qkv_dtype=2), "qkv_dtype"),
    (dict(qkv_stride=8), "qkv_stride"), (dict(qkv_stride=12 * 128 + 4), "qkv_stride"), (dict(qkv_stride=-8), "qkv_stride"),
    (dict(rope_max_pos=0), "rope_max_pos"), (dict(qkv=0), "NULL"), (dict(base_pos=0), "NULL"), (dict(q=0), "NULL"),
    (dict(rope_cs=0), "NULL"), (dict(kb=0), "both"), (dict(vb=0), "both"), (dict(q=4100), "aligned"),
    (dict(qkv=4104), "aligned"), (dict(q_norm=4098), "aligned"), (dict(kb=0, vb=0, k=0), "NULL cache"),
    (dict(kb=0, vb=0, window=512), "window"), (dict(kb=0, vb=0, capacity=0), "capacity"),
    (dict(kb=0, vb=0, v=4104), "aligned"), (dict(kb=0, vb=0, capacity=1 << 29), "2^31"),
    (dict(kb=0, vb=0, pages=4096, page_size=100, max_pages=4, pool_pages=9), "page_size"),
    (dict(head_dim=96), "head_dim"), (dict(n_kv_heads=3), "n_kv_heads"), (dict(dtype=7), "dtype"),
])
def test_qk_norm_refusals(D, change, word):
    _refuse(D, "dflash_qk_norm_rope", qk_args(D, **change), word)


def test_qk_norm_takes_no_8_bit_cache(D):
    _refuse(D, "dflash_qk_norm_rope", qk_args(D, kb=0, vb=0, k_exp=4096, v_exp=4096), "8-bit", D.DFLASH_ERR_UNSUPPORTED)


def prompt_args(D, **kw):
    a = D.dflash_prompt_attention_args()
    a.dims = D.dflash_dims(256, 8, 2, 128, 512, 1000, 1e4, 1e-6, D.DFLASH_BF16)
    a.n_seqs, a.n_rows, a.max_pos = 3, 100, 512
    a.row_start = a.base_pos = a.q = a.kb = a.vb = a.out = 4096
    a.kv = D.dflash_kv(4096, 4096, 512, 0)
    return _change(a, kw)


@pytest.mark.parametrize("change,word", [
    (dict(n_seqs=0), "n_seqs"), (dict(n_rows=0), "n_rows"), (dict(n_rows=-5), "n_rows"), (dict(max_pos=513), "max_pos"),
    (dict(max_pos=-1), "max_pos"), (dict(window=512), "window"), (dict(capacity=0), "capacity"),
    (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(q=0), "NULL"), (dict(row_start=0), "NULL"), (dict(kb=0), "NULL"), (dict(out=4104), "aligned"),
    (dict(k=0), "NULL"), (dict(k=4104), "aligned"), (dict(n_rows=1 << 27), "too many query vectors"),
    (dict(pages=4096, page_size=100, max_pages=4, pool_pages=9), "page_size"),
    (dict(pages=4096, page_size=128, max_pages=3, pool_pages=9), "max_pages"),
    (dict(capacity=1 << 30, max_pos=16), "2^31"), (dict(head_dim=80), "head_dim"),
])
def test_prompt_attention_refusals(D, change, word):
    _refuse(D, "dflash_prompt_attention", prompt_args(D, **change), word)


@pytest.mark.parametrize("change,word", [
    (dict(k_exp=4096, v_exp=4096), "8-bit"), (dict(n_q_heads=129, n_kv_heads=1), "query heads"),
    (dict(n_seqs=1 << 21, base_pos=0), "pieces"), (dict(n_rows=1 << 23, max_pos=0), "pieces"),
])
def test_prompt_attention_unsupported(D, change, word):
    _refuse(D, "dflash_prompt_attention", prompt_args(D, **change), word, D.DFLASH_ERR_UNSUPPORTED)


def test_prompt_attention_workspace(D):
    """Sized from the shapes alone; a smaller one is refused."""
    for dtype in (D.DFLASH_BF16, D.DFLASH_F32):
        a = prompt_args(D, dtype=dtype, q=0, k=0)
        n = D.dflash_workspace_bytes(D.DFLASH_OP_PROMPT_ATTENTION, a)
        assert n > 0
        a = prompt_args(D, dtype=dtype)
        assert D.lib().dflash_prompt_attention(C.byref(a), C.c_void_p(256), n - 1, None) == D.DFLASH_ERR_WORKSPACE
        assert D.lib().dflash_prompt_attention(C.byref(a), None, n, None) == D.DFLASH_ERR_INVALID_ARG
        assert D.lib().dflash_prompt_attention(C.byref(a), C.c_void_p(264), n, None) == D.DFLASH_ERR_INVALID_ARG
    assert D.dflash_workspace_bytes(D.DFLASH_OP_PROMPT_ATTENTION, prompt_args(D, n_rows=0)) == 0


def score_args(D, **kw):
    a = D.dflash_token_logprobs_args()
    a.dims.vocab = 1000
    a.n_rows, a.temperature, a.topk = 4, 1.0, 5
    a.logits = a.tokens = a.logprob = a.entropy = a.top_ids = a.top_logprobs = 4096
    return _change(a, kw)


@pytest.mark.parametrize("change,word", [
    (dict(n_rows=0), "n_rows"), (dict(n_rows=(1 << 24) + 1), "n_rows"), (dict(vocab=0), "vocab"),
    (dict(vocab=1 << 28), "vocab"), (dict(temperature=0.0), "temperature"), (dict(temperature=-1.0), "temperature"),
    (dict(temperature=float("nan")), "temperature"), (dict(temperature=float("inf")), "temperature"),
    (dict(topk=-1), "topk"), (dict(topk=33), "topk"), (dict(topk=6, vocab=5), "topk"), (dict(logits=0), "logits"),
    (dict(logits=4098), "aligned"), (dict(tokens=0), "go together"), (dict(logprob=0), "go together"),
    (dict(top_ids=0), "top_ids"), (dict(top_logprobs=0), "top_logprobs"),
    (dict(topk=0, tokens=0, logprob=0, entropy=0), "no output"),
])
def test_token_logprobs_refusals(D, change, word):
    _refuse(D, "dflash_token_logprobs", score_args(D, **change), word)


def test_null_arguments_and_small_workspaces(D):
    for name, op, make in (("dflash_qk_norm_rope", D.DFLASH_OP_QK_NORM_ROPE, qk_args),
                           ("dflash_prompt_attention", D.DFLASH_OP_PROMPT_ATTENTION, prompt_args),
                           ("dflash_token_logprobs", D.DFLASH_OP_TOKEN_LOGPROBS, score_args)):
        assert getattr(D.lib(), name)(None, None, 0, None) == D.DFLASH_ERR_INVALID_ARG
        assert "NULL args" in D.dflash_last_error()
        n = D.dflash_workspace_bytes(op, make(D))
        assert n > 0
        a = make(D)
        assert getattr(D.lib(), name)(C.byref(a), C.c_void_p(256), n - 256, None) == D.DFLASH_ERR_WORKSPACE
