"""include/svd_tree.h without a GPU: layouts, sizes, argument checks before any launch, and the
refusals of the Python entry points."""
import ctypes
import os
import subprocess

import pytest
import torch

from speculative_decoding_verify_distill_b200 import api
from speculative_decoding_verify_distill_b200 import build as svd_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, WS = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x10000)   # never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    svd_build.build()
    return api.lib()


@pytest.mark.parametrize("struct,mirror", [("svd_tree_attention_args", api.TreeAttentionArgs),
                                           ("svd_logits_process_args", api.LogitsProcessArgs),
                                           ("svd_tree_verify_args", api.TreeVerifyArgs),
                                           ("svd_cache_append_args", api.CacheAppendArgs)])
def test_ctypes_mirrors_match_the_c_layout(struct, mirror, tmp_path):
    names = [f[0] for f in mirror._fields_]
    src = tmp_path / "layout.c"
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "svd_tree.h"', "int main(void) {",
             '  printf("%%zu\\n", sizeof(%s));' % struct]
    lines += ['  printf("%%zu\\n", offsetof(%s, %s));' % (struct, f) for f in names]
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert out[0] == ctypes.sizeof(mirror)
    assert out[1:] == [getattr(mirror, f).offset for f in names]


def test_status_names(L):
    assert L.svd_status_string(8).decode() == "SVD_ERR_PAGE_RANGE"
    assert L.svd_status_string(9).decode() == "SVD_ERR_TREE"


def test_workspace_sizes(L):
    assert L.svd_tree_attention_workspace_bytes(4, 65, 8, 8, 128) == 0
    assert L.svd_tree_attention_workspace_bytes(4, 8, 9, 8, 128) == 0
    assert L.svd_tree_attention_workspace_bytes(4, 8, 8, 8, 128) >= 256
    assert L.svd_logits_process_workspace_bytes(4, 0) == 0
    assert L.svd_logits_process_workspace_bytes(4, 9) >= 256 + 4 * 9 * 8 + 4 * 4
    assert L.svd_tree_verify_workspace_bytes(4, 9) >= 256 + 4 * 9 * 8 + 4 * 4
    assert L.svd_cache_append_workspace_bytes(-1) == 0
    assert L.svd_cache_append_workspace_bytes(1000) >= 256 + 4000


def _args(cls, base, kw):
    a = cls()
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return ctypes.byref(a)


ATT = dict(q=FAKE, k_new=FAKE, v_new=FAKE, cache_k=FAKE, cache_v=FAKE, page_stride_k=16 * 4 * 64, page_stride_v=16 * 4 * 64,
           page_table=FAKE, cache_len=FAKE, B=2, n=5, Hq=8, Hkv=4, D=64, n_pages=10, page_size=16, max_pages=5, dtype=0,
           scale=0.125, out=FAKE)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), 1), (dict(n=65), 1), (dict(B=-1), 1), (dict(Hq=9), 1), (dict(Hkv=0), 1), (dict(D=0), 1), (dict(dtype=2), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(n_pages=-1), 1), (dict(max_pages=-1), 1),
    (dict(page_size=0), 1), (dict(max_pages=1 << 28), 1), (dict(max_pages=(1 << 26) + 1), 1), (dict(page_stride_k=1 << 39), 6), (dict(page_table=None), 1), (dict(cache_k=None), 1),
    (dict(page_stride_k=16 * 4 * 64 - 8), 1), (dict(page_stride_v=-8), 1), (dict(q=None), 1), (dict(k_new=None), 1),
    (dict(cache_len=None), 1), (dict(out=None), 1), (dict(D=136, page_stride_k=BIG, page_stride_v=BIG), 6),
    (dict(D=60), 6), (dict(page_size=4), 6), (dict(page_size=24, page_stride_k=BIG, page_stride_v=BIG), 6), (dict(Hq=2048), 6),
    (dict(q=ctypes.c_void_p(0x1008)), 2), (dict(cache_v=ctypes.c_void_p(0x1002)), 2),
    (dict(page_stride_k=16 * 4 * 64 + 4), 2)])
def test_attention_refusals(L, kw, code):
    assert L.svd_tree_attention(_args(api.TreeAttentionArgs, ATT, kw), WS, BIG, None) == code


def test_attention_workspace_refusals_and_empty_batch(L):
    a = lambda **kw: _args(api.TreeAttentionArgs, ATT, kw)  # noqa: E731
    assert L.svd_tree_attention(None, WS, BIG, None) == 1
    assert L.svd_tree_attention(a(), None, BIG, None) == 1
    assert L.svd_tree_attention(a(), ctypes.c_void_p(0x10010), BIG, None) == 2
    assert L.svd_tree_attention(a(), WS, 16, None) == 3
    assert L.svd_tree_attention(a(B=0, q=None, out=None), None, 0, None) == 0


PROC = dict(logits=FAKE, B=2, n=5, V=100, history=FAKE, hist_stride=10, node_tok=FAKE, bias_tok=FAKE, bias_val=FAKE, n_bias=3,
            mask=FAKE, mask_rows=5, mask_value=-1.0, out=FAKE, dz=FAKE, dlogits=FAKE)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), 1), (dict(n=65), 1), (dict(B=-1), 1), (dict(V=0), 1), (dict(V=400000), 6), (dict(B=70000), 6),
    (dict(hist_stride=-1), 1), (dict(hist_stride=1 << 24), 1), (dict(bias_val=None), 1), (dict(n_bias=-1), 1),
    (dict(n_bias=5000), 1), (dict(mask_rows=0), 1), (dict(mask_rows=4), 1), (dict(logits=None), 1)])
def test_process_refusals(L, kw, code):
    a = lambda **more: _args(api.LogitsProcessArgs, PROC, {**kw, **more})  # noqa: E731
    assert L.svd_logits_process(a(), WS, BIG, None) == code
    assert L.svd_logits_process_grad(a(), WS, BIG, None) == code


def test_process_own_refusals(L):
    a = lambda **kw: _args(api.LogitsProcessArgs, PROC, kw)  # noqa: E731
    assert L.svd_logits_process(None, WS, BIG, None) == 1
    assert L.svd_logits_process(a(mask_value=float("nan")), WS, BIG, None) == 1
    assert L.svd_logits_process(a(out=None, argmax=None), WS, BIG, None) == 1
    assert L.svd_logits_process(a(), ctypes.c_void_p(0x10001), BIG, None) == 2
    assert L.svd_logits_process(a(), WS, 255, None) == 3
    assert L.svd_logits_process(a(B=0), None, 0, None) == 0
    assert L.svd_logits_process_grad(None, WS, BIG, None) == 1
    assert L.svd_logits_process_grad(a(dz=None), WS, BIG, None) == 1
    assert L.svd_logits_process_grad(a(dlogits=None), WS, BIG, None) == 1
    assert L.svd_logits_process_grad(a(grad_fp32=2), WS, BIG, None) == 1
    assert L.svd_logits_process_grad(a(B=0), None, 0, None) == 0


def test_verify_refusals(L):
    base = dict(T=FAKE, node_tok=FAKE, B=2, n=5, V=100, path=FAKE, n_path=FAKE, accept_len=FAKE, emitted=FAKE, n_emitted=FAKE)
    a = lambda **kw: _args(api.TreeVerifyArgs, base, kw)  # noqa: E731
    for kw, code in ((dict(n=0), 1), (dict(n=65), 1), (dict(B=-1), 1), (dict(V=0), 1), (dict(V=400000), 6), (dict(B=70000), 6),
                     (dict(target_tok=FAKE), 1), (dict(T=None), 1), (dict(node_tok=None), 1), (dict(path=None), 1),
                     (dict(n_emitted=None), 1)):
        assert L.svd_tree_verify(a(**kw), WS, BIG, None) == code, kw
    assert L.svd_tree_verify(None, WS, BIG, None) == 1
    assert L.svd_tree_verify(a(), ctypes.c_void_p(0x10010), BIG, None) == 2
    assert L.svd_tree_verify(a(), WS, 300, None) == 3
    assert L.svd_tree_verify(a(B=0), None, 0, None) == 0


def test_append_refusals(L):
    base = dict(k_new=FAKE, v_new=FAKE, cache_k=FAKE, cache_v=FAKE, page_stride_k=10 * 128, page_stride_v=10 * 128,
                page_table=FAKE, cache_len=FAKE, count=FAKE, B=2, n=5, Hkv=2, D=64, n_pages=9, page_size=10, max_pages=4)
    a = lambda **kw: _args(api.CacheAppendArgs, base, kw)  # noqa: E731
    for kw, code in ((dict(n=0), 1), (dict(B=-1), 1), (dict(Hkv=0), 1), (dict(D=0), 1), (dict(D=3), 6), (dict(B=70000), 6),
                     (dict(page_size=0), 1), (dict(n_pages=-1), 1), (dict(page_table=None), 1), (dict(cache_v=None), 1),
                     (dict(page_stride_k=8), 1), (dict(count=None), 1), (dict(k_new=None), 1),
                     (dict(k_new=ctypes.c_void_p(0x1004)), 2), (dict(page_stride_v=1284), 2)):
        assert L.svd_cache_append(a(**kw), WS, BIG, None) == code, kw
    assert L.svd_cache_append(None, WS, BIG, None) == 1
    assert L.svd_cache_append(a(), ctypes.c_void_p(0x10010), BIG, None) == 2
    assert L.svd_cache_append(a(), WS, 256, None) == 3
    assert L.svd_cache_append(a(B=0), None, 0, None) == 0


def test_python_refuses_cpu_tensors():
    """Every entry point wants CUDA tensors; wrong types and ranks are named before that."""
    bf, i32 = torch.bfloat16, torch.int32
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)  # noqa: E731
    with pytest.raises(TypeError):
        api.TreeAttention(z(1, 1, 8, 64, dt=torch.float32), z(1, 1, 8, 64), z(1, 1, 8, 64), z(4, 16, 8, 64), z(4, 16, 8, 64),
                          z(1, 4, dt=i32), z(1, dt=i32))
    with pytest.raises(ValueError):
        api.TreeAttention(z(1, 1, 8, 64), z(1, 1, 8, 64), z(1, 1, 8, 64), z(4, 16, 8, 64), z(4, 16, 8, 64), z(1, 4, dt=i32),
                          z(1, dt=i32))
    with pytest.raises(ValueError):
        api.LogitsProcess(z(2, 3, 100))
    with pytest.raises(ValueError):
        api.LogitsProcessGrad(z(2, 3, 100), z(2, 3, 100))
    with pytest.raises(ValueError):
        api.TreeVerify(z(2, 3, dt=i32))
    with pytest.raises(ValueError):
        api.TreeVerify(z(2, 3, dt=i32), logits=z(2, 3, 100))
    with pytest.raises(TypeError):
        api.CacheAppend(z(1, 1, 8, 64, dt=torch.float32), None, None, None, None, None, None)
    with pytest.raises(ValueError):
        api.CacheAppend(z(1, 1, 8, 64), z(1, 1, 8, 64), z(4, 16, 8, 64), z(4, 16, 8, 64), z(1, 4, dt=i32), z(1, dt=i32),
                        z(1, dt=i32))
