"""Refusals at the edges of include/svd_tree.h, without a GPU."""
import ctypes

import pytest

from speculative_decoding_verify_distill_b200 import api
from speculative_decoding_verify_distill_b200 import build as svd_build
from tests.test_tree_abi import ATT, BIG, WS, _args


@pytest.fixture(scope="module")
def L():
    svd_build.build()
    return api.lib()


@pytest.mark.parametrize("sign", [1, -1])
def test_attention_refuses_scales_that_overflow(L, sign):
    """The scale is brought to base 2: scale * log2(e) has to be finite as well, or 0 * inf spoils rows of zeros."""
    call = lambda scale: L.svd_tree_attention(_args(api.TreeAttentionArgs, ATT, dict(scale=sign * scale)), WS, 16, None)  # noqa: E731
    assert call(2.0 ** 127) == 3            # taken: the next check is the workspace's size
    assert call(2.0 ** -149) == 3
    for scale in (2.0 ** 127 * 1.5, 3e38, 3.4e38):
        assert ctypes.c_float(scale).value < float("inf")
        assert call(scale) == 1


def test_empty_batches_have_no_page_table(L):
    """The page table of no sequences is an empty tensor, whose pointer is NULL."""
    none = dict(B=0, page_table=None)
    assert L.svd_tree_attention(_args(api.TreeAttentionArgs, ATT, none), WS, BIG, None) == 0
    append = dict(k_new=None, v_new=None, cache_k=WS, cache_v=WS, page_stride_k=10 * 128, page_stride_v=10 * 128, n=5, Hkv=2,
                  D=64, n_pages=9, page_size=10, max_pages=4)
    assert L.svd_cache_append(_args(api.CacheAppendArgs, append, none), WS, BIG, None) == 0
    assert L.svd_cache_append(_args(api.CacheAppendArgs, append, dict(B=1, page_table=None)), WS, BIG, None) == 1
