"""The size limits of gpt2_attention_paged_draft as documented, on both sides, by its
refusals (nothing is launched: the workspace pointer is left out)."""
import ctypes

import pytest

import gpt_pre_ln_gb300 as G
from test_paged_abi_cpu import _cache

ARG, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def L():
    from gpt_pre_ln_gb300 import build
    build.build()
    return G.lib()


def _call(L, T, heads, kv, **cache):
    c = _cache(n_kv_head=kv, n_layer=1, n_pages=64, **cache)
    return L.gpt2_attention_paged_draft(ctypes.byref(c), 0, 256, 64 * heads, None, None, 0, 4096, 64 * heads, None, T, None,
                                        None, heads, 0.125, 0, 0, None, 0, None)


@pytest.mark.parametrize("T, heads, kv, blocks", [(1, 1, 1, 1), (8, 1, 1, 1), (9, 1, 1, 1), (64, 1, 1, 1), (33, 4, 2, 2),
                                                  (64, 8, 2, 4), (13, 10, 1, 3), (64, 1024, 1, 1024)])
def test_places_times_blocks_of_rows(L, T, heads, kv, blocks):
    """n_seq * n_kv_head * max_pages * page_size * blocks of 64 query rows below 2^34."""
    n_seq, page = 256, 64
    most = ((1 << 34) - 1) // (n_seq * kv * page * blocks)
    assert _call(L, T, heads, kv, n_seq=n_seq, page_size=page, max_pages=most) == ARG  # no workspace
    assert _call(L, T, heads, kv, n_seq=n_seq, page_size=page, max_pages=most + 1) == UNSUPPORTED
