"""Pointers that the paged-cache and scoring calls may not follow are refused
on the host: an int32 or fp32 array off its 4-byte boundary is a misaligned
access on the GPU.  So are pools whose bytes do not fit 64 bits.  Nothing is
launched (no GPU needed)."""
import ctypes

import pytest

import gpt_pre_ln_gb300 as G

ARG = 1
ODD = 258  # 2 bytes off


@pytest.fixture(scope="module")
def L():
    from gpt_pre_ln_gb300 import build
    build.build()
    return G.lib()


CACHE = G.PagedCache(256, 256, 256, 256, 10, 16, 2, 2, 4, 8, G.BF16)


def test_page_calls(L):
    c, big = ctypes.byref(CACHE), 1 << 30
    assert L.gpt2_pages_reserve(c, ODD, 256, big, None) == ARG
    assert L.gpt2_pages_fork(c, ODD, 256, 1, None) == ARG
    assert L.gpt2_pages_fork(c, 256, ODD, 1, None) == ARG
    assert L.gpt2_pages_free(c, ODD, 1, 0, 0, None) == ARG
    assert L.gpt2_pages_compact(c, ODD, 256, big, None) == ARG
    assert L.gpt2_pages_write(c, 0, 256, 256, 384, 1, ODD, None) == ARG


def test_model_calls(L):
    d = G.make_dims(2, 128, 2, 512, 1000, 64)
    blk = G.BlockWeights(*([256] * 12))
    blocks = (G.BlockWeights * 2)(blk, blk)
    mw = ctypes.byref(G.ModelWeights(256, 256, 256, 256, ctypes.cast(blocks, ctypes.POINTER(G.BlockWeights))))
    for tokens, nxt in ((ODD, 256), (256, ODD)):
        assert L.gpt2_decode_step_paged(ctypes.byref(d), mw, ctypes.byref(CACHE), 0, 0, tokens, nxt, None, 0, 256,
                                        1 << 40, None) == ARG
        assert L.gpt2_prefill_paged(ctypes.byref(d), mw, ctypes.byref(CACHE), tokens, 8, nxt, None, 0, 256, 1 << 40,
                                    None) == ARG


@pytest.mark.parametrize("which", ["tok", "lp", "ent", "lse", "ids", "tlp"])
def test_scores(L, which):
    p = dict(tok=256, lp=256, ent=256, lse=256, ids=256, tlp=256)
    p[which] = ODD
    assert L.gpt2_token_logprobs(256, 1000, G.F32, 4, 1000, p["tok"], p["lp"], p["ent"], p["lse"], 5, p["ids"],
                                 p["tlp"], None) == ARG


@pytest.mark.parametrize("n_pages, fits", [(1 << 20, True), (1 << 22, False), (2 ** 31 - 1, False)])
def test_pools_beyond_64_bits(L, n_pages, fits):
    """4096 layers of 1024 heads, pages of 4096: 2^42 bytes each."""
    c = G.PagedCache(256, 256, 256, 256, n_pages, 4096, 4096, 1024, 4, 8, G.BF16)
    assert G.gpt2_paged_cache_bytes(c) == (n_pages << 42 if fits else 0)
    assert L.gpt2_pages_fork(ctypes.byref(c), None, None, 0, None) == (0 if fits else 2)
