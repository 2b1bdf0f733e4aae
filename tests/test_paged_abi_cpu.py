"""Host-side checks of the paged cache and scoring entry points that need no
GPU: struct layout, size queries, and refusals before anything is launched
(pointers here are never dereferenced)."""
import ctypes

import pytest

import gpt_pre_ln_gb300 as G

ARG, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from gpt_pre_ln_gb300 import build
    build.build()
    return G.lib()


def _cache(**kw):
    f = dict(pages=256, refs=256, table=256, lens=256, n_pages=10, page_size=16, n_layer=2, n_kv_head=2, n_seq=4,
             max_pages=8, dtype=G.BF16)
    f.update(kw)
    return G.PagedCache(*[f[k] for k in ("pages", "refs", "table", "lens", "n_pages", "page_size", "n_layer",
                                         "n_kv_head", "n_seq", "max_pages", "dtype")])


def test_struct_layout(L):
    assert ctypes.sizeof(G.PagedCache) == 4 * 8 + 7 * 4 + 4
    assert G.PagedCache.n_pages.offset == 32 and G.PagedCache.dtype.offset == 56


def test_sizes(L):
    c = _cache(n_pages=7, page_size=32, n_layer=3, n_kv_head=5)
    assert G.gpt2_paged_cache_bytes(c) == 7 * 3 * 2 * 5 * 32 * 64 * 2
    assert G.gpt2_pages_workspace_bytes(c) > 0
    assert G.gpt2_attention_paged_workspace_bytes(c, 10) > 0
    assert G.gpt2_attention_paged_workspace_bytes(c, 11) == 0
    bad = _cache(page_size=24)
    assert G.gpt2_paged_cache_bytes(bad) == 0 and G.gpt2_pages_workspace_bytes(bad) == 0
    d = G.make_dims(2, 128, 2, 512, 1000, 64)
    assert G.gpt2_decode_step_paged_workspace_bytes(d, _cache()) > G.gpt2_decode_workspace_bytes(d, 4)
    assert G.gpt2_prefill_paged_workspace_bytes(d, _cache(), 8) == G.gpt2_prefill_workspace_bytes(d, 4, 8)


@pytest.mark.parametrize("change, status", [
    (dict(pages=0), ARG), (dict(refs=0), ARG), (dict(table=0), ARG), (dict(lens=0), ARG), (dict(pages=264), ARG),
    (dict(table=258), ARG), (dict(n_pages=0), ARG), (dict(n_pages=-1), ARG), (dict(page_size=0), ARG),
    (dict(n_layer=0), ARG), (dict(n_kv_head=0), ARG), (dict(n_seq=-1), ARG), (dict(max_pages=0), ARG),
    (dict(dtype=7), ARG), (dict(dtype=G.F32), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
    (dict(page_size=4112), UNSUPPORTED), (dict(n_seq=1025), UNSUPPORTED),
    (dict(page_size=4096, max_pages=1 << 19), UNSUPPORTED)])
def test_cache_refusals(L, change, status):
    c = ctypes.byref(_cache(**change))
    assert L.gpt2_pages_reserve(c, 256, 256, 1 << 30, None) == status
    assert L.gpt2_pages_fork(c, 256, 256, 1, None) == status
    assert L.gpt2_pages_free(c, 256, 1, 0, 0, None) == status
    assert L.gpt2_pages_compact(c, 256, 256, 1 << 30, None) == status
    assert L.gpt2_pages_write(c, 0, 256, 256, 384, 1, None, None) == status
    assert L.gpt2_attention_paged(c, 0, 256, 384, None, None, 0, 4096, 128, None, 2, 0.125, 0, 0, 256, 1 << 30,
                                  None) == status
    assert L.gpt2_pages_reserve(None, 256, 256, 1 << 30, None) == ARG


def test_page_call_refusals(L):
    c = ctypes.byref(_cache())
    need = G.gpt2_pages_workspace_bytes(_cache())
    assert L.gpt2_pages_reserve(c, None, 256, need, None) == ARG
    assert L.gpt2_pages_reserve(c, 256, 0, need, None) == ARG
    assert L.gpt2_pages_reserve(c, 256, 272, need, None) == ARG  # workspace not 256-byte aligned
    assert L.gpt2_pages_reserve(c, 256, 256, need - 1, None) == WORKSPACE
    assert L.gpt2_pages_compact(c, None, 256, need, None) == ARG
    assert L.gpt2_pages_compact(c, 256, 256, need - 1, None) == WORKSPACE
    for n in (-1, 5):
        assert L.gpt2_pages_fork(c, 256, 256, n, None) == ARG
        assert L.gpt2_pages_free(c, 256, n, 0, 0, None) == ARG
    assert L.gpt2_pages_fork(c, None, 256, 1, None) == ARG
    assert L.gpt2_pages_fork(c, 256, None, 1, None) == ARG
    assert L.gpt2_pages_fork(c, 256, 256, 0, None) == 0
    assert L.gpt2_pages_free(c, None, 1, 0, 0, None) == ARG
    assert L.gpt2_pages_free(c, 256, 1, -1, 0, None) == ARG
    assert L.gpt2_pages_free(c, 256, 1, 0, -1, None) == ARG
    assert L.gpt2_pages_write(c, 2, 256, 256, 384, 1, None, None) == ARG  # layer
    assert L.gpt2_pages_write(c, -1, 256, 256, 384, 1, None, None) == ARG
    assert L.gpt2_pages_write(c, 0, 256, 256, 120, 1, None, None) == ARG  # rows overlap
    assert L.gpt2_pages_write(c, 0, 256, 256, 132, 1, None, None) == UNSUPPORTED
    assert L.gpt2_pages_write(c, 0, 264, 256, 384, 1, None, None) == ARG
    assert L.gpt2_pages_write(c, 0, 256, None, 384, 1, None, None) == ARG
    assert L.gpt2_pages_write(c, 0, 256, 256, 384, -1, None, None) == ARG
    assert L.gpt2_pages_write(c, 0, 256, 256, 384, 1 << 30, None, None) == ARG  # n_seq * T
    assert L.gpt2_pages_write(c, 0, None, None, 384, 0, None, None) == 0
    e = ctypes.byref(_cache(n_seq=0))
    assert L.gpt2_pages_reserve(e, None, None, 0, None) == 0
    assert L.gpt2_attention_paged(e, 0, None, 128, None, None, 0, None, 128, None, 2, 0.125, 0, 0, None, 0, None) == 0


def test_attention_refusals(L):
    c = ctypes.byref(_cache())
    need = G.gpt2_attention_paged_workspace_bytes(_cache(), 4)

    def call(layer=0, q=256, ldq=512, k=256, v=256, ldkv=512, out=4096, ldo=256, lse=None, heads=4, scale=0.125,
             window=0, sinks=0, ws=256, ws_bytes=need):
        return L.gpt2_attention_paged(c, layer, q, ldq, k, v, ldkv, out, ldo, lse, heads, scale, window, sinks, ws,
                                      ws_bytes, None)

    for kw in (dict(layer=2), dict(layer=-1), dict(heads=0), dict(window=-1), dict(sinks=-1), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(k=None), dict(v=None), dict(ldq=248),
               dict(ldo=248), dict(ldkv=120), dict(q=None), dict(out=None), dict(q=264), dict(out=264), dict(k=264),
               dict(v=264), dict(lse=258), dict(ws=None), dict(ws=272)):
        assert call(**kw) == ARG, kw
    for kw in (dict(heads=3), dict(ldq=260), dict(ldo=260), dict(ldkv=132)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(ws_bytes=need - 1) == WORKSPACE
    big = ctypes.byref(_cache(n_seq=1024, max_pages=1 << 17, n_kv_head=25))  # tiles beyond 32 bits
    assert L.gpt2_attention_paged(big, 0, 256, 1600, None, None, 0, 4096, 1600, None, 25, 0.125, 0, 0, 256, 1 << 40,
                                  None) == UNSUPPORTED


def test_model_call_refusals(L):
    d = G.make_dims(2, 128, 2, 512, 1000, 64)
    blk = G.BlockWeights(*([256] * 12))
    blocks = (G.BlockWeights * 2)(blk, blk)
    mw = ctypes.byref(G.ModelWeights(256, 256, 256, 256, ctypes.cast(blocks, ctypes.POINTER(G.BlockWeights))))

    def step(dims=d, cache=None, window=0, sinks=0, tokens=256, nxt=256, logits=None, ld=0, ws=256, have=1 << 40):
        return L.gpt2_decode_step_paged(ctypes.byref(dims), mw, ctypes.byref(cache or _cache()), window, sinks, tokens,
                                        nxt, logits, ld, ws, have, None)

    def prompt(dims=d, cache=None, T=8, tokens=256, nxt=256, logits=None, ld=0, ws=256, have=1 << 40):
        return L.gpt2_prefill_paged(ctypes.byref(dims), mw, ctypes.byref(cache or _cache()), tokens, T, nxt, logits,
                                    ld, ws, have, None)

    for call in (step, prompt):
        assert call(dims=G.make_dims(2, 128, 2, 512, 1000, 64, dtype=G.F32)) == UNSUPPORTED
        for c in (_cache(dtype=G.F16), _cache(n_layer=3), _cache(n_kv_head=1), _cache(lens=0)):
            assert call(cache=c) == ARG
        assert call(tokens=None) == ARG and call(nxt=None) == ARG and call(ws=None) == ARG
        assert call(logits=256, ld=999) == ARG and call(logits=256, ld=1001) == UNSUPPORTED
        assert call(have=1000) == WORKSPACE
        assert call(cache=_cache(n_seq=0)) == 0
    assert step(window=-1) == ARG and step(sinks=-1) == ARG
    assert prompt(T=0) == ARG and prompt(T=65) == ARG and prompt(T=-1) == ARG
    assert prompt(cache=_cache(max_pages=1), T=17) == ARG


def test_logprobs_refusals(L):
    def call(logits=256, ld=1000, t=G.F32, M=4, V=1000, tok=256, lp=256, ent=256, lse=256, n=5, ids=256, tlp=256):
        return L.gpt2_token_logprobs(logits, ld, t, M, V, tok, lp, ent, lse, n, ids, tlp, None)

    for kw in (dict(t=7), dict(M=-1), dict(V=0), dict(ld=996), dict(n=-1), dict(tok=None), dict(lp=None),
               dict(ids=None), dict(tlp=None), dict(logits=None), dict(logits=264), dict(V=4, ld=8, n=5),
               dict(tok=None, lp=None, ent=None, lse=None, n=0)):
        assert call(**kw) == ARG, kw
    for kw in (dict(n=33), dict(ld=1002), dict(t=G.BF16, ld=1004)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(M=0, logits=None) == 0


def test_paged_cache_helper_checks_shapes():
    torch = pytest.importorskip("torch")
    pages = torch.zeros(5, 2, 2, 3, 16, 64, dtype=torch.bfloat16)
    refs, table, lens = (torch.zeros(s, dtype=torch.int32) for s in ((5,), (4, 7), (4,)))
    c = G.paged_cache(pages, refs, table, lens)
    assert (c.n_pages, c.n_layer, c.n_kv_head, c.page_size, c.n_seq, c.max_pages) == (5, 2, 3, 16, 4, 7)
    assert c.dtype == G.BF16 and c.pages == pages.data_ptr() and c.lens == lens.data_ptr()
    for args in ((pages.float(), refs, table, lens), (pages[:, :, :1], refs, table, lens), (pages, refs[:4], table, lens),
                 (pages, refs, table, lens[:3]), (pages, refs.long(), table, lens), (pages, refs, table.t(), lens),
                 (pages[:, :1], refs, table, lens)):
        with pytest.raises(ValueError):
            G.paged_cache(*args)
