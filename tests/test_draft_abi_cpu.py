"""Host-side checks of the drafted-token and sampling entry points that need no
GPU: size queries, and refusals before anything is launched (pointers here are
never dereferenced)."""
import ctypes

import pytest

import gpt_pre_ln_gb300 as G
from test_paged_abi_cpu import _cache

ARG, UNSUPPORTED, WORKSPACE = 1, 2, 3
ODD = 258  # 2 bytes off a 4-byte boundary


@pytest.fixture(scope="module")
def L():
    from gpt_pre_ln_gb300 import build
    build.build()
    return G.lib()


def test_sizes(L):
    c = _cache()
    need = [G.gpt2_attention_paged_draft_workspace_bytes(c, T, 4) for T in (1, 4, 8, 16, 64)]
    assert all(n > 0 for n in need)
    for T, heads in ((0, 4), (-1, 4), (65, 4), (8, 0), (8, 3), (8, 1026)):
        assert G.gpt2_attention_paged_draft_workspace_bytes(c, T, heads) == 0
    assert G.gpt2_attention_paged_draft_workspace_bytes(_cache(page_size=24), 8, 4) == 0
    d = G.make_dims(2, 128, 2, 512, 1000, 64)
    assert (G.gpt2_draft_step_paged_workspace_bytes(d, c, 8)
            == G.gpt2_workspace_bytes(d, 4, 8) + G.gpt2_attention_paged_draft_workspace_bytes(c, 8, 2))
    assert G.gpt2_draft_step_paged_workspace_bytes(d, c, 65) == 0
    assert G.gpt2_draft_step_paged_workspace_bytes(G.make_dims(2, 128, 2, 512, 1000, 64, dtype=G.F32), c, 8) == 0


def _attn(L, c=None, layer=0, q=256, ldq=512, k=256, v=256, ldkv=512, out=4096, ldo=256, lse=None, T=8, parents=256,
          n=256, heads=4, scale=0.125, window=0, sinks=0, ws=256, ws_bytes=1 << 40):
    return L.gpt2_attention_paged_draft(ctypes.byref(c or _cache()), layer, q, ldq, k, v, ldkv, out, ldo, lse, T,
                                        parents, n, heads, scale, window, sinks, ws, ws_bytes, None)


def test_attention_refusals(L):
    for kw in (dict(layer=2), dict(layer=-1), dict(heads=0), dict(window=-1), dict(sinks=-1), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(k=None), dict(v=None), dict(ldq=248),
               dict(ldo=248), dict(ldkv=120), dict(q=None), dict(out=None), dict(q=264), dict(out=264), dict(k=264),
               dict(v=264), dict(lse=ODD), dict(parents=ODD), dict(n=ODD), dict(ws=None), dict(ws=272), dict(T=-1)):
        assert _attn(L, **kw) == ARG, kw
    for kw in (dict(heads=3), dict(heads=1026), dict(ldq=260), dict(ldo=260), dict(ldkv=132), dict(T=65)):
        assert _attn(L, **kw) == UNSUPPORTED, kw
    assert _attn(L, ws_bytes=G.gpt2_attention_paged_draft_workspace_bytes(_cache(), 8, 4) - 1) == WORKSPACE
    assert _attn(L, T=0, q=None, out=None, ws=None) == 0
    assert _attn(L, c=_cache(n_seq=0), q=None, out=None, ws=None) == 0
    big = _cache(n_seq=1024, max_pages=1 << 17, n_kv_head=25)  # tiles beyond 32 bits
    assert _attn(L, c=big, heads=25, ldq=4800, ldkv=4800, ldo=1600) == UNSUPPORTED
    rows = _cache(n_pages=1 << 20, n_layer=64, n_kv_head=2)  # rows of the pool beyond 32 bits
    assert _attn(L, c=rows) == UNSUPPORTED
    for change, status in ((dict(pages=0), ARG), (dict(dtype=7), ARG), (dict(dtype=G.F32), UNSUPPORTED),
                           (dict(page_size=24), UNSUPPORTED), (dict(n_seq=1025), UNSUPPORTED)):
        assert _attn(L, c=_cache(**change)) == status, change


def test_accept_refusals(L):
    def call(c=None, T=8, tokens=256, parents=256, n=256, chosen=256, path=256, kept=256, nxt=256):
        return L.gpt2_draft_accept(ctypes.byref(c or _cache()), T, tokens, parents, n, chosen, path, kept, nxt, None)

    for name in ("tokens", "chosen", "path", "kept", "nxt"):
        for bad in (None, ODD):
            assert call(**{name: bad}) == ARG, name
    assert call(parents=ODD) == ARG and call(n=ODD) == ARG and call(T=-1) == ARG
    assert call(T=65) == UNSUPPORTED
    assert call(T=0, tokens=None) == 0 and call(c=_cache(n_seq=0), tokens=None) == 0
    assert call(c=_cache(lens=0)) == ARG and call(c=_cache(dtype=G.F32)) == UNSUPPORTED


def test_model_refusals(L):
    d = G.make_dims(2, 128, 2, 512, 1000, 64)
    blk = G.BlockWeights(*([256] * 12))
    blocks = (G.BlockWeights * 2)(blk, blk)
    mw = ctypes.byref(G.ModelWeights(256, 256, 256, 256, ctypes.cast(blocks, ctypes.POINTER(G.BlockWeights))))

    def call(dims=d, c=None, T=8, tokens=256, parents=256, n=256, window=0, sinks=0, logits=256, ld=1000, t=G.F32,
             ws=256, have=1 << 40):
        return L.gpt2_draft_step_paged(ctypes.byref(dims), mw, ctypes.byref(c or _cache()), T, tokens, parents, n,
                                       window, sinks, logits, ld, t, ws, have, None)

    for kw in (dict(tokens=None), dict(tokens=ODD), dict(parents=ODD), dict(n=ODD), dict(window=-1), dict(sinks=-1),
               dict(logits=None), dict(logits=264), dict(ld=996), dict(t=7), dict(T=-1), dict(ws=None), dict(ws=272),
               dict(c=_cache(dtype=G.F16)), dict(c=_cache(n_layer=3)), dict(c=_cache(n_kv_head=1))):
        assert call(**kw) == ARG, kw
    for kw in (dict(T=65), dict(t=G.F16), dict(ld=1001), dict(t=G.BF16, ld=1004),
               dict(dims=G.make_dims(2, 128, 2, 512, 1000, 64, dtype=G.F32))):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(have=1000) == WORKSPACE
    assert call(T=0) == 0 and call(c=_cache(n_seq=0)) == 0


def test_sample_refusals(L):
    def call(logits=256, ld=1000, t=G.F32, M=4, V=1000, temp=256, k=256, p=256, m=256, u=256, tok=256, lp=256):
        return L.gpt2_sample_tokens(logits, ld, t, M, V, temp, k, p, m, u, tok, lp, None)

    for kw in (dict(t=7), dict(M=-1), dict(V=0), dict(V=-1), dict(ld=996), dict(logits=None), dict(logits=264),
               dict(u=None), dict(tok=None)) + tuple({k: ODD} for k in ("temp", "k", "p", "m", "u", "tok", "lp")):
        assert call(**kw) == ARG, kw
    for kw in (dict(ld=1001), dict(t=G.BF16, ld=1004), dict(M=1 << 30), dict(V=(1 << 21) + 4, ld=(1 << 21) + 4)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(M=0, logits=None, u=None, tok=None) == 0
