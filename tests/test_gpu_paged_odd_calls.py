"""Calls on the paged cache that its description allows and that stand between
the other tests: a captured prompt, a captured step with compaction and forks
between its replays, two caches served at once, 1024 slots, slots further on,
large pages, limits of the integer arguments, logits in a wider buffer."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402
from test_gpu_logprobs import _logits, _run  # noqa: E402
from test_gpu_paged_attention import Case, _go  # noqa: E402
from test_gpu_paged_model import Server, _built, _i32, _ref_last, _rel  # noqa: E402,F401
from test_gpu_pages import Both  # noqa: E402

pytestmark = pytest.mark.gpu
RANGE = 6
MOST = 2 ** 31 - 1


def _prompt(n, T, seed=0):
    return np.random.default_rng(seed).integers(0, 1000, (n, T))


def test_a_captured_prompt():
    """Reserve and prefill in one graph; replayed once the slots are begun again, with other tokens."""
    a, b = Server(3), Server(3)
    tokens, new, stream = _i32(_prompt(3, 20).tolist()), _i32([20] * 3), torch.cuda.Stream()
    a.prefill(0, _prompt(3, 20))  # (one call that sets kernel attributes up)
    b.lens.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        G.gpt2_pages_reserve(b.cache, new, b.ws, b.ws.numel())
        G.gpt2_prefill_paged(b.cd, b.mw, b.cache, tokens, 20, b.next, b.logits, 1000, b.ws, b.ws.numel())
    for seed in (0, 1, 2):
        p = _prompt(3, 20, seed)
        tokens.copy_(_i32(p.tolist()))
        if seed:
            G.gpt2_pages_free(b.cache, _i32([0, 1, 2]), 3)
            b.lens.zero_()
        torch.cuda.synchronize()
        graph.replay()
        got = b.got()
        for k in range(3):
            assert _rel(got[k], _ref_last(b, list(p[k]))) < 1e-2
        assert b.lens.cpu().tolist() == [20] * 3
        b.step(b.next)  # and the cache serves
        assert b.lens.cpu().tolist() == [21] * 3


def test_a_captured_step_with_forks_frees_and_compaction_between_its_replays():
    s, e = Server(4, n_pages=30), Server(4, n_pages=30)
    ones, stream = _i32([1] * 4), torch.cuda.Stream()
    for x in (s, e):
        x.prefill(0, _prompt(4, 15))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        G.gpt2_pages_reserve(s.cache, ones, s.ws, s.ws.numel())
        s.step(s.next, reserve=False)
    for turn in range(9):
        graph.replay()
        e.step(e.next)
        live = [b for b in range(4) if int(e.lens[b]) >= 0]
        assert np.array_equal(s.got()[live], e.got()[live]) and torch.equal(s.lens, e.lens)
        if turn == 2:  # beams change places; the graph knows nothing of it
            for x in (s, e):
                G.gpt2_pages_fork(x.cache, _i32([1, 0, 1]), _i32([0, 1, 3]), 3)
                x.next[[0, 1, 3]] = x.next[[1, 0, 1]]
        if turn == 4:
            for x in (s, e):
                G.gpt2_pages_free(x.cache, _i32([2]), 1)
        if turn == 5:  # only one of them: where its pages are makes no difference
            n = _i32([0])
            G.gpt2_pages_compact(s.cache, n, s.ws, s.ws.numel())
            assert int(n) == int((s.refs > 0).sum())
        torch.cuda.synchronize()
    assert s.lens.cpu().tolist()[2] == -1 and torch.equal(s.next, e.next)


def test_two_caches_served_at_once():
    """Steps of two caches on two streams, a workspace each, through the library's launch graphs."""
    many = dict(n_seq=60, n_pages=200)
    a, b = Server(**many), Server(**many, seed=78)
    ra, rb = Server(**many), Server(**many, seed=78)
    for k, x in enumerate((a, b, ra, rb)):
        x.prefill(0, _prompt(60, 12, k % 2))
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ones = _i32([1] * 60)
    for _ in range(6):
        for x, s in ((a, sa), (b, sb)):
            G.gpt2_pages_reserve(x.cache, ones, x.ws, x.ws.numel(), s)
            x.step(x.next, reserve=False, stream=s)
        torch.cuda.synchronize()
        for x, r in ((a, ra), (b, rb)):
            r.step(r.next)
            assert np.array_equal(x.got(), r.got()) and torch.equal(x.next, r.next)


def test_all_slots():
    """1024 sequences: prompts, forks of every slot, a step, and all of them given back."""
    s = Server(1024, n_pages=1300, max_pages=4)
    s.prefill(0, _prompt(8, 20))
    parents = [k % 8 for k in range(1024)]
    G.gpt2_pages_fork(s.cache, _i32(parents), _i32(list(range(1024))), 1024)
    s.next.copy_(s.next[:8].repeat(128))
    torch.cuda.synchronize()
    assert int(s.refs[s.table[0, 0]]) == 128
    s.step(s.next)  # every sequence writes into a shared page: 1016 copies
    got = s.got()
    assert s.lens.cpu().tolist() == [21] * 1024 and int((s.refs > 0).sum()) == 8 + 1024
    for k in range(8):
        # (the same work, cut into runs at other places)
        assert _rel(got[k::8], np.repeat(got[k:k + 1], 128, 0)) < 5e-3
    G.gpt2_pages_free(s.cache, _i32(list(range(1024))), 1024)
    torch.cuda.synchronize()
    assert int(s.refs.abs().sum()) == 0 and int((s.table >= 0).sum()) == 0 and int((s.lens != -1).sum()) == 0


def test_a_step_of_later_slots_leaves_the_others():
    s, full = Server(5), Server(5)
    for x in (s, full):
        x.prefill(0, _prompt(5, 30))
    view = G.paged_cache(s.pages, s.refs, s.table[2:4], s.lens[2:4])
    s.reserve([0, 0, 1, 1, 0])
    before = s.next.clone()
    tok = s.next[2:4].clone()
    other = s.logits[[0, 1, 4]].clone()
    G.gpt2_decode_step_paged(s.cd, s.mw, view, 0, 0, tok, s.next[2:4], s.logits[2:4], 1000, s.ws, s.ws.numel())
    full.step(full.next)
    got, ref = s.got(), full.got()
    assert torch.equal(s.logits[[0, 1, 4]], other)
    assert _rel(got[2:4], ref[2:4]) < 5e-3 and s.lens.cpu().tolist() == [30, 30, 31, 31, 30]
    assert torch.equal(s.next[[0, 1, 4]], before[[0, 1, 4]])


@pytest.mark.parametrize("page", [16, 48, 128, 4096])
def test_page_sizes_of_a_served_model(page):
    """Where the positions lie changes nothing but roundings."""
    cols = -(-128 // page)
    a, s = Server(2), Server(2, n_pages=20, page=page, max_pages=cols)
    for x in (a, s):
        x.prefill(0, _prompt(2, 45))
    for _ in range(5):
        tok = a.next.clone()
        a.step(tok)
        s.step(tok)
        assert _rel(s.got(), a.got()) < 5e-3
    assert torch.equal(a.lens, s.lens)


@pytest.mark.parametrize("window, sinks", [(MOST, 0), (MOST, MOST), (1, MOST), (0, MOST)])
@pytest.mark.parametrize("max_pages", [None, 300])
def test_windows_at_the_integers_end(window, sinks, max_pages):
    c = Case([0, 1, 90, 200, -1], heads=4, kv_heads=2, window=window, sinks=sinks, seed=1, max_pages=max_pages)
    _go(c)


def test_counts_at_the_integers_end():
    x = Both(20, 16, 3, 4)
    x.begin(0)
    x.begin(1)
    x.grow([20, 16, 0])
    x.reserve([MOST, 0, 0], ok=False)
    x.reserve([1, MOST, MOST], ok=False)
    x.reserve([-MOST, 0, MOST], ok=True)  # nothing wanted: the idle slot's count is not looked at
    x.free([0, 1], MOST, 0)
    x.free([0, 1], 0, MOST)
    x.free([0, 1], MOST, MOST)
    x.check()
    rows = torch.ones(3 * 2, 192, dtype=torch.bfloat16, device="cuda")
    before = x.pages.clone()
    G.gpt2_pages_write(x.cache, 0, rows, rows, 192, 2, _i32([-MOST, 0, MOST]))
    torch.cuda.synchronize()
    assert torch.equal(x.pages, before) and G.gpt2_last_error()[0] == 0
    x.lens[0] = MOST  # a length that no table holds: nothing is written, forked pages are those there are
    G.gpt2_pages_write(x.cache, 0, rows, rows, 192, 2, _i32([2, 0, 0]))
    assert G.gpt2_last_error()[0] == RANGE and torch.equal(x.pages, before)
    G.gpt2_pages_reserve(x.cache, _i32([1, 0, 0]), x.ws, x.ws_bytes)
    assert G.gpt2_last_error()[0] == RANGE
    x.lens[0] = 20
    x.check()


def test_empty_sequences_keep_what_was_reserved():
    x = Both(20, 16, 2, 4)
    x.begin(0)
    x.begin(1)
    x.reserve([30, 5])
    x.free([0, 1], 4, 1)
    x.check()
    assert x.m.table[0][:2] == [0, 1]
    x.fork([0], [1])  # nothing to share: the child is an empty sequence without pages
    x.check()
    assert x.m.lens[1] == 0 and x.m.table[1] == [-1] * 4
    x.append([30, 0])
    x.check()


def test_attention_of_sequences_that_share_their_pages():
    """Query only, several sequences and different lengths over the same pages."""
    c = Case([300, 300, 300, 300], heads=12, kv_heads=4, append=False, seed=2)
    c.table[1:] = c.table[0]
    c.refs.fill_(4)
    for b in range(1, 4):
        c.k[b], c.v[b] = c.k[0], c.v[0]
    lens = [300, 1, 0, 177]
    c.lens.copy_(_i32(lens))
    c.lens_l = c.totals = lens
    before = c.pages.clone()
    c.run()
    c.check()
    assert torch.equal(c.pages.view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("dtype, V", [("bf16", 50257), ("bf16", 1003), ("f32", 50257), ("f16", 300)])
def test_scores_of_rows_within_a_wider_buffer(dtype, V):
    """A view of every third row of a buffer, from a column that stands on 16 bytes, NaN all around."""
    z = _logits(4, V, dtype, seed=9)
    wide = torch.full((12, z.shape[1] + 64), float("nan"), dtype=z.dtype, device="cuda")
    view = wide.view(4, 3, -1)[:, 1, 32:32 + z.shape[1]]
    view.copy_(z)
    ld = 3 * wide.shape[1]
    t = {"bf16": G.BF16, "f32": G.F32, "f16": G.F16}[dtype]
    tokens = torch.tensor([0, 5, V - 1, 7], dtype=torch.int32, device="cuda")
    ref = _run(z, V, dtype, 9, tokens)
    lp, ent, lse = (torch.empty(4, device="cuda") for _ in range(3))
    ids, lps = torch.empty((4, 9), dtype=torch.int32, device="cuda"), torch.empty((4, 9), device="cuda")
    G.gpt2_token_logprobs(view.data_ptr(), ld, t, 4, V, tokens, lp, ent, lse, 9, ids, lps)
    torch.cuda.synchronize()
    for k, v in dict(logprob=lp, entropy=ent, lse=lse, ids=ids, lps=lps).items():
        assert torch.equal(v.cpu(), ref[k]), k


def test_scores_on_two_streams_at_once():
    a, b = _logits(900, 50257, "bf16", seed=1), _logits(900, 50257, "bf16", seed=2)
    tokens = torch.arange(900, dtype=torch.int32, device="cuda")
    refs = [_run(z, 50257, "bf16", 8, tokens) for z in (a, b)]
    outs = [dict(logprob=torch.empty(900, device="cuda"), entropy=torch.empty(900, device="cuda"),
                 lse=torch.empty(900, device="cuda"), ids=torch.empty((900, 8), dtype=torch.int32, device="cuda"),
                 lps=torch.empty((900, 8), device="cuda")) for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for z, o, s in zip((a, b), outs, streams):
            G.gpt2_token_logprobs(z, z.shape[1], G.BF16, 900, 50257, tokens, o["logprob"], o["entropy"], o["lse"], 8,
                                  o["ids"], o["lps"], s)
    torch.cuda.synchronize()
    for o, ref in zip(outs, refs):
        assert all(torch.equal(v.cpu(), ref[k]) for k, v in o.items())
