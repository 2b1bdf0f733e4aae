"""A model served from a paged cache, on the GPU: gpt2_prefill_paged and
gpt2_decode_step_paged with the page calls and gpt2_token_logprobs around
them, against the contiguous-cache calls and the float64 oracle.

Gates: logits against the oracle within the relative L2 of 1e-2 that the other
model tests use for bf16 (a wrong page, position or head is an error of order
1); log probabilities and entropies are checked against the GPU's own logits
in float64 to fp32 rounding (2e-5 for a vocabulary of 1000)."""
import numpy as np
import pytest

import oracle as O
import synth

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402

pytestmark = pytest.mark.gpu
RANGE = 6


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gpt_pre_ln_gb300 import build
    build.build()
    G.lib()
    yield
    st, site = G.gpt2_last_error()
    assert st == 0, f"device error {st} at site {site}"


def _i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _rel(got, ref):
    return float(np.linalg.norm(got - ref) / np.linalg.norm(ref))


class Server:
    def __init__(self, n_seq, n_pages=60, page=16, max_pages=8, seed=77, dtype=G.BF16):
        self.dims = synth.Dims(n_layer=2, d_model=192, n_head=3, d_ff=512, vocab=1000, n_pos=128)
        self.params, _ = synth.draw_model(self.dims, "bf16", seed)
        d = self.dims
        self.dev = G.to_device(self.params, dtype)
        self.mw, self.keep = G.model_weights(self.dev)
        self.cd = G.make_dims(d.n_layer, d.d_model, d.n_head, d.d_ff, d.vocab, d.n_pos, d.eps, dtype)
        tdt = torch.float16 if dtype == G.F16 else torch.bfloat16
        self.n = n_seq
        self.pages = torch.full((n_pages, d.n_layer, 2, d.n_head, page, 64), float("nan"), dtype=tdt, device="cuda")
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((n_seq, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.full((n_seq,), -1, dtype=torch.int32, device="cuda")
        self.cache = G.paged_cache(self.pages, self.refs, self.table, self.lens)
        need = max(G.gpt2_pages_workspace_bytes(self.cache),
                   G.gpt2_decode_step_paged_workspace_bytes(self.cd, self.cache),
                   G.gpt2_prefill_paged_workspace_bytes(self.cd, self.cache, d.n_pos))
        self.ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        self.logits = torch.zeros(n_seq, 1000, device="cuda")
        self.next = torch.full((n_seq,), -1, dtype=torch.int32, device="cuda")

    def reserve(self, n_new):
        G.gpt2_pages_reserve(self.cache, _i32(n_new), self.ws, self.ws.numel())

    def prefill(self, first, tokens):
        """Prompts of equal length into slots first, first + 1, ..."""
        B, T = tokens.shape
        self.lens[first:first + B] = 0
        self.reserve([T if first <= b < first + B else 0 for b in range(self.n)])
        view = G.paged_cache(self.pages, self.refs, self.table[first:first + B], self.lens[first:first + B])
        G.gpt2_prefill_paged(self.cd, self.mw, view, _i32(tokens.tolist()), T, self.next[first:first + B],
                             self.logits[first:first + B], 1000, self.ws, self.ws.numel())

    def step(self, tokens, window=0, sinks=0, reserve=True, stream=None):
        if reserve:
            self.reserve([1] * self.n)
        G.gpt2_decode_step_paged(self.cd, self.mw, self.cache, window, sinks, tokens, self.next, self.logits, 1000,
                                 self.ws, self.ws.numel(), stream)

    def got(self):
        torch.cuda.synchronize()
        return self.logits.double().cpu().numpy()


def _ref_last(s, tokens):
    return O.forward_logits(np.asarray([tokens]), s.params, s.dims)[0, -1]


@pytest.mark.parametrize("dtype", [G.BF16, G.F16])
def test_prefill_and_decode_follow_the_oracle(dtype):
    s = Server(5, dtype=dtype)
    g = np.random.default_rng(1)
    a, b = g.integers(0, 1000, (2, 21)), g.integers(0, 1000, (1, 40))
    s.prefill(0, a)
    s.prefill(3, b)  # slots 2 and 4 stay empty
    seqs = {0: list(a[0]), 1: list(a[1]), 3: list(b[0])}
    got = s.got()
    for k, t in seqs.items():
        assert _rel(got[k], _ref_last(s, t)) < 1e-2
        assert int(s.next[k]) == int(np.argmax(got[k]))
    assert s.lens.cpu().tolist() == [21, 21, -1, 40, -1]
    for _ in range(12):  # across page borders
        tok = s.next.clone()
        tok[2] = -5  # an idle slot's token is not looked at
        for k in seqs:
            seqs[k].append(int(tok[k]))
        s.step(tok)
        got = s.got()
        for k, t in seqs.items():
            assert _rel(got[k], _ref_last(s, t)) < 1e-2
            assert int(s.next[k]) == int(np.argmax(got[k]))
    assert s.lens.cpu().tolist() == [33, 33, -1, 52, -1]
    assert int(s.next[2]) == -1


def test_paged_and_contiguous_caches_agree():
    """The same prompt and steps through both caches: they differ in the attention's rounding alone."""
    s = Server(3)
    g = np.random.default_rng(2)
    prompt = g.integers(0, 1000, (3, 50))
    s.prefill(0, prompt)
    d = s.dims
    kv = torch.zeros(d.n_layer, 2, 3, d.n_head, 128, 64, dtype=torch.bfloat16, device="cuda")
    past, nxt, lg = _i32([0] * 3), _i32([0] * 3), torch.zeros(3, 1000, device="cuda")
    need = G.gpt2_prefill_workspace_bytes(s.cd, 3, 50)
    ws = torch.empty(max(need, G.gpt2_decode_workspace_bytes(s.cd, 3)), dtype=torch.uint8, device="cuda")
    G.gpt2_prefill(s.cd, s.mw, _i32(prompt.tolist()), 3, 50, kv, 128, past, nxt, lg, 1000, ws, ws.numel())
    assert np.array_equal(s.got(), lg.double().cpu().numpy())
    for _ in range(3):
        tok = nxt.clone()
        s.step(tok)
        G.gpt2_decode_step(s.cd, s.mw, kv, 3, 128, past, tok, nxt, lg, 1000, ws, ws.numel())
        assert _rel(s.got(), lg.double().cpu().numpy()) < 5e-3
    assert torch.equal(past, s.lens)


def test_beams_share_a_prompt_diverge_and_are_scored():
    """Prompt, fork, diverging steps with permuted beams, scores of the chosen tokens, compaction: every beam stands
    where the oracle's forward over its tokens does."""
    s = Server(6, n_pages=40)
    g = np.random.default_rng(3)
    prompt = g.integers(0, 1000, (1, 37))
    s.prefill(0, prompt)
    seqs = [list(prompt[0]) for _ in range(4)]
    G.gpt2_pages_fork(s.cache, _i32([0, 0, 0]), _i32([1, 2, 3]), 3)
    lp, ent, ids = (torch.zeros(6, device="cuda"), torch.zeros(6, device="cuda"),
                    torch.zeros((6, 4), dtype=torch.int32, device="cuda"))
    lps = torch.zeros((6, 4), device="cuda")
    for turn in range(14):
        tok = g.integers(0, 1000, 6)
        for b in range(4):
            seqs[b].append(int(tok[b]))
        s.step(_i32(tok.tolist()))
        nxt = g.integers(0, 1000, 6)
        G.gpt2_token_logprobs(s.logits, 1000, G.F32, 4, 1000, _i32(nxt.tolist()), lp, ent, None, 4, ids, lps)
        got = s.got()[:4]
        z = torch.log_softmax(torch.from_numpy(got), 1)
        assert (lp[:4].cpu() - z[torch.arange(4), torch.from_numpy(nxt[:4])]).abs().max() < 2e-5
        assert (ent[:4].cpu() + (z.exp() * z).sum(1)).abs().max() < 2e-5
        order = torch.sort(torch.from_numpy(got), dim=1, descending=True, stable=True)[1][:, :4]
        assert torch.equal(ids[:4].long().cpu(), order)
        for b in range(4):
            assert _rel(got[b], _ref_last(s, seqs[b])) < 1e-2, (turn, b)
        if turn % 4 == 1:
            perm = [int(x) for x in g.integers(0, 4, 4)]
            G.gpt2_pages_fork(s.cache, _i32(perm), _i32([0, 1, 2, 3]), 4)
            seqs = [list(seqs[p]) for p in perm]
        if turn == 9:
            n = _i32([0])
            G.gpt2_pages_compact(s.cache, n, s.ws, s.ws.numel())
            used = int((s.refs > 0).sum())
            assert int(n) == used and bool((s.refs[:used] > 0).all())
    G.gpt2_pages_free(s.cache, _i32([0, 1, 2, 3]), 4)
    torch.cuda.synchronize()
    assert int(s.refs.abs().sum()) == 0 and s.lens.cpu().tolist() == [-1] * 6


def test_sliding_window_with_pages_given_back():
    """Decode under a window and sinks while pages behind the window are freed: the same logits as with every page
    kept, bit for bit; and a window as long as the sequence changes nothing."""
    g = np.random.default_rng(4)
    prompt = g.integers(0, 1000, (2, 30))
    toks = [_i32(g.integers(0, 1000, 2).tolist()) for _ in range(60)]
    outs = []
    for trim in (False, True):
        s = Server(2)
        s.prefill(0, prompt)
        rows = []
        for t in toks:
            s.step(t, window=24, sinks=3)
            if trim:
                G.gpt2_pages_free(s.cache, _i32([0, 1]), 2, 3, 23)
            rows.append(s.got())
        outs.append(rows)
        if trim:
            assert int((s.table[0] >= 0).sum()) <= 4  # the sinks' page and the window's
    assert all(np.array_equal(x, y) for x, y in zip(*outs))
    s, w = Server(2), Server(2)
    s.prefill(0, prompt)
    w.prefill(0, prompt)
    for t in toks[:20]:
        s.step(t)
        w.step(t, window=100, sinks=0)
        assert np.array_equal(s.got(), w.got())


def test_step_captured_with_its_reservation():
    """Reserve and decode in one graph, replayed across page borders, equals the eager loop."""
    g = np.random.default_rng(5)
    prompt = g.integers(0, 1000, (3, 14))
    a, b = Server(3), Server(3)
    for s in (a, b):
        s.prefill(0, prompt)
    ones, stream = _i32([1] * 3), torch.cuda.Stream()
    tok = b.next.clone()
    eager = []
    for _ in range(8):
        a.step(a.next)
        eager.append(a.got())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        G.gpt2_pages_reserve(b.cache, ones, b.ws, b.ws.numel())
        b.step(b.next, reserve=False)
    del tok
    for ref in eager:
        graph.replay()
        assert np.array_equal(b.got(), ref)
    assert torch.equal(a.lens, b.lens) and torch.equal(a.next, b.next)


def test_repeated_calls_replay_and_see_the_new_state():
    """On a stream of its own the third call and later replay the library's launch graph."""
    g = np.random.default_rng(6)
    prompt = g.integers(0, 1000, (2, 10))
    a, b = Server(2), Server(2)
    for s in (a, b):
        s.prefill(0, prompt)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for _ in range(6):
        a.step(a.next)
        ref = a.got()
        b.reserve([1, 1])
        torch.cuda.synchronize()
        b.step(b.next, reserve=False, stream=stream)
        assert np.array_equal(b.got(), ref)


def test_faults_are_reported():
    s = Server(3)
    g = np.random.default_rng(7)
    s.prefill(0, g.integers(0, 1000, (2, 10)))
    torch.cuda.synchronize()
    # a prompt into a sequence that already holds positions
    before, held = s.lens.clone(), s.pages.clone()
    G.gpt2_prefill_paged(s.cd, s.mw, G.paged_cache(s.pages, s.refs, s.table[:1], s.lens[:1]), _i32([[1, 2, 3]]), 3,
                         s.next[:1], None, 0, s.ws, s.ws.numel())
    assert G.gpt2_last_error()[0] == RANGE and torch.equal(s.lens, before)
    assert torch.equal(s.pages.view(torch.int16), held.view(torch.int16))
    # a token out of range leaves its sequence alone
    nxt = s.next.clone()
    s.step(_i32([5, 1000, 0]))
    torch.cuda.synchronize()
    assert G.gpt2_last_error()[0] == RANGE
    assert s.lens.cpu().tolist() == [11, 10, -1] and int(s.next[1]) == int(nxt[1])
    # the end of the positions
    s.lens[0] = 128
    s.step(_i32([5, 6, 0]), reserve=False)
    assert G.gpt2_last_error()[0] == RANGE
    assert s.lens.cpu().tolist() == [128, 11, -1]


def test_more_rows_than_the_few_row_gemm_takes():
    """130 slots, three of them in use: the tiled GEMMs and the argmax over stored logits."""
    s = Server(130, n_pages=40, max_pages=4)
    g = np.random.default_rng(8)
    first, last = g.integers(0, 1000, (1, 18)), g.integers(0, 1000, (2, 31))
    s.prefill(7, first)
    s.prefill(128, last)
    seqs = {7: list(first[0]), 128: list(last[0]), 129: list(last[1])}
    for _ in range(3):
        tok = s.next.clone()
        for k in seqs:
            seqs[k].append(int(tok[k]))
        s.step(tok)
        got = s.got()
        for k, t in seqs.items():
            assert _rel(got[k], _ref_last(s, t)) < 1e-2
            assert int(s.next[k]) == int(np.argmax(got[k]))
    assert int((s.lens >= 0).sum()) == 3 and int(s.next[0]) == -1


def test_a_pool_that_runs_short_leaves_its_sequences():
    """A sequence without a page for its next position takes no step, the others do; once there is a page it takes
    the step with the result it would have had."""
    s, full = Server(3, n_pages=5), Server(3)
    g = np.random.default_rng(9)
    a, b, c = g.integers(0, 1000, (1, 32)), g.integers(0, 1000, (1, 20)), g.integers(0, 1000, (1, 5))
    for x in (s, full):
        x.prefill(0, a)
        x.prefill(1, b)
        x.prefill(2, c)
    G.gpt2_pages_free(s.cache, _i32([2]), 1)
    G.gpt2_pages_fork(s.cache, _i32([1]), _i32([2]), 1)  # shares b's pages: sequence 2 may not write either
    torch.cuda.synchronize()
    assert G.gpt2_last_error()[0] == 0
    assert int((s.refs == 0).sum()) == 1
    s.reserve([1, 1, 1])  # two entries want another page, one is free
    assert G.gpt2_last_error()[0] == RANGE
    tok = _i32([3, 4, 4])
    before = s.next.clone()
    s.step(tok, reserve=False)
    torch.cuda.synchronize()
    assert G.gpt2_last_error()[0] == RANGE
    assert s.lens.cpu().tolist() == [32, 20, 20] and torch.equal(s.next, before)
    G.gpt2_pages_free(s.cache, _i32([2]), 1)
    s.reserve([0, 1, 0])
    s.step(tok, reserve=False)  # sequence 0 still has none, sequence 1 steps
    assert G.gpt2_last_error()[0] == RANGE
    assert s.lens.cpu().tolist() == [32, 21, -1] and int(s.next[0]) == int(before[0])
    s.step(tok)
    torch.cuda.synchronize()
    assert G.gpt2_last_error()[0] == 0 and s.lens.cpu().tolist() == [33, 22, -1]
    full.step(tok)
    got, ref = s.got()[0], full.got()[0]
    assert np.array_equal(got, ref) and int(s.next[0]) == int(full.next[0])
    assert _rel(got, _ref_last(s, list(a[0]) + [3])) < 1e-2


def test_a_prompt_without_its_pages_is_not_taken():
    s = Server(2, n_pages=3)
    g = np.random.default_rng(10)
    prompt = g.integers(0, 1000, (2, 20))
    s.prefill(0, prompt)  # four pages wanted
    assert G.gpt2_last_error()[0] == RANGE
    assert s.lens.cpu().tolist() == [0, 0] and s.next.cpu().tolist() == [-1, -1] and int(s.refs.sum()) == 0
    s.reserve([20, 0])
    G.gpt2_prefill_paged(s.cd, s.mw, s.cache, _i32(prompt.tolist()), 20, s.next, s.logits, 1000, s.ws, s.ws.numel())
    assert G.gpt2_last_error()[0] == RANGE
    assert s.lens.cpu().tolist() == [20, 0] and int(s.next[1]) == -1
    assert _rel(s.got()[0], _ref_last(s, list(prompt[0]))) < 1e-2
