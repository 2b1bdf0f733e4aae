"""Steps of speculative decoding with a model, as they are run together on the
GPU: pages reserved, trees of drafted tokens through gpt2_draft_step_paged, a
choice per token by gpt2_sample_tokens, the confirmed path kept by
gpt2_draft_accept, and on with the next tree or a plain decode step.

Gates: logits against the float64 oracle over each token's own path within the
relative L2 of 1e-2 that the other model tests use (a wrong page, position or
ancestor is an error of order 1)."""
import numpy as np
import pytest

from test_gpu_draft_attention import path_to, tree
from test_gpu_paged_model import Server, _i32, _ref_last, _rel

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


class Drafts:
    """A server's buffers for steps of T drafted tokens."""

    def __init__(self, s, T, logits_t=G.F32):
        self.s, self.T, self.t = s, T, logits_t
        tdt = {G.F32: torch.float32, G.BF16: torch.bfloat16, G.F16: torch.float16}[logits_t]
        self.logits = torch.zeros(s.n * T, 1000, dtype=tdt, device="cuda")
        self.need = G.gpt2_draft_step_paged_workspace_bytes(s.cd, s.cache, T)
        self.ws = torch.full((self.need,), 255, dtype=torch.uint8, device="cuda")
        i = lambda *z: torch.zeros(z, dtype=torch.int32, device="cuda")  # noqa: E731
        self.tokens, self.parents, self.counts = i(s.n, T), i(s.n, T), i(s.n)
        self.chosen, self.path, self.kept = i(s.n, T), i(s.n, T), i(s.n)
        self.u = torch.full((s.n * T,), 0.5, device="cuda")
        self.zero = torch.zeros(s.n * T, device="cuda")

    def put(self, tokens, parents, counts):
        for x, v in ((self.tokens, tokens), (self.parents, parents), (self.counts, counts)):
            x.copy_(_i32(v))

    def step(self, window=0, sinks=0, temperature=None):
        s = self.s
        G.gpt2_pages_reserve(s.cache, self.counts, s.ws, s.ws.numel())
        G.gpt2_draft_step_paged(s.cd, s.mw, s.cache, self.T, self.tokens, self.parents, self.counts, window, sinks,
                                self.logits, 1000, self.t, self.ws, self.need)
        G.gpt2_sample_tokens(self.logits, 1000, self.t, s.n * self.T, 1000,
                             self.zero if temperature is None else temperature, None, None, None, self.u, self.chosen)

    def accept(self):
        s = self.s
        G.gpt2_draft_accept(s.cache, self.T, self.tokens, self.parents, self.counts, self.chosen, self.path, self.kept,
                            s.next)


def _drafts(s, seqs, T, counts, g):
    """Trees whose tokens are partly what the model will choose (by the oracle), so that paths of several stay."""
    tokens, parents = np.zeros((s.n, T), int), np.full((s.n, T), -1)
    for b in range(s.n):
        parents[b, :counts[b]] = tree(g, counts[b])
        tokens[b] = g.integers(0, 1000, T)
    for b, have in seqs.items():
        if counts[b] <= 0:
            continue
        tokens[b, 0] = have[-1]
        for t in range(1, counts[b]):
            up = path_to(parents[b].tolist(), int(parents[b, t]))
            if g.random() < 0.75:
                tokens[b, t] = int(np.argmax(_ref_last(s, have[:-1] + [int(tokens[b, u]) for u in up])))
    return tokens, parents


@pytest.mark.parametrize("dtype, T, logits_t", [(G.BF16, 7, G.F32), (G.F16, 12, G.F16), (G.BF16, 40, G.BF16)])
def test_steps_follow_the_oracle(dtype, T, logits_t):
    s = Server(4, dtype=dtype)
    g = np.random.default_rng(T)
    a, b = g.integers(0, 1000, (2, 17)), g.integers(0, 1000, (1, 30))
    s.prefill(0, a)
    s.prefill(3, b)  # slot 2 stays empty
    seqs = {0: list(a[0]), 1: list(a[1]), 3: list(b[0])}
    for k in seqs:
        seqs[k].append(int(s.next[k]))  # chosen, not in the cache yet
    d = Drafts(s, T, logits_t)
    kept = 0
    for _ in range(3):
        counts = [T, max(1, T // 2), 3, T - 1]
        tokens, parents = _drafts(s, seqs, T, counts, g)
        d.put(tokens.tolist(), parents.tolist(), counts)
        d.step()
        torch.cuda.synchronize()
        got = d.logits.double().cpu().numpy().reshape(4, T, 1000)
        for k, have in seqs.items():
            for t in range(counts[k]):
                path = path_to(parents[k].tolist(), t)
                ref = _ref_last(s, have[:-1] + [int(tokens[k, u]) for u in path])
                assert _rel(got[k, t], ref) < 1e-2, (k, t)
                assert int(d.chosen[k, t]) == int(np.argmax(got[k, t]))
        before = s.lens.tolist()
        d.accept()
        torch.cuda.synchronize()
        for k, have in seqs.items():
            n = int(d.kept[k])
            path = d.path[k, :n].tolist()
            assert path[0] == 0 and s.lens.tolist()[k] == before[k] + n
            for x, y in zip(path, path[1:]):
                assert int(d.chosen[k, x]) == int(tokens[k, y])
            have += [int(d.chosen[k, t]) for t in path]
            assert have[-1] == int(s.next[k])
            kept += n - 1
        assert s.lens.tolist()[2] == -1
    assert kept >= 6  # the moves had something to do
    # what is in the cache now is what a plain decode step needs
    for _ in range(2):
        s.step(s.next.clone())
        got = s.got()
        for k, have in seqs.items():
            assert _rel(got[k], _ref_last(s, have)) < 1e-2
            have.append(int(s.next[k]))


@pytest.mark.parametrize("window, sinks", [(0, 0), (10, 0), (24, 3), (3, 2)])
def test_one_drafted_token_is_a_decode_step(window, sinks):
    """The same logits as gpt2_decode_step_paged, up to its rounding."""
    x, y = Server(3), Server(3)
    g = np.random.default_rng(5)
    prompt = g.integers(0, 1000, (3, 45))
    for s in (x, y):
        s.prefill(0, prompt)
    d = Drafts(y, 1)
    for _ in range(4):
        tok = x.next.clone()
        x.step(tok, window, sinks)
        d.put(tok.tolist() if tok.dim() > 1 else [[int(t)] for t in tok], [[-1]] * 3, [1] * 3)
        d.step(window, sinks)
        d.accept()
        torch.cuda.synchronize()
        a, b = x.got(), d.logits.double().cpu().numpy()
        for k in range(3):
            assert _rel(b[k], a[k]) < 5e-3
        y.next.copy_(x.next)
        assert x.lens.tolist() == y.lens.tolist() and d.kept.tolist() == [1] * 3


def test_a_chain_under_a_window_is_decode_steps_in_one():
    x, y = Server(2), Server(2)
    g = np.random.default_rng(6)
    prompt, more = g.integers(0, 1000, (2, 30)), g.integers(0, 1000, (2, 9))
    for s in (x, y):
        s.prefill(0, prompt)
    d = Drafts(y, 9)
    d.put(more.tolist(), [list(range(-1, 8))] * 2, [9, 9])
    d.step(window=6, sinks=2)
    torch.cuda.synchronize()
    got = d.logits.double().cpu().numpy().reshape(2, 9, 1000)
    for t in range(9):
        x.step(_i32(more[:, t].tolist()), 6, 2)
        a = x.got()
        for k in range(2):
            assert _rel(got[k, t], a[k]) < 5e-3


def test_a_token_or_position_out_of_range():
    s = Server(2, max_pages=9)  # room for more places than the model has positions
    g = np.random.default_rng(7)
    prompt = g.integers(0, 1000, (2, 125))
    s.prefill(0, prompt)
    d = Drafts(s, 2)
    d.put([[5, 1000], [5, 6]], [[-1, 0]] * 2, [2, 2])
    d.step()
    torch.cuda.synchronize()
    assert G.gpt2_last_error() == (RANGE, 12)
    got = d.logits.double().cpu().numpy().reshape(2, 2, 1000)
    for k, t, path in ((0, 0, [5]), (1, 0, [5]), (1, 1, [5, 6])):
        assert _rel(got[k, t], _ref_last(s, list(prompt[k]) + path)) < 1e-2
    d = Drafts(s, 4)  # positions 125 .. 128 of 128
    d.put([[5, 6, 7, 8]] * 2, [[-1, 0, 1, 2], [-1, 0, 0, 0]], [4, 4])
    d.step()
    torch.cuda.synchronize()
    assert G.gpt2_last_error() == (RANGE, 11)
    got = d.logits.double().cpu().numpy().reshape(2, 4, 1000)
    assert _rel(got[0, 2], _ref_last(s, list(prompt[0]) + [5, 6, 7])) < 1e-2
    assert _rel(got[1, 3], _ref_last(s, list(prompt[1]) + [5, 8])) < 1e-2


def test_a_whole_step_captured_and_replayed():
    """Reserve, model, choice and acceptance as one graph, replayed with other trees; eager calls beside it."""
    x, y = Server(3), Server(3)
    g = np.random.default_rng(8)
    prompt = g.integers(0, 1000, (3, 20))
    stream = torch.cuda.Stream()
    for s in (x, y):
        s.prefill(0, prompt)
    dx, dy = Drafts(x, 6), Drafts(y, 6)
    torch.cuda.synchronize()

    def both(d):
        d.step()
        d.accept()

    graph = None
    for i in range(4):
        tokens = g.integers(0, 1000, (3, 6))
        tokens[:, 0] = x.next.cpu().numpy()
        args = (tokens.tolist(), [tree(g, 6) for _ in range(3)], [6, 4, 5])
        for d in (dx, dy):
            d.put(*args)
        torch.cuda.synchronize()
        both(dx)
        with torch.cuda.stream(stream):
            if graph is None:
                both(dy)  # sets the kernels' attributes
            else:
                graph.replay()
        torch.cuda.synchronize()
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            lens, table, refs = y.lens.clone(), y.table.clone(), y.refs.clone()
            with torch.cuda.graph(graph, stream=stream):
                both(dy)
            assert torch.equal(lens, y.lens) and torch.equal(table, y.table) and torch.equal(refs, y.refs)
        for p, q in ((x.lens, y.lens), (x.next, y.next), (dx.path, dy.path)):
            assert torch.equal(p, q), i
        for k, n in enumerate((6, 4, 5)):  # (rows behind them are not defined)
            assert torch.equal(dx.logits[6 * k:6 * k + n], dy.logits[6 * k:6 * k + n]), i


def test_the_pool_runs_short_and_the_step_is_taken_again():
    s = Server(2, n_pages=5)
    g = np.random.default_rng(9)
    prompt = g.integers(0, 1000, (2, 30))  # two pages each
    s.prefill(0, prompt)
    d = Drafts(s, 4)
    tokens = g.integers(0, 1000, (2, 4))
    d.put(tokens.tolist(), [[-1, 0, 1, 2]] * 2, [4, 4])
    d.step()  # places 30 .. 33: one page short
    torch.cuda.synchronize()
    assert G.gpt2_last_error()[0] == RANGE
    d.chosen.copy_(_i32(np.roll(tokens, -1, 1).tolist()))  # all four would stay
    d.accept()
    torch.cuda.synchronize()
    assert G.gpt2_last_error() == (RANGE, 21)
    assert s.lens.tolist() == [30, 30] and d.kept.tolist() == [0, 0]
    G.gpt2_pages_free(s.cache, _i32([1]), 1)
    d.step()
    torch.cuda.synchronize()
    got = d.logits.double().cpu().numpy().reshape(2, 4, 1000)
    assert _rel(got[0, 3], _ref_last(s, list(prompt[0]) + tokens[0].tolist())) < 1e-2
    d.accept()
    torch.cuda.synchronize()
    assert int(s.lens[0]) >= 31 and int(s.lens[1]) == -1


def test_drawn_tokens_of_every_node():
    """Temperature 1 over the nodes of a batch of trees: each token is where its number falls in its own row."""
    s = Server(2)
    g = np.random.default_rng(10)
    s.prefill(0, g.integers(0, 1000, (2, 25)))
    d = Drafts(s, 30)
    d.put(g.integers(0, 1000, (2, 30)).tolist(), [tree(g, 30) for _ in range(2)], [30, 30])
    d.u.copy_(torch.from_numpy(g.random(60, dtype=np.float32)))
    d.step(temperature=torch.ones(60, device="cuda"))
    torch.cuda.synchronize()
    z, u = d.logits.double().cpu().numpy(), d.u.double().cpu().numpy()
    for m in range(60):
        part = np.cumsum(np.exp(z[m] - z[m].max()))
        assert int(d.chosen.view(-1)[m]) == int(np.searchsorted(part, u[m] * part[-1], side="right"))
