"""gpt2_attention_paged_draft on the GPU against float64, element by element.

Bounds as for one new token: half a step of the 16-bit result, eps / 2 |ref| +
(smallest normal) eps, plus what the sums may be off.  A score is a dot product
of 64 exact products accumulated in fp32 in four groups, each off by at most 17
2^-23 of the sum of magnitudes: |dz| <= 2^-16 A, A = scale sum |q k| (its
largest over the places seen).  A probability is off by a factor within 2 |dz| +
2^-21, its two 16-bit parts carry it to 2^-16 (bf16; fp16 more), the fp32 sums
over positions add less than 2^-16.  So |out - ref| <= eps / 2 |ref| + (2^-15 A +
2^-14) sum p |v|, and the log-sum-exp (log2 units) is off by at most log2(e) 2^-16
A + 2^-14 + 2^-22 |lse|.

Whatever must not be read or must not count holds NaN."""
import math

import numpy as np
import pytest

import paged_ref as R

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
RANGE = 6


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gpt_pre_ln_gb300 import build
    build.build()
    G.lib()
    yield
    st, site = G.gpt2_last_error()
    assert st == 0, f"device error {st} at site {site}"


def tree(g, n, kind="tree"):
    """Parents of n tokens: random, a chain, all after the first, or several that follow the cached positions."""
    if kind == "chain":
        return [t - 1 for t in range(n)]
    if kind == "star":
        return [-1 if t == 0 else 0 for t in range(n)]
    if kind == "roots":
        return [-1 if t == 0 or g.random() < 0.3 else int(g.integers(0, t)) for t in range(n)]
    return [-1 if t == 0 else t - 1 if g.random() < 0.4 else int(g.integers(0, t)) for t in range(n)]


def path_to(parents, t):
    return (path_to(parents, parents[t]) if parents[t] >= 0 else []) + [t]


def places(n, path, window, sinks):
    """The places (cached positions, n + token) that the token at the path's end sees."""
    end = n + len(path)
    ok = lambda p: window == 0 or p >= end - window or p < sinks  # noqa: E731
    return [p for p in range(n) if ok(p)] + [n + t for d, t in enumerate(path) if ok(n + d)]


class Case:
    def __init__(self, lens, T, heads=2, kv=2, page=16, window=0, sinks=0, kind="tree", counts=None, stored=False,
                 dtype="bf16", scale=0.125, layers=2, layer=1, seed=0, pad=0, grow=0.0, max_pages=None, extra=0):
        g = np.random.default_rng(seed)
        self.lens_l, self.T, self.heads, self.kv, self.page, self.window, self.sinks = lens, T, heads, kv, page, window, sinks
        self.scale, self.layer, self.dtype, self.stored = scale, layer, dtype, stored
        tdt, n_seq = DT[dtype], len(lens)
        self.counts_l = counts or [T] * n_seq
        self.tree = [tree(g, max(0, min(c, T)), kind) for c in self.counts_l]
        live = [(b, n, len(self.tree[b])) for b, n in enumerate(lens) if n >= 0 and self.tree[b]]
        cols = (max_pages or max([1] + [-(-(n + c) // page) for _, n, c in live])) + extra
        want = set()
        self.seen = {}
        for b, n, c in live:
            for t in range(c):
                self.seen[b, t] = places(n, path_to(self.tree[b], t), window, sinks)
                want |= {(b, p // page) for p in self.seen[b, t]} | {(b, (n + t) // page)}
        want = sorted(want)
        self.n_pages = len(want) + 5
        table = np.full((n_seq, cols), -1, np.int64)
        for (b, c), p in zip(want, g.permutation(self.n_pages)):
            table[b, c] = p
        r16 = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).to(tdt)  # noqa: E731
        self.q = r16(n_seq, T, heads, 64)
        self.kn, self.vn = r16(n_seq, T, kv, 64), r16(n_seq, T, kv, 64)
        pages = torch.full((self.n_pages, layers, 2, kv, page, 64), float("nan"), dtype=tdt)
        self.kc, self.vc = {}, {}
        for b, n, c in live:
            used = sorted({p for t in range(c) for p in self.seen[b, t] if p < n})
            self.kc[b], self.vc[b] = r16(n, kv, 64), r16(n, kv, 64)
            self.kc[b] = (self.kc[b].float() * (1 + grow * torch.arange(n))[:, None, None]).to(tdt)
            for p in used:
                pages[table[b, p // page], layer, 0, :, p % page] = self.kc[b][p]
                pages[table[b, p // page], layer, 1, :, p % page] = self.vc[b][p]
            if stored:
                for t in range(c):
                    pages[table[b, (n + t) // page], layer, 0, :, (n + t) % page] = self.kn[b, t]
                    pages[table[b, (n + t) // page], layer, 1, :, (n + t) % page] = self.vn[b, t]
        self.live, self.table_np = live, table
        self.pages = pages.cuda()
        self.before = self.pages.clone()
        self.table = torch.from_numpy(table.astype(np.int32)).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.refs = torch.ones(self.n_pages, dtype=torch.int32, device="cuda")
        self.parents = torch.tensor([p + [99] * (T - len(p)) for p in self.tree], dtype=torch.int32).reshape(n_seq, T).cuda()
        self.counts = torch.tensor(self.counts_l, dtype=torch.int32).cuda()
        self.ld = (heads + 2 * kv) * 64 + pad
        row = torch.full((n_seq * T, self.ld), float("nan"), dtype=tdt)
        row[:, :heads * 64] = self.q.reshape(n_seq * T, -1)
        row[:, heads * 64:(heads + kv) * 64] = self.kn.reshape(n_seq * T, -1)
        row[:, (heads + kv) * 64:(heads + 2 * kv) * 64] = self.vn.reshape(n_seq * T, -1)
        for b in range(n_seq):  # rows that must not be looked at
            used = len(self.tree[b]) if lens[b] >= 0 else 0
            row[b * T + used:(b + 1) * T] = float("nan")
        self.qkv = row.cuda()
        self.ldo = heads * 64 + pad
        self.out = torch.full((n_seq * T, self.ldo), 7.0, dtype=tdt, device="cuda")
        self.lse = torch.full((n_seq * T, heads), 7.0, device="cuda")
        self.cache = G.paged_cache(self.pages, self.refs, self.table, self.lens)
        self.need = G.gpt2_attention_paged_draft_workspace_bytes(self.cache, T, heads)
        self.ws = torch.full((self.need,), 255, dtype=torch.uint8, device="cuda")

    def run(self, lse=True, parents=True, counts=True, stream=None, ws=None):
        at, w = self.qkv.data_ptr(), self.heads * 128
        k, v = (None, None) if self.stored else (at + w, at + w + self.kv * 128)
        G.gpt2_attention_paged_draft(self.cache, self.layer, at, self.ld, k, v, self.ld, self.out, self.ldo,
                                     self.lse if lse else None, self.T, self.parents if parents else None,
                                     self.counts if counts else None, self.heads, self.scale, self.window, self.sinks,
                                     self.ws if ws is None else ws, self.need, stream)
        return self

    def expect(self, b, t, head, only=None):
        g, n = head // (self.heads // self.kv), self.lens_l[b]
        seen = [p for p in self.seen[b, t] if only is None or only(p)]
        pick = lambda c, d: np.stack([(c[b][p, g] if p < n else d[b, p - n, g]).double().numpy() for p in seen]) if seen else np.zeros((0, 64))  # noqa: E731,E501
        return R.attention(self.q[b, t, head].double().numpy(), pick(self.kc, self.kn), pick(self.vc, self.vn), self.scale)

    def check(self, stored=True, only=None, seqs=None):
        torch.cuda.synchronize()
        out, lse = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        info, T = torch.finfo(DT[self.dtype]), self.T
        rows = {(b, t) for b, _, c in self.live for t in range(c) if seqs is None or b in seqs}
        for b in range(len(self.lens_l)):
            for t in range(T):
                m = b * T + t
                assert (out[m, self.heads * 64:] == 7.0).all()
                if (b, t) not in rows:
                    assert (out[m] == 7.0).all() and (lse[m] == 7.0).all(), (b, t)
                    continue
                for h in range(self.heads):
                    ref, rl, mag, A = self.expect(b, t, h, only)
                    got = out[m, h * 64:h * 64 + 64]
                    bound = info.eps / 2 * np.abs(ref) + info.tiny * info.eps + (2 ** -15 * A + 2 ** -14) * mag
                    assert (np.abs(got - ref) <= bound).all(), (b, t, h, np.abs(got - ref).max())
                    if math.isinf(rl):
                        assert lse[m, h] == rl
                    else:
                        assert abs(lse[m, h] - rl) <= math.log2(math.e) * 2 ** -16 * A + 2 ** -14 + 2 ** -22 * abs(rl)
        want = self.before.clone()
        if stored and not self.stored:
            for b, n, c in self.live:
                for t in range(c):
                    p = self.table_np[b, (n + t) // self.page]
                    if p >= 0 and (seqs is None or b in seqs):
                        want[p, self.layer, 0, :, (n + t) % self.page] = self.kn[b, t].cuda()
                        want[p, self.layer, 1, :, (n + t) % self.page] = self.vn[b, t].cuda()
        assert torch.equal(self.pages.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 33, 48, 49, 64])
def test_drafts(T, dtype):
    Case([70, 0, -1, 16, 15, 131], T, dtype=dtype, seed=T).run().check()


@pytest.mark.parametrize("heads, kv", [(1, 1), (3, 3), (8, 1), (16, 1), (12, 4), (25, 1), (20, 5), (40, 2)])
@pytest.mark.parametrize("T", [1, 3, 11])
def test_grouped_heads(heads, kv, T):
    Case([40, 3, 97], T, heads=heads, kv=kv, seed=heads + T, dtype="f16").run().check()


@pytest.mark.parametrize("kind", ["chain", "star", "roots", "tree"])
@pytest.mark.parametrize("T", [5, 64])
def test_trees(kind, T):
    Case([33, 200], T, kind=kind, seed=T).run().check()


def test_a_chain_without_parents():
    Case([20, 0, 47], 12, kind="chain").run(parents=False).check()


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("pad", [0, 8])
def test_pages_and_strides(page, pad):
    Case([page - 1, page, 3 * page - 2, 1], 20, page=page, pad=pad, layers=3, layer=page % 3, seed=page).run().check()


@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 3), (2, 0), (5, 2), (16, 4), (17, 0), (40, 33), (64, 1), (300, 4)])
@pytest.mark.parametrize("T, kind", [(4, "chain"), (24, "tree"), (64, "chain")])
def test_windows(window, sinks, T, kind):
    Case([100, 0, 3, 39, 261], T, window=window, sinks=sinks, kind=kind, seed=window + T, page=32).run().check()


@pytest.mark.parametrize("stored", [False, True])
def test_ragged_counts(stored):
    """Counts of 0 and below, and above T (T of them); rows behind them are left as they were."""
    Case([50, 9, 31, -1, 64, 16], 19, counts=[19, 0, 1, 7, 25, 18], stored=stored, seed=5).run().check()
    Case([50, 9], 6, counts=[-3, 6], stored=stored, seed=6).run().check()


def test_without_counts_and_lse():
    c = Case([50, 9], 6, seed=6).run(lse=False, counts=False)
    c.lse.copy_(Case([50, 9], 6, seed=6).run().lse)
    c.check()


@pytest.mark.parametrize("n_seq", [129, 300])
def test_many_sequences(n_seq):
    g = np.random.default_rng(n_seq)
    lens = [int(x) for x in g.integers(-1, 40, n_seq)]
    counts = [int(x) for x in g.integers(0, 5, n_seq)]
    Case(lens, 4, heads=1, kv=1, counts=counts, seed=n_seq).run().check()


@pytest.mark.parametrize("T, heads, kv", [(8, 1, 1), (16, 1, 1), (30, 1, 1), (64, 1, 1), (40, 4, 1)])
def test_long_caches_are_split_and_joined(T, heads, kv):
    Case([9001, 5, 2500], T, heads=heads, kv=kv, page=256, layers=1, layer=0, seed=T).run().check()


@pytest.mark.parametrize("T, group", [(7, 1), (12, 1), (24, 1), (60, 1), (20, 3)])
@pytest.mark.parametrize("window, sinks", [(0, 0), (500, 20)])
def test_more_work_than_runs_of_eight_tiles(T, group, window, sinks):
    # the CTAs' parts are longer than the shortest there are, and run over the items' ends
    g = np.random.default_rng(T)
    lens = [int(x) for x in g.integers(0, 1500, 28)]
    lens[3], lens[11], lens[12] = -1, 0, 15
    counts = [int(x) for x in g.integers(0, 7, 28)]
    counts[5] = T
    Case(lens, T, heads=7 * group, kv=7, page=64, counts=counts, window=window, sinks=sinks, layers=1, layer=0,
         seed=T).run().check()


def test_growing_scores_rescale():
    Case([300, 77], 40, grow=0.05, seed=3).run().check()
    Case([300, 77], 5, grow=0.05, seed=3, dtype="f16").run().check()


@pytest.mark.parametrize("T, group", [(6, 1), (12, 1), (30, 1), (60, 1), (20, 3)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_stay_with_those_who_see_them(T, group, what):
    """A token with such a K, another with such a V: the tokens that do not follow it are as without it."""
    c = Case([37, 20], T, heads=group, kv=1, kind="star", window=0, seed=T)
    bad_k, bad_v = 2, 4  # leaves of the star: nobody follows them
    row = c.qkv.view(2, T, -1)
    row[:, bad_k, group * 64 + 5] = what
    row[:, bad_v, (group + 1) * 64 + 9] = what
    row[:, bad_v, (group + 1) * 64 + 50] = what
    c.run()
    torch.cuda.synchronize()
    out = c.out.view(2, T, -1)
    for b in range(2):
        for h in range(group):
            at = out[b, bad_v, h * 64:h * 64 + 64].float().cpu()
            assert not torch.isfinite(at[[9, 50]]).any() and torch.isfinite(at[:9]).all()
            assert torch.isnan(at[9]) if math.isnan(what) else at[9] == what
        for t in (bad_k, bad_v):  # looked at above, or with a score that is not finite
            out[b, t] = 7.0
            c.lse[b * T + t] = 7.0
    keep = {(b, t): s for (b, t), s in c.seen.items() if t not in (bad_k, bad_v)}
    for (b, t), seen in keep.items():
        for h in range(group):
            ref, rl, mag, A = c.expect(b, t, h)
            got = out[b, t, h * 64:h * 64 + 64].double().cpu().numpy()
            assert (np.abs(got - ref) <= torch.finfo(DT["bf16"]).eps / 2 * np.abs(ref) + 1e-40
                    + (2 ** -15 * A + 2 ** -14) * mag).all(), (b, t, h)


def test_values_that_are_not_finite_behind_the_window():
    """A cached V that only the shallow tokens still see."""
    c = Case([40], 6, heads=1, kv=1, window=8, kind="chain", seed=1)
    p = 40 + 1 - 8  # seen by the first token alone
    c.pages[c.table_np[0, p // 16], 1, 1, :, p % 16, 3] = float("inf")
    c.before = c.pages.clone()
    c.run()
    torch.cuda.synchronize()
    assert c.out[0, 3] == float("inf")
    c.vc[0][p, :, 3] = 0  # what the others do not see does not matter
    c.out[0] = 7.0
    c.lse[0] = 7.0
    for t in range(1, 6):
        ref, rl, mag, A = c.expect(0, t, 0)
        got = c.out[t].double().cpu().numpy()
        assert (np.abs(got - ref) <= 2 ** -8 * np.abs(ref) + 1e-40 + (2 ** -15 * A + 2 ** -14) * mag).all()


def test_scores_of_minus_infinity():
    c = Case([0], 3, heads=1, kv=1, kind="star", scale=1.0, seed=2)
    c.qkv[:, :64] = 1.0
    c.qkv[:, 64:128] = -float("inf")
    c.run()
    torch.cuda.synchronize()
    assert (c.out == 0).all() and (c.lse == -float("inf")).all()


def test_missing_page():
    """Places on a page that the table does not name are left out."""
    for T, gone in ((5, 1), (40, 5), (40, 6)):
        c = Case([70], T, seed=T)
        p = int(c.table_np[0, gone])
        c.table[0, gone] = -1
        c.before[p] = c.pages[p]
        c.table_np[0, gone] = -1
        c.run()
        c.check(only=lambda x: x // 16 != gone)
        assert G.gpt2_last_error() == (RANGE, 21)


def test_entry_beyond_the_pool():
    c = Case([70], 5, seed=1)
    c.table[0, 2] = c.n_pages
    c.run()
    c.check(only=lambda x: x // 16 != 2)
    assert G.gpt2_last_error() == (RANGE, 21)


def test_shared_page():
    """A page that others read too: the tokens are attended over but not stored there."""
    c = Case([20], 20, seed=4)  # places 20 .. 39 on pages 1 and 2
    c.refs[int(c.table_np[0, 1])] = 2
    p2 = int(c.table_np[0, 2])
    c.run()
    for t in range(20):
        if 20 + t >= 32:
            for i, src in enumerate((c.kn, c.vn)):
                c.before[p2, 1, i, :, (20 + t) % 16] = src[0, t].cuda()
    c.check(stored=False)
    assert G.gpt2_last_error() == (RANGE, 28)


def test_parents_out_of_range():
    """They count as -1."""
    for bad in (7, 12, -2, 2 ** 31 - 1, -2 ** 31):
        c = Case([20], 9, kind="tree", seed=4)
        c.parents[0, 7] = bad
        c.tree[0][7] = -1
        for t in range(9):
            c.seen[0, t] = places(20, path_to(c.tree[0], t), 0, 0)
        c.run().check()
        assert G.gpt2_last_error() == (RANGE, 29)


@pytest.mark.parametrize("length", [100, 10 ** 9, 2 ** 31 - 20, 2 ** 31 - 1])
def test_sequence_longer_than_its_table_row(length):
    c = Case([30, 20], 8, seed=4, max_pages=3)
    c.lens[0] = length
    c.run().check(seqs=[1])
    assert G.gpt2_last_error() == (RANGE, 20)


def test_results_do_not_depend_on_timing_or_stream():
    a = Case([500, 77, 0, 1024], 24, heads=3, kv=3, seed=9).run()
    s = torch.cuda.Stream()
    b = Case([500, 77, 0, 1024], 24, heads=3, kv=3, seed=9)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        b.run()
        b.run(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse) and torch.equal(a.pages.view(torch.int16), b.pages.view(torch.int16))


def test_captured_and_replayed_at_other_lengths():
    c = Case([100, 70], 10, seed=8)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        c.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.run()
    d = Case([61, 97], 10, seed=18, max_pages=c.table.shape[1])
    torch.cuda.synchronize()
    c.pages[:d.n_pages].copy_(d.pages[:c.n_pages])
    assert c.n_pages >= d.n_pages
    for x in ("lens", "parents", "qkv"):
        getattr(c, x).copy_(getattr(d, x))
    c.table.copy_(d.table)
    c.out.fill_(7.0)
    with torch.cuda.stream(s):
        graph.replay()
    torch.cuda.synchronize()
    d.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, d.out) and torch.equal(c.lse, d.lse)


def test_two_calls_at_once():
    """Two streams, two caches, a workspace each."""
    xs = [Case([700, 300], 16, heads=4, kv=4, seed=20 + i) for i in range(2)]
    ss = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, s in zip(xs, ss):
            x.run(stream=s)
    for x in xs:
        x.check()


def test_one_token_agrees_with_gpt2_attention_paged():
    """T = 1 is gpt2_attention_paged: the same within two of its steps (the sums run in another order)."""
    c = Case([700, 31, 0], 1, heads=12, kv=12, seed=2).run()
    other = Case([700, 31, 0], 1, heads=12, kv=12, seed=2)
    need = G.gpt2_attention_paged_workspace_bytes(other.cache, 12)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    at = other.qkv.data_ptr()
    G.gpt2_attention_paged(other.cache, 1, at, other.ld, at + 12 * 128, at + 24 * 128, other.ld, other.out, other.ldo,
                           other.lse, 12, 0.125, 0, 0, ws, need)
    torch.cuda.synchronize()
    assert torch.equal(c.pages.view(torch.int16), other.pages.view(torch.int16))
    x, y = c.out.double(), other.out.double()
    assert ((x - y).abs() <= 2 * 2.0 ** -8 * y.abs() + 1e-4).all()


def test_a_cache_of_later_slots():
    """A struct whose table and lens point at a later slot is a cache of those slots alone."""
    c = Case([40, 50, 60], 6, seed=12)
    view = G.paged_cache(c.pages, c.refs, c.table[1:], c.lens[1:])
    at, w = c.qkv[6:].data_ptr(), c.heads * 128
    G.gpt2_attention_paged_draft(view, 1, at, c.ld, at + w, at + w + c.kv * 128, c.ld, c.out[6:], c.ldo, c.lse[6:], 6,
                                 c.parents[1:], c.counts[1:], c.heads, c.scale, 0, 0, c.ws, c.need)
    c.check(seqs=[1, 2])
