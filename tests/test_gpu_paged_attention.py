"""gpt2_attention_paged on the GPU against float64, element by element.

Bound of an output element: half a step of the 16-bit result,
eps / 2 |ref| + eps_sub (the smallest normal times eps, for results near 0), plus what the sums
may be off.  A score is a dot product of 64 exact products accumulated in
fp32 in four groups, each off by at most 17 2^-23 of the sum of magnitudes:
|dz| <= 4 * 17 * 2^-23 A < 2^-16 A with A = scale sum |q k| (its largest over the
positions).  A probability is then off by a factor within 2 |dz| + 2^-21
(exponential), its two 16-bit parts carry it to 2^-16 (bf16; fp16 more), and
the fp32 sums over positions add less than 2^-16 for the lengths here.  So
|out - ref| <= eps/2 |ref| + (2^-15 A + 2^-14) sum p |v|.  The log-sum-exp (log2
units) is off by at most log2(e) |dz| + 2^-14 + 2^-22 |lse|.

Whatever must not be read or must not count holds NaN: pages nobody owns,
positions behind a sequence's end, positions in front of its window.
"""
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


class Case:
    def __init__(self, lens, heads=2, kv_heads=2, page=16, window=0, sinks=0, append=True, dtype="bf16", scale=0.125,
                 layers=2, layer=1, seed=0, grow=0.0, junk_entry=-1, drop_hidden=True, pad=0, max_pages=None):
        g = np.random.default_rng(seed)
        self.lens_l, self.heads, self.kv, self.page, self.window, self.sinks = lens, heads, kv_heads, page, window, sinks
        self.append, self.dtype, self.scale, self.layer = append, dtype, scale, layer
        n_seq = len(lens)
        totals = [(n + 1 if append else n) if n >= 0 else 0 for n in lens]
        cols = max_pages or max(1, max(-(-t // page) for t in totals))
        want = []
        for b, n in enumerate(totals):
            seen = set(p // page for p in R.visible(n, window, sinks)) if drop_hidden else set(range(-(-n // page)))
            want += [(b, c) for c in sorted(seen)]
        self.n_pages = len(want) + 5
        ids = g.permutation(self.n_pages)
        table = np.full((n_seq, cols), junk_entry, np.int64)
        for (b, c), p in zip(want, ids):
            table[b, c] = p
        tdt = DT[dtype]
        # values as the 16-bit type holds them
        q = torch.from_numpy(g.standard_normal((n_seq, heads, 64)).astype(np.float32)).to(tdt)
        self.k = [torch.from_numpy((g.standard_normal((t, kv_heads, 64)) *
                                    (1 + grow * np.arange(t)[:, None, None])).astype(np.float32)).to(tdt)
                  for t in totals]
        self.v = [torch.from_numpy(g.standard_normal((t, kv_heads, 64)).astype(np.float32)).to(tdt) for t in totals]
        self.q = q
        pages = torch.full((self.n_pages, layers, 2, kv_heads, page, 64), float("nan"), dtype=tdt)
        for b, n in enumerate(totals):
            for p in R.visible(n, window, sinks):
                if append and p == n - 1:
                    continue
                pages[table[b, p // page], layer, 0, :, p % page] = self.k[b][p]
                pages[table[b, p // page], layer, 1, :, p % page] = self.v[b][p]
        self.totals, self.table_np = totals, table
        self.pages = pages.cuda()
        self.table = torch.from_numpy(table.astype(np.int32)).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.refs = torch.ones(self.n_pages, dtype=torch.int32, device="cuda")
        # one row per sequence: q | k | v, as c_attn writes it, with optional padding
        self.ld = (heads + 2 * kv_heads) * 64 + pad
        row = torch.full((n_seq, self.ld), float("nan"), dtype=tdt)
        row[:, :heads * 64] = q.reshape(n_seq, -1)
        for b, n in enumerate(totals):
            if append and n > 0:
                row[b, heads * 64:(heads + kv_heads) * 64] = self.k[b][n - 1].reshape(-1)
                row[b, (heads + kv_heads) * 64:(heads + 2 * kv_heads) * 64] = self.v[b][n - 1].reshape(-1)
        self.qkv = row.cuda()
        self.ldo = heads * 64 + pad
        self.out = torch.full((n_seq, self.ldo), 7.0, dtype=tdt, device="cuda")
        self.lse = torch.full((n_seq, heads), 7.0, device="cuda")
        self.cache = G.paged_cache(self.pages, self.refs, self.table, self.lens)
        self.ws_bytes = G.gpt2_attention_paged_workspace_bytes(self.cache, heads)
        self.ws = torch.full((self.ws_bytes,), 255, dtype=torch.uint8, device="cuda")

    def run(self, lse=True, stream=None):
        at, w = self.qkv.data_ptr(), self.heads * 128
        G.gpt2_attention_paged(self.cache, self.layer, at, self.ld, at + w if self.append else None,
                               at + w + self.kv * 128 if self.append else None, self.ld, self.out, self.ldo,
                               self.lse if lse else None, self.heads, self.scale, self.window, self.sinks, self.ws,
                               self.ws_bytes, stream)

    def check(self, rows=None):
        torch.cuda.synchronize()
        out = self.out.float().cpu().numpy().astype(np.float64)
        lse = self.lse.cpu().numpy().astype(np.float64)
        info = torch.finfo(DT[self.dtype])
        group = self.heads // self.kv
        for b in rows if rows is not None else range(len(self.lens_l)):
            assert (out[b, self.heads * 64:] == 7.0).all()
            if self.lens_l[b] < 0:
                assert (out[b] == 7.0).all() and (lse[b] == 7.0).all()
                continue
            vis = R.visible(self.totals[b], self.window, self.sinks)
            k, v = self.k[b][vis].double().numpy(), self.v[b][vis].double().numpy()
            for h in range(self.heads):
                ref, rl, pv, a = R.attention(self.q[b, h].double().numpy(), k[:, h // group], v[:, h // group],
                                             self.scale)
                got = out[b, h * 64:(h + 1) * 64]
                tol = info.eps / 2 * np.abs(ref) + info.smallest_normal * info.eps + (2 ** -15 * a + 2 ** -14) * pv
                assert (np.abs(got - ref) <= tol).all(), (b, h, np.abs(got - ref).max(), tol.min())
                if vis:
                    assert abs(lse[b, h] - rl) <= 1.45 * 2 ** -16 * a + 2 ** -14 + 2 ** -22 * abs(rl), (b, h)
                else:
                    assert lse[b, h] == -math.inf

    def check_cache(self, before):
        """The new rows stand in their slots, nothing else in the pool changed."""
        want = before.clone()
        if self.append:
            for b, n in enumerate(self.lens_l):
                if n >= 0:
                    p = int(self.table_np[b, n // self.page])
                    want[p, self.layer, 0, :, n % self.page] = self.k[b][n].cuda()
                    want[p, self.layer, 1, :, n % self.page] = self.v[b][n].cuda()
        assert torch.equal(self.pages.view(torch.int16), want.view(torch.int16))


def _go(c):
    before = c.pages.clone()
    c.run()
    c.check()
    c.check_cache(before)
    return c


EDGES = [0, 1, 14, 15, 16, 17, 30, 31, 32, 33, 47, 63, 64, 65, 127, 128, -1, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("append", [True, False])
@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_lengths_and_pages(dtype, append, page):
    _go(Case(EDGES, page=page, append=append, dtype=dtype, seed=page))


@pytest.mark.parametrize("heads, kv_heads", [(1, 1), (3, 3), (8, 1), (9, 1), (16, 1), (12, 4), (17, 1), (20, 1), (32, 2),
                                             (25, 1), (25, 25), (40, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_head_layouts(heads, kv_heads, dtype):
    _go(Case([5, 100, 31], heads=heads, kv_heads=kv_heads, dtype=dtype, seed=heads, pad=24))


@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (16, 0), (16, 4), (17, 16), (17, 17), (40, 33), (100, 1),
                                           (64, 64), (1000, 4), (5, 1000)])
@pytest.mark.parametrize("append", [True, False])
def test_windows(window, sinks, append):
    """Pages that the window hides are not in the table: their entries name no page."""
    _go(Case(EDGES + [500], window=window, sinks=sinks, append=append, junk_entry=1 << 30, seed=window))
    _go(Case([90, 200], window=window, sinks=sinks, append=append, page=32, drop_hidden=False, heads=12, kv_heads=4))


WIDE = 4096  # positions of a table row: more than one CTA takes per item, so the work is split and joined


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("append", [True, False])
@pytest.mark.parametrize("page", [16, 48, 256])
@pytest.mark.parametrize("heads, kv_heads", [(2, 2), (12, 4), (20, 1)])
def test_lengths_in_wide_tables(dtype, append, page, heads, kv_heads):
    _go(Case(EDGES + [1000, 2, 2500], page=page, append=append, dtype=dtype, seed=page, max_pages=WIDE // page + 1,
             heads=heads, kv_heads=kv_heads))


@pytest.mark.parametrize("window, sinks", [(1, 1), (16, 4), (17, 17), (100, 1), (5, 1000), (700, 33)])
@pytest.mark.parametrize("append", [True, False])
def test_windows_in_wide_tables(window, sinks, append):
    _go(Case(EDGES + [500, 3000], window=window, sinks=sinks, append=append, junk_entry=1 << 30, seed=window,
             max_pages=WIDE // 16))


def test_infinite_scores_and_missing_pages_in_wide_tables():
    c = Case([40, 2000, 600], heads=2, kv_heads=2, seed=16, max_pages=WIDE // 16)
    # two pages that are not there are left out, and so is a whole first half
    c.table[2, :20] = c.n_pages
    # sequence 1, head 0: every score -inf
    c.qkv[1, :64] = 0.0
    c.qkv[1, 0] = 1.0
    at = torch.arange(2001, device="cuda")
    rows = c.table[1].long()[at // 16], at % 16
    c.pages[rows[0][:2000], 1, 0, 0, rows[1][:2000]] = 0.0
    c.pages[rows[0][:2000], 1, 0, 0, rows[1][:2000], 0] = -math.inf
    c.qkv[1, 128:192] = 0.0
    c.qkv[1, 128] = -math.inf
    c.run()
    torch.cuda.synchronize()
    assert G.gpt2_last_error()[0] == RANGE
    assert (c.out[1, :64] == 0).all() and c.lse[1, 0] == -math.inf
    ref = R.attention(c.q[2, 1].double().numpy(), c.k[2][320:, 1].double().numpy(), c.v[2][320:, 1].double().numpy(),
                      0.125)
    assert np.abs(c.out[2, 64:128].double().cpu().numpy() - ref[0]).max() < 0.01
    assert abs(float(c.lse[2, 1]) - ref[1]) < 1e-3
    c.check(rows=[0])


@pytest.mark.parametrize("lens, heads, kv_heads", [([5000], 1, 1), ([5000], 12, 12), ([4097, 3, 2000], 4, 1),
                                                   ([20000], 2, 2), ([9000, 0, -1, 8999], 16, 1)])
def test_long_lengths_are_split_and_joined(lens, heads, kv_heads):
    _go(Case(lens, heads=heads, kv_heads=kv_heads, page=64, seed=heads))


def test_many_sequences():
    g = np.random.default_rng(3)
    lens = [int(n) for n in g.integers(-1, 80, 1024)]
    _go(Case(lens, heads=3, kv_heads=3, seed=4))


def test_scores_that_grow_raise_the_maximum_in_every_tile():
    """Keys that grow along the sequence, and a large scale: the running maximum moves on and on."""
    _go(Case([400, 33], heads=4, kv_heads=2, grow=0.02, scale=0.5, seed=5))
    _go(Case([400, 33], heads=4, kv_heads=2, grow=0.02, scale=0.5, seed=5, dtype="f16"))


def test_infinite_scores():
    c = Case([40, 20], heads=2, kv_heads=2, seed=6)
    # every visible key of sequence 0, head 0 gives a score of -inf: nothing is left, as for an empty sequence
    c.qkv[0, :128] = 0.0
    c.qkv[0, 0] = 1.0
    for p in range(40):
        c.pages[c.table_np[0, p // 16], 1, 0, 0, p % 16, :] = 0.0
        c.pages[c.table_np[0, p // 16], 1, 0, 0, p % 16, 0] = -math.inf
    c.qkv[0, 128:192] = 0.0
    c.qkv[0, 128] = -math.inf
    # one key of sequence 1, head 1 holds NaN: the head's row is NaN, the other head is not
    c.pages[c.table_np[1, 0], 1, 0, 1, 3, 5] = math.nan
    c.run()
    torch.cuda.synchronize()
    assert (c.out[0, :64] == 0).all() and c.lse[0, 0] == -math.inf
    assert torch.isnan(c.out[1, 64:128]).all() and torch.isnan(c.lse[1, 1])
    assert torch.isfinite(c.out[1, :64]).all()


def test_without_lse_and_repeated_calls_give_the_same_bits():
    c = Case([700, 3, 64, 1200], heads=12, kv_heads=12, seed=7)
    c.run()
    torch.cuda.synchronize()
    first, lse = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.out.fill_(7.0)
        c.ws.random_(0, 256)
        c.run(lse=False)
        torch.cuda.synchronize()
        assert torch.equal(c.out, first) and torch.equal(c.lse, lse)


def test_pages_behind_four_gigabytes():
    """Element offsets beyond 32 bits in the pool and in the table's row."""
    page, layers, kv = 4096, 4, 16
    per = layers * 2 * kv * page * 64
    n_pages = (1 << 32) // per + 3
    pages = torch.empty((n_pages, layers, 2, kv, page, 64), dtype=torch.bfloat16, device="cuda")
    assert pages.numel() > 1 << 32
    small = Case([150], heads=16, kv_heads=16, page=4096, layers=layers, layer=3, seed=8, append=True)
    pages[n_pages - 1] = small.pages[int(small.table_np[0, 0])]
    small.table.fill_(n_pages - 1)
    refs = torch.ones(n_pages, dtype=torch.int32, device="cuda")
    small.cache = G.paged_cache(pages, refs, small.table, small.lens)
    small.run()
    small.check()
    assert torch.equal(pages[n_pages - 1, 3, 0, :, 150], small.k[0][150].cuda())


def test_bad_pages_and_lengths_are_reported_and_the_rest_is_right():
    c = Case([40, 50, 600, 60], heads=2, kv_heads=2, seed=9, max_pages=40)
    c.table[1, 1] = c.n_pages  # out of range
    c.table[1, 2] = -1
    c.lens[2] = 640  # does not fit 40 pages of 16 with the new token
    c.run()
    c.check(rows=[0, 3])
    assert (c.out[2] == 7.0).all()
    assert G.gpt2_last_error()[0] == RANGE
    # the two pages that are not there are left out
    vis = [p for p in range(51) if p // 16 not in (1, 2)]
    ref = R.attention(c.q[1, 0].double().numpy(), c.k[1][vis][:, 0].double().numpy(),
                      c.v[1][vis][:, 0].double().numpy(), 0.125)[0]
    assert np.abs(c.out[1, :64].double().cpu().numpy() - ref).max() < 0.02


def test_lengths_far_out_of_range_are_reported():
    c = Case([40, 50], heads=2, kv_heads=2, seed=17)
    c.lens[1] = 2 ** 31 - 1
    c.run()
    c.check(rows=[0])
    assert (c.out[1] == 7.0).all()
    assert G.gpt2_last_error()[0] == RANGE


def test_view_of_later_slots():
    c = Case([40, 50, 60], heads=2, kv_heads=2, seed=10)
    c.cache = G.paged_cache(c.pages, c.refs, c.table[1:], c.lens[1:])
    c.qkv, full = c.qkv[1:], c.out
    c.out, lse = full[1:], c.lse
    c.lse = lse[1:]
    c.run()
    c.out, c.lse = full, lse
    c.check(rows=[1, 2])
    assert (full[0] == 7.0).all()


def test_graphs_and_streams():
    """Two captured calls with a workspace each, replayed on two streams at once, with lengths changed in place."""
    cases = [Case([500, 90, 7], heads=12, kv_heads=12, seed=s, max_pages=40, drop_hidden=True) for s in (11, 12)]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for c, s in zip(cases, streams):
        c.run(stream=s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run(stream=torch.cuda.current_stream())
        graphs.append(g)
    for c in cases:
        c.out.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    for c in cases:
        c.check()
    # shorter sequences through the same graph: position 64 takes the new token, what is behind counts no more
    for c, g in zip(cases, graphs):
        c.lens.copy_(torch.tensor([64, -1, 7], dtype=torch.int32))
        c.lens_l, c.totals = [64, -1, 7], [65, 0, 8]
        for kv in (c.k, c.v):
            kv[0][64] = kv[0][500]
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        c.check()
