"""Page bookkeeping on the GPU against a model of it that works one entry at a
time on Python lists: tables, reference counts and lengths must be equal, and
every position that is defined must hold its K and V bit for bit."""
import numpy as np
import pytest

import paged_ref as R

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


class Both:
    """The library's cache and the model, driven alike."""

    def __init__(self, n_pages, page, n_seq, max_pages, layers=2, kv=3, dtype=torch.bfloat16, seed=0):
        self.m = R.Pool(n_pages, page, n_seq, max_pages)
        self.layers, self.kv, self.dtype = layers, kv, dtype
        self.rng = np.random.default_rng(seed)
        self.pages = torch.full((n_pages, layers, 2, kv, page, 64), 9.0, dtype=dtype, device="cuda")
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((n_seq, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.full((n_seq,), -1, dtype=torch.int32, device="cuda")
        self.cache = G.paged_cache(self.pages, self.refs, self.table, self.lens)
        self.ws_bytes = G.gpt2_pages_workspace_bytes(self.cache)
        self.ws = torch.full((self.ws_bytes,), 255, dtype=torch.uint8, device="cuda")
        self.values = {}  # id -> [layers, 2, kv, 64]

    def begin(self, b):
        self.m.lens[b] = 0
        self.lens[b] = 0

    def reserve(self, n_new, ok=True):
        G.gpt2_pages_reserve(self.cache, _i32(n_new), self.ws, self.ws_bytes)
        assert self.m.reserve(n_new) == ok
        assert G.gpt2_last_error()[0] == (0 if ok else RANGE)

    def append(self, n_new, T=None, counts=True):
        """New tokens of every sequence, in all layers."""
        T = T or max(max(n_new), 1)
        n_seq, w = self.m.n_seq, self.kv * 64
        rows = torch.from_numpy(self.rng.standard_normal((self.layers, n_seq * T, 3 * w)).astype(np.float32))
        rows = rows.to(self.dtype).cuda()
        for l in range(self.layers):
            at = rows[l].data_ptr()
            G.gpt2_pages_write(self.cache, l, at + 2 * w, at + 4 * w, 3 * w, T, _i32(n_new) if counts else None)
        for b, add in enumerate(n_new):
            if self.m.lens[b] < 0:
                continue
            for t in range(add):
                key = len(self.values)
                self.values[key] = rows[:, b * T + t, w:].view(self.layers, 2, self.kv, 64)
                self.m.put(b, self.m.lens[b] + t, key)
            self.m.lens[b] += max(add, 0)
        self.lens.copy_(_i32(self.m.lens))

    def grow(self, n_new):
        self.reserve(n_new)
        self.append(n_new)

    def fork(self, parents, children):
        G.gpt2_pages_fork(self.cache, _i32(parents), _i32(children), len(parents))
        self.m.fork(parents, children)

    def free(self, seqs, first=0, last=0):
        G.gpt2_pages_free(self.cache, _i32(seqs), len(seqs), first, last)
        self.m.free(seqs, first, last)

    def compact(self):
        n = _i32([-5])
        G.gpt2_pages_compact(self.cache, n, self.ws, self.ws_bytes)
        assert int(n) == self.m.compact()

    def check(self):
        torch.cuda.synchronize()
        assert G.gpt2_last_error()[0] == 0
        assert self.table.cpu().tolist() == self.m.table
        assert self.lens.cpu().tolist() == self.m.lens
        assert self.refs.cpu().tolist() == self.m.refs
        count = [0] * self.m.n_pages
        for row in self.m.table:
            for p in row:
                if p >= 0:
                    count[p] += 1
        assert count == self.m.refs  # the model itself
        at, off, keys = [], [], []
        for b in range(self.m.n_seq):
            for pos in range(max(self.m.lens[b], 0)):
                p = self.m.table[b][pos // self.m.page]
                if p >= 0:
                    at.append(p)
                    off.append(pos % self.m.page)
                    keys.append(self.m.content[p][pos % self.m.page])
        assert None not in keys
        if keys:
            got = self.pages[torch.tensor(at), :, :, :, torch.tensor(off)]
            assert torch.equal(got, torch.stack([self.values[k] for k in keys]))


def test_write_reserve_and_read_back_ragged_prompts():
    x = Both(40, 16, 5, 8, dtype=torch.float16)
    for b in (0, 1, 3, 4):
        x.begin(b)
    x.grow([17, 1, 5, 16, 0])
    x.check()
    x.grow([1, 15, 9, 33, 2])
    x.check()


def test_write_without_counts_and_odd_page_size():
    x = Both(12, 48, 3, 3, kv=5)
    x.begin(0)
    x.begin(2)
    x.reserve([50, 0, 50])
    x.append([50, 50, 50], T=50, counts=False)  # slot 1 is idle: skipped
    x.check()


def test_write_to_positions_without_a_page_is_reported():
    x = Both(12, 16, 2, 2)
    x.begin(0)
    x.begin(1)
    x.reserve([16, 32])
    rows = torch.ones(2 * 40, 3 * 64, dtype=torch.bfloat16, device="cuda")
    before = x.pages.clone()
    x.append([16, 32])
    assert G.gpt2_last_error()[0] == 0
    before = x.pages.clone()
    G.gpt2_pages_write(x.cache, 0, rows, rows, 192, 40, None)  # lens 16 and 32: no page, and behind the table
    assert G.gpt2_last_error()[0] == RANGE
    assert torch.equal(x.pages, before)


def test_samples_share_a_prompt_and_split_when_they_write():
    x = Both(30, 16, 6, 4)
    x.begin(0)
    x.grow([21, 0, 0, 0, 0, 0])
    x.fork([0] * 5, [1, 2, 3, 4, 5])
    x.check()
    assert x.m.refs.count(6) == 2
    x.grow([1] * 6)  # all six write: five copies, the last keeps the page
    x.check()
    assert x.m.table[5][1] == 1
    x.grow([0, 1, 1, 1, 0, 0])
    x.check()


def test_only_some_holders_write():
    x = Both(30, 16, 4, 4)
    x.begin(0)
    x.grow([20, 0, 0, 0])
    x.fork([0, 0], [1, 2])
    x.grow([0, 1, 1, 0])  # sequence 0 still reads the page: both split off
    x.check()
    x.fork([0], [3])
    x.free([0])
    x.grow([0, 0, 0, 1])  # the last holder: no copy
    x.check()


def test_fork_at_a_page_border_copies_nothing():
    x = Both(10, 16, 2, 4)
    x.begin(0)
    x.grow([32, 0])
    x.fork([0], [1])
    x.grow([1, 1])
    x.check()
    assert x.m.refs[:2] == [2, 2]


def test_fork_permutes_beams_and_copies_onto_itself():
    x = Both(64, 16, 5, 6)
    for b in range(4):
        x.begin(b)
    x.grow([20, 35, 3, 16, 0])
    x.fork([1, 2, 0, 3, 1], [0, 1, 2, 3, 4])  # cycle, itself, and a copy
    x.check()
    x.grow([2] * 5)
    x.check()
    x.fork([4, 4, 4, 4, 4], [0, 1, 2, 3, 4])
    x.check()
    x.fork([0], [0])
    x.check()


def test_fork_of_an_idle_slot_empties_the_child_and_reserved_pages_stay_behind():
    x = Both(20, 16, 3, 5)
    x.begin(0)
    x.begin(1)
    x.grow([40, 5, 0])
    x.reserve([30, 0, 0])  # pages without positions
    x.fork([2, 0], [1, 2])
    x.check()
    assert x.m.lens[1] == -1


def test_a_sequence_cut_back_splits_every_page_it_writes_to():
    x = Both(20, 16, 2, 6)
    x.begin(0)
    x.grow([60, 0])
    x.fork([0], [1])
    x.m.lens[1] = 20
    x.lens[1] = 20
    x.grow([0, 30])
    x.check()


def test_free_whole_sequences_and_behind_a_window():
    x = Both(60, 16, 4, 10)
    for b in range(4):
        x.begin(b)
    x.grow([150, 40, 16, 0])
    x.reserve([10, 0, 0, 5])
    x.free([0, 1, 3], 4, 39)
    x.check()
    assert x.m.table[0][0] >= 0 and x.m.table[0][1] == -1
    x.free([0], 0, 1)
    x.check()
    x.free([2, 0])
    x.check()
    x.begin(2)
    x.grow([0, 3, 20, 2])
    x.check()


def test_refusals_change_nothing():
    x = Both(8, 16, 4, 4)
    x.begin(0)
    x.begin(1)
    x.grow([40, 16, 0, 0])
    state = (x.table.clone(), x.refs.clone(), x.lens.clone())
    for parents, children in (([0, 0], [2, 2]), ([0], [4]), ([4], [2]), ([-1], [2]), ([0], [-1])):
        G.gpt2_pages_fork(x.cache, _i32(parents), _i32(children), len(parents))
        assert G.gpt2_last_error()[0] == RANGE
    for seqs in ([1, 1], [4], [-1]):
        G.gpt2_pages_free(x.cache, _i32(seqs), len(seqs), 0, 0)
        assert G.gpt2_last_error()[0] == RANGE
    x.reserve([0, 25, 0, 0], ok=True)
    x.check()
    x.begin(2)
    x.reserve([0, 0, 60, 0], ok=False)  # four pages wanted, two left
    x.reserve([25, 0, 0, 0], ok=False)  # 40 + 25 positions do not fit four pages of 16
    x.check()
    keep = int(x.table[0, 2])
    x.table[0, 2] = 8  # names no page
    G.gpt2_pages_reserve(x.cache, _i32([1, 0, 1, 0]), x.ws, x.ws_bytes)
    assert G.gpt2_last_error()[0] == RANGE
    G.gpt2_pages_compact(x.cache, _i32([0]), x.ws, x.ws_bytes)
    assert G.gpt2_last_error()[0] == RANGE
    x.table[0, 2] = keep
    x.check()
    del state


def test_free_pages_are_taken_lowest_first_from_a_large_pool():
    n = 30000
    x = Both(n, 16, 3, 8, layers=1, kv=1)
    x.refs.fill_(1)
    x.m.refs = [1] * n
    for p in (29999, 5, 17000, 8191, 8192, 16384, 12345):
        x.refs[p] = 0
        x.m.refs[p] = 0
    x.begin(1)
    x.reserve([0, 97, 0])
    assert x.m.table[1][:7] == [5, 8191, 8192, 12345, 16384, 17000, 29999]
    assert x.table.cpu().tolist() == x.m.table and x.refs.cpu().tolist() == x.m.refs


def test_reserve_of_many_entries():
    """More entries than one CTA has threads: prompts of many pages, some of them shared and all rewritten."""
    x = Both(1600, 16, 40, 64, layers=1, kv=1)
    for b in range(20):
        x.begin(b)
    x.grow([500 + 7 * b if b < 20 else 0 for b in range(40)])
    x.check()
    x.fork(list(range(20)), list(range(20, 40)))
    x.m.lens = [n - 300 if b % 3 else n for b, n in enumerate(x.m.lens)]  # cut back: shared pages behind the end
    x.lens.copy_(_i32(x.m.lens))
    x.grow([301 if b % 5 else 350 for b in range(40)])
    x.check()
    x.reserve([900 - n for n in x.m.lens], ok=False)  # too few pages left
    x.check()


def test_fork_of_many_rows():
    """Tables beyond what one CTA takes: the cluster."""
    x = Both(4000, 16, 300, 64, layers=1, kv=1)
    for b in range(100):
        x.begin(b)
    x.grow([200 + b if b < 100 else 0 for b in range(300)])
    g = np.random.default_rng(1)
    x.fork([int(p) for p in g.integers(0, 120, 250)], [int(c) for c in g.permutation(300)[:250]])
    x.check()
    x.fork([int(p) for p in g.integers(0, 300, 300)], [int(c) for c in g.permutation(300)])
    x.check()


@pytest.mark.parametrize("T, kv", [(200, 3), (130, 1), (33, 70)])
def test_writes_of_many_rows(T, kv):
    """Several rows per CTA, ragged, across pages, and more heads than a CTA has threads for."""
    x = Both(150, 16, 20, 30, layers=1, kv=kv)
    for b in range(18):
        x.begin(b)
    x.grow([b % 7 for b in range(20)])
    n = [min(T, (b * 37) % (T + 1)) if b % 4 else T for b in range(20)]
    n = [c if b < 10 else 0 for b, c in enumerate(n)]
    x.reserve(n)
    x.append(n, T=T)
    x.check()


def test_writes_to_shared_pages_are_refused():
    x = Both(20, 16, 3, 4)
    x.begin(0)
    x.grow([20, 0, 0])
    x.fork([0], [1])
    before = x.pages.clone()
    rows = torch.ones(3 * 2, 3 * 64, dtype=torch.bfloat16, device="cuda")
    G.gpt2_pages_write(x.cache, 1, rows, rows, 192, 2, _i32([2, 0, 0]))
    assert G.gpt2_last_error()[0] == RANGE and torch.equal(x.pages, before)
    need = G.gpt2_attention_paged_workspace_bytes(x.cache, 3)
    ws, out = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.zeros(3, 192, dtype=torch.bfloat16, device="cuda")
    G.gpt2_attention_paged(x.cache, 1, rows, 192, rows, rows, 192, out, 192, None, 3, 0.125, 0, 0, ws, need)
    assert G.gpt2_last_error()[0] == RANGE and torch.equal(x.pages, before)
    x.reserve([1, 0, 0])
    G.gpt2_pages_write(x.cache, 1, rows, rows, 192, 2, _i32([1, 0, 0]))
    assert G.gpt2_last_error()[0] == 0


@pytest.mark.parametrize("n_pages, used", [(1, 0), (1, 1), (7, 3), (50, 49), (50, 50), (4097, 2000), (9000, 8500), (16384, 9000), (16385, 9000),
                                           (40000, 39990)])
def test_compact(n_pages, used):
    page = 16
    g = np.random.default_rng(n_pages + used)
    x = Both(n_pages, page, 4, max(1, -(-used // 4)), layers=1, kv=1)
    ids = g.permutation(n_pages)[:used]
    tags = torch.arange(n_pages, dtype=torch.int32, device="cuda")  # each page's number, in its first two values
    x.pages.view(torch.int32).view(n_pages, -1)[:, 0] = tags
    x.pages.view(torch.int32).view(n_pages, -1)[:, -1] = tags
    for k, p in enumerate(ids):
        x.m.table[k % 4][k // 4] = int(p)
        x.m.refs[p] = 1
    if used:
        x.m.refs[int(ids[0])] = 2
        x.m.table[3][-1] = int(ids[0]) if x.m.table[3][-1] < 0 else x.m.table[3][-1]
        if x.m.table[3][-1] != int(ids[0]):
            x.m.refs[int(ids[0])] = 1
    x.m.content = [[p] * page for p in range(n_pages)]
    x.table.copy_(_i32(x.m.table))
    x.refs.copy_(_i32(x.m.refs))
    x.compact()
    torch.cuda.synchronize()
    assert x.table.cpu().tolist() == x.m.table and x.refs.cpu().tolist() == x.m.refs
    for col in (0, -1):
        got = x.pages.view(torch.int32).view(n_pages, -1)[:used, col].cpu().tolist()
        assert got == [x.m.content[p][0] for p in range(used)]


@pytest.mark.parametrize("seed", range(6))
def test_random_histories(seed):
    """Sequences begin, grow, are shared, trimmed, given back and compacted in random order."""
    g = np.random.default_rng(100 + seed)
    page = int(g.choice([16, 32, 48]))
    n_seq = int(g.integers(2, 12))
    x = Both(int(g.integers(60, 120)), page, n_seq, 8, layers=2, kv=2, seed=seed)
    trimmed = set()
    for _ in range(60):
        op = g.integers(0, 10)
        live = [b for b in range(n_seq) if x.m.lens[b] >= 0]
        if op <= 1:
            for b in range(n_seq):
                if x.m.lens[b] < 0 and g.random() < 0.5:
                    x.begin(b)
        elif op <= 5:
            add = [int(g.integers(0, 40)) if g.random() < 0.6 else 0 for _ in range(n_seq)]
            add = [min(a, 8 * page - x.m.lens[b]) if x.m.lens[b] >= 0 else a for b, a in enumerate(add)]
            if sum(-(-a // page) + 1 for a in add) <= x.m.refs.count(0):
                x.grow(add)
        elif op <= 7 and live:
            n = int(g.integers(1, n_seq + 1))
            x.fork([int(b) for b in g.choice(live, n)], [int(b) for b in g.permutation(n_seq)[:n]])
        elif op == 8 and live:
            seqs = [int(b) for b in g.permutation(n_seq)[:int(g.integers(1, n_seq + 1))]]
            if g.random() < 0.5:
                x.free(seqs)
            else:
                x.free(seqs, int(g.integers(0, 20)), int(g.integers(1, 60)))
                trimmed.update(seqs)
        elif op == 9:
            x.compact()
        x.check()


def test_captured_step_of_a_serving_loop():
    """Fork, reserve and write inside one CUDA graph: replays split the pages anew from the state they find."""
    x = Both(40, 16, 4, 6, seed=5)
    x.begin(0)
    x.grow([21, 0, 0, 0])
    parents, children, new = _i32([0, 0, 0]), _i32([1, 2, 3]), _i32([0, 1, 1, 1])
    x.fork([0, 0, 0], [1, 2, 3])
    x.reserve([0, 1, 1, 1])
    x.check()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        G.gpt2_pages_free(x.cache, children, 3, 0, 0)
        G.gpt2_pages_fork(x.cache, parents, children, 3)
        G.gpt2_pages_reserve(x.cache, new, x.ws, x.ws_bytes)
    for _ in range(3):
        g.replay()
        x.m.free([1, 2, 3])
        x.m.fork([0, 0, 0], [1, 2, 3])
        assert x.m.reserve([0, 1, 1, 1])
        x.check()
