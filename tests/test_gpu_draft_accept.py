"""gpt2_draft_accept on the GPU against the walk and the moves made one at a
time in Python; everything is compared bit for bit."""
import numpy as np
import pytest

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


class Case:
    def __init__(self, lens, T, page=16, layers=3, kv=2, counts=None, likely=0.7, chain=False, seed=0, vocab=50,
                 dtype=torch.bfloat16):
        g = np.random.default_rng(seed)
        n_seq = len(lens)
        self.lens_l, self.T, self.page = list(lens), T, page
        self.counts_l = counts or [T] * n_seq
        cols = max([1] + [-(-(n + T) // page) for n in lens if n >= 0])
        ids = g.permutation(n_seq * cols + 3)
        self.table_l = [[int(ids[b * cols + c]) for c in range(cols)] for b in range(n_seq)]
        self.parents_l = [[-1 if t == 0 else t - 1 if chain else int(g.integers(0, t)) for t in range(T)]
                          for _ in range(n_seq)]
        self.tokens_l = g.integers(0, vocab, (n_seq, T)).tolist()
        self.chosen_l = g.integers(0, vocab, (n_seq, T)).tolist()
        for b in range(n_seq):  # most tokens are followed by one of their children
            for t in range(T):
                down = [u for u in range(T) if self.parents_l[b][u] == t]
                if down and g.random() < likely:
                    self.chosen_l[b][t] = self.tokens_l[b][int(g.choice(down))]
        self.pages = torch.randint(-32768, 32767, (n_seq * cols + 3, layers, 2, kv, page, 64), dtype=torch.int16,
                                   device="cuda").view(dtype)
        self.before = self.pages.clone()
        self.refs, self.table, self.lens = _i32([1] * (n_seq * cols + 3)), _i32(self.table_l), _i32(self.lens_l)
        self.cache = G.paged_cache(self.pages, self.refs, self.table, self.lens)
        self.path, self.kept, self.next = (torch.full(s, -7, dtype=torch.int32, device="cuda")
                                           for s in ((n_seq, T), (n_seq,), (n_seq,)))

    def upload(self):
        self.tokens, self.parents, self.chosen = _i32(self.tokens_l), _i32(self.parents_l), _i32(self.chosen_l)
        self.counts = _i32(self.counts_l)

    def run(self, parents=True, counts=True, stream=None):
        self.upload()
        G.gpt2_draft_accept(self.cache, self.T, self.tokens, self.parents if parents else None,
                            self.counts if counts else None, self.chosen, self.path, self.kept, self.next, stream)
        return self

    def check(self, left=(), gone=()):
        """left: sequences that stay as they were, with n_kept 0."""
        torch.cuda.synchronize()
        want = self.before.clone()
        for b, n in enumerate(self.lens_l):
            count = min(self.counts_l[b], self.T)
            if n < 0 or count <= 0 or b in left:
                assert self.path[b].tolist() == [-7] * self.T and int(self.next[b]) == -7
                assert int(self.kept[b]) == (0 if b in left else -7) and int(self.lens[b]) == n
                continue
            path = [0]
            while True:
                down = [u for u in range(path[-1] + 1, count) if self.parents_l[b][u] == path[-1]
                        and self.tokens_l[b][u] == self.chosen_l[b][path[-1]]]
                if not down:
                    break
                path.append(down[0])
            assert self.path[b].tolist() == path + [-1] * (self.T - len(path))
            assert int(self.kept[b]) == len(path) and int(self.next[b]) == self.chosen_l[b][path[-1]]
            assert int(self.lens[b]) == n + len(path)
            for j, t in enumerate(path):
                a, z = n + t, n + j
                want[self.table_l[b][z // self.page], :, :, :, z % self.page] = \
                    want[self.table_l[b][a // self.page], :, :, :, a % self.page]
        assert torch.equal(self.pages.view(torch.int16), want.view(torch.int16))
        return self


@pytest.mark.parametrize("T", [1, 2, 5, 16, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("likely", [0.0, 0.7, 1.0])
def test_paths(T, likely):
    Case([70, 0, -1, 15, 16, 3], T, likely=likely, seed=T).run().check()


@pytest.mark.parametrize("page", [16, 48, 256])
@pytest.mark.parametrize("layers, kv", [(1, 1), (12, 5), (2, 70)])
def test_pages(page, layers, kv):
    Case([page - 1, 5, 2 * page], 40, page=page, layers=layers, kv=kv, likely=0.95, seed=page,
         dtype=torch.float16).run().check()


def test_a_chain_that_stays_whole_moves_nothing():
    c = Case([20, 7], 64, chain=True, likely=1.0, seed=3).run(parents=False).check()
    assert c.kept.tolist() == [64, 64] and torch.equal(c.pages.view(torch.int16), c.before.view(torch.int16))


def test_the_longest_moves():
    """Every second token stays: rows move over one another."""
    c = Case([9], 64, seed=4)
    c.parents_l[0] = [-1] + [(t - 1) // 2 * 2 for t in range(1, 64)]
    c.tokens_l[0] = list(range(64))
    c.chosen_l[0] = [t + 2 if t + 2 < 64 else 99 for t in range(64)]
    c.run().check()
    assert c.kept.tolist() == [32] and c.next.tolist() == [99]


def test_the_lowest_of_equal_children():
    c = Case([9], 6, seed=4)
    c.parents_l[0], c.tokens_l[0], c.chosen_l[0] = [-1, 0, 0, 0, 3, 2], [5, 1, 8, 8, 9, 9], [8, 0, 9, 9, 2, 3]
    c.run().check()
    assert c.path.tolist() == [[0, 2, 5, -1, -1, -1]] and c.next.tolist() == [3]


def test_ragged_counts():
    Case([50, 9, 31, -1, 64], 19, counts=[19, 0, 1, 7, 25], likely=1.0, seed=5).run().check()
    Case([50, 9], 7, counts=[-2, 3], likely=1.0, seed=6).run().check()
    Case([50, 9], 7, likely=1.0, seed=6).run(counts=False).check()


def test_parents_out_of_range_have_no_part_in_a_path():
    c = Case([50], 8, seed=5)
    c.parents_l[0] = [0, 0, 2, 9, -5, 1, 2 ** 31 - 1, 4]
    c.tokens_l[0] = [3] * 8
    c.chosen_l[0] = [3] * 8
    c.run().check()
    assert c.path.tolist() == [[0, 1, 5] + [-1] * 5]


def test_a_missing_page_leaves_the_sequence():
    c = Case([14, 14], 8, chain=True, likely=1.0, seed=5)
    c.table[0, 1] = -1
    c.run().check(left=[0])
    assert G.gpt2_last_error() == (RANGE, 21)
    c = Case([14, 14], 8, chain=True, likely=1.0, seed=5)
    c.table[1, 1] = c.pages.shape[0]
    c.run().check(left=[1])
    assert G.gpt2_last_error() == (RANGE, 21)


def test_a_shared_page_leaves_the_sequence():
    c = Case([14, 14], 8, chain=True, likely=1.0, seed=5)
    c.refs[c.table_l[0][1]] = 2
    c.run().check(left=[0])
    assert G.gpt2_last_error() == (RANGE, 28)
    c = Case([14, 14], 8, likely=0.0, seed=5)  # one token kept, on the page before
    c.refs[c.table_l[0][1]] = 2
    c.chosen_l = [[1000] * 8] * 2
    c.run().check()


@pytest.mark.parametrize("length", [41, 10 ** 9, 2 ** 31 - 1])
def test_a_sequence_longer_than_its_table_row(length):
    c = Case([40, 12], 8, seed=5)  # three pages: 48 places
    c.lens[0] = length
    c.lens_l[0] = length
    c.run().check(left=[0])
    assert G.gpt2_last_error() == (RANGE, 20)


@pytest.mark.parametrize("n_seq", [1, 200, 1024])
def test_many_sequences(n_seq):
    g = np.random.default_rng(n_seq)
    Case([int(x) for x in g.integers(-1, 30, n_seq)], 6, layers=1, kv=1, likely=0.9, seed=n_seq).run().check()


def test_captured_and_replayed():
    c = Case([20, 40], 12, likely=1.0, seed=8)
    s = torch.cuda.Stream()
    c.upload()
    torch.cuda.synchronize()
    call = lambda: G.gpt2_draft_accept(c.cache, 12, c.tokens, c.parents, c.counts, c.chosen, c.path, c.kept, c.next)  # noqa: E731,E501
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
        graph.replay()
    c.check()
