"""gpt2_attention_paged and gpt2_decode_step_paged on the GPU where the work is
split into runs and joined: tables too wide, or sequences too many, for one CTA
per item.  Elements against float64 with the bounds of the other attention
tests; the workspace holding anything, captured calls and replays equal to eager
ones bit for bit.

An item is one block of query heads (at most 16) of one key-value head of one
sequence.  More items than SMs are joined a warp each; fewer a CTA each, for
1, 2, 4 or 8 heads of it at a time."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402
from test_gpu_paged_attention import Case, _built, _go  # noqa: E402,F401
from test_gpu_paged_model import Server, _i32  # noqa: E402

pytestmark = pytest.mark.gpu
COLS = 300  # pages of 16 a table row: 4800 positions, beyond what one CTA takes


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _items(n_seq, heads, kv_heads):
    return n_seq * kv_heads * -(-(heads // kv_heads) // 16)


def _ragged(n, seed, most=400):
    """Empty, idle, single, long and ordinary sequences."""
    g = np.random.default_rng(seed)
    lens = [int(x) for x in g.integers(0, most, n)]
    for k, v in zip(g.permutation(n), (-1, 0, 1, 15, 16, 17, -1, 2900, 1500, 0)):
        lens[int(k)] = v
    return lens


MANY = [(2, 1, 200), (6, 3, 60), (9, 3, 60), (16, 4, 64), (5, 1, 170), (12, 1, 160), (17, 1, 90), (25, 1, 80),
        (32, 2, 80), (40, 1, 60)]


@pytest.mark.parametrize("heads, kv_heads, n_seq", MANY)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_more_items_than_sms(heads, kv_heads, n_seq, dtype):
    assert _items(n_seq, heads, kv_heads) > _sms()
    _go(Case(_ragged(n_seq, heads), heads=heads, kv_heads=kv_heads, dtype=dtype, seed=heads, pad=8, max_pages=COLS))


@pytest.mark.parametrize("heads, kv_heads, n_seq", [(6, 3, 60), (25, 1, 80)])
@pytest.mark.parametrize("append", [True, False])
def test_more_items_than_sms_under_a_window(heads, kv_heads, n_seq, append):
    _go(Case(_ragged(n_seq, 7), heads=heads, kv_heads=kv_heads, window=150, sinks=5, append=append, junk_entry=1 << 30,
             seed=heads, max_pages=COLS))


@pytest.mark.parametrize("heads, kv_heads, n_seq, width", [(3, 3, 12, 1), (16, 1, 15, 1), (16, 1, 30, 2),
                                                           (16, 1, 60, 4), (11, 1, 80, 4), (16, 1, 100, 8),
                                                           (20, 1, 70, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_fewer_items_than_sms(heads, kv_heads, n_seq, width, dtype):
    items, group = _items(n_seq, heads, kv_heads), heads // kv_heads
    block = -(-group // -(-group // 16))
    assert items <= _sms()
    if _sms() == 152:  # the number of heads side by side that these sizes are here for
        assert width == next(w for w in (1, 2, 4, 8) if w == 8 or items * -(-block // w) <= 2 * 152)
    _go(Case(_ragged(n_seq, n_seq), heads=heads, kv_heads=kv_heads, dtype=dtype, seed=n_seq, max_pages=COLS))


SPLIT = [dict(heads=12, kv_heads=12, n=4), dict(heads=16, kv_heads=1, n=60), dict(heads=12, kv_heads=4, n=50),
         dict(heads=25, kv_heads=1, n=90)]


def _split_case(heads, kv_heads, n, seed, dtype="bf16"):
    g = np.random.default_rng(seed)
    lens = [2500] + [int(x) for x in g.integers(70, 600, n - 1)]
    return Case(lens, heads=heads, kv_heads=kv_heads, seed=seed, max_pages=COLS, dtype=dtype)


@pytest.mark.parametrize("kw", SPLIT, ids=lambda k: "-".join(str(v) for v in k.values()))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_workspace_may_hold_anything_and_calls_give_the_same_bits(kw, dtype):
    c = _split_case(**kw, seed=3, dtype=dtype)
    c.run()
    c.check()
    first, lse = c.out.clone(), c.lse.clone()
    for fill in (0, 255, None):
        c.out.fill_(7.0)
        if fill is None:
            c.ws.random_(0, 256)
        else:
            c.ws.fill_(fill)
        c.run(lse=False)
        torch.cuda.synchronize()
        assert torch.equal(c.out, first) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("kw", SPLIT, ids=lambda k: "-".join(str(v) for v in k.values()))
def test_captured_calls_on_two_streams_follow_the_lengths(kw):
    """Two captured calls with a workspace each, replayed on two streams at once; then with lengths changed in place
    and the workspaces scrambled."""
    cases = [_split_case(**kw, seed=s) for s in (11, 12)]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for c, s in zip(cases, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run(stream=torch.cuda.current_stream())
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    for c in cases:
        c.check()
    for c, cut in zip(cases, (lambda b, n: -1 if b % 5 == 3 else n - 64 if b % 2 else n,
                              lambda b, n: 0 if b % 7 == 2 else n // 2)):
        new = [cut(b, n) for b, n in enumerate(c.lens_l)]
        for b, (n, was) in enumerate(zip(new, c.lens_l)):
            if n >= 0:  # the new token's rows go to position n
                for kv in (c.k, c.v):
                    kv[b][n] = kv[b][was]
        c.lens_l, c.totals = new, [n + 1 if n >= 0 else 0 for n in new]
        c.lens.copy_(_i32(new))
        c.ws.random_(0, 256)
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    for c in cases:
        c.check()


SERVERS = [dict(n_seq=3, max_pages=136), dict(n_seq=60, n_pages=200, max_pages=8)]  # wide tables; many sequences


@pytest.mark.parametrize("kw", SERVERS, ids=["wide", "many"])
@pytest.mark.parametrize("window, sinks", [(0, 0), (9, 2)])
@pytest.mark.parametrize("dtype", [G.BF16, G.F16])
def test_decode_steps_captured_and_replayed_equal_eager_ones(kw, window, sinks, dtype):
    """Eager on the default stream; reserve and step captured by the caller; the library's own launch graph, which a
    repeated call on a stream of its own replays.  Lengths grow from step to step."""
    n = kw["n_seq"]
    prompt = np.random.default_rng(5).integers(0, 1000, (n, 14))
    a, b, c = (Server(dtype=dtype, **kw) for _ in range(3))
    for s in (a, b, c):
        s.prefill(0, prompt)
    eager = []
    for _ in range(7):
        a.step(a.next, window=window, sinks=sinks)
        eager.append(a.got())
    ones, stream = _i32([1] * n), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        G.gpt2_pages_reserve(b.cache, ones, b.ws, b.ws.numel())
        b.step(b.next, window=window, sinks=sinks, reserve=False)
    own = torch.cuda.Stream()
    for ref in eager:
        graph.replay()
        assert np.array_equal(b.got(), ref)
        c.reserve([1] * n)
        torch.cuda.synchronize()
        c.ws.random_(0, 256)
        torch.cuda.synchronize()
        c.step(c.next, window=window, sinks=sinks, reserve=False, stream=own)
        assert np.array_equal(c.got(), ref)
    assert torch.equal(a.lens, b.lens) and torch.equal(a.lens, c.lens)
    assert torch.equal(a.next, b.next) and torch.equal(a.next, c.next)
