"""gpt2_sample_tokens on the GPU against float64.

Ids must be those of float64 arithmetic.  Its sums of at most 2^21 weights are
good to 2^-50 of the row's weight, and the random numbers here are fp32 numbers,
some of them the nearest to a border: a border's own rounding to fp32 leaves
2^-25 of it, so the two sides of a border that the nearest fp32 numbers fall on are
told apart unless the border is within 2^-36 of one (the kernel's own bound);
such numbers are left out of the borders' test.  Log probabilities: 2^-24 of
themselves, a rounded logarithm of the sum (2^-22) and its sum (4e-6): 1e-5 in all
as documented, for |log p| up to 60."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"f32": (torch.float32, G.F32), "bf16": (torch.bfloat16, G.BF16), "f16": (torch.float16, G.F16)}
RANGE = 6


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gpt_pre_ln_gb300 import build
    build.build()
    G.lib()
    yield
    st, site = G.gpt2_last_error()
    assert st == 0, f"device error {st} at site {site}"


def kept(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Ids that a row keeps, in their order, and their weights.  z float64."""
    order = np.argsort(-z, kind="stable")
    if temperature == 0:
        return order[:1], np.ones(1)
    t = min(max(temperature, 2.0 ** -100), 2.0 ** 100)
    d = z[order] - z[order[0]]
    w = np.exp(d / t)
    n = min(top_k, len(z)) if top_k else len(z)
    if top_p < 1:
        part = np.concatenate([[0.0], np.cumsum(w[:n])])
        n = max(1, int((part[:-1] < top_p * part[-1]).sum()))
    if min_p > 0:
        n = max(1, min(n, int((d >= temperature * math.log(min_p)).sum())))
    ids = np.sort(order[:n])
    return ids, np.exp((z[ids] - z[order[0]]) / t)


def expect(z, u, **kw):
    ids, w = kept(z, **kw)
    part = np.cumsum(w)
    at = min(int(np.searchsorted(part, u * part[-1], side="right")), len(ids) - 1)
    return int(ids[at]), math.log(w[at] / part[-1]) if w[at] > 0 else -math.inf


def run(z, V, dtype, u, temperature=None, top_k=None, top_p=None, min_p=None, logprob=True, stream=None):
    """z [M, ld] on the GPU; settings as lists, arrays or None."""
    M, ld = z.shape
    f = lambda v: None if v is None else torch.tensor(np.asarray(v, np.float32)).cuda()  # noqa: E731
    k = None if top_k is None else torch.tensor(np.asarray(top_k, np.int32)).cuda()
    tok = torch.full((M,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((M,), 7.0, device="cuda")
    keep = [f(temperature), k, f(top_p), f(min_p), f(u)]
    G.gpt2_sample_tokens(z, ld, DT[dtype][1], M, V, *keep, tok, lp if logprob else None, stream)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), lp.cpu().numpy().astype(np.float64)


def check(z, V, dtype, u, **kw):
    tok, lp = run(z, V, dtype, u, **kw)
    x = z[:, :V].double().cpu().numpy()
    for m in range(len(u)):
        one = {k: (np.float32(v[m]).item() if k != "top_k" else int(v[m])) for k, v in kw.items() if v is not None}
        want, wlp = expect(x[m], float(np.float32(u[m])), **one)
        assert tok[m] == want, (m, tok[m], want, one, float(u[m]))
        assert abs(lp[m] - wlp) <= 1e-5, (m, lp[m], wlp)


def logits(M, V, dtype, seed=0, scale=2.5, kind="normal"):
    g = np.random.default_rng(seed)
    ld = -(-V // 8) * 8 + 8
    z = np.full((M, ld), np.nan, np.float32)  # what stands behind the vocabulary must not count
    z[:, :V] = scale * (g.standard_normal((M, V)) if kind == "normal" else g.exponential(size=(M, V)))
    return torch.from_numpy(z).to(DT[dtype][0]).cuda()


def uniforms(M, seed=0):
    return np.random.default_rng(seed + 99).random(M, dtype=np.float32)


def settings(M, seed=0):
    g = np.random.default_rng(seed + 7)
    pick = lambda p, on, off: np.where(g.random(M) < p, on, off)  # noqa: E731
    return dict(temperature=pick(0.1, 0.0, g.uniform(0.3, 2.0, M)).astype(np.float32),
                top_k=pick(0.4, g.integers(1, 400, M), 0).astype(np.int32),
                top_p=pick(0.5, g.uniform(0.05, 0.999, M), 1.0).astype(np.float32),
                min_p=pick(0.3, g.uniform(0.001, 0.3, M), 0.0).astype(np.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 33, 127, 513, 4096, 4097, 8192, 8193, 28000, 50257])
def test_sizes(V, dtype):
    M = 24
    check(logits(M, V, dtype, seed=V), V, dtype, uniforms(M, V), **settings(M, V))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", [{}, dict(top_p=0.9), dict(top_k=50), dict(min_p=0.05), dict(top_p=0.999),
                                  dict(top_k=3000), dict(top_k=1000, top_p=0.95), dict(temperature=0.0),
                                  dict(temperature=0.2, top_p=0.5), dict(temperature=20.0, top_p=0.7),
                                  dict(top_p=1 - 2.0 ** -24), dict(top_p=1e-6), dict(top_k=1), dict(top_p=0.0)])
def test_each_setting(dtype, what):
    M, V = 64, 10007
    kw = {k: np.full(M, v, np.int32 if k == "top_k" else np.float32) for k, v in what.items()}
    for kind in ("normal", "exponential"):
        check(logits(M, V, dtype, seed=5, scale=1.3, kind=kind), V, dtype, uniforms(M, 3), **kw)


@pytest.mark.parametrize("dtype, V", [("f32", 60001), ("bf16", 120001), ("f32", 200003), ("f16", 300000),
                                      ("bf16", 1 << 21), ("f32", 1 << 21)])
def test_large_vocabularies(dtype, V):
    M = 5
    check(logits(M, V, dtype, seed=1), V, dtype, uniforms(M, V), temperature=[1.0, 0.7, 1.0, 3.0, 0.0],
          top_p=[1.0, 0.9, 0.99, 0.6, 1.0], top_k=[0, 0, 5000, 0, 0])


@pytest.mark.parametrize("dtype, V", [("f32", 53000), ("f32", 53500), ("f32", 25600), ("f32", 25610), ("bf16", 51100),
                                      ("bf16", 51300), ("bf16", 106000), ("bf16", 107500), ("f32", 54000)])
def test_each_side_of_the_kernels_borders(dtype, V):
    M = 6
    check(logits(M, V, dtype, seed=V), V, dtype, uniforms(M, V), **settings(M, V))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kw", [{}, dict(top_p=0.9), dict(top_k=700)])
@pytest.mark.parametrize("V", [300, 30011])
def test_random_numbers_next_to_a_border(dtype, kw, V):
    """The nearest fp32 numbers to the border between two tokens' shares, and their neighbours."""
    z = logits(1, V, dtype, seed=V, scale=1.5)
    x = z[0, :V].double().cpu().numpy()
    ids, w = kept(x, **kw)
    part = np.cumsum(w) / w.sum()
    g = np.random.default_rng(1)
    us = []
    for i in g.integers(0, len(ids) - 1, 200):
        u = np.float32(part[i])
        us += [v for v in (u, np.nextafter(u, np.float32(0)), np.nextafter(u, np.float32(2)))
               if 0 <= v < 1 and np.abs(part - float(v)).min() > 2.0 ** -35]
    full = {k: np.full(len(us), v, np.int32 if k == "top_k" else np.float32) for k, v in kw.items()}
    check(z.expand(len(us), -1).contiguous(), V, dtype, us, **full)


@pytest.mark.parametrize("V", [4, 1000, 5000, 50257])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_logits(V, dtype):
    """Every weight is 1: sums are whole numbers and borders are met exactly; a list of them does not fit one round."""
    M = 12
    z = torch.full((M, -(-V // 8) * 8), 3.0, dtype=DT[dtype][0], device="cuda")
    u = [0.0, 0.5, 0.25, 0.75, 1 - 2.0 ** -24, 1 / 3, 0.0, 0.5, 0.9, 0.125, 0.5, 0.999]
    check(z, V, dtype, u)
    check(z, V, dtype, u, top_p=[0.5, 0.25, 0.75, 0.5, 0.5, 0.3, 1e-9, 0.125, 0.9, 0.99, 0.0, 1.0])
    check(z, V, dtype, u, top_k=[1, 2, 3, V // 2, V, V - 1, 2 * V, 600, 1025, 0, V // 3 + 1, 513])
    check(z, V, dtype, u, min_p=[1.0] * 12, top_k=[700] * 12, top_p=[0.5] * 12)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_few_values(dtype):
    """Thousands of ties on either side of a border, 0 of both signs among them."""
    g = np.random.default_rng(2)
    M, V = 40, 20000
    z = torch.from_numpy(g.choice(np.float32([-2, -1, -0.0, 0.0, 0.5, 0.75]), (M, V))).to(DT[dtype][0]).cuda()
    s = settings(M, 4)
    s["top_k"] = np.where(s["top_k"] > 0, s["top_k"] * 40, 0).astype(np.int32)
    check(z, V, dtype, uniforms(M, 1), **s)


def test_crowded_values():
    """fp32 logits that differ in their last bits: 20000 of them in one bin of the first histogram."""
    g = np.random.default_rng(3)
    M, V = 16, 20000
    z = torch.from_numpy((7 + 1e-5 * g.standard_normal((M, V))).astype(np.float32)).cuda()
    check(z, V, "f32", uniforms(M, 2), top_k=g.integers(1, V, M).astype(np.int32))
    check(z, V, "f32", uniforms(M, 2), top_p=g.uniform(0.1, 0.99, M).astype(np.float32))


@pytest.mark.parametrize("V", [20000, 1 << 20])
def test_tails_far_below_the_maximum(V):
    """The border of top_p lies among tokens of 2^-30 and less of the maximum's weight."""
    g = np.random.default_rng(4)
    z = (-(20.0 + 12.0 * g.random((4, V)))).astype(np.float32)
    z[:, 5] = 0.0
    z[2:, 77] = -20.5
    for p in (1 - 2.0 ** -24, 1 - 2.0 ** -22, 1 - 2.0 ** -20, 1 - 2.0 ** -16):
        check(torch.from_numpy(z).cuda(), V, "f32", [1 - 2.0 ** -24, 0.3, 1 - 2.0 ** -23, 0.99999],
              top_p=np.full(4, p, np.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_masks(dtype):
    """-inf and the type's lowest value never come, unless nothing else is there."""
    M, V = 30, 5000
    z = logits(M, V, dtype, seed=6)
    gone = torch.rand(M, V, device="cuda") < 0.95
    z[:, :V][gone] = -math.inf
    z[:10, :V][gone[:10]] = torch.finfo(z.dtype).min
    z[:, 3] = 1.0
    s = settings(M, 3)
    check(z, V, dtype, uniforms(M, 1), **s)
    check(z, V, dtype, np.full(M, 0.0, np.float32))
    check(z, V, dtype, np.full(M, 1 - 2.0 ** -24, np.float32))
    alone = torch.full((2, 5000), -math.inf, dtype=z.dtype, device="cuda")
    alone[0, 4999] = -5.0
    alone[1, 0] = torch.finfo(z.dtype).min
    check(alone, V, dtype, [0.7, 0.2], top_k=[50, 50], top_p=[0.9, 0.9])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_without_a_distribution(dtype):
    z = logits(5, 700, dtype, seed=1)
    z[0, 699] = math.nan
    z[1, 0] = math.inf
    z[2, :700] = -math.inf
    z[3, 5] = -math.nan
    tok, lp = run(z, 700, dtype, uniforms(5), top_k=[0, 5, 0, 0, 0])
    assert tok[:4].tolist() == [-1] * 4 and np.isnan(lp[:4]).all() and tok[4] >= 0 and lp[4] < 0
    tok, lp = run(z, 700, dtype, uniforms(5), temperature=[0.0] * 5)
    assert tok[:4].tolist() == [-1] * 4 and np.isnan(lp[:4]).all() and tok[4] == int(z[4, :700].float().argmax())


@pytest.mark.parametrize("bad", [dict(temperature=-1.0), dict(temperature=math.nan), dict(temperature=math.inf),
                                 dict(top_k=-1), dict(top_p=-0.1), dict(top_p=math.nan), dict(min_p=-0.1),
                                 dict(min_p=1.5), dict(min_p=math.nan), dict(u=1.0), dict(u=-0.1), dict(u=math.nan)])
def test_settings_out_of_range(bad):
    z = logits(3, 700, "bf16", seed=1)
    kw = dict(u=[0.5] * 3, temperature=[1.0] * 3, top_k=[0] * 3, top_p=[1.0] * 3, min_p=[0.0] * 3)
    for k, v in bad.items():
        kw[k] = [kw[k][0], v, kw[k][0]]
    tok, lp = run(z, 700, "bf16", **kw)
    assert tok[1] == -1 and np.isnan(lp[1]) and (tok[[0, 2]] >= 0).all()
    assert G.gpt2_last_error() == (RANGE, 30)


def test_extreme_numbers():
    """Logits near the ends of fp32 and temperatures near those of the clamps."""
    big = np.float32(3e38)
    z = np.zeros((8, 8), np.float32)
    z[0] = [big, -big, 0, big, -big, 1, 2, 3]
    z[1] = z[0]
    z[2] = [1e-38, 2e-38, 0, -1e-38, 3e-38, 0, 0, 1e-45]
    z[3] = [1, 1, 1 - 2.0 ** -24, 1, 0, 0, 0, 0]
    z[4] = [5, 4, 3, 2, 1, 0, -1, -2]
    z[5], z[6], z[7] = z[4], z[4], z[4]
    t = [1.0, 1e38, 1e-38, 1e-30, 1e30, 1e-45, 3e38, 2.0 ** -100]
    for u in (0.1, 0.6, 0.95):
        check(torch.from_numpy(z).cuda(), 8, "f32", [u] * 8, temperature=t)
        check(torch.from_numpy(z).cuda(), 8, "f32", [u] * 8, temperature=t, top_p=[0.8] * 8)


def test_defaults_and_what_is_left_out():
    z = logits(50, 3000, "bf16", seed=9)
    u = uniforms(50)
    a, la = run(z, 3000, "bf16", u)
    b, lb = run(z, 3000, "bf16", u, temperature=np.ones(50), top_k=np.zeros(50), top_p=np.ones(50), min_p=np.zeros(50))
    c, lc = run(z, 3000, "bf16", u, logprob=False)
    assert (a == b).all() and (la == lb).all() and (a == c).all() and (lc == 7.0).all()


@pytest.mark.parametrize("V", [2000, 50257])
def test_many_rows_twice(V):
    """Equal results of equal calls, on another stream too, and on rows of a wider array."""
    M = 700
    z, s, u = logits(M, V, "bf16", seed=3, scale=1.0), settings(M, 2), uniforms(M, 5)
    a, la = run(z, V, "bf16", u, **s)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    b, lb = run(z, V, "bf16", u, stream=st, **s)
    wide = torch.zeros(M, z.shape[1] + 24, dtype=z.dtype, device="cuda")
    wide[:, :z.shape[1]] = z
    c, lc = run(wide, V, "bf16", u, **s)
    assert (a == b).all() and (a == c).all() and (la == lb).all() and (la == lc).all()
    pick = np.random.default_rng(1).permutation(M)[:60]
    check(z[torch.from_numpy(pick).cuda()], V, "bf16", u[pick], **{k: v[pick] for k, v in s.items()})


def test_captured_and_replayed():
    M, V = 9, 5000
    z, u = logits(M, V, "f32", seed=3), torch.rand(M, device="cuda")
    tok = torch.zeros(M, dtype=torch.int32, device="cuda")
    p = torch.full((M,), 0.9, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = lambda: G.gpt2_sample_tokens(z, z.shape[1], G.F32, M, V, None, None, p, None, u, tok)  # noqa: E731
    with torch.cuda.stream(s):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    for seed in range(3):
        torch.cuda.synchronize()
        z.copy_(logits(M, V, "f32", seed=50 + seed))
        u.copy_(torch.from_numpy(uniforms(M, seed)))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        x = z[:, :V].double().cpu().numpy()
        assert tok.tolist() == [expect(x[m], float(u[m]), top_p=float(np.float32(0.9)))[0] for m in range(M)]


def test_shares_of_many_draws():
    """65536 draws from one row: each token's count is within 6 standard deviations of its share."""
    M, V = 65536, 40
    row = logits(1, V, "f32", seed=2, scale=1.0)
    u = (np.arange(M, dtype=np.float64) + 0.5) / M
    tok, _ = run(row.expand(M, -1).contiguous(), V, "f32", u.astype(np.float32), temperature=np.full(M, 0.8))
    ids, w = kept(row[0, :V].double().cpu().numpy(), temperature=float(np.float32(0.8)))
    count = np.bincount(tok, minlength=V)
    assert np.abs(count - M * w / w.sum()).max() <= 1.5  # evenly spaced numbers: off by the two ends of a share


def test_log_probabilities_of_shares_near_one():
    # 20 tokens, 7 below the largest: the others' weight is 0.0009 to 0.02.  The sums of two floats are off by 2^-36,
    # the logarithm, the exponent and its product by two steps of 2^-23 each.
    V, M = 20, 8
    g = np.random.default_rng(5)
    z = torch.from_numpy((g.standard_normal((M, V)) * 0.3 - 7).astype(np.float32))
    z[torch.arange(M), torch.arange(M)] = 0.0
    z[:, 10:] -= torch.linspace(0, 3, M)[:, None]
    tok, lp = run(z.cuda(), V, "f32", [0.5] * M)[:2]
    for m in range(M):
        t, ref = expect(z[m].double().numpy(), 0.5)
        assert int(tok[m]) == t == m
        assert abs(float(lp[m]) - ref) <= 2 ** -20 * abs(ref), (m, float(lp[m]), ref)
