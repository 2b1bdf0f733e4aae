"""gpt2_sample_tokens on the GPU at the ends of what it promises."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402
from test_gpu_sample import expect, kept, run  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gpt_pre_ln_gb300 import build
    build.build()
    G.lib()
    yield
    st, site = G.gpt2_last_error()
    assert st == 0, f"device error {st} at site {site}"


# ---- clusters
def _cluster_logits(one, share_sign):
    """Logits whose weight counts a whole step too much (share_sign 1) or too little of `one` where
    2^(b / 64) t is rounded to whole numbers twice (b the bin of t = z log2 e)."""
    z = -np.random.default_rng(1).uniform(0.3, 1.2, 400000).astype(np.float32)
    t = (z.astype(np.float64) * math.log2(math.e)).astype(np.float32).astype(np.float64)
    b = np.rint(-64 * t)
    unit = float(np.float32(np.float32(0.010830424696249145) * np.float32(one)))
    n = np.rint(np.rint(b * unit + one) + t * 64 * unit)
    over = n / one * 2.0 ** (-b / 64) / 2.0 ** t - 1
    return z[np.argsort(-share_sign * over)[:4]]


@pytest.mark.parametrize("V, one", [(1 << 21, 512), (150000, 8192), (65536, 16384)])
@pytest.mark.parametrize("sign", [1, -1])
def test_a_border_behind_a_cluster(V, one, sign):
    """A thousand equal logits with most of the weight, whose share the histogram of whole numbers misses by as much as
    it can, and the border of top_p behind them.  Wrongly kept tokens show in the log probability."""
    g = np.random.default_rng(7)
    n_tail, M = 12000, 48
    for zc in _cluster_logits(one, sign):
        ids = np.sort(g.permutation(V)[:1001 + n_tail])
        place = g.permutation(1001 + n_tail)
        x = np.empty(1001 + n_tail, np.float32)
        x[place[0]], x[place[1:1001]] = 0.0, zc
        w_c = math.exp(float(zc))
        tail = -3.0 * g.random(n_tail)
        x[place[1001:]] = tail + math.log(1000 * w_c * 0.06 / np.exp(tail).sum())
        w = np.exp(x.astype(np.float64))
        ahead = (1 + 1000 * w_c) / w.sum()
        top_p = (ahead + g.uniform(1e-4, 0.99 * (1 - ahead), M)).astype(np.float32)
        u = np.where(np.arange(M) % 4 == 0, 1 - 2.0 ** -24, g.random(M)).astype(np.float32)
        z = torch.full((V,), -math.inf, device="cuda")
        z[torch.from_numpy(ids).cuda()] = torch.from_numpy(x).cuda()
        tok, lp = run(z.expand(M, -1).contiguous(), V, "f32", u, top_p=top_p)
        for m in range(M):
            want, ref = expect(x.astype(np.float64), float(u[m]), top_p=float(top_p[m]))
            assert tok[m] == ids[want], (float(zc), m, tok[m], ids[want], float(top_p[m]))
            assert abs(lp[m] - ref) <= 1e-5, (float(zc), m, lp[m], ref, float(top_p[m]))


# ---- the very borders
def _neighbours(z, V, u, left, **kw):
    """Rows drawn with numbers next to the end of token left[m]'s share: the token is that one or the next one kept, and
    the log probability its own."""
    full = {k: np.full(len(u), v, np.int32 if k == "top_k" else np.float32) for k, v in kw.items()}
    tok, lp = run(z, V, "f32", u, **full)
    x = z[:, :V].double().cpu().numpy()
    for m in range(len(u)):
        ids, w = kept(x[m], **{k: np.float32(v).item() if k != "top_k" else v for k, v in kw.items()})
        at = int(np.searchsorted(ids, left[m]))
        assert tok[m] in ids[at:at + 2], (m, tok[m], ids[at:at + 2])
        ref = math.log(w[np.searchsorted(ids, tok[m])] / w.sum())
        assert abs(lp[m] - ref) <= 1e-5, (m, lp[m], ref)


def test_each_row_belongs_to_one_token():
    """Rows of 512 whose target falls between two sums that differ only by their roundings (found by trying 4e8)."""
    V = 512
    cases = [(261, 42, 0.8920871019363403, 435), (177, 5147, 0.26442840695381165, 113),
             (187, 8942, 0.03250562772154808, 30), (703, 12524, 0.9267133474349976, 479),
             (316, 15120, 0.9688754081726074, 470)]
    rows = [2 * np.random.default_rng(s).standard_normal((m + 1, V), dtype=np.float32)[m] for s, m, _, _ in cases]
    _neighbours(torch.from_numpy(np.stack(rows)).cuda(), V, np.float32([c[2] for c in cases]), [c[3] for c in cases],
                top_k=256)


@pytest.mark.parametrize("V, kw", [(512, dict(top_k=256)), (300, {}), (5000, dict(top_k=200)),
                                   (30011, dict(top_p=0.9)), (30011, {}), (50257, dict(top_p=0.2))])
def test_the_fp32_numbers_nearest_to_borders(V, kw):
    """However near: either neighbour will do, but one of them it has to be."""
    g = np.random.default_rng(V)
    x = 1.5 * g.standard_normal(V, dtype=np.float32)
    ids, w = kept(x.astype(np.float64), **{k: np.float32(v).item() if k != "top_k" else v for k, v in kw.items()})
    part = np.cumsum(w) / w.sum()
    dist = np.abs(part[:-1].astype(np.float32).astype(np.float64) - part[:-1])
    at = np.argsort(dist)[:400]
    u = part[at].astype(np.float32)
    at, u = at[u < 1], u[u < 1]
    z = torch.nn.functional.pad(torch.from_numpy(x), (0, -V % 4)).cuda().expand(len(u), -1).contiguous()
    _neighbours(z, V, u, ids[at], **kw)


# ---- min_p and the ends of the temperatures
def test_min_p_goes_by_the_temperature_that_counts():
    """Temperatures below 2^-100 and above 2^100 count as these, for min_p too."""
    hi, lo = 2.0 ** 100, 2.0 ** -100
    z = np.zeros((6, 8), np.float32)
    z[:, 1:] = -np.inf
    z[0, 3] = z[1, 3] = z[2, 3] = -hi  # weights e^-1
    z[3, 3] = z[4, 3] = z[5, 3] = -0.5 * lo  # e^-0.5
    t = [2.0 ** 127, 2.0 ** 101, hi, 1e-38, 2.0 ** -101, lo]
    u = [0.95] * 6
    for min_p, stays in ((0.5, [0, 0, 0, 1, 1, 1]), (0.3, [1] * 6), (0.7, [0] * 6)):
        tok, lp = run(torch.from_numpy(z).cuda(), 8, "f32", u, temperature=t, min_p=[min_p] * 6)
        for m in range(6):
            w = math.exp(-1.0 if m < 3 else -0.5)
            assert tok[m] == (3 if stays[m] else 0), (min_p, m)
            assert abs(lp[m] - (math.log(w / (1 + w)) if stays[m] else 0.0)) <= 1e-5


# ---- many equal tokens far below the maximum
@pytest.mark.parametrize("z_tail", [-24.97173, -25.3, -26.7, -28.123, -31.0])
def test_two_million_equal_tokens_far_below_the_maximum(z_tail):
    """The random number falls into the share of 2^21 - 1 equal tokens; the largest weight has the last id.  Their prefix
    sums are multiples of one weight, so that the id is a quotient; the documented bound is 2^-36 of the row's weight."""
    V = 1 << 21
    z = np.full(V, np.float32(z_tail), np.float32)
    z[-1] = 0.0
    w = math.exp(float(np.float32(z_tail)))
    total = 1.0 + (V - 1) * w
    us = np.float32([f * (V - 1) * w / total for f in (0.05, 0.2, 0.35, 0.5, 0.65, 0.8, 0.9, 0.97)])
    tok, _ = run(torch.from_numpy(z).cuda().expand(len(us), -1).contiguous(), V, "f32", us)
    for m, u in enumerate(us):
        at = float(u) * total / w  # the id is its whole part
        off = max(0.0, tok[m] - at, at - (tok[m] + 1)) * w / total
        assert off <= 2.0 ** -36, (m, tok[m], at, math.log2(off))


# ---- log probabilities
def test_log_probabilities_of_unlikely_tokens():
    """u = 0 draws the lowest id, however small its share.  Half a step of the result, one of the logarithm of the sum
    (below 4), and sums of two floats."""
    M, V = 4096, 40
    g = np.random.default_rng(8)
    z = (0.5 * g.standard_normal((M, V))).astype(np.float32)
    z[:, 0] = -g.uniform(20, 66, M).astype(np.float32)
    tok, lp = run(torch.from_numpy(z).cuda(), V, "f32", np.zeros(M, np.float32))
    for m in range(M):
        want, ref = expect(z[m].astype(np.float64), 0.0)
        assert tok[m] == want == 0
        step = 2.0 ** (math.floor(math.log2(-ref)) - 23)
        assert abs(lp[m] - ref) <= step / 2 + 2.0 ** -22 + 2.0 ** -30, (m, lp[m], ref)


def test_log_probabilities_where_the_border_is_close():
    """top_p's border is the nearest fp32 number to a token's, or a neighbour of that, and the token has 0.97e-5 to 1e-5
    of the kept weight: fp32 sums may take it for the other side's."""
    V, n, heavy, M = 65536, 50000, 10, 3000
    g = np.random.default_rng(11)
    for _ in range(8):
        z = np.full(V, -np.inf, np.float32)
        ids = g.permutation(V)
        z[ids[:heavy]] = 0.0
        z[ids[heavy:heavy + n]] = (math.log(heavy / n) - 0.05 + 0.1 * g.random(n)).astype(np.float32)
        ranked = np.sort(z.astype(np.float64))[::-1][:n + heavy]
        part = np.concatenate([[0.0], np.cumsum(np.exp(ranked))])
        share = np.diff(part) / part[1:]
        at = part[1:-1][(share[1:] > 0.97e-5) & (share[1:] < 1e-5)] / part[-1]
        p = at.astype(np.float32)
        p = np.concatenate([p, np.nextafter(p, np.float32(0)), np.nextafter(p, np.float32(2))])
        p = p[g.permutation(len(p))[:M]]
        u = g.random(len(p), dtype=np.float32)
        tok, lp = run(torch.from_numpy(z).cuda().expand(len(p), -1).contiguous(), V, "f32", u, top_p=p)
        count = np.searchsorted(part[:-1], p.astype(np.float64) * part[-1], side="left")
        ref = z[tok].astype(np.float64) - np.log(part[count])
        assert (np.abs(lp - ref) <= 1e-5).all(), np.abs(lp - ref).max()


# ---- the same calls
@pytest.mark.parametrize("V", [3000, 50257])
def test_equal_calls_give_equal_bits(V):
    """Rows with 150 to 400 tokens ahead of top_p's border, some listed and some summed by parts, and rows alike."""
    M = 1500
    g = np.random.default_rng(V)
    x = (1.8 * g.exponential(size=(M // 3, V))).astype(np.float32)
    x = np.concatenate([x, x, x])
    w = np.sort(np.exp(x.astype(np.float64) - x.max(1, keepdims=True)), 1)[:, ::-1]
    part = np.cumsum(w, 1) / w.sum(1, keepdims=True)
    n = np.tile(g.integers(150, 400, M // 3), 3)
    p = part[np.arange(M), n].astype(np.float32)
    u = np.tile(g.random(M // 3, dtype=np.float32), 3)
    z = torch.nn.functional.pad(torch.from_numpy(x), (0, -V % 4)).cuda()
    first, lp = run(z, V, "f32", u, top_p=p)
    assert (first.reshape(3, -1) == first[:M // 3]).all() and (lp.reshape(3, -1) == lp[:M // 3]).all()
    for _ in range(5):
        tok, again = run(z, V, "f32", u, top_p=p)
        assert (tok == first).all() and (again == lp).all()
