"""gpt2_sample_tokens on the GPU at the ends of what it promises."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402
from test_gpu_sample import expect, run  # noqa: E402

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
