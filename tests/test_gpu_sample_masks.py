"""gpt2_sample_tokens on the GPU against float64, on rows with finite masks (the
type's lowest value, -1e9) whose top-p border lies among many tokens.

Ids must be those of float64 arithmetic (weights to 2^-52, sums of up to 2^18 of
them in pairs of 2^-50 or better; the kernel's own bound is 2^-36, which the
random numbers here are not within of a border unless by chance of 1e-6).  Log
probabilities within 1e-5, as documented."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402
from test_gpu_sample import DT, check, uniforms  # noqa: E402

pytestmark = pytest.mark.gpu
TOP_P = [0.9, 0.999, 0.9999, 0.99995, 1 - 2.0 ** -20]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gpt_pre_ln_gb300 import build
    build.build()
    G.lib()
    yield
    st, site = G.gpt2_last_error()
    assert st == 0, f"device error {st} at site {site}"


def low(dtype, what):
    return torch.finfo(DT[dtype][0]).min if what == "lowest" else what


def rows(V, dtype, tail, scale, seed, mask, share):
    """One row per top_p: a tail of exponential or normal logits, or tied ones far below one peak; `share` of them
    (or one alone) at the mask's value."""
    g = np.random.default_rng(seed)
    M = len(TOP_P)
    if tail == "ties":
        z = np.full((M, V), -scale)
        z[:, V // 3] = 0.0
    else:
        z = scale * (g.exponential(size=(M, V)) if tail == "exponential" else g.standard_normal((M, V)))
    z = torch.from_numpy(z.astype(np.float32)).to(DT[dtype][0])
    gone = torch.from_numpy(g.random((M, V)) < share) if share else torch.zeros(M, V, dtype=torch.bool)
    gone[:, V // 2] = True
    gone[:, V // 3] = False
    z[gone] = low(dtype, mask)
    ld = -(-V // 8) * 8
    return torch.nn.functional.pad(z, (0, ld - V), value=float("nan")).cuda()


@pytest.mark.parametrize("share", [0.0, 0.3])
@pytest.mark.parametrize("dtype, V, mask", [("f32", 50257, "lowest"), ("f32", 262144, -1e9), ("bf16", 50257, "lowest"),
                                            ("f16", 50257, -65504.0), ("f16", 262144, -65504.0), ("f32", 50257, -1e4)])
@pytest.mark.parametrize("tail, scale", [("exponential", 1.8), ("normal", 2.0), ("ties", 11.5), ("ties", 25.0)])
def test_finite_masks_and_a_border_among_many(tail, scale, dtype, V, mask, share):
    z = rows(V, dtype, tail, scale, V + len(tail), mask, share)
    for seed in range(2):
        check(z, V, dtype, uniforms(len(TOP_P), seed), top_p=TOP_P)
    check(z, V, dtype, [1 - 2.0 ** -24] * len(TOP_P), top_p=TOP_P)  # the last that stays


@pytest.mark.parametrize("dtype, mask", [("f32", -1e9), ("f16", -65504.0)])
def test_finite_masks_with_top_k_and_min_p(dtype, mask):
    V, M = 50257, len(TOP_P)
    z = rows(V, dtype, "exponential", 1.8, 3, mask, 0.3)
    for top_k in (3000, 20000, 40000, 50257):
        check(z, V, dtype, uniforms(M, top_k), top_p=TOP_P, top_k=[top_k] * M)
        check(z, V, dtype, [1 - 2.0 ** -24] * M, top_p=TOP_P, top_k=[top_k] * M)
    check(z, V, dtype, uniforms(M, 1), top_p=TOP_P, min_p=[1e-5, 1e-6, 1e-4, 1e-7, 1e-8])


@pytest.mark.parametrize("temperature", [2.0 ** -100, 1e-6, 0.01, 30.0, 1e6, 1e9, 2.0 ** 100])
def test_finite_masks_at_other_temperatures(temperature):
    """From rows where the maximum alone counts to those where the mask's own tokens come."""
    V, M = 20000, len(TOP_P)
    for mask in (-1e9, "lowest"):
        z = rows(V, "f32", "normal", 2.0, 9, mask, 0.3)
        check(z, V, "f32", uniforms(M, 4), top_p=TOP_P, temperature=[temperature] * M)
