"""The sums of gpt2_token_logprobs where the order of additions shows: a few
large terms that each thread meets first, then thousands of terms below half the
last place of one.  Added one after another to the large ones they would all
be lost (1.7e-5 of the sum).  The tolerance is the one that the other tests of the
scores derive: V / 512 + 40 roundings one after another."""
import pytest

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402,F401
from test_gpu_logprobs import DT, _built, _check  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype, M, V, top", [
    ("bf16", 400, 20480, 0.0), ("f16", 400, 20480, 0.0), ("f32", 400, 10240, 0.0),  # a warp per row
    ("bf16", 3, 4088, 0.0), ("f32", 3, 2044, 0.0),
    ("f32", 400, 10240, 61000.0), ("f32", 400, 10240, -61000.0),  # far out, where the kernel sums another way
    ("bf16", 3, 50257, 0.0), ("f32", 3, 50257, 0.0), ("f32", 3, 50257, 61000.0)])  # a CTA per row
def test_small_terms_behind_large_ones_are_not_lost(dtype, M, V, top):
    n = 16 // DT[dtype][0].itemsize  # logits that a thread takes at a time
    z = torch.full((M, -(-V // 8) * 8), top - 16.75, dtype=DT[dtype][0], device="cuda")
    for v in range(32):  # one for each of the two sums that a thread may keep
        z[:, v * n:v * n + 2] = top
    _check(z, V, dtype, 5)
