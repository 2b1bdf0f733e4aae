"""Long streams under a sliding window on the GPU, their pages given back as
they go by the header's rule for gpt2_pages_free: keep_first = sinks,
keep_last = max(window - 1, 1).

What is compared is equal bit for bit: the pages that go hold nothing that a
later query sees, so the logits may not change."""
import pathlib
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402
from test_gpu_paged_model import Server, _i32  # noqa: E402


@pytest.fixture(scope="module")
def built():
    from gpt_pre_ln_gb300 import build
    build.build()
    G.lib()
    yield
    st, site = G.gpt2_last_error()
    assert st == 0, f"device error {st} at site {site}"


def rule(window, sinks):
    return sinks, max(window - 1, 1)


def test_the_header_gives_this_rule():
    text = (pathlib.Path(__file__).resolve().parent.parent / "include" / "gpt2gb.h").read_text()
    assert "keep_first = sinks and keep_last = max(window - 1, 1)" in re.sub(r"\s*\n \* ?", " ", text)


@pytest.mark.parametrize("window", [1, 2, 3, 16, 17, 1000])
@pytest.mark.parametrize("sinks", [0, 1, 16])
def test_the_rule_never_ends_a_sequence_and_keeps_what_is_seen(window, sinks):
    first, last = rule(window, sinks)
    assert (first, last) != (0, 0) and first >= 0 and last >= 0
    for n in (0, 1, 15, 16, 40, 1200):  # cached positions; the new token is the n-th
        seen = {p for p in range(n) if p >= n + 1 - window or p < sinks}
        assert seen <= {p for p in range(n) if p < first or p >= n - last}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [G.BF16, G.F16])
@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (2, 0), (2, 17), (16, 0), (17, 3), (40, 0)])
def test_streams_whose_pages_are_given_back(window, sinks, dtype, built):
    g = np.random.default_rng(window)
    prompt = g.integers(0, 1000, (2, 14))  # page borders at the second and at later steps
    toks = [_i32(g.integers(0, 1000, 2).tolist()) for _ in range(36)]
    first, last = rule(window, sinks)
    kept, trimmed = Server(2, dtype=dtype), Server(2, dtype=dtype)
    for s in (kept, trimmed):
        s.prefill(0, prompt)
    for i, t in enumerate(toks):
        kept.step(t, window=window, sinks=sinks)
        trimmed.step(t, window=window, sinks=sinks)
        G.gpt2_pages_free(trimmed.cache, _i32([0, 1]), 2, first, last)
        assert np.array_equal(kept.got(), trimmed.got()), i
        assert trimmed.lens.cpu().tolist() == [15 + i] * 2
        held = (trimmed.table >= 0).sum(1).cpu().tolist()
        assert max(held) <= -(-sinks // 16) + -(-last // 16) + 1
    G.gpt2_pages_free(trimmed.cache, _i32([0, 1]), 2)
    torch.cuda.synchronize()
    assert int(trimmed.refs.abs().sum()) == 0 and trimmed.lens.cpu().tolist() == [-1, -1]
