"""The largest vocabulary of gpt2_token_logprobs: one limit in the header and
in the code, checked before anything is launched (no GPU needed)."""
import pathlib

import pytest

import gpt_pre_ln_gb300 as G

UNSUPPORTED = 2
LIMIT = 1 << 21


@pytest.fixture(scope="module")
def L():
    from gpt_pre_ln_gb300 import build
    build.build()
    return G.lib()


@pytest.mark.parametrize("dtype", [G.F32, G.BF16, G.F16])
def test_vocabularies_beyond_the_limit_are_refused(L, dtype):
    def call(V):
        # no rows: nothing is launched, but the sizes are checked
        return L.gpt2_token_logprobs(256, (V + 7) // 8 * 8, dtype, 0, V, 256, 256, 256, 256, 5, 256, 256, None)

    assert call(LIMIT) == 0
    for V in (LIMIT + 1, 10 * LIMIT, 2 ** 31 - 17):
        assert call(V) == UNSUPPORTED, V


def test_the_header_names_the_limit():
    assert "V <= 2^21" in (pathlib.Path(__file__).resolve().parent.parent / "include" / "gpt2gb.h").read_text()
