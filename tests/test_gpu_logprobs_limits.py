"""gpt2_token_logprobs at its largest vocabulary on the GPU, with the rows that
take it longest: thousands of distinct likely tokens in few threads' parts, so
that the alternatives come from passes over the row, and several such rows to
each CTA, whose warps wait for one another.  No wait may run out."""
import pytest

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402

pytestmark = pytest.mark.gpu
V = 1 << 21
TOP = 32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gpt_pre_ln_gb300 import build
    build.build()
    G.lib()
    yield
    st, site = G.gpt2_last_error()
    assert st == 0, f"device error {st} at site {site}"


@pytest.mark.parametrize("M", [1, 700])
def test_rows_that_are_ranked_by_passes(M):
    g = torch.Generator(device="cuda").manual_seed(M)
    base = torch.randn((2, V), device="cuda", generator=g)
    # every 128th vector of four logits: however the row is cut into runs of whole warps, few threads hold them
    tall = (torch.arange(V, device="cuda") // 4) % 128 == 3
    base[:, tall] += 20 + 10 * torch.rand((2, int(tall.sum())), device="cuda", generator=g)
    z = base.repeat(-(-M // 2), 1)[:M].contiguous()
    ids = torch.zeros((M, TOP), dtype=torch.int32, device="cuda")
    lps, lse = torch.zeros((M, TOP), device="cuda"), torch.zeros(M, device="cuda")
    G.gpt2_token_logprobs(z, V, G.F32, M, V, None, None, None, lse, TOP, ids, lps)
    torch.cuda.synchronize()
    assert G.gpt2_last_error()[0] == 0
    ref_ids = torch.sort(base, dim=1, descending=True, stable=True)[1][:, :TOP]
    d = base.double() - base.amax(1, keepdim=True)
    S = d.exp().sum(1)
    ref_lse, D = base.amax(1) + S.log(), (d.exp() * -d).sum(1) / S
    for k in range(min(M, 2)):
        assert (ids[k::2] == ref_ids[k].int()).all()
        # as for smaller rows: V / 512 + 40 roundings of the sum, the exponentials, the result's own
        tol = (V / 512 + 40) * 2.0 ** -24 + 2.0 ** -22 * (1 + D[k]) + 2.0 ** -22 * ref_lse[k]
        assert ((lse[k::2].double() - ref_lse[k]).abs() <= tol).all()
