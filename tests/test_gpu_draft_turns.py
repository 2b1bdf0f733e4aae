"""gpt2_attention_paged_draft on the GPU where each CTA takes many short items one
after another: the slots of its ring hold tiles with drafted tokens, which lanes
copy, and whole tiles of a page, which the TMA unit brings, in turn.  Bounds as in
test_gpu_draft_attention.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402
from test_gpu_draft_attention import Case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gpt_pre_ln_gb300 import build
    build.build()
    G.lib()
    yield
    st, site = G.gpt2_last_error()
    assert st == 0, f"device error {st} at site {site}"


def check(c):
    """Case.check's bounds for whole sequences at a time."""
    torch.cuda.synchronize()
    info, group = torch.finfo(c.out.dtype), c.heads // c.kv
    out = c.out.view(len(c.lens_l), c.T, -1)[:, :, :c.heads * 64].double()
    left = torch.ones(len(c.lens_l), c.T, dtype=torch.bool, device="cuda")
    for b, n, count in c.live:
        left[b, :count] = False
        both = lambda cache, new: torch.cat([cache[b], new[b, :count]]).cuda().double().repeat_interleave(group, 1)  # noqa: E731,E501
        k, v, q = both(c.kc, c.kn), both(c.vc, c.vn), c.q[b, :count].cuda().double()
        seen = torch.zeros(count, n + count, dtype=torch.bool)
        for t in range(count):
            seen[t, c.seen[b, t]] = True
        seen = seen.cuda()[:, None]
        p = torch.softmax((c.scale * torch.einsum("thd,phd->thp", q, k)).masked_fill(~seen, -torch.inf), 2)
        A = (c.scale * torch.einsum("thd,phd->thp", q.abs(), k.abs())).masked_fill(~seen, 0.0).amax(2)[..., None]
        ref, mag = torch.einsum("thp,phd->thd", p, v), torch.einsum("thp,phd->thd", p, v.abs())
        bound = info.eps / 2 * ref.abs() + info.tiny * info.eps + (2 ** -15 * A + 2 ** -14) * mag
        off = (out[b, :count].view(count, c.heads, 64) - ref).abs()
        assert (off <= bound).all(), (b, float((off - bound).max()))
    assert (out[left] == 7.0).all()


@pytest.mark.parametrize("T, group, dtype", [(6, 1, "bf16"), (13, 1, "f16"), (20, 1, "bf16"), (31, 1, "f16"),
                                             (7, 4, "bf16"), (40, 1, "bf16"), (64, 1, "f16")])
@pytest.mark.parametrize("stored", [False, True])
def test_many_short_items_in_turn(T, group, dtype, stored):
    g = np.random.default_rng(T)
    n_seq, kv = min(200, 2500 // (T * group)), 11
    lens = [int(n) for n in np.where(g.random(n_seq) < 0.5, g.integers(0, 40, n_seq), g.integers(40, 700, n_seq))]
    lens[n_seq // 2] = -1
    counts = [int(c) for c in g.integers(max(1, T // 2), T + 1, n_seq)]
    c = Case(lens, T, heads=kv * group, kv=kv, page=48, counts=counts, dtype=dtype, layers=2, layer=1, seed=T,
             stored=stored).run()
    check(c)
    once, lse = c.out.clone(), c.lse.clone()
    for _ in range(10):
        c.pages.copy_(c.before)
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out.view(torch.int16), once.view(torch.int16)) and torch.equal(c.lse, lse)
