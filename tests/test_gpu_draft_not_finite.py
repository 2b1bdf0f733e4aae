"""gpt2_attention_paged_draft on the GPU: values that are not finite in V, at
cached places that every token sees and at places that some do.

An infinite V of a place that a token sees, with a probability above 0, makes
that dimension infinite with its sign; two of opposite signs, or a NaN, make it
NaN; the other dimensions are those of finite numbers (bounds as in
test_gpu_draft_attention.py)."""
import math

import pytest

torch = pytest.importorskip("torch")
import gpt_pre_ln_gb300 as G  # noqa: E402
from test_gpu_draft_attention import Case  # noqa: E402

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gpt_pre_ln_gb300 import build
    build.build()
    G.lib()
    yield
    st, site = G.gpt2_last_error()
    assert st == 0, f"device error {st} at site {site}"


def put(c, b, p, g, d, value):
    """Dimension d of the V of cached position p (key-value head g)."""
    c.vc[b][p, g, d] = value
    c.pages[c.table_np[b, p // c.page], c.layer, 1, g, p % c.page, d] = value
    c.before = c.pages.clone()


def check(c):
    """Like Case.check, whole sequences at a time, with values that are not finite where the formula has them; how many."""
    torch.cuda.synchronize()
    info, group = torch.finfo(c.out.dtype), c.heads // c.kv
    out = c.out.view(len(c.lens_l), c.T, -1)[:, :, :c.heads * 64].double()
    odd = 0
    for b, n, count in c.live:
        both = lambda cache, new: torch.cat([cache[b], new[b, :count]]).cuda().double().repeat_interleave(group, 1)  # noqa: E731,E501
        k, v, q = both(c.kc, c.kn), both(c.vc, c.vn), c.q[b, :count].cuda().double()
        seen = torch.zeros(count, n + count, dtype=torch.bool)
        for t in range(count):
            seen[t, c.seen[b, t]] = True
        seen = seen.cuda()[:, None]
        p = torch.softmax((c.scale * torch.einsum("thd,phd->thp", q, k)).masked_fill(~seen, -INF), 2)
        A = (c.scale * torch.einsum("thd,phd->thp", q.abs(), k.abs())).masked_fill(~seen, 0.0).amax(2)[..., None]
        fine = torch.where(v.isfinite(), v, 0.0)
        ref, mag = torch.einsum("thp,phd->thd", p, fine), torch.einsum("thp,phd->thd", p, fine.abs())
        bound = info.eps / 2 * ref.abs() + info.tiny * info.eps + (2 ** -15 * A + 2 ** -14) * mag
        # how many NaN, infinities of either sign (of NaN both) each token sees in a dimension
        count_of = lambda x: torch.einsum("tp,phd->thd", seen[:, 0].double(), x.double())  # noqa: E731
        up, down = count_of(v.isnan() | (v == INF)) > 0, count_of(v.isnan() | (v == -INF)) > 0
        got = out[b, :count].view(count, c.heads, 64)
        ok = torch.where(up & down, got.isnan(), torch.where(up, got == INF, torch.where(
            down, got == -INF, (got - ref).abs() <= bound)))
        assert ok.all(), (b, (~ok).nonzero()[0].tolist(), got[~ok][0].item(), ref[~ok][0].item())
        odd += int((up | down).sum())
    return odd


SHAPES = [(1, 1, "bf16"), (7, 1, "bf16"), (8, 1, "f16"), (12, 1, "bf16"), (16, 1, "f16"), (30, 1, "bf16"),
          (32, 1, "f16"), (60, 1, "bf16"), (20, 3, "f16")]


@pytest.mark.parametrize("T, group, dtype", SHAPES)
def test_an_infinite_value_that_every_token_sees(T, group, dtype):
    """Wherever it stands: in the first tile, in the middle, next to the drafted tokens, and beside others."""
    for n, at in ((300, (3,)), (300, (150,)), (303, (302,)), (5000, (17, 4000)), (40, (39,))):
        for value in (INF, -INF, NAN):
            c = Case([n, 90], T, heads=group, kv=1, page=32, dtype=dtype, seed=T + n, layers=1, layer=0)
            for p in at:
                put(c, 0, p, 0, p % 64, value)
                put(c, 0, p, 0, 63, value)
            assert check(c.run()) > 0


@pytest.mark.parametrize("T, group, dtype", SHAPES)
def test_infinite_values_of_both_signs(T, group, dtype):
    for p, q in ((20, 21), (20, 400), (3, 500)):
        c = Case([505], T, heads=2 * group, kv=2, dtype=dtype, seed=T, layers=1, layer=0)
        put(c, 0, p, 0, 5, INF)
        put(c, 0, q, 0, 5, -INF)
        put(c, 0, q, 0, 6, -INF)
        put(c, 0, q, 1, 9, INF)
        assert check(c.run()) > 0


@pytest.mark.parametrize("T, group, dtype", SHAPES)
@pytest.mark.parametrize("stored", [False, True])
def test_in_a_row_of_tiles(T, group, dtype, stored):
    """One dimension of every third cached place; drafted places too, seen by the tokens behind them."""
    c = Case([270, -1, 33], T, heads=group, kv=1, kind="roots", dtype=dtype, seed=T, stored=stored, layers=1, layer=0)
    for p in range(0, 270, 3):
        put(c, 0, p, 0, p % 40, INF)
    t = T // 2
    c.vn[0, t, 0, 50] = -INF
    row = c.qkv.view(3, T, -1)
    row[0, t, (group + 1) * 64 + 50] = -INF
    if stored:
        p = 270 + t
        c.pages[c.table_np[0, p // 16], 0, 1, 0, p % 16, 50] = -INF
        c.before = c.pages.clone()
    assert check(c.run()) > 0


@pytest.mark.parametrize("T, group, dtype", SHAPES)
def test_under_a_window(T, group, dtype):
    """Places that leave the window from one depth to the next, the first tokens, and the whole tiles between."""
    c = Case([700], T, heads=group, kv=1, kind="chain", window=200, sinks=20, dtype=dtype, seed=T, layers=1, layer=0)
    for p in (2, 19, 20, 501, 503, 520, 600, 699):
        if any(p in s for s in c.seen.values()):
            put(c, 0, p, 0, p % 64, INF if p % 2 else -INF)
    assert check(c.run()) > 0


@pytest.mark.parametrize("T", [3, 12, 24, 60])
def test_scores_of_minus_infinity_and_values_that_are_not_finite(T):
    """A token that sees nothing but scores of -inf gets zeros, whatever the values are."""
    for n in (0, 64, 3000):
        c = Case([n], T, heads=1, kv=1, kind="star", scale=1.0, seed=2, page=64)
        c.qkv[:, :64] = 1.0
        c.qkv[:, 64:128] = -INF
        c.qkv[:, 128:192] = INF
        c.qkv[0, 130] = NAN
        for p in range(-(-n // 64)):
            c.pages[c.table_np[0, p], 1, 0] = -INF
            c.pages[c.table_np[0, p], 1, 1] = -INF if p % 2 else INF
        c.run()
        torch.cuda.synchronize()
        assert (c.out == 0).all() and (c.lse == -INF).all()


@pytest.mark.parametrize("T, group, dtype", SHAPES)
def test_however_small_its_probability(T, group, dtype):
    """Scores grow with the position: the first places' probabilities are e^-100 and less, in other CTAs' parts too."""
    for n in (400, 9000):
        c = Case([n], T, heads=group, kv=1, page=256, dtype=dtype, seed=T, grow=300 / n, layers=1, layer=0)
        for p in (2, n // 4, n // 2):
            put(c, 0, p, 0, p % 50, INF)
        put(c, 0, 3, 0, 51, -INF)
        put(c, 0, n - 3, 0, 51, INF)
        put(c, 0, n // 3, 0, 52, NAN)
        assert check(c.run()) > 0


@pytest.mark.parametrize("T, group, dtype", SHAPES)
def test_with_a_score_of_minus_infinity(T, group, dtype):
    """0 * inf: NaN for those who see the place, whatever else there is; its other dimensions are finite."""
    c = Case([200], T, heads=group, kv=1, dtype=dtype, seed=T, layers=1, layer=0)
    c.q[..., 7] = 1.0
    c.qkv.view(T, -1)[:, 7:group * 64:64] = 1.0
    for p in (20, 170):
        c.pages[c.table_np[0, p // 16], 0, 0, 0, p % 16, 7] = -INF
        put(c, 0, p, 0, 30, INF)
    put(c, 0, 100, 0, 30, INF)
    c.run()
    torch.cuda.synchronize()
    out = c.out.view(T, group, 64)
    assert torch.isnan(out[:, :, 30]).all()
    rest = [d for d in range(64) if d != 30]
    assert torch.isfinite(out[:, :, rest]).all()


@pytest.mark.parametrize("T, group, dtype", [(6, 1, "bf16"), (12, 1, "f16"), (30, 1, "bf16"), (60, 1, "f16")])
def test_nothing_but_values_that_are_not_finite(T, group, dtype):
    """A whole long cache of NaN or of infinities of one sign, as a model that has overflowed leaves it; the next sequence
    is as it would be."""
    for value in (NAN, INF):
        c = Case([20000, 700], T, heads=group, kv=1, page=256, dtype=dtype, seed=T, layers=1, layer=0)
        for p in range(-(-20000 // 256)):
            c.pages[c.table_np[0, p], 0, 1] = value
        c.vc[0][:] = value
        row = c.qkv.view(2, T, -1)
        row[0, :, (group + 1) * 64:(group + 2) * 64] = value
        c.before = c.pages.clone()
        c.run()
        torch.cuda.synchronize()
        out = c.out.view(2, T, -1)
        assert (torch.isnan(out[0]) if math.isnan(value) else out[0] == value).all()
        c.live = [x for x in c.live if x[0] == 1]
        assert check(c) == 0
