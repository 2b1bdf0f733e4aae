"""gpt2_token_logprobs on the GPU against float64.

d = z - m is rounded once (2^-24 |d|); e^d through the hardware exp2 of the
rounded product d log2(e) is off by a factor within 2^-22 + 2^-23 |d| + 2^-24 |d|; the sum S of
V terms adds at most V / 512 + 40 roundings of partial sums one after another.
With D = sum p |d| the sums are off relatively by
  r = 2^-22 + 2^-22 D + (V / 512 + 40) 2^-24,
so log S is off by r + 2^-23 (log), log p by r + 2^-22 |log p| + 2^-23 |d|, and the entropy by
r (1 + 2 D) + 2^-22 (D + log S).  (d of -inf, or so low that e^d is 0, adds nothing to D.)
The alternatives' ids must be exactly those of a stable descending sort."""
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


def _run(z, V, dtype, top, tokens=None, only=None):
    """z: [M, ld] on the GPU, ld a multiple of 8."""
    M, ld = z.shape
    kw = dict(device="cuda")
    o = dict(logprob=torch.full((M,), 7.0, **kw), entropy=torch.full((M,), 7.0, **kw), lse=torch.full((M,), 7.0, **kw),
             ids=torch.full((M, top), -7, dtype=torch.int32, **kw), lps=torch.full((M, top), 7.0, **kw))
    g = lambda k: o[k] if only is None or k in only else None  # noqa: E731
    G.gpt2_token_logprobs(z, ld, DT[dtype][1], M, V, tokens if g("logprob") is not None else None, g("logprob"),
                          g("entropy"), g("lse"), top, g("ids") if top else None, g("lps") if top else None)
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in o.items()}


def _check(z, V, dtype, top, tokens=None):
    M = z.shape[0]
    if tokens is None:
        tokens = torch.from_numpy(np.random.default_rng(V).integers(0, V, M).astype(np.int32)).cuda()
    o = _run(z, V, dtype, top, tokens)
    x = z[:, :V].double().cpu()
    m = x.amax(1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    S = e.sum(1, keepdim=True)
    p = e / S
    D = torch.where(p > 0, p * d.abs(), 0.0).sum(1)
    lse = (m + torch.log(S))[:, 0]
    H = (torch.log(S))[:, 0] - torch.where(e > 0, e * d, 0.0).sum(1) / S[:, 0]
    r = 2.0 ** -22 * (1 + D) + (V / 512 + 40) * 2.0 ** -24
    assert ((o["lse"] - lse).abs() <= r + 2.0 ** -22 * lse.abs() + 2.0 ** -23 * m[:, 0].abs()).all()
    lp = (d.gather(1, tokens.long().cpu()[:, None]) - torch.log(S))[:, 0]
    fin = torch.isfinite(lp)
    assert (o["logprob"][~fin] == lp[~fin]).all()
    assert ((o["logprob"] - lp).abs() <= r + 2.0 ** -22 * lp.abs())[fin].all()
    assert ((o["entropy"] - H).abs() <= r * (1 + 2 * D) + 2.0 ** -22 * (D + torch.log(S)[:, 0])).all()
    order = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :top]
    assert torch.equal(o["ids"].long(), order)
    best = d.gather(1, order) - torch.log(S)
    fin = torch.isfinite(best)
    assert (o["lps"][~fin] == best[~fin]).all()
    assert ((o["lps"] - best).abs() <= r[:, None] + 2.0 ** -22 * best.abs())[fin].all()


def _logits(M, V, dtype, seed=0, scale=2.5):
    ld = -(-V // 8) * 8 + 8
    z = np.full((M, ld), np.nan, np.float32)  # what stands behind the vocabulary must not count
    z[:, :V] = scale * np.random.default_rng(seed).standard_normal((M, V))
    return torch.from_numpy(z).to(DT[dtype][0]).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 33, 127, 513, 4096, 50257])
def test_sizes(V, dtype):
    for top in sorted({0, min(1, V), min(5, V), min(32, V)}):
        _check(_logits(3, V, dtype, seed=V), V, dtype, top)


@pytest.mark.parametrize("dtype, V", [("f32", 200003), ("bf16", 400009), ("f32", 60001), ("bf16", 120001)])
def test_large_vocabularies(dtype, V):
    _check(_logits(2, V, dtype, seed=1), V, dtype, 20)


@pytest.mark.parametrize("dtype, M, V", [("bf16", 1, 4088), ("bf16", 1, 4089), ("f32", 2, 2049), ("f32", 400, 10240),
                                         ("f32", 400, 10241), ("bf16", 400, 20481), ("f16", 304, 9000),
                                         ("f16", 305, 9000), ("bf16", 5000, 100), ("bf16", 200, 50257)])
def test_each_side_of_the_kernels_borders(dtype, M, V):
    """A warp per row, a CTA per row with one chunk or several, one CTA or two per SM."""
    _check(_logits(M, V, dtype, seed=M), V, dtype, min(20, V))


@pytest.mark.parametrize("M", [1, 17, 64, 700])
def test_many_rows(M):
    _check(_logits(M, 5003, "bf16", seed=M), 5003, "bf16", 20)
    _check(_logits(M, 5003, "f32", seed=M, scale=20.0), 5003, "f32", 3)


@pytest.mark.parametrize("V", [20011, 3001, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["equal", "two values", "sorted", "falling", "one far ahead", "lowest but one",
                                  "lowest but a few", "inf but a few", "inf but one", "inf but thousands",
                                  "huge", "zeros of both signs", "strided", "low ids ahead",
                                  "low ids far ahead"])
def test_shapes_of_rows(kind, dtype, V):
    z = _logits(3, V, dtype, seed=2)
    low = torch.finfo(DT[dtype][0]).min
    g = torch.Generator().manual_seed(1)
    if kind == "equal":
        z[:, :V] = 1.5
    elif kind == "two values":
        z[:, :V] = (torch.rand(3, V, generator=g) < 0.001).to(z.dtype).cuda()
    elif kind in ("sorted", "falling"):
        z[:, :V] = z[:, :V].float().sort(1, descending=kind == "falling")[0].to(z.dtype)
    elif kind == "one far ahead":
        z[:, 77] = 200.0
    elif kind.startswith("lowest"):
        n = 1 if kind.endswith("one") else 9
        keep = torch.randperm(V, generator=g)[:n]
        vals = z[:, keep].clone()
        z[:, :V] = low
        z[:, keep] = vals
    elif kind.startswith("inf"):
        n = {"one": 1, "few": 9, "thousands": V // 7}[kind.split()[-1]]
        # thousands: a contiguous run, so that few of the threads hold any of them
        keep = torch.arange(100, 100 + n) if n > 9 else torch.randperm(V, generator=g)[:n]
        vals = z[:, keep].clone()
        z[:, :V] = -math.inf
        z[:, keep] = vals
    elif kind == "huge":
        z[:, :V] = z[:, :V] * (-low / 64)
    elif kind.startswith("low ids"):
        z[:, :V] -= (torch.arange(V, device="cuda") * (0.1 if "far" in kind else 0.001)).to(z.dtype)
    elif kind == "zeros of both signs":
        z[:, :V] = -5.0
        z[:, 1:280:2] = -0.0
        z[:, 30:280:2] = 0.0
    else:  # the largest all in the columns that one thread reads
        z[:, 5:V:512] = 30.0
        z[:, 8:V:4096] = 31.0
    tokens = torch.tensor([0, 77, V - 1], dtype=torch.int32).cuda()
    _check(z, V, dtype, 20, tokens)
    _check(z, V, dtype, 32, tokens)


def test_rows_without_a_distribution():
    V = 1000
    z = _logits(4, V, "f32", seed=3)
    z[0, 5] = math.nan
    z[1, 6] = math.inf
    z[2, :V] = -math.inf
    tokens = torch.tensor([1, 1, 1, 1], dtype=torch.int32).cuda()
    o = _run(z, V, "f32", 4, tokens)
    for k in ("lse", "logprob", "entropy"):
        assert torch.isnan(o[k][:3]).all() and torch.isfinite(o[k][3]), k
    assert torch.isnan(o["lps"][:3]).all()
    x = torch.where(torch.isnan(z), -math.inf, z)[:, :V].cpu()
    assert torch.equal(o["ids"].long(), torch.sort(x, dim=1, descending=True, stable=True)[1][:, :4])
    assert o["ids"][1, 0] == 6 and o["ids"][2].tolist() == [0, 1, 2, 3]
    # mostly NaN: the rest of the list is the lowest ids among what ranks as -inf
    z[3, :V] = math.nan
    z[3, 500] = 1.0
    o = _run(z, V, "f32", 4, tokens)
    assert o["ids"][3].tolist() == [500, 0, 1, 2]


def test_token_out_of_range():
    z = _logits(3, 100, "bf16")
    tokens = torch.tensor([100, -1, 99], dtype=torch.int32).cuda()
    o = _run(z, 100, "bf16", 0, tokens)
    assert torch.isnan(o["logprob"][:2]).all() and torch.isfinite(o["logprob"][2])
    assert torch.isfinite(o["lse"]).all()
    assert G.gpt2_last_error()[0] == RANGE


def test_outputs_are_optional_and_repeatable():
    z = _logits(5, 3001, "f16", seed=4)
    tokens = torch.arange(5, dtype=torch.int32).cuda()
    full = _run(z, 3001, "f16", 8, tokens)
    for _ in range(3):
        again = _run(z, 3001, "f16", 8, tokens)
        assert all(torch.equal(full[k], again[k]) for k in full)
    for only in (("lse",), ("entropy",), ("logprob",), ("ids", "lps")):
        o = _run(z, 3001, "f16", 8 if "ids" in only else 0, tokens, only)
        for k in full:
            if k in only:
                assert torch.equal(o[k], full[k])
            elif o[k].numel():
                assert (o[k] == (-7 if k == "ids" else 7)).all()


def test_captured_and_on_another_stream():
    z = _logits(64, 5003, "f32", seed=5)
    tokens = torch.arange(64, dtype=torch.int32).cuda()
    out = [torch.empty(64, device="cuda") for _ in range(3)]
    ids, lps = torch.empty((64, 5), dtype=torch.int32, device="cuda"), torch.empty((64, 5), device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        G.gpt2_token_logprobs(z, z.shape[1], G.F32, 64, 5003, tokens, *out, 5, ids, lps)
    z.copy_(_logits(64, 5003, "f32", seed=6))
    g.replay()
    torch.cuda.synchronize()
    ref = _run(z, 5003, "f32", 5, tokens)
    assert torch.equal(ids.cpu(), ref["ids"]) and torch.equal(out[0].cpu(), ref["logprob"])


@pytest.mark.parametrize("dtype, M, V", [("bf16", 6000, 1003), ("f32", 6000, 203), ("f32", 700, 52001),
                                         ("f32", 400, 110003), ("bf16", 300, 300007)])
def test_many_rows_through_the_same_buffers(dtype, M, V):
    """More rows than CTAs (or clusters) are resident: each takes a dozen or more in turn."""
    _check(_logits(M, V, dtype, seed=V), V, dtype, 20)
