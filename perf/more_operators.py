"""Workloads of speculative decoding and sampling: what is timed, its plain form, and its value in 64 bits.

A case names an operator and its sizes.  ``run`` computes it with elementary torch operations, or, where ``own`` is
true, with the calls a user makes of ``gpt_pre_ln_gb300``.

- draft: attention of a tree of drafted tokens per sequence over a paged key-value cache, storing their K and V
- accept: the path of drafted tokens that the model's own choices confirm; its K and V move together in the cache
- sample: one token per row of logits, under temperature, top-k, top-p and min-p, from a given random number
"""
import math
import random

import numpy as np
import torch

own = False

HD = 64  # head dimension of the whole library
LOG2E = 1.4426950408889634
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one conversation of a GPT-2 small, eight drafted tokens in a small tree (latency)
        dict(name="draft-single", op="draft", seqs=1, heads=12, kv_heads=12, drafts=8, length=777, page=16, window=0,
             sinks=0, dtype="bf16", chain=False),
        # a batch at the benchmark's cache length, sixteen drafted tokens each, ragged
        dict(name="draft-batch32", op="draft", seqs=32, heads=12, kv_heads=12, drafts=16, length=1087, page=16,
             window=0, sinks=0, dtype="bf16", chain=False),
        # wide trees, as several drafting heads give them, at GPT-2 medium width
        dict(name="draft-wide64", op="draft", seqs=16, heads=16, kv_heads=16, drafts=64, length=4096, page=64,
             window=0, sinks=0, dtype="f16", chain=False),
        # long documents with query heads that share key-value heads
        dict(name="draft-long-grouped", op="draft", seqs=8, heads=16, kv_heads=4, drafts=12, length=32768, page=64,
             window=0, sinks=0, dtype="f16", chain=False),
        # endless chat at GPT-2 XL width: a window of 1024 and four first tokens, a chain from a small draft model
        dict(name="draft-window-xl", op="draft", seqs=64, heads=25, kv_heads=25, drafts=7, length=8000, page=32,
             window=1024, sinks=4, dtype="bf16", chain=True),
        # the end of one conversation's step on GPT-2 small (latency)
        dict(name="accept-single", op="accept", seqs=1, layers=12, kv_heads=12, drafts=8, kept=4, length=777, page=16,
             dtype="bf16"),
        # the end of a step of 64 sequences with wide trees on GPT-2 medium
        dict(name="accept-wide64", op="accept", seqs=64, layers=24, kv_heads=16, drafts=64, kept=9, length=90, page=64,
             dtype="f16"),
        # the next token of one conversation (latency)
        dict(name="sample-single", op="sample", rows=1, vocab=50257, dtype="bf16", mode="top_p", masked=False),
        # a decode step's tokens, nucleus sampling, part of the vocabulary masked out
        dict(name="sample-step", op="sample", rows=64, vocab=50257, dtype="f32", mode="top_p", masked=True),
        # many samples from the 20 to 400 most likely tokens
        dict(name="sample-top-k", op="sample", rows=256, vocab=50257, dtype="f16", mode="top_k", masked=False),
        # a small vocabulary at temperature alone
        dict(name="sample-small", op="sample", rows=512, vocab=8000, dtype="f32", mode="plain", masked=False),
        # every node of 16 trees of 64 drafted tokens, each request with settings of its own
        dict(name="sample-trees", op="sample", rows=1024, vocab=50257, dtype="bf16", mode="mixed", masked=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["draft", "draft", "draft", "accept", "sample", "sample", "sample"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    dtype = rng.choice(["bf16", "f16"])
    if op == "draft":
        heads, kv_heads = rng.choice(
            [(12, 12), (16, 16), (20, 20), (25, 25), (16, 4), (12, 1), (20, 5), (25, 1), (32, 4)])
        drafts = rng.choice([1, 4, 8, _log_int(rng, 2, 64), _log_int(rng, 2, 64), 64])
        length = _log_int(rng, 1, 32769) - 1
        window = rng.choice([0, 0, _log_int(rng, 16, 4096)])
        sinks = rng.choice([0, 1, 4, rng.randint(5, 64)]) if window else 0
        seen = min(length, window + sinks) if window else length
        seen += drafts
        most = max(1, min(128, 1000000 // (seen * kv_heads), 67000000 // (seen * heads * drafts)))
        return dict(op=op, seqs=_log_int(rng, 1, most), heads=heads, kv_heads=kv_heads, drafts=drafts, length=length,
                    page=page, window=window, sinks=sinks, dtype=dtype, chain=rng.random() < 0.3)
    if op == "accept":
        layers, kv_heads = rng.choice([(12, 12), (24, 16), (36, 20), (48, 25), (12, 1), (24, 4)])
        drafts = _log_int(rng, 1, 64)
        size = layers * 2 * kv_heads * HD * 2
        length = _log_int(rng, 1, 1024)
        held = (length + drafts) // page * page + page
        most = max(1, min(64, (1200 << 20) // (held * size)))
        return dict(op=op, seqs=_log_int(rng, 1, most), layers=layers, kv_heads=kv_heads, drafts=drafts,
                    kept=rng.randint(1, min(9, (drafts + 1) // 2)), length=length, page=page, dtype=dtype)
    vocab = rng.choice([_log_int(rng, 40, 150000), 50257, 50304])
    dtype = rng.choice(["bf16", "f16", "f32"])
    most = max(1, min(1024, 51000000 // vocab))
    return dict(op=op, rows=_log_int(rng, 1, most), vocab=vocab, dtype=dtype,
                mode=rng.choice(["plain", "top_k", "top_p", "min_p", "mixed", "mixed"]), masked=rng.random() < 0.3)


# ------------------------------------------------------------------ sizes that follow from a case
def _ragged(n, longest):
    """Lengths of n sequences: the longest, and others down to half of it."""
    return [longest - (b * 977) % (longest // 2 + 1) for b in range(n)]


def _lens(case):
    """Cached positions of each slot before the call; one slot of a batch of eight or more is idle (-1)."""
    lens = _ragged(case["seqs"], case["length"])
    if case["seqs"] >= 8:
        lens[5] = -1
    return lens


def _counts(case):
    """Drafted tokens of each sequence: the full count, and others down to half of it."""
    return [max(1, c) for c in _ragged(case["seqs"], case["drafts"])]


def _cached(case, length):
    """Cached positions that the drafted tokens of one sequence attend over (the first of them sees most)."""
    if not case["window"]:
        return length
    behind = max(0, length + 1 - case["window"])
    return length - behind + min(behind, case["sinks"])


def _kept(case):
    """Tokens that each sequence keeps: the case's count, and others down to half of it."""
    return [max(1, min(k, (c + 1) // 2)) for k, c in zip(_ragged(case["seqs"], case["kept"]), _counts(case))]


def work(case):
    op = case["op"]
    if op == "draft":
        bytes_, flops, row = 0, 0, HD * 2
        for n, c in zip(_lens(case), _counts(case)):
            if n < 0:
                continue
            seen = _cached(case, n)
            bytes_ += (seen + 2 * c) * case["kv_heads"] * 2 * row + c * case["heads"] * (2 * row + 4) + 4 * c
            flops += 4 * HD * case["heads"] * c * (seen + (c + 1) // 2)
        return {"bytes": bytes_, "flops": flops}
    if op == "accept":
        live = [(k, c) for k, c, n in zip(_kept(case), _counts(case), _lens(case)) if n >= 0]
        moved = sum(k - 1 for k, _ in live)
        return {"bytes": 2 * moved * case["layers"] * 2 * case["kv_heads"] * HD * 2 + 16 * sum(c for _, c in live),
                "flops": 0}
    elem = 4 if case["dtype"] == "f32" else 2
    return {"bytes": case["rows"] * (case["vocab"] * elem + 24), "flops": 6 * case["rows"] * case["vocab"]}


# ------------------------------------------------------------------ inputs
def _rand(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _tree(rng, count, width, chain):
    """Parents of one sequence's drafted tokens (-1 for the first, which follows the cached ones), padded with -1."""
    parents = [-1] + [t - 1 if chain or rng.random() < 0.4 else rng.randrange(t) for t in range(1, count)]
    return parents + [-1] * (width - count)


def _placed(g, columns, spare):
    """A table whose wanted entries (True in the rows of `columns`) name pages in random order; and the page count."""
    want = torch.tensor(columns, dtype=torch.bool)
    count = int(want.sum())
    ids = torch.randperm(count + spare, generator=g, device="cuda")[:count].to(torch.int32)
    table = torch.full(want.shape, -1, dtype=torch.int32, device="cuda")
    table[want.cuda()] = ids
    return table, count + spare


def _cache_of(state, g, case, rows, layers):
    table, pages = _placed(g, rows, 8)
    shape = (pages, layers, 2, case["kv_heads"], case["page"], HD)
    state["pages"] = torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[case["dtype"]])
    state["refs"] = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
    state["table"] = table


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    state = {"case": dict(case), "op": case["op"]}
    dtype, op = DTYPES[case["dtype"]], case["op"]
    if op == "sample":
        _prepare_sample(state, g, case)
        return state
    lens, counts, page, width = _lens(case), _counts(case), case["page"], case["drafts"]
    state["lens"], state["counts"] = _ints(lens), _ints(counts)
    cols = -(-(case["length"] + width) // page)
    if op == "draft":
        rows = []
        for n, c in zip(lens, counts):
            first = max(0, n + 1 - case["window"]) if case["window"] else 0
            rows.append([n >= 0 and k * page < n + c and ((k + 1) * page > first or k * page < case["sinks"])
                         for k in range(cols)])
        _cache_of(state, g, case, rows, 2)
        state["parents"] = _ints([_tree(rng, c, width, case["chain"]) for c in counts])
        heads = case["heads"] + 2 * case["kv_heads"]  # heads of one row of the fused projection
        state["qkv"] = _rand(g, (case["seqs"] * width, heads * HD), dtype)
        state["out"] = torch.zeros((case["seqs"] * width, case["heads"] * HD), device="cuda", dtype=dtype)
        state["lse"] = torch.zeros((case["seqs"] * width, case["heads"]), device="cuda", dtype=torch.float32)
        state["layer"], state["longest"] = 1, max([1] + [_cached(case, n) + c for n, c in zip(lens, counts) if n >= 0])
    else:
        rows = [[n >= 0 and k * page < n + c for k in range(cols)] for n, c in zip(lens, counts)]
        _cache_of(state, g, case, rows, case["layers"])
        parents, tokens, chosen = [], [], []
        for c, kept in zip(counts, _kept(case)):
            tree = _tree(rng, c, width, False)
            # the tokens that will be kept: the first, and others behind the places that they move to
            path = [0] + sorted(rng.sample(range(kept, c), kept - 1))
            for a, b in zip(path, path[1:]):
                tree[b] = a
            drafted = rng.sample(range(50257), width)
            choice = [rng.choice(drafted[:c]) if t not in path else 50257 for t in range(width)]
            for a, b in zip(path, path[1:]):
                choice[a] = drafted[b]
            parents.append(tree)
            tokens.append(drafted)
            chosen.append(choice)
        state["parents"], state["tokens"], state["chosen"] = _ints(parents), _ints(tokens), _ints(chosen)
        state["lens0"] = state["lens"].clone()
        state["path"] = torch.full((case["seqs"], width), -1, dtype=torch.int32, device="cuda")
        state["kept"] = torch.zeros(case["seqs"], dtype=torch.int32, device="cuda")
        state["next"] = torch.zeros(case["seqs"], dtype=torch.int32, device="cuda")
    if own:
        import gpt_pre_ln_gb300 as G
        state["cache"] = G.paged_cache(state["pages"], state["refs"], state["table"], state["lens"])
        if op == "draft":
            need = G.gpt2_attention_paged_draft_workspace_bytes(state["cache"], width, case["heads"])
            state["ws"], state["ws_bytes"] = torch.empty(need, device="cuda", dtype=torch.uint8), need
    return state


def _prepare_sample(state, g, case):
    rows, vocab, mode = case["rows"], case["vocab"], case["mode"]

    def uniform(lo=0.0, hi=1.0):
        return lo + (hi - lo) * torch.rand(rows, generator=g, device="cuda")

    # probabilities that fall with a power of the rank, as a language model's do, sharper in some rows than in others
    ld = -(-vocab // 8) * 8
    logits = torch.empty((rows, ld), device="cuda").exponential_(generator=g).mul_(uniform(0.9, 2.5)[:, None])
    logits += 0.5 * torch.randn((rows, ld), generator=g, device="cuda")
    if case["masked"]:  # constrained decoding: three in ten entries cannot come next
        gone = torch.rand(ld, generator=g, device="cuda") < 0.3
        gone[vocab // 2] = False
        logits[:, gone] = -math.inf
    state["logits"], state["ld"] = logits.to(DTYPES[case["dtype"]]), ld
    mixed = mode == "mixed"
    state["temperature"] = uniform(0.5, 1.3)
    if mixed:
        state["temperature"].masked_fill_(uniform() < 0.1, 0.0)  # some requests are greedy
    off = torch.zeros(rows, device="cuda")
    k = torch.randint(20, 401, (rows,), generator=g, device="cuda", dtype=torch.int32)
    state["top_k"] = torch.where(uniform() < 0.4, k, 0) if mixed else k if mode == "top_k" else k * 0
    p = uniform(0.8, 0.99)
    state["top_p"] = torch.where(uniform() < 0.5, p, off + 1) if mixed else p if mode == "top_p" else off + 1
    m = uniform(0.02, 0.1)
    state["min_p"] = torch.where(uniform() < 0.3, m, off) if mixed else m if mode == "min_p" else off
    state["uniform"] = uniform().clamp_(max=1 - 2.0 ** -24)
    state["token"] = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    state["logprob"] = torch.zeros(rows, device="cuda")


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["op"]](state)


def _run_own(s):
    import gpt_pre_ln_gb300 as G
    c, op = s["case"], s["op"]
    if op == "draft":
        h, kv, ld = c["heads"], c["kv_heads"], s["qkv"].shape[1]
        at = s["qkv"].data_ptr()
        G.gpt2_attention_paged_draft(s["cache"], s["layer"], at, ld, at + 2 * HD * h, at + 2 * HD * (h + kv), ld,
                                     s["out"], h * HD, s["lse"], c["drafts"], s["parents"], s["counts"], h, 0.125,
                                     c["window"], c["sinks"], s["ws"], s["ws_bytes"])
        return {"out": s["out"], "lse": s["lse"], "pages": s["pages"]}
    if op == "accept":
        s["lens"].copy_(s["lens0"])
        G.gpt2_draft_accept(s["cache"], c["drafts"], s["tokens"], s["parents"], s["counts"], s["chosen"], s["path"],
                            s["kept"], s["next"])
        return {k: s[k] for k in ("path", "kept", "next", "lens", "pages")}
    kinds = {"bf16": G.BF16, "f16": G.F16, "f32": G.F32}
    G.gpt2_sample_tokens(s["logits"], s["ld"], kinds[c["dtype"]], c["rows"], c["vocab"], s["temperature"], s["top_k"],
                         s["top_p"], s["min_p"], s["uniform"], s["token"], s["logprob"])
    return {"token": s["token"], "logprob": s["logprob"]}


def _reached(steps):
    """[b, t, u]: whether steps of `steps`, at most one from each t, lead from t to u (at most 64 of them)."""
    stay = torch.eye(steps.shape[2], device="cuda")
    return torch.matrix_power(steps.float() + stay, 64) > 0


def _plain_draft(s):
    c, table, lens, pages, layer = s["case"], s["table"].long(), s["lens"].long(), s["pages"], s["layer"]
    h, kv, page, width, seqs = c["heads"], c["kv_heads"], c["page"], c["drafts"], c["seqs"]
    q, k_new, v_new = s["qkv"].view(seqs, width, -1, HD).split([h, kv, kv], 2)
    t = torch.arange(width, device="cuda")
    live = (lens >= 0)[:, None] & (t[None, :] < s["counts"][:, None])
    # the drafted tokens' K and V into their places
    b, node = live.nonzero(as_tuple=True)
    at, off = table[b, (lens[b] + node) // page], (lens[b] + node) % page
    pages[at, layer, 0, :, off] = k_new[b, node]
    pages[at, layer, 1, :, off] = v_new[b, node]
    # ancestors of each drafted token, itself among them
    above = _reached((s["parents"].long()[:, :, None] == t) & live[:, :, None])
    depth = above.sum(2) - 1
    # places that some drafted token of a sequence may see, in order; the position that each stands for
    i = torch.arange(s["longest"], device="cuda")[None, :]
    if c["window"]:
        behind = (lens + 1 - c["window"]).clamp(min=0)[:, None]
        first = behind.clamp(max=c["sinks"])
        i = torch.where(i < first, i, i - first + behind)
    i = i.expand(seqs, -1)
    there = (i < (lens + s["counts"])[:, None]) & (lens >= 0)[:, None]
    new = i - lens[:, None]  # >= 0: a drafted token
    of = new.clamp(0, width - 1)
    position = torch.where(new < 0, i, lens[:, None] + depth.gather(1, of))
    mine = (lens[:, None] + depth)[:, :, None]  # [seqs, width, 1]
    seen = there[:, None] & ((new < 0)[:, None] | above.gather(2, of[:, None].expand(-1, width, -1)))
    if c["window"]:
        seen &= (position[:, None] > mine - c["window"]) | (position < c["sinks"])[:, None]
    i = torch.where(there, i, 0)
    at = table.gather(1, i // page).clamp(min=0)
    k = pages[at, layer, 0, :, i % page].float()  # [seqs, places, kv heads, 64]
    v = pages[at, layer, 1, :, i % page].float().masked_fill(~there[:, :, None, None], 0.0)
    qf = q.float().view(seqs, width, kv, h // kv, HD)
    z = torch.einsum("bthgd,bnhd->bthgn", qf, k) * 0.125
    z = z.masked_fill(~seen[:, :, None, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bthgn,bnhd->bthgd", p, v) / torch.where(total == 0, 1.0, total)
    lse = ((m + torch.log(total)) * LOG2E).view(seqs * width, h)
    rows = live.view(-1, 1)
    s["out"].copy_(torch.where(rows, out.reshape(seqs * width, h * HD).to(q.dtype), s["out"]))
    s["lse"].copy_(torch.where(rows, lse, s["lse"]))
    return {"out": s["out"], "lse": s["lse"], "pages": pages}


def _plain_accept(s):
    c, pages, page, width = s["case"], s["pages"], s["case"]["page"], s["case"]["drafts"]
    s["lens"].copy_(s["lens0"])
    lens, t = s["lens"].long(), torch.arange(width, device="cuda")
    on = lens >= 0
    # [b, t, u]: u is the first child of t that is the token chosen behind t
    match = (s["parents"][:, None, :] == t[:, None]) & (s["tokens"][:, None, :] == s["chosen"][:, :, None])
    match &= (t < s["counts"][:, None])[:, None]
    child = torch.where(match, t, width).amin(2)
    kept = _reached(child[:, :, None] == t)[:, 0] & on[:, None]  # a child stands behind its parent: in order
    count = kept.sum(1)
    path = torch.sort(torch.where(kept, t, width), 1)[0]
    last = s["chosen"].gather(1, torch.where(kept, t, 0).amax(1, keepdim=True))[:, 0]
    path = torch.where(path < width, path, -1)
    b, j = ((path >= 0) & (path != t)).nonzero(as_tuple=True)
    table = s["table"].long()
    source, target = lens[b] + path[b, j], lens[b] + j
    pages[table[b, target // page], :, :, :, target % page] = pages[table[b, source // page], :, :, :, source % page]
    s["path"].copy_(torch.where(on[:, None], path.to(torch.int32), s["path"]))
    s["kept"].copy_(torch.where(on, count.to(torch.int32), s["kept"]))
    s["next"].copy_(torch.where(on, last, s["next"]))
    s["lens"].copy_(lens + count)
    return {k: s[k] for k in ("path", "kept", "next", "lens", "pages")}


def _plain_sample(s):
    # in 64 bits: a token's part of a long sum decides which one a random number falls on
    c = s["case"]
    x, index = torch.sort(s["logits"][:, :c["vocab"]].float(), dim=1, descending=True, stable=True)
    x = x.double()
    x = x - x[:, :1]  # the most likely token at 0
    temperature = s["temperature"].double().clamp(min=2.0 ** -100)[:, None]
    w = torch.exp(x / temperature)
    rank = torch.arange(c["vocab"], device="cuda")[None, :]
    k = torch.where(s["top_k"] == 0, c["vocab"], s["top_k"])
    k = torch.where(s["temperature"] == 0, 1, k)[:, None]
    keep = rank < k
    w = torch.where(keep, w, 0.0)
    part = torch.cumsum(w, 1)
    top_p = s["top_p"].double()[:, None]
    keep &= (top_p >= 1) | (part - w < top_p * part[:, -1:]) | (rank == 0)
    least = temperature * torch.log(s["min_p"].double())[:, None]  # -inf without a min_p
    keep &= x >= least
    w = torch.zeros_like(w).scatter_(1, index, torch.where(keep, w, 0.0))  # in the order of the ids
    part = torch.cumsum(w, 1)
    target = s["uniform"].double()[:, None] * part[:, -1:]
    token = (part <= target).sum(1, keepdim=True)
    s["token"].copy_(token[:, 0])
    s["logprob"].copy_(torch.log(w.gather(1, token) / part[:, -1:])[:, 0])
    return {"token": s["token"], "logprob": s["logprob"]}


_PLAIN = {"draft": _plain_draft, "accept": _plain_accept, "sample": _plain_sample}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_draft(c, s):
    table, pages, page, layer, width = s["table"].tolist(), s["pages"], c["page"], s["layer"], c["drafts"]
    h, kv = c["heads"], c["kv_heads"]
    out, lse = s["out"].double(), s["lse"].double()
    parents, counts = s["parents"].tolist(), s["counts"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        if n < 0:
            continue
        paths = []  # slots of the drafted tokens from the first to each
        for t in range(counts[b]):
            paths.append((paths[parents[b][t]] if parents[b][t] >= 0 else []) + [t])
            row = s["qkv"][b * width + t].view(-1, HD)
            at = table[b][(n + t) // page]
            pages[at, layer, 0, :, (n + t) % page] = row[h:h + kv]
            pages[at, layer, 1, :, (n + t) % page] = row[h + kv:]
        start = max(0, n + 1 - c["window"]) if c["window"] else 0
        slots = list(range(min(c["sinks"], start) if c["window"] else 0)) + list(range(start, n + counts[b]))
        place = {p: i for i, p in enumerate(slots)}
        seen = torch.zeros(counts[b], len(slots), dtype=torch.bool)
        for t, path in enumerate(paths):
            end = n + len(path)  # positions up to and with its own
            from_ = max(0, end - c["window"]) if c["window"] else 0
            seen[t, [place[p] for p in slots if p < n and (p >= from_ or p < c["sinks"])]] = True
            seen[t, [place[n + a] for d, a in enumerate(path) if n + d >= from_ or n + d < c["sinks"]]] = True
        seen = seen.cuda()
        at = torch.tensor([table[b][p // page] for p in slots], device="cuda")
        off = torch.tensor([p % page for p in slots], device="cuda")
        rows = slice(b * width, b * width + counts[b])
        for head in range(h):
            g = head // (h // kv)
            k, v = pages[at, layer, 0, g, off].double(), pages[at, layer, 1, g, off].double()
            q = s["qkv"][rows, head * HD:(head + 1) * HD].double()
            z = (q @ k.t() / 8).masked_fill(~seen, -math.inf)
            lse[rows, head] = torch.logsumexp(z, 1) / math.log(2)
            out[rows, head * HD:(head + 1) * HD] = torch.softmax(z, 1) @ v
    return {"out": out, "lse": lse, "pages": pages}


def _exact_accept(c, s):
    table, pages, page, lens = s["table"].tolist(), s["pages"], c["page"], s["lens0"].tolist()
    out = {k: s[k].tolist() for k in ("path", "kept", "next")}
    tokens, parents, chosen = s["tokens"].tolist(), s["parents"].tolist(), s["chosen"].tolist()
    for b, count in enumerate(s["counts"].tolist()):
        if lens[b] < 0:
            continue
        path = [0]
        while True:
            down = [t for t in range(count) if parents[b][t] == path[-1] and tokens[b][t] == chosen[b][path[-1]]]
            if not down:
                break
            path.append(down[0])
        out["next"][b], out["kept"][b] = chosen[b][path[-1]], len(path)
        out["path"][b] = path + [-1] * (c["drafts"] - len(path))
        for j, t in enumerate(path):
            a, z = lens[b] + t, lens[b] + j
            pages[table[b][z // page], :, :, :, z % page] = pages[table[b][a // page], :, :, :, a % page]
        lens[b] += len(path)
    return {"path": _ints(out["path"]), "kept": _ints(out["kept"]), "next": _ints(out["next"]), "lens": _ints(lens),
            "pages": pages}


def _exact_sample(c, s):
    z = s["logits"][:, :c["vocab"]].float().cpu().numpy().astype(np.float64)
    get = {k: s[k].cpu().numpy().astype(np.float64) for k in ("temperature", "top_k", "top_p", "min_p", "uniform")}
    tokens, logprobs = [], []
    for m in range(c["rows"]):
        order = np.argsort(-z[m], kind="stable")
        t = get["temperature"][m]
        if t == 0:
            tokens.append(int(order[0]))
            logprobs.append(0.0)
            continue
        x = z[m][order] - z[m][order[0]]
        w = np.exp(x / t)
        n = int(get["top_k"][m]) or c["vocab"]
        n = min(n, c["vocab"])
        if get["top_p"][m] < 1:
            part = np.cumsum(w[:n])
            n = max(1, int(np.searchsorted(part, get["top_p"][m] * part[-1])) + 1)
        if get["min_p"][m] > 0:
            n = min(n, int((x >= t * math.log(get["min_p"][m])).sum()))
        ids = np.sort(order[:n])
        part = np.cumsum(np.exp((z[m][ids] - z[m][order[0]]) / t))
        tokens.append(int(ids[np.searchsorted(part, get["uniform"][m] * part[-1], side="right")]))
        logprobs.append((z[m][tokens[-1]] - z[m][order[0]]) / t - math.log(part[-1]))
    return {"token": _ints(tokens), "logprob": torch.tensor(logprobs, dtype=torch.float64).cuda()}


def exact(case, seed):
    return {"draft": _exact_draft, "accept": _exact_accept, "sample": _exact_sample}[case["op"]](
        dict(case), prepare(case, seed))
