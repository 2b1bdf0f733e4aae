"""Workloads of the paged-cache and scoring operators: what is timed, its plain form, and its value in 64 bits.

A case names an operator and its sizes.  ``run`` computes it with elementary torch operations, or, where ``own`` is
true, with the calls a user makes of ``gpt_pre_ln_gb300``.
"""
import math

import torch

own = False

HD = 64  # head dimension of the whole library
LOG2E = 1.4426950408889634
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # attention of one new token: one conversation of a GPT-2 small, mid-context (latency)
        dict(name="attn-single", op="attn", seqs=1, heads=12, kv_heads=12, length=777, page=16, window=0, sinks=0,
             dtype="bf16", append=True),
        # a decode batch at the benchmark's cache length, ragged
        dict(name="attn-batch64", op="attn", seqs=64, heads=12, kv_heads=12, length=1087, page=16, window=0, sinks=0,
             dtype="bf16", append=True),
        # long documents with query heads that share key-value heads; the query reads only (scoring a probe token)
        dict(name="attn-long-grouped", op="attn", seqs=16, heads=16, kv_heads=4, length=32768, page=64, window=0,
             sinks=0, dtype="f16", append=False),
        # endless chat at GPT-2 XL width: a window of 1024 and four first tokens, older pages given back
        dict(name="attn-window-xl", op="attn", seqs=128, heads=25, kv_heads=25, length=8000, page=32, window=1024,
             sinks=4, dtype="bf16", append=True),
        # the new token's K and V of a decode batch into the cache (latency)
        dict(name="write-step", op="write", seqs=64, kv_heads=12, tokens=1, length=1087, page=16, dtype="bf16"),
        # ragged prompts of a GPT-2 XL batch into the cache
        dict(name="write-prompts", op="write", seqs=16, kv_heads=25, tokens=1023, length=0, page=32, dtype="bf16"),
        # eight samples drawn from one prompt on GPT-2 small: share its pages, split off the last one
        dict(name="fork-samples8", op="fork", layers=12, kv_heads=12, page=16, prompts=1, samples=8, length=1019,
             dtype="bf16"),
        # sixteen prompts with seven samples each, GPT-2 medium, larger pages
        dict(name="fork-samples112", op="fork", layers=24, kv_heads=16, page=64, prompts=16, samples=7, length=700,
             dtype="bf16"),
        # a small pool after half of its sequences ended
        dict(name="compact-small", op="compact", layers=12, kv_heads=12, page=16, pages=256, used=128, seqs=16,
             dtype="bf16"),
        # a GPT-2 medium pool, 60 percent in use
        dict(name="compact-large", op="compact", layers=24, kv_heads=16, page=16, pages=1500, used=900, seqs=64,
             dtype="f16"),
        # scores of a decode step's tokens, part of the vocabulary masked out (latency)
        dict(name="logprobs-step", op="logprobs", rows=64, vocab=50257, top=5, dtype="f32", masked=True),
        # scores of a whole batch of texts, 8 x 1024 positions
        dict(name="logprobs-texts", op="logprobs", rows=8192, vocab=50257, top=20, dtype="bf16", masked=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "write", "fork", "compact", "logprobs", "logprobs"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    dtype = rng.choice(["bf16", "f16"])
    if op == "attn":
        heads, kv_heads = rng.choice(
            [(12, 12), (16, 16), (20, 20), (25, 25), (16, 4), (12, 1), (20, 5), (25, 1), (32, 4)])
        length = _log_int(rng, 1, 32768)
        window = rng.choice([0, 0, _log_int(rng, 16, 4096)])
        sinks = rng.choice([0, 1, 4, rng.randint(5, 64)]) if window else 0
        seen = min(length, window + sinks) if window else length
        most = max(1, min(128, (3 << 20) // (seen * kv_heads + 1)))
        return dict(op=op, seqs=_log_int(rng, 1, most), heads=heads, kv_heads=kv_heads, length=length, page=page,
                    window=window, sinks=sinks, dtype=dtype, append=rng.random() < 0.7)
    if op == "write":
        seqs, kv_heads = _log_int(rng, 1, 128), rng.choice([1, 4, 12, 16, 20, 25])
        most = max(1, min(1024, 409600 // (seqs * kv_heads)))
        return dict(op=op, seqs=seqs, kv_heads=kv_heads, tokens=_log_int(rng, 1, most), length=rng.randint(0, 300),
                    page=page, dtype=dtype)
    layers, kv_heads = rng.choice([(12, 12), (24, 16), (36, 20), (12, 1), (24, 4)])
    if op == "fork":
        size = layers * 2 * kv_heads * page * HD * 2
        most = max(1, min(128, (350 << 20) // size))
        prompts = _log_int(rng, 1, min(16, most))
        length = _log_int(rng, 1, max(2, min(1024, page * (1 << 30) // (size * prompts))))
        return dict(op=op, layers=layers, kv_heads=kv_heads, page=page, prompts=prompts,
                    samples=rng.randint(1, max(1, most // prompts)), length=length, dtype=dtype)
    if op == "compact":
        size = layers * 2 * kv_heads * page * HD * 2
        pages = _log_int(rng, 8, max(9, min(4000, (2 << 30) // size)))
        used = max(1, int(pages * rng.uniform(0.1, 0.95)))
        return dict(op=op, layers=layers, kv_heads=kv_heads, page=page, pages=pages, used=used,
                    seqs=rng.randint(1, min(64, used)), dtype=dtype)
    vocab = rng.choice([_log_int(rng, 40, 150000), 50257, 50304])
    dtype = rng.choice(["bf16", "f16", "f32"])
    most = max(1, min(8192, (800 << 20) // (vocab * (4 if dtype == "f32" else 2))))
    return dict(op=op, rows=_log_int(rng, 1, most), vocab=vocab, top=rng.choice([0, 1, 5, 20, 32]), dtype=dtype,
                masked=rng.random() < 0.4)


# ------------------------------------------------------------------ sizes that follow from a case
def _ragged(n, longest):
    """Lengths of n sequences: the longest, and others down to half of it."""
    return [longest - (b * 977) % (longest // 2 + 1) for b in range(n)]


def _attn_lens(case):
    """Cached positions of each slot before the call; one slot of a batch of eight or more is idle (-1)."""
    lens = _ragged(case["seqs"], case["length"])
    if case["seqs"] >= 8:
        lens[5] = -1
    return lens


def _seen(case, length):
    """Positions that the query of one sequence attends over."""
    n = length + 1 if case["append"] else length
    return max(0, min(n, case["window"] + case["sinks"]) if case["window"] else n)


def _row_bytes(case):
    return HD * (4 if case["dtype"] == "f32" else 2)


def work(case):
    op = case["op"]
    if op == "attn":
        row, seen, bytes_, active = _row_bytes(case), 0, 0, 0
        for n in _attn_lens(case):
            if n >= 0:
                seen += _seen(case, n)
                active += 1
        new = active * case["kv_heads"] * 2 * row if case["append"] else 0
        old = (seen - active if case["append"] else seen) * case["kv_heads"] * 2 * row
        bytes_ = old + 2 * new + 2 * active * case["heads"] * row + 4 * active * case["heads"]
        return {"bytes": bytes_, "flops": 4 * HD * case["heads"] * seen}
    if op == "write":
        rows = sum(_new_counts(case))
        return {"bytes": 2 * rows * case["kv_heads"] * 2 * _row_bytes(case), "flops": 0}
    if op == "fork":
        rows = sum(n % case["page"] for n in _ragged(case["prompts"], case["length"])) * case["samples"]
        tables = 8 * case["prompts"] * (1 + case["samples"]) * (case["length"] // case["page"] + 1)
        return {"bytes": 2 * rows * case["layers"] * 2 * case["kv_heads"] * _row_bytes(case) + tables, "flops": 0}
    if op == "compact":
        size = case["layers"] * 2 * case["kv_heads"] * case["page"] * _row_bytes(case)
        return {"bytes": 2 * _moves(case) * size + 8 * (case["used"] + case["pages"]), "flops": 0}
    elem = 4 if case["dtype"] == "f32" else 2
    return {"bytes": case["rows"] * (case["vocab"] * elem + 16 + 8 * case["top"]),
            "flops": 6 * case["rows"] * case["vocab"]}


def _new_counts(case):
    """New tokens of each sequence of a prompt batch: the full count, and others down to half of it."""
    return _ragged(case["seqs"], case["tokens"])


def _moves(case):
    """Pages in use that lie behind the first `used` places of the pool."""
    used, pages = case["used"], case["pages"]
    return min(pages - used, used, round(used * (1 - used / pages)))


# ------------------------------------------------------------------ inputs
def _rand(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _pool(g, pages, layers, kv_heads, page, dtype):
    return torch.randn((pages, layers, 2, kv_heads, page, HD), generator=g, device="cuda", dtype=dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _cache(state):
    """The cache's handle and the workspace that a program keeps beside its buffers."""
    import gpt_pre_ln_gb300 as G
    if state["op"] == "logprobs":
        return
    cache = G.paged_cache(state["pages"], state["refs"], state["table"], state["lens"])
    need = G.gpt2_pages_workspace_bytes(cache)
    if state["op"] == "attn":
        need = max(need, G.gpt2_attention_paged_workspace_bytes(cache, state["case"]["heads"]))
    state["cache"], state["ws"], state["ws_bytes"] = cache, torch.empty(need, device="cuda", dtype=torch.uint8), need


def _placed(g, columns, spare):
    """A table whose wanted entries (True in the rows of `columns`) name pages in random order; and the page count."""
    want = torch.tensor(columns, dtype=torch.bool)
    count = int(want.sum())
    ids = torch.randperm(count + spare, generator=g, device="cuda")[:count].to(torch.int32)
    table = torch.full(want.shape, -1, dtype=torch.int32, device="cuda")
    table[want.cuda()] = ids
    return table, count + spare


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": dict(case), "op": case["op"]}
    dtype = DTYPES[case["dtype"]]
    op = case["op"]
    if op == "attn":
        page, lens, layers = case["page"], _attn_lens(case), 2
        cols = max(1, (case["length"] + 1 + page - 1) // page)
        rows = []
        for n in lens:
            total = n + 1 if case["append"] else n
            first = max(0, total - case["window"]) if case["window"] else 0
            sinks = case["sinks"] if case["window"] else 0
            rows.append([c * page < total and ((c + 1) * page > first or c * page < sinks) for c in range(cols)])
        table, pages = _placed(g, rows, 8)
        state["pages"] = _pool(g, pages, layers, case["kv_heads"], page, dtype)
        state["refs"] = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
        state["table"], state["lens"] = table, _ints(lens)
        width = case["heads"] + 2 * case["kv_heads"]  # heads of one row of the fused projection
        state["qkv"] = _rand(g, (case["seqs"], width * HD), dtype)
        state["out"] = torch.zeros((case["seqs"], case["heads"] * HD), device="cuda", dtype=dtype)
        state["lse"] = torch.zeros((case["seqs"], case["heads"]), device="cuda", dtype=torch.float32)
        state["layer"], state["longest"] = 1, max([1] + [_seen(case, n) for n in lens if n >= 0])
    elif op == "write":
        page, seqs = case["page"], case["seqs"]
        counts, lens = _new_counts(case), _ragged(seqs, case["length"])
        cols = max(-(-(n + c) // page) for n, c in zip(lens, counts))
        rows = [[c * page < n + t for c in range(cols)] for n, t in zip(lens, counts)]
        table, pages = _placed(g, rows, 4)
        state["pages"] = _pool(g, pages, 2, case["kv_heads"], page, dtype)
        state["refs"] = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
        state["table"], state["lens"], state["counts"] = table, _ints(lens), _ints(counts)
        state["qkv"] = _rand(g, (seqs * case["tokens"], 3 * case["kv_heads"] * HD), dtype)
        state["layer"] = 1
    elif op == "fork":
        page, prompts = case["page"], case["prompts"]
        lens = _ragged(prompts, case["length"])
        cols = case["length"] // page + 1
        rows = [[c * page < n for c in range(cols)] for n in lens]
        rows += [[False] * cols] * (prompts * case["samples"])
        table, pages = _placed(g, rows, prompts * case["samples"] + 8)
        state["pages"] = _pool(g, pages, case["layers"], case["kv_heads"], page, dtype)
        state["refs"] = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
        state["table"], state["lens"] = table, _ints(lens + [-1] * (prompts * case["samples"]))
        state["parents"] = _ints([i // case["samples"] for i in range(prompts * case["samples"])])
        state["children"] = _ints(list(range(prompts, prompts * (1 + case["samples"]))))
        state["new"] = _ints([0] * prompts + [1] * (prompts * case["samples"]))
    elif op == "compact":
        used, pages, moves = case["used"], case["pages"], _moves(case)
        low = torch.randperm(used, generator=g, device="cuda")[:used - moves]
        high = used + torch.randperm(pages - used, generator=g, device="cuda")[:moves]
        ids = torch.cat([low, high])[torch.randperm(used, generator=g, device="cuda")].to(torch.int32)
        cols = -(-used // case["seqs"])
        table = torch.full((case["seqs"] * cols,), -1, dtype=torch.int32, device="cuda")
        table[:used] = ids
        state["pages"] = _pool(g, pages, case["layers"], case["kv_heads"], case["page"], dtype)
        state["table0"] = table.view(case["seqs"], cols)
        state["refs0"] = torch.bincount(ids.long(), minlength=pages).to(torch.int32)
        state["table"], state["refs"] = state["table0"].clone(), state["refs0"].clone()
        state["lens"] = ((state["table"] >= 0).sum(1) * case["page"]).to(torch.int32)
        state["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        rows, vocab = case["rows"], case["vocab"]
        ld = -(-vocab // 8) * 8
        logits = _rand(g, (rows, ld), dtype).mul_(2.5)
        tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        if case["masked"]:  # constrained decoding: three in ten entries cannot come next, the chosen token can
            gone = torch.rand(ld, generator=g, device="cuda") < 0.3
            keep = logits.gather(1, tokens[:, None])
            logits[:, gone] = -math.inf
            logits.scatter_(1, tokens[:, None], keep)
        state["logits"], state["tokens"], state["ld"] = logits, tokens.to(torch.int32), ld
        for k in ("logprob", "entropy", "lse"):
            state[k] = torch.empty(rows, device="cuda", dtype=torch.float32)
        state["top_ids"] = torch.empty((rows, case["top"]), device="cuda", dtype=torch.int32)
        state["top_logprobs"] = torch.empty((rows, case["top"]), device="cuda", dtype=torch.float32)
    if own:
        _cache(state)
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["op"]](state)


def _run_own(s):
    import gpt_pre_ln_gb300 as G
    c, op = s["case"], s["op"]
    kinds = {"bf16": G.BF16, "f16": G.F16, "f32": G.F32}
    if op == "attn":
        h, kv, ld = c["heads"], c["kv_heads"], s["qkv"].shape[1]
        at = s["qkv"].data_ptr()
        k_new = at + 2 * HD * h if c["append"] else None
        v_new = at + 2 * HD * (h + kv) if c["append"] else None
        G.gpt2_attention_paged(s["cache"], s["layer"], at, ld, k_new, v_new, ld, s["out"], h * HD, s["lse"], h, 0.125,
                               c["window"], c["sinks"], s["ws"], s["ws_bytes"])
        return {"out": s["out"], "lse": s["lse"], "pages": s["pages"]}
    if op == "write":
        kv, at = c["kv_heads"], s["qkv"].data_ptr()
        G.gpt2_pages_write(s["cache"], s["layer"], at + 2 * HD * kv, at + 4 * HD * kv, 3 * kv * HD, c["tokens"],
                           s["counts"])
        return {"pages": s["pages"]}
    if op == "fork":
        n = c["prompts"] * c["samples"]
        G.gpt2_pages_free(s["cache"], s["children"], n, 0, 0)
        G.gpt2_pages_fork(s["cache"], s["parents"], s["children"], n)
        G.gpt2_pages_reserve(s["cache"], s["new"], s["ws"], s["ws_bytes"])
        return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "pages": s["pages"]}
    if op == "compact":
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        G.gpt2_pages_compact(s["cache"], s["count"], s["ws"], s["ws_bytes"])
        return {"table": s["table"], "refs": s["refs"], "count": s["count"], "pages": s["pages"]}
    G.gpt2_token_logprobs(s["logits"], s["ld"], kinds[c["dtype"]], c["rows"], c["vocab"], s["tokens"], s["logprob"],
                          s["entropy"], s["lse"], c["top"], s["top_ids"], s["top_logprobs"])
    return {k: s[k] for k in ("logprob", "entropy", "lse", "top_ids", "top_logprobs")}


def _plain_attn(s):
    c, table, lens, pages, layer = s["case"], s["table"].long(), s["lens"].long(), s["pages"], s["layer"]
    h, kv, page = c["heads"], c["kv_heads"], c["page"]
    q, k_new, v_new = s["qkv"].view(c["seqs"], -1, HD).split([h, kv, kv], 1)
    active = lens >= 0
    n = lens + 1 if c["append"] else lens
    if c["append"]:
        rows = active.nonzero()[:, 0]
        at = table[rows, lens[rows] // page]
        pages[at, layer, 0, :, lens[rows] % page] = k_new[rows]
        pages[at, layer, 1, :, lens[rows] % page] = v_new[rows]
    i = torch.arange(s["longest"], device="cuda")[None, :]
    if c["window"]:
        behind = (n - c["window"]).clamp(min=0)[:, None]
        first = behind.clamp(max=c["sinks"])
        i = torch.where(i < first, i, i - first + behind)
    seen = (i < n[:, None])
    i = torch.where(seen, i, 0).expand(c["seqs"], -1)
    at = table.gather(1, i // page).clamp(min=0)
    k = pages[at, layer, 0, :, i % page].float()  # [seqs, positions, kv heads, 64]
    v = pages[at, layer, 1, :, i % page].float()
    qf = q.float().view(c["seqs"], kv, h // kv, HD)
    z = torch.einsum("bhgd,bnhd->bhgn", qf, k) * 0.125
    z = z.masked_fill(~seen[:, None, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgn,bnhd->bhgd", p, v.masked_fill(~seen[:, :, None, None], 0.0))
    out = out / torch.where(total == 0, 1.0, total)
    lse = ((m + torch.log(total)) * LOG2E).view(c["seqs"], h)
    s["out"].copy_(torch.where(active[:, None], out.reshape(c["seqs"], h * HD).to(q.dtype), s["out"]))
    s["lse"].copy_(torch.where(active[:, None], lse, s["lse"]))
    return {"out": s["out"], "lse": s["lse"], "pages": pages}


def _plain_write(s):
    c, pages, layer, lens = s["case"], s["pages"], s["layer"], s["lens"].long()
    t = torch.arange(c["tokens"], device="cuda")[None, :]
    b, t = (t < s["counts"][:, None]).nonzero(as_tuple=True)
    pos = lens[b] + t
    at = s["table"].long()[b, pos // c["page"]]
    _, k, v = s["qkv"].view(c["seqs"], c["tokens"], 3, c["kv_heads"], HD).unbind(2)
    pages[at, layer, 0, :, pos % c["page"]] = k[b, t]
    pages[at, layer, 1, :, pos % c["page"]] = v[b, t]
    return {"pages": pages}


def _counted(refs, ids, by):
    refs.index_add_(0, ids.reshape(-1), torch.full((ids.numel(),), by, dtype=refs.dtype, device=refs.device))


def _plain_fork(s):
    c, table, lens, refs, pages, page = s["case"], s["table"], s["lens"], s["refs"], s["pages"], s["case"]["page"]
    parents, children = s["parents"].long(), s["children"].long()
    # the children's slots are given back ...
    old = table[children]
    _counted(refs, old[old >= 0].long(), -1)
    table[children] = -1
    lens[children] = -1
    # ... and share their parents' pages
    column = torch.arange(table.shape[1], device="cuda")[None, :]
    mine = torch.where(column * page < lens[parents][:, None], table[parents], -1)
    _counted(refs, mine[mine >= 0].long(), 1)
    table[children] = mine
    lens[children] = lens[parents]
    # room for the new tokens: a page where there is none, and one of its own where the page is shared (the last
    # writer of a page that nobody else reads keeps it)
    new = s["new"]
    wants = (lens >= 0) & (new > 0)
    first, last = lens.div(page, rounding_mode="floor"), (lens + new - 1).div(page, rounding_mode="floor")
    span = wants[:, None] & (column >= first[:, None]) & (column <= last[:, None])
    entry = table.long()
    shared = span & (entry >= 0) & (refs[entry.clamp(min=0)] > 1)
    flat = torch.arange(table.numel(), device="cuda").view_as(entry)
    writers = torch.zeros(refs.numel(), dtype=torch.int32, device="cuda")
    _counted(writers, entry[shared], 1)
    final = torch.full((refs.numel(),), -1, dtype=torch.long, device="cuda")
    final.scatter_reduce_(0, entry[shared], flat[shared], "amax")
    safe = entry.clamp(min=0)
    keeps = (writers[safe] == refs[safe]) & (final[safe] == flat)
    split = shared & ~keeps
    b, col = (split | (span & (entry < 0))).nonzero(as_tuple=True)
    fresh = (refs == 0).nonzero()[:b.numel(), 0]
    was = entry[b, col]
    _counted(refs, was[was >= 0], -1)
    refs[fresh] = 1
    table[b, col] = fresh.to(torch.int32)
    held = (lens[b] - col * page).clamp(min=0, max=page)  # positions of a split page that hold something
    moved = ((was >= 0) & (held > 0) & (col == first[b])).nonzero()[:, 0]
    pair, row = (torch.arange(page, device="cuda")[None, :] < held[moved][:, None]).nonzero(as_tuple=True)
    pages[fresh[moved][pair], :, :, :, row] = pages[was[moved][pair], :, :, :, row]
    return {"table": table, "lens": lens, "refs": refs, "pages": pages}


def _plain_compact(s):
    table, refs, pages = s["table"], s["refs"], s["pages"]
    table.copy_(s["table0"])
    refs.copy_(s["refs0"])
    used = refs > 0
    count = used.sum()
    index = torch.arange(refs.numel(), device="cuda")
    holes = (~used & (index < count)).nonzero()[:, 0]
    movers = (used & (index >= count)).nonzero()[:, 0].flip(0)  # the first hole takes the last page
    pages[holes] = pages[movers]
    refs[holes] = refs[movers]
    refs[movers] = 0
    now = index.to(torch.int32)
    now[movers] = holes.to(torch.int32)
    table.copy_(torch.where(table >= 0, now[table.clamp(min=0).long()], table))
    s["count"].copy_(count.view(1))
    return {"table": table, "refs": refs, "count": s["count"], "pages": pages}


def _plain_logprobs(s):
    c = s["case"]
    x = s["logits"][:, :c["vocab"]].float()
    m = x.amax(1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    entropy = log_total - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / total
    logprob = d.gather(1, s["tokens"].long()[:, None]) - log_total
    out = {"logprob": logprob[:, 0], "entropy": entropy[:, 0], "lse": (m + log_total)[:, 0]}
    value, index = torch.sort(d, dim=1, descending=True, stable=True)
    out["top_ids"] = index[:, :c["top"]].to(torch.int32)
    out["top_logprobs"] = value[:, :c["top"]] - log_total
    return out


_PLAIN = {"attn": _plain_attn, "write": _plain_write, "fork": _plain_fork, "compact": _plain_compact,
          "logprobs": _plain_logprobs}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    def attn(c, s):
        table, pages, page, layer = s["table"].tolist(), s["pages"], c["page"], s["layer"]
        h, kv = c["heads"], c["kv_heads"]
        out, lse = s["out"].double(), s["lse"].double()
        for b, n in enumerate(s["lens"].tolist()):
            if n < 0:
                continue
            row = s["qkv"][b].view(-1, HD)
            if c["append"]:
                at = table[b][n // page]
                pages[at, layer, 0, :, n % page] = row[h:h + kv]
                pages[at, layer, 1, :, n % page] = row[h + kv:]
                n += 1
            seen = [p for p in range(n) if not c["window"] or p >= n - c["window"] or p < c["sinks"]]
            if not seen:
                out[b], lse[b] = 0, -math.inf
                continue
            at = torch.tensor([table[b][p // page] for p in seen], device="cuda")
            off = torch.tensor([p % page for p in seen], device="cuda")
            for g in range(kv):
                k, v = pages[at, layer, 0, g, off].double(), pages[at, layer, 1, g, off].double()
                mine = slice(g * (h // kv), (g + 1) * (h // kv))
                z = row[:h][mine].double() @ k.t() / 8
                lse[b, mine] = torch.logsumexp(z, 1) / math.log(2)
                out[b].view(h, HD)[mine] = torch.softmax(z, 1) @ v
        return {"out": out, "lse": lse, "pages": pages}

    def write(c, s):
        table, pages, page = s["table"].tolist(), s["pages"], c["page"]
        for b, (n, count) in enumerate(zip(s["lens"].tolist(), s["counts"].tolist())):
            rows = s["qkv"][b * c["tokens"]:b * c["tokens"] + count].view(count, 3, c["kv_heads"], HD)
            t = 0
            while t < count:  # the tokens that share a page
                off = (n + t) % page
                end = min(count, t + page - off)
                at = pages[table[b][(n + t) // page], s["layer"]]
                at[:, :, off:off + end - t] = rows[t:end, 1:].permute(1, 2, 0, 3)
                t = end
        return {"pages": pages}

    def fork(c, s):
        table, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
        pages, page = s["pages"], c["page"]
        for child, parent in zip(s["children"].tolist(), s["parents"].tolist()):
            table[child], lens[child] = list(table[parent]), lens[parent]
            for p in table[child]:
                if p >= 0:
                    refs[p] += 1
        free = [p for p, r in enumerate(refs) if r == 0]
        for b, new in enumerate(s["new"].tolist()):
            for pos in range(lens[b], lens[b] + new):
                p = table[b][pos // page]
                if p < 0 or refs[p] > 1:
                    fresh = free.pop(0)
                    if p >= 0:
                        refs[p] -= 1
                        pages[fresh, :, :, :, :pos % page] = pages[p, :, :, :, :pos % page]
                    table[b][pos // page], refs[fresh] = fresh, 1
        return {"table": _ints(table), "lens": _ints(lens), "refs": _ints(refs), "pages": pages}

    def compact(c, s):
        table, refs, pages = s["table0"].tolist(), s["refs0"].tolist(), s["pages"]
        low, high, now = 0, len(refs) - 1, {}
        while True:
            while low < len(refs) and refs[low]:
                low += 1
            while high >= 0 and not refs[high]:
                high -= 1
            if low >= high:
                break
            pages[low] = pages[high]
            refs[low], refs[high], now[high] = refs[high], 0, low
        table = [[now.get(p, p) for p in row] for row in table]
        return {"table": _ints(table), "refs": _ints(refs), "count": _ints([low]), "pages": pages}

    def logprobs(c, s):
        x = s["logits"][:, :c["vocab"]].double()
        lse = torch.logsumexp(x, 1)
        x -= lse[:, None]
        logprob = x[torch.arange(c["rows"], device="cuda"), s["tokens"].long()]
        entropy = torch.special.entr(torch.exp(x)).sum(1)
        ids, values = [], []
        index = torch.arange(c["vocab"], dtype=torch.int32, device="cuda")[None, :]
        left = torch.ones(x.shape, dtype=torch.bool, device="cuda")
        for _ in range(c["top"]):
            best = x.amax(1, keepdim=True)
            at = torch.where((x == best) & left, index, c["vocab"]).amin(1, keepdim=True)
            ids.append(at.int())
            values.append(best)
            x.scatter_(1, at.long(), -math.inf)
            left.scatter_(1, at.long(), False)
        top = torch.cat(ids, 1) if ids else torch.empty((c["rows"], 0), dtype=torch.int32, device="cuda")
        top_logprobs = torch.cat(values, 1) if ids else torch.empty((c["rows"], 0), dtype=torch.float64, device="cuda")
        return {"logprob": logprob, "entropy": entropy, "lse": lse, "top_ids": top, "top_logprobs": top_logprobs}

    return {"attn": attn, "write": write, "fork": fork, "compact": compact, "logprobs": logprobs}[case["op"]](
        dict(case), prepare(case, seed))
