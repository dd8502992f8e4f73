"""The paged key-value cache operators and the attention that reads the cache,
as measured workloads: one listed case per use, and drawn cases of the same
ranges.

``run`` makes one pass.  With ``own`` false it computes the operators from
their definitions with elementary torch operations in 32 bits, rounded once at
the end; with ``own`` true it makes the calls a program makes of
w4a4_block_scaled_amd.  ``exact`` gives the attention outputs and the appended
cache in 64 bits.

Notation: a cache holds pages of `page` tokens, [pages, page, kv_heads, dim];
a sequence's token p is on page tables[s, p // page], row p % page; lens[s] is
its number of tokens, those of the present call included.  A query at position
p sees token t if t <= p and (window == 0, or t > p - window, or t < sinks).
"""
import math

import torch

own = False

NEG = float("-inf")
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}


def listed():
    llama = {"q_heads": 32, "kv_heads": 8, "dim": 128}
    qwen = {"q_heads": 28, "kv_heads": 4, "dim": 128}
    return [
        # one chat, a few hundred tokens in: the call is as short as its launches
        {"name": "decode one short", "op": "decode", **llama, "seqs": 1, "low": 513, "high": 513, "page": 16,
         "type": "bf16", "window": 0, "sinks": 0},
        # an ordinary serving batch, every sequence of another length
        {"name": "decode ragged batch", "op": "decode", **llama, "seqs": 48, "low": 37, "high": 8191, "page": 16,
         "type": "bf16", "window": 0, "sinks": 0},
        # a few very long documents with an 8-bit cache: few rows, a long axis
        {"name": "decode long fp8", "op": "decode", **qwen, "seqs": 3, "low": 90001, "high": 131071, "page": 64,
         "type": "fp8", "window": 0, "sinks": 0},
        # a large batch that sees a window and the first tokens
        {"name": "decode window sinks", "op": "decode", "q_heads": 16, "kv_heads": 16, "dim": 64, "seqs": 128,
         "low": 300, "high": 6000, "page": 24, "type": "fp16", "window": 1024, "sinks": 4},
        # a short prompt, nothing in the cache before it
        {"name": "prefill short prompt", "op": "prefill", **llama, "seqs": 1, "q_low": 82, "q_high": 82, "past_low": 0,
         "past_high": 0, "page": 16, "type": "bf16", "window": 0, "sinks": 0},
        # a whole prompt under a window with sinks
        {"name": "prefill window sinks", "op": "prefill", **llama, "seqs": 1, "q_low": 8192, "q_high": 8192,
         "past_low": 0, "past_high": 0, "page": 16, "type": "fp16", "window": 1024, "sinks": 4},
        # a ragged batch of prompt chunks on top of what the cache holds
        {"name": "prefill ragged chunks", "op": "prefill", **qwen, "seqs": 5, "q_low": 17, "q_high": 3001, "past_low": 0,
         "past_high": 6001, "page": 32, "type": "bf16", "window": 0, "sinks": 0},
        # a few tokens (drafted, or the rest of a prompt) on a long 8-bit cache: few rows
        {"name": "prefill few on long fp8", "op": "prefill", **llama, "seqs": 2, "q_low": 5, "q_high": 9,
         "past_low": 30000, "past_high": 33333, "page": 64, "type": "fp8", "window": 0, "sinks": 0},
        # one new token of every sequence of a decoding batch into the cache
        {"name": "append one token each", "op": "append", **llama, "seqs": 16, "q_low": 1, "q_high": 1,
         "past_low": 100, "past_high": 4000, "page": 16, "type": "bf16"},
        # whole prompts into an 8-bit cache
        {"name": "append prompts fp8", "op": "append", **qwen, "seqs": 7, "q_low": 33, "q_high": 4096, "past_low": 0,
         "past_high": 100, "page": 32, "type": "fp8"},
        # a step of parallel sampling over all layers: branches are dropped, forked again, and get room for a token
        {"name": "fork branches", "op": "fork", **llama, "layers": 16, "parents": 4, "branches": 8, "low": 100,
         "high": 2050, "page": 16, "type": "bf16"},
        # a cache left full of holes by finished requests is closed up
        {"name": "compact", "op": "compact", **llama, "layers": 4, "seqs": 64, "low": 30, "high": 3000, "page": 64,
         "type": "bf16", "dropped": 3},
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    g, kv, dim = rng.choice([(4, 8, 128), (7, 4, 128), (1, 16, 64), (8, 2, 128), (5, 3, 64), (1, 4, 256), (16, 1, 128)])
    case = {"op": rng.choice(["decode", "decode", "prefill", "prefill", "append", "fork", "compact"]), "q_heads": g * kv,
            "kv_heads": kv, "dim": dim, "page": rng.choice([8, 16, 16, 24, 32, 64, 128, 11]),
            "type": rng.choice(["bf16", "bf16", "fp16", "fp8"])}
    masks = {"window": rng.choice([0, 0, _log(rng, 16, 4096)]), "sinks": rng.choice([0, 4, rng.randrange(1, 130)])}
    if case["op"] == "decode":
        seqs = _log(rng, 1, 128)
        high = _log(rng, 64, min(131072, 400000 // seqs))
        return {**case, "seqs": seqs, "low": rng.randrange(1, high + 1), "high": high, **masks}
    if case["op"] == "prefill":
        seqs = _log(rng, 1, 5)
        q, past = _log(rng, 2, 2200), rng.choice([0, _log(rng, 16, 4000)])
        return {**case, "seqs": seqs, "q_low": rng.randrange(1, q + 1), "q_high": q, "past_low": rng.randrange(0, past + 1),
                "past_high": past, **masks}
    if case["op"] == "append":
        seqs = _log(rng, 1, 64)
        q, past = _log(rng, 1, 16384 // seqs), _log(rng, 1, 4000)
        return {**case, "seqs": seqs, "q_low": rng.randrange(1, q + 1), "q_high": q, "past_low": rng.randrange(0, past + 1),
                "past_high": past}
    high = _log(rng, 40, 2500)
    case = {**case, "layers": _log(rng, 1, 8), "low": rng.randrange(1, high + 1), "high": high}
    if case["op"] == "fork":
        return {**case, "parents": rng.randrange(1, 5), "branches": rng.randrange(1, 9)}
    return {**case, "seqs": rng.randrange(8, 65), "dropped": rng.randrange(2, 5)}


def _spread(n, low, high, turn):
    """n whole numbers over low..high, both ends among them, in a mixed order that the case fixes."""
    step = next(k for k in (turn, 11, 13, 17, 1) if math.gcd(k, n) == 1)
    return [low + ((i * step) % n) * (high - low) // max(1, n - 1) for i in range(n)] if n > 1 else [high]


def _lengths(case):
    """(tokens of each sequence, new ones included; new tokens of each)."""
    if case["op"] in ("prefill", "append"):
        q = _spread(case["seqs"], case["q_low"], case["q_high"], 5)
        past = _spread(case["seqs"], case["past_low"], case["past_high"], 7)
        return [a + b for a, b in zip(q, past)], q
    if case["op"] == "fork":
        return _spread(case["parents"], case["low"], case["high"], 3), None
    return _spread(case["seqs"], case["low"], case["high"], 7), None


def _values(shape, kind, gen):
    x = torch.empty(shape, dtype=torch.float16 if kind == "fp16" else torch.bfloat16, device="cuda")
    x.normal_(generator=gen)
    return x.to(TORCH[kind]) if kind == "fp8" else x


def _tables(lens, page, pages, rows, width, gen):
    """Block tables of `rows` sequences (those past len(lens) empty) over shuffled pages."""
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    held = [-(-n // page) for n in lens]
    tables = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(held):
        tables[s, :n] = order[at:at + n]
        at += n
    return tables


def _device(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens, new = _lengths(case)
    page, kv, dim, kind = case["page"], case["kv_heads"], case["dim"], case["type"]
    held = sum(-(-n // page) for n in lens)
    state = {"case": case, "lens": _device(lens)}
    if case["op"] in ("decode", "prefill", "append"):
        width = -(-max(lens) // page) + 1
        pages = held + 3
        state["k"] = _values((pages, page, kv, dim), kind, gen)
        state["v"] = _values((pages, page, kv, dim), kind, gen)
        state["tables"] = _tables(lens, page, pages, len(lens), width, gen)
        for name in ("k_scale", "v_scale"):
            state[name] = torch.rand(kv, generator=gen, device="cuda") + 0.5 if kind == "fp8" else None
        high = "fp16" if kind == "fp16" else "bf16"
        if case["op"] == "decode":
            state["q"] = _values((len(lens), case["q_heads"], dim), high, gen)
        else:
            ends = [0]
            for n in new:
                ends.append(ends[-1] + n)
            state["cu"] = _device(ends)
            # queries, keys and values as a fused projection leaves them: slices of one row per token
            rows = _values((ends[-1], case["q_heads"] + 2 * kv, dim), high, gen)
            state["q"], state["k_new"], state["v_new"] = rows.split([case["q_heads"], kv, kv], dim=1)
        return state
    if case["op"] == "fork":
        children = case["parents"] * case["branches"]
        rows, width = case["parents"] + children, -(-max(lens) // page) + 2
        pages = held + rows + children + 5
        state["children"] = _device(range(case["parents"], rows))
        state["parents"] = state["children"] % case["parents"]
        state["lens"] = _device(lens + [0] * children)
    else:
        rows, width, pages = case["seqs"], -(-max(lens) // page) + 1, held + held // 3 + 5
    pool = _values((case["layers"], 2, pages, page, kv, dim), kind, gen)
    tables = _tables(lens, page, pages, rows, width, gen)
    if case["op"] == "compact":
        tables[torch.arange(rows, device="cuda") % case["dropped"] == 1] = -1  # those that have finished
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[tables[tables >= 0].long()] = 1
    state.update(pool=pool, tables=tables, refs=refs)
    if case["op"] == "compact":  # the bookkeeping as it is before: each pass starts from it
        state["before"] = torch.cat([tables.flatten(), refs])
        state["work"] = state["before"].clone()
        state["tables"], state["refs"] = state["work"][: tables.numel()].view_as(tables), state["work"][tables.numel():]
    return state


def run(state):
    case = state["case"]
    if own:
        import w4a4_block_scaled_amd as w4
        return _run_own(w4, case, state)
    return {"decode": _decode, "prefill": _prefill, "append": _append, "fork": _fork, "compact": _compact}[case["op"]](case, state)


def _run_own(w4, case, s):
    if case["op"] == "decode":
        return w4.attn_decode(s["q"], s["k"], s["v"], s["tables"], s["lens"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                              window=case["window"], sinks=case["sinks"])
    if case["op"] == "prefill":
        return w4.attn_prefill(s["q"], s["cu"], s["k"], s["v"], s["tables"], s["lens"], k_scale=s["k_scale"],
                               v_scale=s["v_scale"], window=case["window"], sinks=case["sinks"])
    if case["op"] == "append":
        w4.kv_append(s["k_new"], s["v_new"], s["k"], s["v"], s["tables"], s["lens"], cu_seqlens=s["cu"],
                     k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["k"], s["v"]
    if case["op"] == "fork":
        w4.kv_free(s["tables"], s["lens"], s["refs"], s["children"])
        w4.kv_fork(s["pool"], s["tables"], s["lens"], s["refs"], s["parents"], s["children"])
        s["lens"] += 1
        w4.kv_reserve(s["tables"], s["lens"], s["refs"], case["page"])
        s["lens"] -= 1
        return s["pool"], s["tables"], s["lens"], s["refs"]
    s["work"].copy_(s["before"])
    remap = w4.kv_compact(s["pool"], s["tables"], s["refs"])
    return s["pool"], s["tables"], s["refs"], remap


# The plain forms.

def _gathered(cache, tables, scale):
    """The cache of every sequence in order, [seqs, kv_heads, tokens, dim] in 32 bits."""
    raw = cache.view(torch.uint8) if cache.element_size() == 1 else cache
    x = raw[tables.clamp(min=0).long()].view(cache.dtype).float()
    x = x.flatten(1, 2).transpose(1, 2)
    return (x if scale is None else x * scale[:, None, None]).contiguous()


def _seen(position, tokens, case):
    t = torch.arange(tokens, device="cuda")
    seen = t <= position[..., None]
    if case["window"]:
        seen &= (t > position[..., None] - case["window"]) | (t < case["sinks"])
    return seen


def _weights(scores, seen):
    scores = scores.masked_fill_(~seen, NEG)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = scores.sub_(top).exp_()
    return p.div_(p.sum(-1, keepdim=True).clamp(min=1e-38))


def _decode(case, s):
    k, v = _gathered(s["k"], s["tables"], s["k_scale"]), _gathered(s["v"], s["tables"], s["v_scale"])
    seqs, kv, tokens, dim = k.shape
    q = s["q"].float().view(seqs, kv, -1, dim)
    seen = _seen(s["lens"].long() - 1, tokens, case)[:, None, None, :]
    p = _weights(torch.matmul(q, k.transpose(2, 3)) / math.sqrt(dim), seen)
    return torch.matmul(p, v).reshape(seqs, -1, dim).to(s["q"].dtype)


def _rows(s):
    """For every new token: its sequence, its place among the sequence's new ones, its position."""
    count = s["cu"][1:] - s["cu"][:-1]
    seq = torch.repeat_interleave(torch.arange(len(count), device="cuda"), count.long())
    place = torch.arange(len(seq), device="cuda") - s["cu"][seq].long()
    return seq, place, (s["lens"] - count)[seq].long() + place


def _prefill(case, s):
    k, v = _gathered(s["k"], s["tables"], s["k_scale"]), _gathered(s["v"], s["tables"], s["v_scale"])
    seqs, kv, tokens, dim = k.shape
    seq, place, position = _rows(s)
    most = case["q_high"]
    q = torch.zeros(seqs, most, kv, case["q_heads"] // kv, dim, device="cuda")
    q[seq, place] = s["q"].float().view(len(seq), kv, -1, dim)
    at = torch.full((seqs, most), -1, device="cuda")
    at[seq, place] = position
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3).contiguous()  # [seqs, kv, heads of the group x rows, dim]
    scores = torch.matmul(q, k.transpose(2, 3)).div_(math.sqrt(dim)).view(seqs, kv, -1, most, tokens)
    p = _weights(scores, _seen(at, tokens, case)[:, None, None]).flatten(2, 3)
    out = torch.matmul(p, v).view(seqs, kv, -1, most, dim).permute(0, 3, 1, 2, 4)
    return out[seq, place].reshape(len(seq), -1, dim).to(s["q"].dtype)


def _append(case, s):
    seq, _, position = _rows(s)
    page = s["tables"][seq, position // case["page"]].long()
    for cache, new, scale in ((s["k"], s["k_new"], s["k_scale"]), (s["v"], s["v_new"], s["v_scale"])):
        if scale is not None:
            new = (new.float() / scale[:, None]).clamp(-448, 448).to(cache.dtype).view(torch.uint8)
            cache = cache.view(torch.uint8)
        cache[page, position % case["page"]] = new
    return s["k"], s["v"]


def _free_pages(refs):
    return (refs == 0).nonzero()[:, 0]


def _fork(case, s):
    tables, lens, refs, page = s["tables"], s["lens"], s["refs"], case["page"]
    parents, children = s["parents"].long(), s["children"].long()
    pool = s["pool"].view(torch.uint8) if s["pool"].element_size() == 1 else s["pool"]
    # the branches' pages are let go
    old = tables[children]
    refs.index_add_(0, old[old >= 0].long(), torch.full_like(old[old >= 0], -1))
    # whole pages are shared, the last one is copied to the lowest free page
    n = lens[parents].long()
    index = torch.arange(tables.shape[1], device="cuda")
    rows = torch.where(index < (n // page)[:, None], tables[parents], -1)
    refs.index_add_(0, rows[rows >= 0].long(), torch.ones_like(rows[rows >= 0]))
    cut = n % page != 0
    source = tables[parents[cut], (n // page)[cut]].long()
    target = _free_pages(refs)[: len(source)]
    pool[:, :, target] = pool[:, :, source]
    rows[cut, (n // page)[cut]] = target.int()
    refs[target] = 1
    tables[children] = rows
    lens[children] = n.int()
    # room for one more token of every sequence
    last = lens.long() // page
    lack = tables.gather(1, last[:, None])[:, 0] < 0
    target = _free_pages(refs)[: int(lack.sum())]
    tables[lack.nonzero()[:, 0], last[lack]] = target.int()
    refs[target] = 1
    return s["pool"], tables, lens, refs


def _compact(case, s):
    s["work"].copy_(s["before"])
    tables, refs = s["tables"], s["refs"]
    pool = s["pool"].view(torch.uint8) if s["pool"].element_size() == 1 else s["pool"]
    live = (refs > 0).nonzero()[:, 0]
    source = live[live >= len(live)]
    target = _free_pages(refs)[: len(source)]
    pool[:, :, target] = pool[:, :, source]
    remap = torch.full((len(refs),), -1, dtype=torch.int32, device="cuda")
    remap[live] = live.int()
    remap[source] = target.int()
    refs[target] = refs[source]
    refs[source] = 0
    tables.copy_(torch.where(tables >= 0, remap[tables.clamp(min=0).long()], tables))
    return s["pool"], tables, refs, remap


def _visible(case, lens, new):
    """(query-token pairs that are visible, tokens that any query sees), summed over the sequences."""
    pairs = tokens = 0
    window, sinks = case["window"], case["sinks"]
    for n, m in zip(lens, new):
        first = n - m
        if not window:
            pairs += m * (first + 1 + n) // 2
            tokens += n
            continue
        # the query at p sees min(p + 1, window) tokens, and the sinks that lie before those
        ps = torch.arange(first, n, dtype=torch.int64)
        low = (ps - window + 1).clamp(min=0)
        pairs += int((ps + 1 - low + low.clamp(max=sinks)).sum())
        low = max(0, first - window + 1)
        tokens += n - low + min(low, sinks)
    return pairs, tokens


def work(case):
    lens, new = _lengths(case)
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    small = 1 if case["type"] == "fp8" else 2
    if case["op"] in ("decode", "prefill"):
        new = new or [1] * len(lens)
        pairs, tokens = _visible(case, lens, new)
        moved = tokens * (kv * dim * 2 * small + 4 / page) + sum(new) * case["q_heads"] * dim * 2 * 2
        return {"bytes": moved, "flops": pairs * case["q_heads"] * dim * 4}
    if case["op"] == "append":
        return {"bytes": sum(new) * kv * dim * 2 * (2 + small), "flops": 0}
    held = [-(-n // page) for n in lens]
    if case["op"] == "fork":
        pages = sum(n % page != 0 for n in lens) * case["branches"]
        book = sum(held) * (1 + case["branches"]) * 4 * 2
    else:
        left = [n for s, n in enumerate(held) if s % case["dropped"] != 1]
        # pages are shuffled over the cache: this share of the live ones lies behind the place where they end
        pages, total = sum(left), sum(held) + sum(held) // 3 + 5
        pages, book = int(pages * (total - pages) / total), (sum(left) + total) * 4 * 2
    return {"bytes": pages * case["layers"] * 2 * page * kv * dim * small * 2 + book, "flops": 0}


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    lens, new = _lengths(case)
    page, kv, dim = case["page"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        return tuple(_exact_cache(case, s, name, lens, new) for name in ("k", "v"))
    new = new or [1] * len(lens)
    outs, at = [], 0
    for i, (n, m) in enumerate(zip(lens, new)):
        p = torch.arange(n, device="cuda")
        where = s["tables"][i].long()[p // page] * page + p % page
        query = torch.arange(n - m, n, device="cuda")[:, None]
        hidden = p[None, :] > query
        if case["window"]:
            hidden = hidden | ((query - p[None, :] >= case["window"]) & (p[None, :] >= case["sinks"]))
        out = torch.empty(m, case["q_heads"], dim, dtype=torch.float64, device="cuda")
        for h in range(case["q_heads"]):
            j = h // (case["q_heads"] // kv)
            k, v = (s[c].flatten(0, 1)[:, j].double()[where] * (s[c + "_scale"][j].double() if small else 1.0)
                    for c, small in (("k", case["type"] == "fp8"), ("v", case["type"] == "fp8")))
            a = (s["q"][at:at + m, h].double() @ k.t()) * dim ** -0.5
            a[hidden] = NEG
            out[:, h] = torch.softmax(a, dim=-1) @ v
        outs.append(out)
        at += m
    return torch.cat(outs)


def _exact_cache(case, s, name, lens, new):
    """The cache after the new rows, from the nearest value of the 8-bit type in 64 bits (ties to the even one)."""
    cache = s[name].to(torch.float64)
    at = 0
    for i, (n, m) in enumerate(zip(lens, new)):
        p = torch.arange(n - m, n, device="cuda")
        x = s[name + "_new"][at:at + m].double()
        if case["type"] == "fp8":
            x = x / s[name + "_scale"].double()[:, None]
            exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
            step = torch.exp2(exponent - 3)
            x = (torch.round(x / step) * step).clamp(-448, 448)
        cache[s["tables"][i].long()[p // case["page"]], p % case["page"]] = x
        at += m
    return cache
