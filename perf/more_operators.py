"""Rotary positions, the paged cache held in 4 bits and what reads it, as
measured workloads: one listed case per use, and drawn cases of the same ranges.

``run`` makes one pass.  With ``own`` false it computes the operators from
their definitions with elementary torch operations in 32 bits (angles and
values that are rounded to 8 or 4 bits in 64), rounded once at the end; with
``own`` true it makes the calls a program makes of w4a4_block_scaled_amd.
``exact`` gives the outputs in 64 bits.

rope      x' = factor R(position * freqs) x on pairs (i, i + rot / 2), or (2 i, 2 i + 1)
          where interleaved, of the first `rot` values of every head; the rest stays
append    q and k of new tokens rotated by their places in their sequences, q to an
          output, k and v into a paged cache of 16, 8 or 4 bits
read      rows of the cache in 16 bits, in the order of their tokens
decode    attention of one token per sequence over a 4-bit cache
prefill   attention of chunks of new tokens over a 4-bit cache

A 4-bit page holds, for each kv head and token, dim / 2 bytes of E2M1 codes (low
nibble first): [heads, page, dim / 2]; behind them a scale byte b for every 32
values, standing for 2^(b - 127): [heads, dim / 32, page].  Pages begin at
multiples of 16 bytes.  A block's exponent is floor(log2 of its largest
magnitude) - 2.

A sequence's token p is on page tables[s, p // page], row p % page; lens[s] is
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
        # queries and keys of a small decoding batch, far into long sequences: as short as its launch
        {"name": "rope decoding batch", "op": "rope", "tokens": 16, "heads": 40, "dim": 128, "rot": 128,
         "interleaved": False, "type": "bf16", "base": 500000.0, "stretch": 1.0, "far": 131071, "scattered": True},
        # a long prompt, half of every head in adjacent pairs, positions compressed for a longer context
        {"name": "rope prompt part of head", "op": "rope", "tokens": 8191, "heads": 32, "dim": 128, "rot": 64,
         "interleaved": True, "type": "fp16", "base": 10000.0, "stretch": 4.0, "far": 8190, "scattered": False},
        # a decoding step of a ragged batch: rotate and store one token each
        {"name": "append one token each", "op": "append", **llama, "rot": 128, "interleaved": False, "base": 500000.0,
         "stretch": 1.0, "seqs": 48, "q_low": 1, "q_high": 1, "past_low": 36, "past_high": 8190, "page": 16,
         "type": "bf16", "rows": "bf16"},
        # prompt chunks into an 8-bit cache with pages of 24, a quarter of the head in adjacent pairs
        {"name": "append chunks fp8", "op": "append", "q_heads": 16, "kv_heads": 16, "dim": 64, "rot": 16,
         "interleaved": True, "base": 10000.0, "stretch": 1.0, "seqs": 5, "q_low": 17, "q_high": 701, "past_low": 0,
         "past_high": 3000, "page": 24, "type": "fp8", "rows": "fp16"},
        # whole prompts into a 4-bit cache, whose new rows are then copied out (for a cache elsewhere)
        {"name": "append prompts 4 bit", "op": "append", **qwen, "rot": 128, "interleaved": False, "base": 1000000.0,
         "stretch": 1.0, "seqs": 7, "q_low": 33, "q_high": 4096, "past_low": 0, "past_high": 100, "page": 32,
         "type": "fp4", "rows": "bf16"},
        # one short sequence leaves the cache
        {"name": "read one short", "op": "read", **llama, "seqs": 1, "q_low": 513, "q_high": 513, "past_low": 0,
         "past_high": 0, "page": 16, "rows": "bf16"},
        # a few long documents leave the cache
        {"name": "read long", "op": "read", **qwen, "seqs": 3, "q_low": 9001, "q_high": 32767, "past_low": 0,
         "past_high": 0, "page": 64, "rows": "fp16"},
        # one chat, a few hundred tokens in: the call is as short as its launches
        {"name": "decode one short", "op": "decode", **llama, "seqs": 1, "low": 513, "high": 513, "page": 16,
         "rows": "bf16", "window": 0, "sinks": 0},
        # an ordinary serving batch, every sequence of another length
        {"name": "decode ragged batch", "op": "decode", **llama, "seqs": 48, "low": 37, "high": 8191, "page": 16,
         "rows": "bf16", "window": 0, "sinks": 0},
        # a few very long documents: few rows, a long axis
        {"name": "decode long", "op": "decode", **qwen, "seqs": 3, "low": 90001, "high": 131071, "page": 64,
         "rows": "fp16", "window": 0, "sinks": 0},
        # a few drafted tokens on long documents: few rows
        {"name": "prefill few on long", "op": "prefill", **llama, "seqs": 2, "q_low": 5, "q_high": 9, "past_low": 30000,
         "past_high": 33333, "page": 64, "rows": "bf16", "window": 0, "sinks": 0},
        # a ragged batch of prompt chunks on top of what the cache holds
        {"name": "prefill ragged chunks", "op": "prefill", **qwen, "seqs": 5, "q_low": 17, "q_high": 3001, "past_low": 0,
         "past_high": 6001, "page": 32, "rows": "bf16", "window": 0, "sinks": 0},
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(["rope", "append", "append", "read", "decode", "decode", "prefill", "prefill"])
    g, kv, dim = rng.choice([(4, 8, 128), (7, 4, 128), (1, 16, 64), (8, 2, 128), (5, 3, 64), (1, 4, 256), (16, 1, 128)])
    turn = {"interleaved": rng.random() < 0.4, "base": rng.choice([10000.0, 500000.0]), "stretch": rng.choice([1.0, 1.0, 4.0, 8.0])}
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        tokens = _log(rng, 1, 8192)
        return {"op": op, "tokens": tokens, "heads": rng.choice([1, 5, 16, 32, 40]), "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2, 2 * rng.randrange(1, dim // 2 + 1)]), **turn,
                "type": rng.choice(["bf16", "fp16"]), "far": max(tokens, _log(rng, 64, 131071)),
                "scattered": rng.random() < 0.5}
    case = {"op": op, "q_heads": g * kv, "kv_heads": kv, "dim": dim, "page": rng.choice([8, 16, 16, 24, 32, 64, 128, 11]),
            "rows": rng.choice(["bf16", "bf16", "fp16"])}
    masks = {"window": rng.choice([0, 0, _log(rng, 16, 4096)]), "sinks": rng.choice([0, 4, rng.randrange(1, 130)])}
    if op == "decode":
        seqs = _log(rng, 1, 128)
        high = _log(rng, 64, min(131072, 400000 // seqs))
        return {**case, "seqs": seqs, "low": rng.randrange(1, high + 1), "high": high, **masks}
    if op == "prefill":
        seqs = _log(rng, 1, 5)
        q, past = _log(rng, 2, 2200), rng.choice([0, _log(rng, 16, 4000)])
        return {**case, "seqs": seqs, "q_low": rng.randrange(1, q + 1), "q_high": q, "past_low": rng.randrange(0, past + 1),
                "past_high": past, **masks}
    seqs = _log(rng, 1, 64)
    q, past = _log(rng, 1, 16384 // seqs), _log(rng, 1, 4000)
    case = {**case, "seqs": seqs, "q_low": rng.randrange(1, q + 1), "q_high": q, "past_low": rng.randrange(0, past + 1),
            "past_high": past}
    if op == "read":
        return case
    return {**case, "rot": rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randrange(1, dim // 2 + 1)]), **turn,
            "type": rng.choice([case["rows"], "fp8", "fp4", "fp4"])}


def _spread(n, low, high, turn):
    """n whole numbers over low..high, both ends among them, in a mixed order that the case fixes."""
    step = next(k for k in (turn, 11, 13, 17, 1) if math.gcd(k, n) == 1)
    return [low + ((i * step) % n) * (high - low) // max(1, n - 1) for i in range(n)] if n > 1 else [high]


def _lengths(case):
    """(tokens of each sequence, new ones included; new tokens of each)."""
    if case["op"] == "decode":
        lens = _spread(case["seqs"], case["low"], case["high"], 7)
        return lens, [1] * len(lens)
    q = _spread(case["seqs"], case["q_low"], case["q_high"], 5)
    past = _spread(case["seqs"], case["past_low"], case["past_high"], 7)
    return [a + b for a, b in zip(q, past)], q


def _device(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _values(shape, kind, gen):
    x = torch.empty(shape, dtype=torch.float16 if kind == "fp16" else torch.bfloat16, device="cuda")
    x.normal_(generator=gen)
    return x.to(TORCH[kind]) if kind == "fp8" else x


def _page_bytes(case):
    """(bytes of codes, bytes of scales, page stride) of a 4-bit page."""
    n = case["page"] * case["kv_heads"] * case["dim"]
    return n // 2, n // 32, -(-(n // 2 + n // 32) // 16) * 16


def _split(case, cache):
    """(codes [pages, heads, page, dim / 2], scales [pages, heads, dim / 32, page]) of 4-bit pages, as views."""
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    codes, scales, stride = _page_bytes(case)
    raw = torch.as_strided(cache, (cache.shape[0], codes + scales), (stride, 1))
    return raw[:, :codes].unflatten(1, (heads, page, dim // 2)), raw[:, codes:].unflatten(1, (heads, dim // 32, page))


def _encode(x):
    """E2M1 codes and scale bytes of blocks of 32 along the last dimension."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top)[1] - 3).clamp(-127, 127) * (top > 0) - 127 * (top == 0)
    a = torch.ldexp(b.abs(), -e)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    a = ((a / step).round() * step).clamp(max=6)       # halves go to the even code
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(b).to(torch.uint8)).flatten(-2)
    return code[..., ::2] | code[..., 1::2] << 4, (e[..., 0] + 127).to(torch.uint8)


def _fp4_pages(case, pages, gen):
    """A 4-bit cache of normal values."""
    codes, scales, stride = _page_bytes(case)
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    store = torch.zeros(pages, stride, dtype=torch.uint8, device="cuda")
    width = dim * 17 // 32
    cache = torch.as_strided(store, (pages, page, heads, width), (stride, heads * width, width, 1))
    c, s = _encode(torch.randn(pages, heads, page, dim, generator=gen, device="cuda"))
    into = _split(case, cache)
    into[0].copy_(c)
    into[1].copy_(s.transpose(2, 3))
    return cache


def _frequencies(case):
    """Radians per position of every pair, for positions compressed by `stretch`."""
    i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda")
    return (case["base"] ** (-i / case["rot"]) / case["stretch"]).float()


def _factor(case):
    """The rotated values' factor that goes with a stretched context."""
    return 0.1 * math.log(case["stretch"]) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"case": case}
    if case["op"] in ("rope", "append"):
        state["freqs"], state["factor"] = _frequencies(case), _factor(case)
    if case["op"] == "rope":
        n = case["tokens"]
        # queries and keys as a fused projection leaves them: in front of the values of the same row
        rows = _values((n, case["heads"] + 2, case["dim"]), case["type"], gen)
        state["x"] = rows[:, :case["heads"]]
        at = torch.arange(n, device="cuda") + (case["far"] - n + 1)
        if case["scattered"]:
            at = torch.randint(0, case["far"] + 1, (n,), generator=gen, device="cuda")
        state["positions"] = at.int().clamp(min=0)
        return state
    lens, new = _lengths(case)
    page, kv, dim, kind = case["page"], case["kv_heads"], case["dim"], case.get("type", "fp4")
    held = [-(-n // page) for n in lens]
    pages = sum(held) + 3
    # tables over shuffled pages
    order, at = torch.randperm(pages, generator=gen, device="cuda").int(), 0
    state["tables"] = torch.full((len(lens), max(held) + 1), -1, dtype=torch.int32, device="cuda")
    for s, n in enumerate(held):
        state["tables"][s, :n] = order[at:at + n]
        at += n
    state["lens"] = _device(lens)
    ends = [0]
    for n in new:
        ends.append(ends[-1] + n)
    state["cu"], state["tokens"] = _device(ends), ends[-1]
    for name in ("k", "v"):
        state[name] = _fp4_pages(case, pages, gen) if kind == "fp4" else _values((pages, page, kv, dim), kind, gen)
    for name in ("k_scale", "v_scale"):
        state[name] = torch.rand(kv, generator=gen, device="cuda") + 0.5 if kind == "fp8" else None
    if case["op"] != "read":
        rows = _values((ends[-1], case["q_heads"] + 2 * kv, dim), case["rows"], gen)
        state["q"], state["k_new"], state["v_new"] = rows.split([case["q_heads"], kv, kv], dim=1)
    return state


def run(state):
    case = state["case"]
    if own:
        import w4a4_block_scaled_amd as w4
        return _run_own(w4, case, state)
    return {"rope": _rope, "append": _append, "read": _read, "decode": _decode, "prefill": _prefill}[case["op"]](case, state)


def _run_own(w4, case, s):
    if case["op"] == "rope":
        return w4.rope(s["x"], s["positions"], s["freqs"], interleaved=case["interleaved"], factor=s["factor"])
    if case["op"] == "append":
        q = w4.kv_append_rope(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["tables"], s["lens"], s["freqs"],
                              cu_seqlens=s["cu"], interleaved=case["interleaved"], factor=s["factor"],
                              k_scale=s["k_scale"], v_scale=s["v_scale"])
        if case["type"] != "fp4":
            return q, s["k"], s["v"]
        return (q, *w4.kv_read(s["k"], s["v"], s["tables"], s["lens"], s["cu"], s["tokens"], dtype=q.dtype))
    if case["op"] == "read":
        return w4.kv_read(s["k"], s["v"], s["tables"], s["lens"], s["cu"], s["tokens"], dtype=TORCH[case["rows"]])
    if case["op"] == "decode":
        return w4.attn_decode(s["q"], s["k"], s["v"], s["tables"], s["lens"], window=case["window"], sinks=case["sinks"])
    return w4.attn_prefill(s["q"], s["cu"], s["k"], s["v"], s["tables"], s["lens"], window=case["window"], sinks=case["sinks"])


# The plain forms.

def _rotated(case, x, positions, s, kind):
    """x with its rotated values, in `kind` bits."""
    angle = positions.double()[:, None] * s["freqs"].double()
    cos, sin = ((f(angle) * s["factor"]).to(kind)[:, None] for f in (torch.cos, torch.sin))
    rot = case["rot"]
    y = x.to(kind, copy=True)
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = y[..., one].clone(), y[..., two].clone()
    y[..., one] = a * cos - b * sin
    y[..., two] = a * sin + b * cos
    return y


def _rope(case, s):
    return _rotated(case, s["x"], s["positions"], s, torch.float32).to(s["x"].dtype)


def _rows(s):
    """For every new token: its sequence, its place among the sequence's new ones, its position."""
    count = s["cu"][1:] - s["cu"][:-1]
    seq = torch.repeat_interleave(torch.arange(len(count), device="cuda"), count.long())
    place = torch.arange(len(seq), device="cuda") - s["cu"][seq].long()
    return seq, place, (s["lens"] - count)[seq].long() + place


def _decode_codes(codes, exponents):
    """Values in 32 bits of codes [..., dim / 2] with scale bytes [..., dim / 32]."""
    grid = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    x = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, 32)) * torch.exp2(exponents.float() - 127)[..., None]).flatten(-2)


def _append(case, s):
    seq, _, position = _rows(s)
    page, slot = s["tables"][seq, position // case["page"]].long(), position % case["page"]
    out = [_rotated(case, s["q"], position, s, torch.float32).to(s["q"].dtype)]
    small = case["type"] in ("fp8", "fp4")
    k_new = _rotated(case, s["k_new"], position, s, torch.float64 if small else torch.float32)
    for cache, new, scale in ((s["k"], k_new, s["k_scale"]), (s["v"], s["v_new"], s["v_scale"])):
        if case["type"] == "fp4":
            codes, scales = _split(case, cache)
            codes[page, :, slot], scales[page, :, :, slot] = _encode(new.double())
            out.append(_decode_codes(codes[page, :, slot], scales[page, :, :, slot]).to(TORCH[case["rows"]]))
            continue
        if case["type"] == "fp8":
            x = (new.double() / scale.double()[:, None]).clamp(-448, 448).float().to(cache.dtype)
            cache.view(torch.uint8)[page, slot] = x.view(torch.uint8)
        else:
            cache[page, slot] = new.to(cache.dtype)
        out.append(cache)
    return tuple(out)


def _read(case, s):
    seq, _, position = _rows(s)
    page, slot = s["tables"][seq, position // case["page"]].long(), position % case["page"]
    out = []
    for cache in (s["k"], s["v"]):
        codes, scales = _split(case, cache)
        out.append(_decode_codes(codes[page, :, slot], scales[page, :, :, slot]).to(TORCH[case["rows"]]))
    return tuple(out)


def _gathered(case, cache, tables):
    """The cache of every sequence in order, [seqs, kv_heads, tokens, dim] in 32 bits."""
    at = tables.clamp(min=0).long()
    codes, scales = _split(case, cache)
    x = _decode_codes(codes[at], scales[at].transpose(-1, -2))      # [seqs, pages, heads, page, dim]
    return x.transpose(1, 2).flatten(2, 3).contiguous()


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
    k, v = _gathered(case, s["k"], s["tables"]), _gathered(case, s["v"], s["tables"])
    seqs, kv, tokens, dim = k.shape
    q = s["q"].float().reshape(seqs, kv, -1, dim)
    seen = _seen(s["lens"].long() - 1, tokens, case)[:, None, None, :]
    p = _weights(torch.matmul(q, k.transpose(2, 3).contiguous()) / math.sqrt(dim), seen)
    return torch.matmul(p, v).reshape(seqs, -1, dim).to(s["q"].dtype)


def _prefill(case, s):
    k, v = _gathered(case, s["k"], s["tables"]), _gathered(case, s["v"], s["tables"])
    seqs, kv, tokens, dim = k.shape
    seq, place, position = _rows(s)
    most = case["q_high"]
    q = torch.zeros(seqs, most, kv, case["q_heads"] // kv, dim, device="cuda")
    q[seq, place] = s["q"].float().reshape(len(seq), kv, -1, dim)
    at = torch.full((seqs, most), -1, device="cuda")
    at[seq, place] = position
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3).contiguous()  # [seqs, kv, heads of the group x rows, dim]
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()).div_(math.sqrt(dim)).view(seqs, kv, -1, most, tokens)
    p = _weights(scores, _seen(at, tokens, case)[:, None, None]).flatten(2, 3)
    out = torch.matmul(p, v).view(seqs, kv, -1, most, dim).permute(0, 3, 1, 2, 4)
    return out[seq, place].reshape(len(seq), -1, dim).to(s["q"].dtype)


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
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * case["dim"] * 4 + case["tokens"] * 4, "flops": n * case["rot"] * 3}
    lens, new = _lengths(case)
    kv, dim, page, heads = case["kv_heads"], case["dim"], case["page"], case["q_heads"]
    row = {"fp4": dim // 2 + dim // 32, "fp8": dim}.get(case.get("type", "fp4"), 2 * dim)      # bytes of a head's row
    if case["op"] in ("decode", "prefill"):
        pairs, tokens = _visible(case, lens, new)
        moved = tokens * (kv * row * 2 + 4 / page) + sum(new) * heads * dim * 2 * 2
        return {"bytes": moved, "flops": pairs * heads * dim * 4}
    copied = kv * 2 * (row + 2 * dim)      # of a token: its rows in the cache, and in 16 bits
    if case["op"] == "read":
        return {"bytes": sum(new) * copied, "flops": 0}
    copied += heads * dim * 4 + (copied if case["type"] == "fp4" else 0)
    return {"bytes": sum(new) * copied, "flops": sum(new) * (heads + kv) * case["rot"] * 3}


# The same in 64 bits.

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_turned(case, s, x, positions):
    """The pairs as complex numbers times factor exp(i angle)."""
    rot = case["rot"]
    angle = torch.outer(positions.to(torch.float64), s["freqs"].to(torch.float64))
    turn = torch.polar(torch.full_like(angle, s["factor"]), angle).unsqueeze(1)
    x = x.to(torch.float64)
    pairs = x[..., :rot].unflatten(-1, (rot // 2, 2) if case["interleaved"] else (2, rot // 2))
    if not case["interleaved"]:
        pairs = pairs.transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = (y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _exact_e2m1(x):
    """The values that a 4-bit cache holds in the place of x: the nearest point of the grid, the even one of two."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = b.abs().max(-1, keepdim=True).values
    unit = torch.exp2(torch.floor(torch.log2(top)) - 2)
    unit = torch.where(torch.exp2(torch.floor(torch.log2(top))) > top, unit / 2, unit)      # log2 rounded up to a whole number
    unit = torch.where(top > 0, unit, torch.ones_like(unit))
    a = b.abs() / unit
    code = torch.zeros_like(a)
    for i in range(7):
        middle = (E2M1[i] + E2M1[i + 1]) / 2
        code = code + ((a >= middle) if i % 2 else (a > middle))
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    return torch.copysign(grid[code.long()], b).mul(unit).reshape(x.shape)


def _exact_e4m3(x):
    exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.exp2(exponent - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_rows(case, s, cache, page, slot):
    """Rows of the 4-bit cache at (page, slot)."""
    codes, scales = _split(case, cache)
    byte = codes[page, :, slot].to(torch.int64)
    code = torch.stack([byte % 16, byte // 16], dim=-1).flatten(-2)
    value = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[code % 8] * (1 - 2 * (code // 8))
    unit = torch.pow(2.0, scales[page, :, :, slot].to(torch.float64) - 127)
    return value * unit.repeat_interleave(32, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turned(case, s, s["x"], s["positions"])
    lens, new = _lengths(case)
    kv, dim, size = case["kv_heads"], case["dim"], case["page"]
    places = [torch.arange(n - m, n, device="cuda") for n, m in zip(lens, new)]
    if case["op"] in ("append", "read"):
        page = torch.cat([s["tables"][i].long()[p // size] for i, p in enumerate(places)])
        slot = torch.cat(places) % size
        if case["op"] == "read":
            return _exact_rows(case, s, s["k"], page, slot), _exact_rows(case, s, s["v"], page, slot)
        at = torch.cat(places)
        out = [_exact_turned(case, s, s["q"], at)]
        for name, x in (("k", _exact_turned(case, s, s["k_new"], at)), ("v", s["v_new"].to(torch.float64))):
            if case["type"] == "fp4":
                out.append(_exact_e2m1(x))
                continue
            cache = s[name].to(torch.float64)
            cache[page, slot] = x if case["type"] != "fp8" else _exact_e4m3(x / s[name + "_scale"].to(torch.float64)[:, None])
            out.append(cache)
        return tuple(out)
    outs, at = [], 0
    for i, (n, m) in enumerate(zip(lens, new)):
        p = torch.arange(n, device="cuda")
        page, slot = s["tables"][i].long()[p // size], p % size
        k, v = _exact_rows(case, s, s["k"], page, slot), _exact_rows(case, s, s["v"], page, slot)
        query = places[i][:, None]
        hidden = p[None, :] > query
        if case["window"]:
            hidden = hidden | ((query - p[None, :] >= case["window"]) & (p[None, :] >= case["sinks"]))
        out = torch.empty(m, case["q_heads"], dim, dtype=torch.float64, device="cuda")
        for h in range(case["q_heads"]):
            j = h // (case["q_heads"] // kv)
            a = (s["q"][at:at + m, h].double() @ k[:, j].t()) * dim ** -0.5
            a[hidden] = NEG
            out[:, h] = torch.softmax(a, dim=-1) @ v[:, j]
        outs.append(out)
        at += m
    return torch.cat(outs)
