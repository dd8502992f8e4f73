"""Every way that the attention's entry points go, by name, over the types, head
dimensions and page sizes that reach a kernel of their own: decoding, a few rows
per sequence, row tiles with the keys whole and with the keys split.  Each case
states the rule that takes it there, and the accuracy that the way promises: the
weights in two 16-bit parts everywhere but in row tiles with the keys whole."""
import numpy as np
import pytest
import torch

import w4a4_block_scaled_amd as w4
from gpu_common import device, say
from kv_common import as_f64, check_attention, ints, on_device, table_of, values
from test_gpu_attn_decode import ORDERS
from test_gpu_attn_edges import attend
from test_gpu_attn_prefill import chunks

pytestmark = pytest.mark.gpu


def way_of(c):
    """The way of attn_prefill, by its rules on sizes."""
    seqs, tokens = len(c["lens"]), len(c["q"])
    page, heads = c["kd"].shape[1:3]
    group = c["q"].shape[1] // heads
    if page % 8 == 0 and tokens * group <= 16 * seqs:
        return "few"
    tiles = tokens * group // 128 + seqs
    return "split" if c["tables"].shape[1] * page > 1000 and tiles * heads < 256 else "whole"


# past, new (both per sequence), of a group of 4 unless given
SIZES = {"few": ([500, 40, 1300], [3, 4, 1]), "whole": ([300, 0], [90, 45]), "split": ([1500, 20], [37, 20])}
TYPES = [("bf16", "bf16"), ("fp16", "fp16"), ("fp8", "bf16"), ("fp8", "fp16")]


@pytest.mark.parametrize("way", ["decode", *SIZES])
@pytest.mark.parametrize("kind,high", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 24, 11])
def test_types_and_dimensions(way, kind, high, dim, page):
    say(f"[ways] {way}, {kind} cache, {high} queries, D = {dim}, page {page}")
    past, new = SIZES.get(way, ([700, 0, 37], [1, 1, 1]))
    if way == "few" and page % 8:
        pytest.skip("few rows go as row tiles where pages are no multiple of 8")
    c = chunks(kind, 2, 4, dim, page, past, new, seed=dim + page, high=high)
    assert way == "decode" or way_of(c) == way
    assert c["q"].dtype == {"bf16": torch.bfloat16, "fp16": torch.float16}[high]
    for window, sinks in ((0, 0), (100, 5)):
        y, lse = attend(c, way, window, sinks)
        rows = sorted({0, 1, len(c["q"]) - 1, int(c["cu"][1]) - 1, int(c["cu"][1])})
        check_attention(y, lse.cpu(), c["q"], c["f64"], c["tables"], c["lens"], c["pos"], c["seqs"], c["high"],
                        dim ** -0.5, window, sinks, "once" if way == "whole" else "two", f"window {window}", rows)


@pytest.mark.parametrize("kind,high,group,dim,past,new", [
    ("bf16", "bf16", 1, 64, [300] * 3, [16, 10, 20]),       # 16 rows per head on average, 20 of one
    ("fp16", "fp16", 7, 128, [64, 900], [2, 2]),
    ("fp8", "fp16", 16, 256, [700, 10], [1, 1]),
    ("bf16", "bf16", 20, 128, [33, 0, 500, 7], [1, 2, 0, 0]),   # more rows per token than a unit has
    ("fp8", "bf16", 3, 64, [5000, 2], [5, 5]),
])
def test_few_rows(kind, high, group, dim, past, new):
    say(f"[ways] few rows, {kind}, group {group}, D = {dim}, new {new}")
    c = chunks(kind, 2, group, dim, 16, past, new, seed=sum(past) + dim, high=high)
    assert way_of(c) == "few"
    for window, sinks in ((0, 0), (40, 3)):
        y, lse = attend(c, "few", window, sinks)
        check_attention(y, lse.cpu(), c["q"], c["f64"], c["tables"], c["lens"], c["pos"], c["seqs"], c["high"],
                        dim ** -0.5, window, sinks, "two", f"window {window}")


@pytest.mark.parametrize("idle", [True, False])
def test_one_chunk_among_many_sequences(idle):
    """A chunk of a prompt among sequences with no new token, or with one each: few
    rows on average, many of one sequence."""
    past = [(37 * s) % 300 for s in range(63)]
    new = [0 if idle else 1] * 63
    past.insert(20, 400)
    new.insert(20, 200)
    say(f"[ways] 200 tokens of one of 64 sequences, {'none' if idle else 'one'} of the others")
    c = chunks("bf16", 2, 4, 64, 16, past, new, seed=9)
    assert way_of(c) == ("few" if 4 * sum(new) <= 1024 else "whole")
    y, lse = attend(c, "few")
    at = int(c["cu"][20])
    rows = sorted({0, at, at + 7, at + 100, at + 199, len(c["q"]) - 1})
    check_attention(y, lse.cpu(), c["q"], c["f64"], c["tables"], c["lens"], c["pos"], c["seqs"], "bf16", 0.125, 0, 0, "once",
                    "mixed", rows)


@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("kind,dim,page", [("bf16", 128, 16), ("fp8", 128, 24), ("fp16", 256, 11), ("fp8", 64, 8)])
@pytest.mark.parametrize("way", ["whole", "split", "few"])
def test_memory_orders(way, order, kind, dim, page):
    say(f"[ways] {way}, {order}, {kind}, D = {dim}, page {page}")
    if way == "few" and page % 8:
        pytest.skip("few rows go as row tiles where pages are no multiple of 8")
    past, new = SIZES[way]
    plain = chunks(kind, 3, 4, dim, page, past, new, seed=dim)
    c = chunks(kind, 3, 4, dim, page, past, new, seed=dim, order=order)
    assert way_of(c) == way
    want, lse = attend(plain, way, 200, 9)
    y, l2 = attend(c, way, 200, 9)
    assert torch.equal(y, want) and torch.equal(lse, l2)


@pytest.mark.parametrize("kind,dim,page", [("bf16", 128, 11), ("fp16", 64, 24), ("fp8", 128, 16), ("fp8", 256, 11), ("bf16", 256, 16)])
def test_row_tiles_ignore_masked_values(kind, dim, page):
    """Inf and NaN where no row sees them: bit for bit the result of clean caches, with
    the keys whole."""
    say(f"[ways] masked values, {kind}, D = {dim}, page {page}")
    past, new, window, sinks = [0, 300], [150, 70], 80, 3
    c = chunks(kind, 2, 4, dim, page, past, new, seed=8)
    assert way_of(c) == "whole"
    clean, lse = attend(c, "whole", window, sinks)
    seen = np.zeros(c["f64"][0].shape[:2], bool)
    for s, n in enumerate(c["lens"]):
        for t in range(n):
            if t > past[s] - window or t < sinks:
                seen[c["tables"][s, t // page], t % page] = True
    hidden = torch.from_numpy(~seen).to(c["dev"])
    for x, odd in ((c["kd"], float("nan")), (c["vd"], float("inf"))):
        if kind == "fp8":
            x.view(torch.uint8)[hidden] = 0x7f
        else:
            x[hidden] = odd
    y, l2 = attend(c, "whole", window, sinks)
    assert torch.equal(y, clean) and torch.equal(lse, l2)


@pytest.mark.parametrize("way,order", [("whole", "page token head"), ("split", "page token head"), ("few", "page token head"),
                                       ("whole", "token page head"), ("split", "token page head")])
@pytest.mark.parametrize("far", ["pages", "rows"])
def test_offsets_past_32_bits(way, order, far):
    """Pages beyond 2^31 elements, and rows of a page that lie up to 2^31 bytes apart
    (the page axis inside the token axis: just below and just above the row stride
    where offsets inside a page are kept in 32 bits)."""
    dev = device()
    page, kv, dim = 16, 4, 128
    if far == "pages":
        pages = 2 ** 31 // (page * kv * dim) + 60
    else:
        if order == "page token head":
            pytest.skip("rows of a page lie side by side in this order")
        pages = 2 ** 26 // (kv * dim) + (-3 if way == "whole" else 3)
    past, new = SIZES[way]
    c = chunks("bf16", kv, 4, dim, page, past, new, seed=3)
    assert way_of(c) == way
    want, lse = attend(c, way)
    shape = (pages, page, kv, dim) if order == "page token head" else (page, pages, kv, dim)
    big = [torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    if order != "page token head":
        big = [x.transpose(0, 1) for x in big]
    say(f"[ways] {way}, {order}, {pages} pages, row stride {big[0].stride(1)}")
    t = np.full_like(c["tables"], -1)
    n = 0
    for s in range(len(past)):
        for j in range(-(-c["lens"][s] // page)):
            at = pages - 1 - 3 * n if n % 4 else n
            for x, y in zip(big, (c["kd"], c["vd"])):
                x[at] = y[int(c["tables"][s, j])]
            t[s, j] = at
            n += 1
    c["kd"], c["vd"], c["tables"] = *big, t
    y, l2 = attend(c, way)
    assert torch.equal(y, want) and torch.equal(lse, l2)


@pytest.mark.parametrize("way", list(SIZES))
def test_prefill_in_a_graph(way):
    """A captured call, replayed with other queries, lengths and tables, the
    program's own work between the replays: every replay equals the eager call."""
    say(f"[graph] {way}")
    past, new = SIZES[way]
    c = chunks("bf16", 2, 4, 128, 16, past, new, seed=5)
    assert way_of(c) == way
    dev = c["dev"]
    q, cu, tables, lens = c["q"].to(dev), ints(c["cu"], dev), ints(c["tables"], dev), ints(c["lens"], dev)
    out = torch.empty_like(q)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=dev)

    def call(o, w):
        return w4.attn_prefill(q, cu, c["kd"], c["vd"], tables, lens, window=300, sinks=4, out=o, workspace=w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    for i in range(5):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(i)).to(q.dtype))
        lens.copy_(ints([n - i for n in c["lens"]], dev))
        want = call(torch.empty_like(q), None).clone()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"
        (want @ want.transpose(1, 2).contiguous()).sum().item()        # other work between the replays


@pytest.mark.parametrize("shape,dtype,gap", [((7, 3, 1, 5), torch.uint8, 0), ((9, 1, 3, 7), torch.bfloat16, 1),
                                             ((6, 2, 1, 4096 + 3), torch.uint8, 0), ((5, 1, 1, 1), torch.uint8, 2)])
def test_copy_pages_of_odd_bytes(shape, dtype, gap):
    """Pages that are no multiple of 16 bytes, side by side or with a gap between them."""
    say(f"[copy] {shape} {dtype}, gap {gap}")
    dev = device()
    gen = torch.Generator().manual_seed(1)
    whole = [torch.randint(0, 255, (shape[0] * (1 + gap), *shape[1:]), generator=gen).to(dtype).to(dev) for _ in range(3)]
    caches = [x[::1 + gap] for x in whole]
    want = [x.clone() for x in whole]
    src, dst = [0, 3, shape[0], 2], [4, 1, 0, -1]
    for x in want:
        x[::1 + gap][4] = x[::1 + gap][0]
        x[::1 + gap][1] = x[::1 + gap][3]
    w4.kv_copy_pages(caches, ints(src, dev), ints(dst, dev))
    assert all(torch.equal(a, b) for a, b in zip(whole, want))
