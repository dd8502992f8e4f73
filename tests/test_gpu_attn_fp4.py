"""Attention over a cache held in 4 bits, every way of the entry points, against
the fp64 oracle: dimensions, groups, pages, types, windows and sinks, lengths from
none to long, masked blocks of NaN, tables without a page, far pages, graphs."""
import numpy as np
import pytest
import torch

import w4a4_block_scaled_amd as w4
from gpu_common import device, say
from kv_common import as_f64, check_attention, ints, values
from oracle import attention as A
from rows_common import chunks_fp4, make_fp4, on_gpu
from test_gpu_attn_decode import check as check_decode
from test_gpu_attn_decode import run as run_decode
from test_gpu_attn_edges import attend
from test_gpu_attn_prefill import check as check_prefill
from test_gpu_attn_prefill import run as run_prefill

pytestmark = pytest.mark.gpu


def way_of(c, page):
    """The way of attn_prefill, by its rules on sizes (the cache's tensor has the page's size)."""
    seqs, tokens = len(c["lens"]), len(c["q"])
    heads = c["kd"].shape[2]
    group = c["q"].shape[1] // heads
    if page % 8 == 0 and tokens * group <= (16 if c["q"].shape[2] == 256 else 48) * seqs:
        return "few"
    return "split" if c["tables"].shape[1] * page > 1000 and (tokens * group // 128 + seqs) * heads < 256 else "whole"


DECODE = [
    # kv heads, group, dim, page, lens, high
    (8, 4, 128, 16, [513], "bf16"), (8, 4, 128, 16, [1], "fp16"), (4, 7, 128, 64, [2000, 3, 129], "bf16"),
    (1, 16, 128, 8, [300, 0, 31], "bf16"), (16, 1, 64, 24, [100, 700, 33, 32], "fp16"), (3, 5, 64, 11, [90, 1, 250], "bf16"),
    (2, 8, 128, 11, [400, 12], "fp16"), (1, 4, 256, 32, [600, 0], "bf16"), (2, 2, 256, 11, [70, 260], "fp16"),
    (1, 20, 64, 16, [77], "bf16"), (1, 40, 128, 1, [130], "bf16"), (2, 4, 64, 8, list(range(0, 66)), "bf16"),
    (2, 3, 256, 128, [1, 127, 128, 129, 255, 256, 257], "bf16"), (4, 1, 128, 16, [5000, 4999], "bf16"),
]


@pytest.mark.parametrize("kv,group,dim,page,lens,high", DECODE)
def test_decode_matches_the_oracle(kv, group, dim, page, lens, high):
    say(f"[decode4] {kv} x {group} heads of {dim}, page {page}, lens {lens[:6]}, {high}")
    c = make_fp4(kv, group, dim, page, lens, seed=sum(lens) + dim, high=high, dev=device(), gap=kv % 2)
    for window, sinks, scale in ((0, 0, None), (100, 5, None), (31, 0, 0.3), (1, 1, None)):
        y, lse = run_decode(c, window, sinks, scale)
        check_decode(c, y, lse, window, sinks, scale, f"window {window}", rows=range(min(len(lens), 8)))


@pytest.mark.parametrize("kv,group,dim,page,lens,high", DECODE)
def test_decode_in_wide_tables(kv, group, dim, page, lens, high):
    """Tables that hold far more than the lengths: units are cut and joined."""
    say(f"[decode4 wide] {kv} x {group} heads of {dim}, page {page}, lens {lens[:6]}, {high}")
    c = make_fp4(kv, group, dim, page, lens, seed=sum(lens) + dim, high=high, dev=device())
    wide = np.full((len(lens), 2100 // page + 1), -1, np.int32)
    n = min(c["tables"].shape[1], wide.shape[1])
    wide[:, :n] = c["tables"][:, :n]
    c["tables"] = wide if n == c["tables"].shape[1] else c["tables"]
    for window, sinks in ((0, 0), (100, 5)):
        y, lse = run_decode(c, window, sinks)
        check_decode(c, y, lse, window, sinks, label=f"window {window}", rows=range(min(len(lens), 8)))


def test_decode_at_the_limit_of_whole_units():
    """Tables of exactly as many tokens as units are left whole for, and of one page more, by
    dimension and units; as many sequences as make more units than workgroups."""
    for kv, dim, page, seqs, tokens in ((2, 128, 16, 2, 1024), (2, 256, 16, 2, 640), (4, 64, 32, 64, 2048), (16, 64, 8, 40, 2048)):
        for pages in (tokens // page, tokens // page + 1):
            say(f"[decode4 limit] {kv} heads of {dim}, {seqs} sequences, {pages} pages of {page}")
            lens = [pages * page] + [(37 * i) % tokens for i in range(1, seqs)]
            c = make_fp4(kv, 2, dim, page, lens, seed=dim, dev=device())
            c["tables"] = np.ascontiguousarray(c["tables"][:, :pages])
            y, lse = run_decode(c, 0, 0)
            check_decode(c, y, lse, 0, 0, label=f"{pages} pages", rows=[0, 1, seqs - 1])


SIZES = {"few": ([500, 40, 1300], [3, 4, 1]), "few, two blocks": ([500, 40, 1300], [3, 9, 8]),
         "few, three blocks": ([500, 40, 1300], [13, 0, 21]), "whole": ([300, 0], [90, 45]), "split": ([1500, 20], [37, 20])}


@pytest.mark.parametrize("way", list(SIZES))
@pytest.mark.parametrize("high", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 24, 11, 64])
def test_prefill_matches_the_oracle(way, high, dim, page):
    say(f"[prefill4] {way}, {high}, D = {dim}, page {page}")
    if way.startswith("few") and (page % 8 or (dim == 256 and way != "few")):
        pytest.skip("these go as row tiles")
    past, new = SIZES[way]
    c = chunks_fp4(2, 4, dim, page, past, new, seed=dim + page, high=high, dev=device(), gap=page % 3)
    assert way_of(c, page) == way.split(",")[0]
    for window, sinks in ((0, 0), (100, 5)):
        y, lse = run_prefill(c, window, sinks)
        rows = sorted({0, 1, len(c["q"]) - 1, int(c["cu"][1]) - 1, int(c["cu"][1])})
        check_attention(y, lse.cpu(), c["q"], c["f64"], c["tables"], c["lens"], c["pos"], c["seqs"], c["high"],
                        dim ** -0.5, window, sinks, "once" if way == "whole" else "two", f"window {window}", rows)


@pytest.mark.parametrize("kv,group,dim,page,past,new", [
    (4, 7, 128, 32, [0, 100, 17], [130, 1, 65]), (1, 20, 64, 24, [7, 0], [33, 64]), (3, 5, 64, 1, [3], [70]),
    (1, 1, 128, 16, [0], [1]), (2, 1, 256, 8, [0, 5, 0], [2, 0, 200]), (1, 16, 128, 128, [1000], [40])])
def test_prefill_groups(kv, group, dim, page, past, new):
    say(f"[prefill4] {kv} x {group} heads of {dim}, page {page}, past {past}, new {new}")
    c = chunks_fp4(kv, group, dim, page, past, new, seed=sum(new) + dim, dev=device())
    for window, sinks in ((0, 0), (64, 0), (7, 4)):
        y, lse = run_prefill(c, window, sinks)
        check_prefill(c, y, lse, window, sinks, label=f"window {window}", most=12)


WAYS = {"decode": ([900, 40], [1, 1], 16), "decode, cut": ([2500, 40], [1, 1], 16), "decode, page 11": ([900, 40], [1, 1], 11), "few": ([900, 40], [3, 2], 16),
        "few, three blocks": ([900, 40], [13, 9], 16),
        "whole": ([700, 40], [150, 60], 16), "whole, page 11": ([700, 40], [150, 60], 11), "split": ([3000, 40], [30, 20], 16)}


def blank(c, page, dim, tokens, s=0, both=True):
    """NaN in the place of every block of those tokens (scale byte 255 over the codes that are there)."""
    heads = c["kd"].shape[2]
    at, per = page * heads * dim // 2, dim // 32
    for x in (c["kd"], c["vd"]) if both else (c["vd"],):
        raw = x.as_strided((x.shape[0], x.stride(0)), (x.stride(0), 1))
        scales = raw[:, at:at + heads * per * page].unflatten(1, (heads, per, page))
        for t in tokens:
            scales[int(c["tables"][s, t // page]), :, :, t % page] = 255


@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("high", ["bf16", "fp16"])
def test_masked_blocks_do_not_count(way, dim, high):
    """Blocks of NaN that no row sees (before the windows, behind the sequences' ends)
    change no bit; one that some rows see makes those NaN and the others no other."""
    say(f"[masked4] {way}, D = {dim}, {high}")
    past, new, page = WAYS[way]
    window, sinks = 200, 3
    c = chunks_fp4(2, 4, dim, page, past, new, seed=dim, high=high, dev=device())
    clean, lse = attend(c, way, window, sinks)
    low = past[0] - window + 1
    blank(c, page, dim, range(sinks, low))
    for s in (0, 1):
        end = c["lens"][s]
        blank(c, page, dim, range(end, -(-end // page) * page), s)
    y, l2 = attend(c, way, window, sinks)
    assert torch.equal(y, clean) and torch.equal(l2, lse)
    if way.startswith("decode"):
        return
    # the token that the first row's window begins with: its values seen by that row alone
    blank(c, page, dim, [low], both=False)
    y, l2 = attend(c, way, window, sinks)
    assert torch.isnan(y[0]).all() and torch.equal(y[1:], clean[1:]) and torch.equal(l2, lse)


@pytest.mark.parametrize("way", list(WAYS))
def test_without_a_page_and_empty(way):
    """A token without a page makes the rows that see it NaN; a length beyond the table's
    pages too; lengths of zero and below give zeros."""
    say(f"[tables4] {way}")
    past, new, page = WAYS[way]
    c = chunks_fp4(2, 4, 128, page, past, new, seed=1, dev=device())
    clean, _ = attend(c, way)
    n = int(c["cu"][1])
    keep = c["tables"].copy()
    for entry in (-1, c["kd"].shape[0], 2 ** 31 - 1):
        c["tables"][0, 3] = entry
        y, _ = attend(c, way)
        assert torch.isnan(y[:n]).all() and torch.equal(y[n:], clean[n:])
        c["tables"] = keep.copy()
    lens = c["lens"]
    for length in (0, -7, -2 ** 31):
        c["lens"] = [length, lens[1]]
        y, l2 = attend(c, way)
        assert torch.all(y[:n] == 0) and torch.all(l2[:n] == -float("inf")) and torch.equal(y[n:], clean[n:])
    c["lens"] = [keep.shape[1] * page + 1, lens[1]]
    y, _ = attend(c, way)
    assert torch.isnan(y[:n]).all() and torch.equal(y[n:], clean[n:])


@pytest.mark.parametrize("way", ["decode", "decode, cut", "few", "whole", "split"])
def test_far_pages(way):
    """Pages past 2^31 and 2^32 bytes."""
    dev = device()
    past, new, page = WAYS[way]
    kv, dim = 2, 128
    c = chunks_fp4(kv, 4, dim, page, past, new, seed=2, dev=dev)
    want, lse = attend(c, way)
    width, t = dim // 32 * 17, np.full_like(c["tables"], -1)
    used = [(s, j) for s in range(len(past)) for j in range(-(-c["lens"][s] // page))]
    stride = (5 << 30) // len(used) // 16 * 16
    say(f"[far4] {way}, {len(used)} pages {stride} bytes apart")
    big = []
    for x in (c["kd"], c["vd"]):
        store = torch.empty(len(used), stride, dtype=torch.uint8, device=dev)
        big.append(store.as_strided((len(used), page, kv, width), (stride, kv * width, width, 1)))
    for i, (s, j) in enumerate(used):
        at = len(used) - 1 - i
        for x, y in zip(big, (c["kd"], c["vd"])):
            x[at] = y[int(c["tables"][s, j])]
        t[s, j] = at
    c["kd"], c["vd"], c["tables"] = *big, t
    y, l2 = attend(c, way)
    assert torch.equal(y, want) and torch.equal(lse, l2)


@pytest.mark.parametrize("way", ["decode", "decode, cut", "few", "whole", "split"])
def test_in_a_graph(way):
    say(f"[graph4] {way}")
    past, new, page = WAYS[way]
    c = chunks_fp4(2, 4, 128, page, past, new, seed=5, dev=device())
    dev = c["dev"]
    q, cu, tables, lens = c["q"].to(dev), ints(c["cu"], dev), ints(c["tables"], dev), ints(c["lens"], dev)
    out, ws = torch.empty_like(q), torch.empty(64 << 20, dtype=torch.uint8, device=dev)

    def call(o, w):
        if way.startswith("decode"):
            return w4.attn_decode(q, c["kd"], c["vd"], tables, lens, window=300, sinks=4, out=o, workspace=w)
        return w4.attn_prefill(q, cu, c["kd"], c["vd"], tables, lens, window=300, sinks=4, out=o, workspace=w)
    call(out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    for i in range(4):
        q.copy_(values(q.shape, "bf16", torch.Generator().manual_seed(i)))
        lens.copy_(ints([n - i for n in c["lens"]], dev))
        want = call(torch.empty_like(q), None).clone()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"
        (want @ want.transpose(1, 2).contiguous()).sum().item()


@pytest.mark.parametrize("way", ["decode", "decode, cut", "few", "few, three blocks", "whole", "split"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("high", ["bf16", "fp16"])
def test_queries_with_outliers(way, dim, high):
    """A value of every block of 32 of the queries 2^11 times the others, where the keys are zero: the scores
    are the others' alone.  Queries enter them within 2^-19 of their block's largest value (four parts
    of 4 bits, the last one's step 2^-17 of the largest value's power of two, rounded to half of it), which is
    added to the bound on the scores' error."""
    if way == "few, three blocks" and dim == 256:
        pytest.skip("these go as row tiles")
    say(f"[outliers4] {way}, D = {dim}, {high}")
    past, new, page = WAYS[way]
    c = chunks_fp4(2, 4, dim, page, past, new, seed=dim, high=high, dev=device())
    q = c["q"].clone()
    q[..., 7::32] = torch.sign(q[..., 7::32]) * 3000
    c["q"] = q
    # the keys' codes of those values: the upper half of a byte each
    at, heads = page * 2 * dim // 2, 2
    raw = c["kd"].as_strided((c["kd"].shape[0], c["kd"].stride(0)), (c["kd"].stride(0), 1))
    raw[:, :at].unflatten(1, (heads, page, dim // 2))[..., 3::16] &= 15
    k64 = c["f64"][0].copy()
    k64[..., 7::32] = 0
    c["f64"] = [k64, c["f64"][1]]
    y, lse = attend(c, way)
    got, lse, q64 = as_f64(y), lse.cpu().numpy().astype(np.float64), as_f64(q)
    u, scale = 2.0 ** -8 if high == "bf16" else 2.0 ** -11, dim ** -0.5
    # decoding and few rows: BF16 weights in two parts whatever the queries' type
    weights = u if way == "whole" else 2.0 ** -20 if way == "split" and high == "fp16" else 2.0 ** -15
    for i in sorted({0, 1, len(q) - 1, int(c["cu"][1]) - 1}):
        s = int(c["seqs"][i])
        for h in (0, 5, 7):
            o, ref, (a, big, size, n) = A.attend(q64[i, h], *c["f64"], c["tables"][s], c["lens"][s], int(c["pos"][i]), h // 4,
                                                 scale, 0, 0)
            keys = np.abs(A.rows(k64, c["tables"][s], range(n), h // 4)).reshape(n, -1, 32).sum(-1)
            parts = (keys * np.abs(q64[i, h]).reshape(-1, 32).max(-1)).sum(-1).max() * scale * 2.0 ** -19
            eta = (dim + 8) * 2.0 ** -23 * (size + parts) + 2.0 ** -22 + parts
            bound = u * np.abs(o) + (1 + u) * (weights + 2 * eta + n * 2.0 ** -22) * a + n * (2.0 ** -24 if high == "fp16" else 0) * big + 2.0 ** -25
            err = np.abs(got[i, h] - o)
            assert np.all(err <= bound), f"row {i} head {h}: off by {err.max():.3e}, bound {bound[err.argmax()]:.3e}"
            assert abs(lse[i, h] - ref) <= eta + n * 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -22 * abs(ref)


def test_a_layer_step_by_step():
    """Rotate and store, then attend, token by token and in one chunk: the 4-bit cache's bytes
    are the same, and the outputs agree with attention over what kv_read gives."""
    dev = device()
    gen = torch.Generator().manual_seed(7)
    page, kv, group, dim, n = 16, 2, 4, 128, 70
    rows = values((n, kv * (group + 2), dim), "bf16", gen).to(dev)
    q, k, v = rows.split([kv * group, kv, kv], dim=1)
    f, _ = w4.rope_freqs(dim, 10000.0, device=dev)
    tables = ints([[4, 0, 3, 1, 2]], dev)
    one, two = (w4.kv_cache_e2m1((2, 5), page, kv, dim, device=dev) for _ in range(2))
    cu, lens = ints([0, n], dev), ints([n], dev)
    turned = w4.kv_append_rope(q, k, v, *one, tables, lens, f, cu_seqlens=cu)
    y = w4.attn_prefill(turned, cu, *one, tables, lens)
    steps = []
    for t in range(n):
        at = ints([t + 1], dev)
        qt = w4.kv_append_rope(q[t:t + 1], k[t:t + 1], v[t:t + 1], *two, tables, at, f)
        steps.append(w4.attn_decode(qt, *two, tables, at))
    assert torch.equal(one, two)
    kr, vr = w4.kv_read(*one, tables, lens, cu, n)
    dense = torch.zeros(2, 5, page, kv, dim, dtype=torch.bfloat16, device=dev)
    w4.kv_append(kr, vr, *dense, tables, lens, cu_seqlens=cu)
    want = w4.attn_prefill(turned, cu, *dense, tables, lens)
    # two roundings of weights and outputs, each half a step, of values below 4
    assert (y.float() - want.float()).abs().max() <= 4 * 2 * 2.0 ** -8
    assert (torch.cat(steps).float() - want.float()).abs().max() <= 4 * 2 * 2.0 ** -8


@pytest.mark.parametrize("page,window", [(16, 128), (8, 20), (24, 60)])
def test_the_example_with_a_cache_of_4_bits(page, window):
    import sys
    from pathlib import Path
    sys.path.insert(0, str(Path(__file__).resolve().parent.parent / "examples"))
    import decoder_attention
    dev = device()
    say(f"[example4] page {page}, window {window}")
    decoder_attention.run(cache_type=torch.uint8, page=page, window=window, device=dev, say=say)
