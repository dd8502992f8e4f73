"""Attention of one new token per sequence over the paged cache
(w4a4_attn_decode) against the fp64 oracle: types, head layouts, page sizes
that end inside a tile, lengths from nothing to several pieces of a sequence,
windows and sinks, memory orders, values in masked places, and tables without
a valid page."""
import numpy as np
import pytest
import torch

import w4a4_block_scaled_amd as w4
from gpu_common import device, say
from kv_common import TYPES, as_f64, check_attention, ints, on_device, table_of, values

pytestmark = pytest.mark.gpu

ORDERS = {"page token head": (0, 1, 2), "page head token": (0, 2, 1), "token page head": (1, 0, 2),
          "head page token": (2, 0, 1)}


def make(kind, kv, group, dim, page, lens, seed, order="page token head", high=None, spare=2):
    dev = device()
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    width = max(1, -(-max(lens) // page)) + 1
    pages = sum(-(-n // page) for n in lens) + spare
    tables = table_of(lens, page, pages, width, rng)
    high = high or ("bf16" if kind == "fp8" else kind)
    q = values((len(lens), kv * group, dim), high, gen)
    k, v = values((pages, page, kv, dim), kind, gen), values((pages, page, kv, dim), kind, gen)
    scales = [torch.rand(kv, generator=gen) + 0.5 if kind == "fp8" else None for _ in range(2)]
    f64 = [as_f64(x) * (1.0 if s is None else as_f64(s)[:, None]) for x, s in zip((k, v), scales)]
    kd, vd = (on_device(x.view(torch.uint8), ORDERS[order], dev).view(x.dtype) if kind == "fp8" else
              on_device(x, ORDERS[order], dev) for x in (k, v))
    return {"q": q, "kd": kd, "vd": vd, "f64": f64, "tables": tables, "lens": lens, "high": high,
            "scales": [None if s is None else s.to(dev) for s in scales], "dev": dev}


def run(c, window=0, sinks=0, scale=None, **more):
    return w4.attn_decode(c["q"].to(c["dev"]), c["kd"], c["vd"], ints(c["tables"], c["dev"]), ints(c["lens"], c["dev"]),
                          k_scale=c["scales"][0], v_scale=c["scales"][1], window=window, sinks=sinks, scale=scale,
                          return_lse=True, **more)


def check(c, y, lse, window=0, sinks=0, scale=None, label="", rows=None):
    dim = c["q"].shape[2]
    check_attention(y, lse.cpu(), c["q"], c["f64"], c["tables"], c["lens"], [n - 1 for n in c["lens"]],
                    range(len(c["lens"])), c["high"], dim ** -0.5 if scale is None else scale, window, sinks, "two",
                    label, rows)


CASES = [
    # (type, kv heads, group, dim, page, lens)
    ("bf16", 8, 4, 128, 16, [1, 513, 128, 0, 77]),
    ("bf16", 4, 7, 128, 32, [300, 31, 32, 33, 129]),
    ("fp16", 2, 1, 64, 16, [1, 2, 127, 500]),
    ("fp16", 1, 16, 128, 8, [260, 9]),
    ("bf16", 1, 20, 64, 24, [200, 65]),                  # more rows than one MFMA block
    ("bf16", 2, 3, 256, 16, [140, 16]),
    ("fp8", 4, 7, 128, 64, [700, 64, 1]),
    ("fp8", 2, 2, 64, 16, [100, 333]),
    ("fp8", 1, 4, 256, 128, [257]),
    ("bf16", 2, 4, 128, 11, [150, 11, 12, 400]),         # pages that are no multiple of 8: a lookup per row
    ("fp16", 3, 5, 64, 1, [70, 5]),                      # one token per page
    ("fp8", 2, 4, 128, 5, [133]),
]


@pytest.mark.parametrize("kind,kv,group,dim,page,lens", CASES)
def test_decode_matches_the_oracle(kind, kv, group, dim, page, lens):
    say(f"[decode] {kind} {kv} x {group} heads of {dim}, page {page}, lens {lens}")
    c = make(kind, kv, group, dim, page, lens, seed=sum(lens) + dim)
    y, lse = run(c)
    check(c, y, lse, label="all visible")
    y, lse = run(c, scale=0.31)
    check(c, y, lse, scale=0.31, label="own scale")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (64, 0), (100, 4), (128, 130), (255, 17), (4000, 4)])
@pytest.mark.parametrize("kind,page", [("bf16", 16), ("fp16", 11), ("fp8", 32)])
def test_decode_window_and_sinks(kind, page, window, sinks):
    say(f"[decode] {kind} page {page} window {window} sinks {sinks}")
    c = make(kind, 2, 4, 128, page, [1, 5, 100, 257, 600, 0], seed=window + sinks)
    y, lse = run(c, window, sinks)
    check(c, y, lse, window, sinks, label=f"window {window} sinks {sinks}")


def test_decode_long_sequences_are_split_and_joined():
    """Sequences longer than one workgroup's piece beside short ones: the piece
    boundaries fall inside units, several workgroups join."""
    say("[decode] lens 20011, 3, 9000")
    c = make("bf16", 1, 4, 64, 16, [20011, 3, 9000], seed=3)
    y, lse = run(c)
    check(c, y, lse, label="split")
    say("[decode] one head, 50000 tokens, fp8")
    c = make("fp8", 1, 16, 128, 64, [50000], seed=4)
    y, lse = run(c)
    check(c, y, lse, label="split fp8")


def test_decode_many_sequences():
    """More sequences than lanes of a wave, most of them short."""
    say("[decode] 150 sequences")
    lens = [(37 * i) % 90 for i in range(150)]
    c = make("fp16", 2, 2, 64, 16, lens, seed=5)
    y, lse = run(c)
    check(c, y, lse, label="many", rows=range(0, 150, 7))


@pytest.mark.parametrize("kind,kv,dim,page,seqs,high", [("fp16", 24, 64, 16, 140, 500), ("fp8", 32, 64, 16, 150, 600),
                                                        ("bf16", 8, 256, 11, 100, 800)])
def test_decode_many_units_per_workgroup(kind, kv, dim, page, seqs, high):
    """So many units that every workgroup takes several, with empty and short
    sequences between long ones."""
    say(f"[decode] {seqs} sequences of up to {high} tokens, {kv} heads of {dim}")
    lens = [0 if i % 13 == 5 else 1 + (101 * i) % 40 if i % 4 == 1 else (173 * i) % high for i in range(seqs)]
    c = make(kind, kv, 1, dim, page, lens, seed=seqs)
    y, lse = run(c)
    check(c, y, lse, label="many units", rows=range(0, seqs, 5))


@pytest.mark.parametrize("order", list(ORDERS))
def test_decode_memory_orders(order):
    say(f"[decode] cache order {order}")
    c = make("bf16", 3, 4, 64, 16, [100, 257], seed=6, order=order)
    y, lse = run(c)
    check(c, y, lse, label=order)


def test_decode_strided_queries_and_output():
    """Queries as a slice of a fused projection, output into a wider buffer:
    the rest of the buffer is untouched."""
    say("[decode] strided q and out")
    c = make("bf16", 2, 4, 128, 16, [100, 257, 31], seed=7)
    wide = torch.randn(3, 12, 128, device=c["dev"]).to(torch.bfloat16)
    wide[:, 2:10] = c["q"].to(c["dev"])
    buf = torch.full((3, 10, 128), 7.0, dtype=torch.bfloat16, device=c["dev"])
    y = w4.attn_decode(wide[:, 2:10], c["kd"], c["vd"], ints(c["tables"], c["dev"]), ints(c["lens"], c["dev"]),
                       out=buf[:, 1:9])
    plain, lse = run(c)
    assert torch.equal(y, plain) and torch.all(buf[:, 0] == 7) and torch.all(buf[:, 9] == 7)
    check(c, y, lse, label="strided")


@pytest.mark.parametrize("kind,page", [("bf16", 16), ("fp16", 11), ("fp8", 32)])
def test_decode_ignores_values_in_masked_places(kind, page):
    """Inf and NaN in rows past the length, before the window and between sinks
    and window: the result is that of clean caches, bit for bit."""
    say(f"[decode] masked values, {kind}")
    c = make(kind, 2, 4, 128, page, [300, 45, 700, 1], seed=8)
    window, sinks = 50, 3
    clean, lse = run(c, window, sinks)
    used = np.zeros(c["f64"][0].shape[:2], bool)
    for s, n in enumerate(c["lens"]):
        for t in range(n):
            if t > n - 1 - window or t < sinks:
                used[c["tables"][s, t // page], t % page] = True
    mask = torch.from_numpy(~used).to(c["dev"])
    for x, codes in ((c["kd"], (float("nan"), float("inf"))), (c["vd"], (float("-inf"), float("nan")))):
        for i, code in enumerate(codes):
            half = mask.clone()
            half[:, i::2] = False
            if kind == "fp8":
                x.view(torch.uint8)[half] = 0x7f if i else 0xff
            else:
                x[half] = code
    dirty, lse2 = run(c, window, sinks)
    assert torch.equal(clean, dirty) and torch.equal(lse, lse2)


def test_decode_visible_infinities_and_nan():
    """Inf and NaN that are seen come through as in the formula."""
    say("[decode] visible Inf and NaN")
    c = make("bf16", 1, 4, 64, 16, [40, 40, 40], seed=9)
    place = [(c["tables"][s, 1], 3) for s in range(3)]
    c["vd"][place[0][0], place[0][1], 0, 5] = float("inf")
    c["vd"][place[1][0], place[1][1], 0, 6] = float("nan")
    c["kd"][place[2][0], place[2][1], 0, 7] = float("nan")
    y, _ = run(c)
    assert torch.all(y[0, :, 5] == float("inf")) and torch.isfinite(y[0, :, :5]).all()
    assert torch.isnan(y[1, :, 6]).all() and torch.isfinite(y[1, :, 7:]).all()
    assert torch.isnan(y[2]).all()


def test_decode_large_scores_do_not_overflow():
    say("[decode] large scores")
    c = make("bf16", 1, 4, 64, 16, [200], seed=10)
    c["q"] = c["q"] * 100
    y, lse = run(c, scale=3.0)
    check(c, y, lse, scale=3.0, label="large")


def test_decode_invalid_pages_give_nan_and_no_access():
    """An entry outside the cache, or a length beyond the table, spoils that
    sequence (NaN) and no other; entries that no query sees do not matter."""
    say("[decode] invalid pages")
    c = make("bf16", 2, 4, 128, 16, [100, 100, 100, 100, 100], seed=11)
    good, lse = run(c)
    pages = c["kd"].shape[0]
    for bad in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        t = c["tables"].copy()
        t[1, 2] = bad
        t[2, 6] = bad                 # holds tokens 96 .. 99 of 100
        t[3, 7] = bad                 # past the end: never read
        y = w4.attn_decode(c["q"].to(c["dev"]), c["kd"], c["vd"], ints(t, c["dev"]), ints(c["lens"], c["dev"]))
        assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
        for s in (0, 3, 4):
            assert torch.equal(y[s], good[s])
    lens = list(c["lens"])
    lens[0], lens[4] = 16 * c["tables"].shape[1] + 1, 2 ** 31 - 1
    y = w4.attn_decode(c["q"].to(c["dev"]), c["kd"], c["vd"], ints(c["tables"], c["dev"]), ints(lens, c["dev"]))
    assert torch.isnan(y[0]).all() and torch.isnan(y[4]).all() and torch.equal(y[1:4], good[1:4])
    lens[0], lens[4] = -5, 100
    y, l2 = w4.attn_decode(c["q"].to(c["dev"]), c["kd"], c["vd"], ints(c["tables"], c["dev"]), ints(lens, c["dev"]),
                           return_lse=True)
    assert torch.all(y[0] == 0) and torch.all(l2[0] == float("-inf")) and torch.equal(y[1:], good[1:])
    # trimmed pages before the window
    t = c["tables"].copy()
    t[:, 1:4] = -1
    seen, _ = run(c, 36, 16)
    y = w4.attn_decode(c["q"].to(c["dev"]), c["kd"], c["vd"], ints(t, c["dev"]), ints(c["lens"], c["dev"]), window=36,
                       sinks=16)
    assert torch.equal(y, seen)


def test_decode_offsets_past_32_bits():
    """Pages beyond 2^31 elements of a cache (bf16, more than 4 GiB)."""
    dev = device()
    page, kv, dim = 64, 8, 128
    pages = 2 ** 31 // (page * kv * dim) + 40
    say(f"[decode] {pages} pages of {page * kv * dim} elements")
    c = make("bf16", kv, 1, dim, page, [300, 64], seed=12)
    high = [pages - 1 - 3 * i for i in range(7)]
    k = torch.empty(pages, page, kv, dim, dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    t = np.full_like(c["tables"], -1)
    n = 0
    for s in range(2):
        for j in range(-(-c["lens"][s] // page)):
            k[high[n]], v[high[n]] = c["kd"][c["tables"][s, j]], c["vd"][c["tables"][s, j]]
            t[s, j] = high[n]
            n += 1
    want, _ = run(c)
    got = w4.attn_decode(c["q"].to(dev), k, v, ints(t, dev), ints(c["lens"], dev))
    assert torch.equal(got, want)


def test_decode_another_stream_and_repeats():
    """On a side stream, and many times: the same bits each time."""
    say("[decode] side stream")
    c = make("bf16", 2, 4, 128, 16, [3000, 45, 700, 1], seed=13)
    want, _ = run(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [run(c)[0] for _ in range(20)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_decode_nothing_to_do():
    dev = device()
    k = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=dev)
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=dev)
    y = w4.attn_decode(q, k, k, torch.zeros(0, 3, dtype=torch.int32, device=dev),
                       torch.zeros(0, dtype=torch.int32, device=dev))
    assert y.shape == (0, 4, 64)
