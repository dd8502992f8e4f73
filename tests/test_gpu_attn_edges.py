"""Attention over the paged cache where values or lengths are extreme: Inf and
NaN in places that the kernels treat apart, lengths far below zero, softmax
weights that span the types' range.  Every way that the entry points go is
taken: decoding, few rows per sequence, row tiles whole and with the keys split
(tables that hold more than 1000 tokens, few row tiles)."""
import numpy as np
import pytest
import torch

import w4a4_block_scaled_amd as w4
from gpu_common import device, say
from kv_common import UNIT, as_f64, ints
from oracle import attention as A
from test_gpu_attn_prefill import check, chunks, run

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def place(c, s, t):
    """Page and row of token t of sequence s."""
    page = c["kd"].shape[1]
    return int(c["tables"][s, t // page]), t % page


# ------------------------------------------------- masked values, keys split --

@pytest.mark.parametrize("kind,dim,page", [("bf16", 128, 16), ("bf16", 64, 24), ("fp16", 256, 16), ("fp16", 128, 11),
                                           ("bf16", 128, 1), ("fp8", 128, 32), ("fp8", 256, 8)])
def test_split_keys_ignore_masked_values_in_their_first_tiles(kind, dim, page):
    """The keys are split, and the first tile of the shares holds Inf and NaN that
    some or all rows do not see (before their windows, between sinks and window):
    the rows that do not see them are those of clean caches, bit for bit, each time."""
    say(f"[split] masked values, {kind}, D = {dim}, page {page}")
    window, sinks, past, new = 1100, 2, 1500, 40
    c = chunks(kind, 1, 4, dim, page, [past], [new], seed=dim + page)
    clean, lse = run(c, window, sinks)
    check(c, clean, lse, window, sinks, label="clean", most=4)
    # the first query's window begins at past - window + 1: tokens below are seen by none (sinks apart), the
    # next ones by ever fewer of the 40 queries
    low = past - window + 1
    hidden = [t for t in range(sinks, low)]
    part = [low + i for i in range(0, 12, 5)]             # token low + i: seen by queries 0 .. i
    for t in hidden + part:
        p, r = place(c, 0, t)
        if kind == "fp8":
            c["vd"].view(torch.uint8)[p, r] = 0x7f
            if t in hidden:
                c["kd"].view(torch.uint8)[p, r] = 0xff
        else:
            c["vd"][p, r] = INF if t % 2 else NAN
            if t in hidden:
                c["kd"][p, r] = NAN
    first = part[-1] - low + 1                            # the first query that sees none of them
    for _ in range(5):
        y, l2 = run(c, window, sinks)
        assert torch.equal(y[first:], clean[first:]) and torch.equal(l2, lse)
        assert not torch.isfinite(y[0]).any()


# -------------------------------------------------------- lengths below zero --

@pytest.mark.parametrize("past,new,group,page", [
    ([0, 20], [300, 50], 4, 16),                # row tiles, the tables hold few tokens: keys whole
    ([2000, 30], [300, 50], 4, 16),             # keys split
    ([2000, 30], [300, 50], 4, 11),
    ([0] * 40, [300] * 40, 4, 16),              # more row tiles than the keys would be split for
    ([600, 30], [3, 2], 4, 16),                 # few rows
    ([600, 30], [8, 8], 1, 16),
])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 3)])
def test_lengths_below_zero(past, new, group, page, window, sinks):
    """A negative length, the lowest of its type among them, puts every query
    before position 0: zeros and -inf, and the other sequences as before."""
    say(f"[lengths] past {past[:2]} new {new[:2]} x {len(new)}, group {group}, page {page}, window {window}")
    c = chunks("bf16", 2, group, 128, page, past, new, seed=new[0])
    good, lse = run(c, window, sinks)
    n = int(c["cu"][1])
    for length in (-1, -5, -299, -2 ** 31, -2 ** 31 + 1, -2 ** 31 + 299, -2 ** 31 + 301):
        lens = [length] + list(c["lens"][1:])
        y, l2 = run(c, window, sinks, lens=lens)
        assert torch.all(y[:n] == 0) and torch.all(l2[:n] == -INF), length
        assert torch.equal(y[n:], good[n:]) and torch.equal(l2[n:], lse[n:]), length


# -------------------------------------------------------- Inf that rows see --

@pytest.mark.parametrize("kind,dim,page,past,new", [("bf16", 128, 16, 2500, 40), ("fp16", 64, 8, 2500, 40),
                                                    ("bf16", 256, 11, 1400, 9), ("fp16", 128, 24, 3000, 5)])
def test_split_keys_with_inf_in_the_first_tile_of_a_share(kind, dim, page, past, new):
    """An Inf among the values of any tile of the split keys, the first one of a
    share among them, comes out as Inf in the rows that see it (its weight is
    positive), and elsewhere nothing changes."""
    say(f"[split] Inf, {kind}, D = {dim}, page {page}, past {past}")
    c = chunks(kind, 2, 4, dim, page, [past], [new], seed=dim + past)
    clean, _ = run(c)
    # a token of every tile of 64, its own column each: some of the tiles begin a share
    tiles = list(range(0, past, 64))[:dim - 1]
    for i, t in enumerate(tiles):
        c["vd"][(*place(c, 0, t + i % 7), 0, i)] = INF if i % 2 else -INF
    y, _ = run(c)
    for i in range(len(tiles)):
        assert torch.all(y[:, :4, i] == (INF if i % 2 else -INF)), f"tile {i}"
    assert torch.equal(y[:, 4:], clean[:, 4:]) and torch.equal(y[:, :4, len(tiles):], clean[:, :4, len(tiles):])


WAYS = {
    # past, new, page: what the table holds and the number of rows choose the way
    "decode": ([900, 40], [1, 1], 16), "decode, page 11": ([900, 40], [1, 1], 11), "decode, long": ([30000, 40], [1, 1], 16),
    "few": ([900, 40], [3, 2], 16), "few, long": ([30000, 40], [3, 2], 16),
    "whole": ([700, 40], [150, 60], 16), "whole, page 11": ([700, 40], [150, 60], 11), "split": ([3000, 40], [30, 20], 16),
    "decode, 131071": ([131070], [1], 16), "few, 131071": ([131068], [3], 16), "split, 131071": ([131051], [20], 16),
}


def attend(c, way, window=0, sinks=0):
    """(out, lse) of the new tokens, in their order, by the entry point of the way."""
    if not way.startswith("decode"):
        return run(c, window, sinks)
    dev = c["dev"]
    return w4.attn_decode(c["q"].to(dev), c["kd"], c["vd"], ints(c["tables"], dev), ints(c["lens"], dev),
                          k_scale=c["scales"][0], v_scale=c["scales"][1], window=window, sinks=sinks, return_lse=True)


def steep(kind, dim, way, seed, gaps, group=4):
    """A case whose queries and keys are zero but in the first element, so that the
    weight of token t of sequence 0 is 2^-gaps(t) of the largest, exactly up to the
    rounding of the scale."""
    past, new, page = WAYS[way]
    c = chunks(kind, 1, group, dim, page, past, new, seed=seed)
    c["q"].zero_()
    c["q"][:, :, 0] = 1.0
    n = c["lens"][0]
    k = torch.zeros_like(c["kd"])
    # score in the exponent of 2: dim^-0.5 / ln 2 * key
    x = torch.tensor([-g * dim ** 0.5 * np.log(2.0) for g in (gaps(t) for t in range(n))]).to(c["kd"].dtype).to(c["dev"])
    t = torch.arange(n, device=c["dev"])
    at = ints(c["tables"][0], c["dev"]).long()[t // page], t % page, 0, 0
    if kind == "fp8":
        k.view(torch.uint8)[at] = x.view(torch.uint8)
        c["scales"][0].fill_(1.0)
    else:
        k[at] = x
    c["kd"].copy_(k)
    c["f64"][0] = as_f64(k)
    return c


SMALL = [w for w in WAYS if not w.startswith("whole") and "131071" not in w]


@pytest.mark.parametrize("way", SMALL)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("gap", [30, 110, 200])
@pytest.mark.parametrize("rest", ["all as small", "others large"])
@pytest.mark.parametrize("first", [True, False])
def test_inf_of_a_small_weight(way, kind, gap, rest, first):
    """A value of Inf whose weight is far below the largest, before the largest and
    behind it, where the running maximum takes one long step and where it does not:
    every positive weight makes it Inf."""
    say(f"[inf] {way}, {kind}, 2^-{gap}, {'before' if first else 'behind'} the largest, {rest}")
    past = WAYS[way][0][0]
    top, at = (past - 5, 3) if first else (3, past - 200)
    c = steep(kind, 64, way, 11, lambda t: 0 if t == top else gap if t == at or rest == "all as small" else 4)
    clean, _ = attend(c, way)
    c["vd"][(*place(c, 0, at), 0, 5)] = INF
    c["vd"][(*place(c, 0, at), 0, 6)] = -INF
    y, _ = attend(c, way)
    n = int(c["cu"][1])
    assert torch.all(y[:n, :, 5] == INF) and torch.all(y[:n, :, 6] == -INF)
    keep = [i for i in range(64) if i not in (5, 6)]
    assert torch.isfinite(y[:n][:, :, keep]).all() and torch.equal(y[n:], clean[n:])
    assert (y[:n][:, :, keep].float() - clean[:n][:, :, keep].float()).abs().max() <= 2.0 ** -6


@pytest.mark.parametrize("way", ["whole", "whole, page 11"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("gap", [30, 110, 200])
@pytest.mark.parametrize("rest", ["all as small", "others large"])
@pytest.mark.parametrize("first", [True, False])
def test_inf_of_a_small_weight_in_row_tiles(way, kind, gap, rest, first):
    """The same where the keys are whole: most tiles are seen whole by all rows."""
    test_inf_of_a_small_weight(way, kind, gap, rest, first)


@pytest.mark.parametrize("kind,dim,page", [("bf16", 128, 16), ("fp16", 256, 16), ("fp16", 64, 11)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 70)])
def test_inf_and_nan_in_row_tiles(kind, dim, page, window, sinks):
    """Row tiles with the keys whole: every row gets the Inf and NaN of the tokens
    that it sees, both signs together as NaN, and no others; the rest as before."""
    say(f"[inf] row tiles, {kind}, D = {dim}, page {page}, window {window}")
    past, new, group = 700, 250, 4
    c = chunks(kind, 1, group, dim, page, [past], [new], seed=dim)
    clean, _ = run(c, window, sinks)
    held = [(2, 3, INF), (65, 4, NAN), (100, 5, -INF), (640, 6, INF), (650, 6, -INF), (699, 7, INF), (720, 8, INF),
            (760, 9, NAN), (800, 10, INF), (949, 11, -INF)]
    for t, d, x in held:
        c["vd"][(*place(c, 0, t), 0, d)] = x
    y, _ = run(c, window, sinks)
    want = clean.float()
    for i in range(new):
        p = past + i
        for t, d, x in held:
            if t <= p and (not window or t > p - window or t < sinks):
                seen = want[i, :, d]
                want[i, :, d] = torch.where(torch.isfinite(seen), torch.full_like(seen, x), seen + x)
    assert torch.equal(torch.nan_to_num(y.float(), nan=12345.0), torch.nan_to_num(want, nan=12345.0))


# ------------------------------------------- weights far below the largest --

@pytest.mark.parametrize("way", [w for w in WAYS if "long" not in w])
@pytest.mark.parametrize("kind,high", [("fp16", "fp16"), ("fp8", "fp16"), ("bf16", "bf16")])
@pytest.mark.parametrize("gap", [16, 22, 26])
def test_many_small_weights_beside_a_large_one(way, kind, high, gap):
    """One token takes nearly all the weight and its value is 0, so that the output is
    the sum of the others, each of about 2^-gap.

    Bound, with u, c, eta, n, A and V as in kv_common, for the types' weights kept at
    2^7 or more where the largest one is: FP16's step of 2^-24 rounds a weight by at
    most 2^-25 / 2^7 of the largest (BF16 has no such step), and the exponents, of up
    to gap + 15, are rounded by 2^-24 of themselves:
    |y - o| <= u |o| + (1 + u) (c + 2 eta + (n / 16 + 64) 2^-23 + (gap + 15) 2^-24) A + n 2^-32 V + 2^-25.
    (An fp32 sum here grows by 8 tokens or an MFMA of at least 16 at a time, n / 16
    steps at most, and is joined from fewer than 64 parts in a row.)"""
    say(f"[small] {way}, {kind}, 2^-{gap}")
    past, new, _ = WAYS[way]
    top = 5
    c = steep(kind, 64, way, 12, lambda t: 0 if t == top else gap)
    if high != c["high"]:
        c["high"], c["q"] = high, c["q"].to(torch.float16)
    p, r = place(c, 0, top)
    v = torch.rand(c["vd"].shape, generator=torch.Generator().manual_seed(gap)).to(c["dev"]) + 0.5
    v[p, r] = 0
    c["vd"].copy_(v.to(c["vd"].dtype))
    c["f64"][1] = as_f64(c["vd"]) * (1.0 if c["scales"][1] is None else as_f64(c["scales"][1])[:, None])
    y, lse = attend(c, way)
    u = UNIT[high]
    weights = 2.0 ** -20 if high == "fp16" else 2.0 ** -15
    if way.startswith("whole"):
        weights = u
    for i in (0, new[0] - 1):
        o, ref_lse, (a, big, size, n) = A.attend(as_f64(c["q"])[i, 0], *c["f64"], c["tables"][0], c["lens"][0],
                                                 past[0] + i, 0, 64 ** -0.5, 0, 0)
        eta = 72 * 2.0 ** -23 * size + 2.0 ** -22
        bound = u * np.abs(o) + (1 + u) * (weights + 2 * eta + (n / 16 + 64) * 2.0 ** -23 + (gap + 15) * 2.0 ** -24) * a
        bound += (n * 2.0 ** -32 * big if high == "fp16" else 0) + 2.0 ** -25
        err = np.abs(as_f64(y)[i, 0] - o)
        assert np.all(err <= bound), f"row {i}: off by {err.max():.3e} ({(err / bound).max():.2f} of the bound)"
        assert abs(lse[i, 0].item() - ref_lse) <= eta + n * 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -22 * abs(ref_lse)
