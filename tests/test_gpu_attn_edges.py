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
from kv_common import ints
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
