"""Attention of chunks of new tokens over the paged cache (w4a4_attn_prefill)
against the fp64 oracle: ragged batches with and without earlier tokens,
windows and sinks, few rows on long caches (the keys split), rows that see
nothing, values in masked places, and tables without a valid page."""
import numpy as np
import pytest
import torch

import w4a4_block_scaled_amd as w4
from gpu_common import device, say
from kv_common import check_attention, ints, values
from test_gpu_attn_decode import ORDERS, make

pytestmark = pytest.mark.gpu


def chunks(kind, kv, group, dim, page, past, new, seed, **more):
    """`new` tokens of each sequence after `past` earlier ones."""
    c = make(kind, kv, group, dim, page, [a + b for a, b in zip(past, new)], seed, **more)
    c["cu"] = np.concatenate([[0], np.cumsum(new)])
    gen = torch.Generator().manual_seed(seed + 1)
    c["q"] = values((int(c["cu"][-1]), kv * group, dim), c["high"], gen)
    c["seqs"] = np.repeat(np.arange(len(new)), new)
    c["pos"] = np.concatenate([np.arange(b) + a for a, b in zip(past, new)])
    return c


def run(c, window=0, sinks=0, scale=None, q=None, tables=None, lens=None, **more):
    dev = c["dev"]
    return w4.attn_prefill(c["q"].to(dev) if q is None else q, ints(c["cu"], dev), c["kd"], c["vd"],
                           ints(c["tables"] if tables is None else tables, dev),
                           ints(c["lens"] if lens is None else lens, dev), k_scale=c["scales"][0],
                           v_scale=c["scales"][1], window=window, sinks=sinks, scale=scale, return_lse=True, **more)


def check(c, y, lse, window=0, sinks=0, scale=None, label="", most=60):
    n = len(c["q"])
    rows = np.unique(np.r_[0, n - 1, c["cu"][1:-1], np.maximum(c["cu"][1:] - 1, 0), np.random.default_rng(n).choice(n, min(n, most))])
    check_attention(y, lse.cpu(), c["q"], c["f64"], c["tables"], c["lens"], c["pos"], c["seqs"], c["high"],
                    c["q"].shape[2] ** -0.5 if scale is None else scale, window, sinks, "once", label,
                    [r for r in rows if r < n])


CASES = [
    # (type, kv heads, group, dim, page, past, new)
    ("bf16", 8, 4, 128, 16, [0], [82]),
    ("bf16", 4, 7, 128, 32, [0, 100, 17], [130, 1, 65]),
    ("fp16", 2, 1, 64, 16, [0, 0, 300], [1, 200, 64]),
    ("fp16", 1, 16, 128, 8, [50], [40]),
    ("bf16", 1, 20, 64, 24, [7, 0], [33, 64]),
    ("bf16", 2, 3, 256, 16, [10, 0], [70, 5]),
    ("fp8", 4, 7, 128, 64, [200, 0], [31, 100]),
    ("fp8", 2, 2, 64, 16, [0, 90], [150, 3]),
    ("fp8", 1, 4, 256, 128, [100], [50]),
    ("bf16", 2, 4, 128, 11, [5, 300], [100, 9]),
    ("fp16", 3, 5, 64, 1, [3], [70]),
]


@pytest.mark.parametrize("kind,kv,group,dim,page,past,new", CASES)
def test_prefill_matches_the_oracle(kind, kv, group, dim, page, past, new):
    say(f"[prefill] {kind} {kv} x {group} heads of {dim}, page {page}, past {past}, new {new}")
    c = chunks(kind, kv, group, dim, page, past, new, seed=sum(new) + dim)
    y, lse = run(c)
    check(c, y, lse, label="causal")
    y, lse = run(c, scale=0.31)
    check(c, y, lse, scale=0.31, label="own scale", most=20)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (64, 0), (100, 4), (128, 130), (255, 17), (4000, 4)])
@pytest.mark.parametrize("kind,page", [("bf16", 16), ("fp16", 11), ("fp8", 32)])
def test_prefill_window_and_sinks(kind, page, window, sinks):
    say(f"[prefill] {kind} page {page} window {window} sinks {sinks}")
    c = chunks(kind, 2, 4, 128, page, [0, 150, 700], [300, 90, 40], seed=window + sinks)
    y, lse = run(c, window, sinks)
    check(c, y, lse, window, sinks, label=f"window {window} sinks {sinks}")


def test_prefill_few_rows_on_a_long_cache():
    """The row tiles leave the card idle, so the keys are split and joined."""
    say("[prefill] 5 and 2 tokens on 9000 and 30")
    c = chunks("bf16", 2, 4, 128, 16, [9000, 30], [5, 2], seed=1)
    y, lse = run(c)
    check(c, y, lse, label="split")
    y, lse = run(c, 6000, 4)
    check(c, y, lse, 6000, 4, label="split, window")
    say("[prefill] 3 tokens on 20000, fp8")
    c = chunks("fp8", 1, 8, 64, 64, [20000], [3], seed=2)
    y, lse = run(c)
    check(c, y, lse, label="split fp8")


def test_prefill_many_row_tiles():
    """Enough row tiles that nothing is split, rows of several tiles."""
    say("[prefill] 1500 tokens, 8 heads of 4")
    c = chunks("bf16", 8, 4, 128, 16, [0, 600], [1000, 500], seed=3)
    y, lse = run(c)
    check(c, y, lse, label="whole", most=12)


def test_prefill_agrees_with_decode():
    """A single token per sequence: both entry points see the same tokens."""
    say("[prefill] against decode")
    c = chunks("bf16", 2, 4, 128, 16, [299, 0, 44], [1, 1, 1], seed=4)
    y, lse = run(c, 100, 4)
    check(c, y, lse, 100, 4, label="one token")
    z, lz = w4.attn_decode(c["q"].to(c["dev"]), c["kd"], c["vd"], ints(c["tables"], c["dev"]), ints(c["lens"], c["dev"]),
                           window=100, sinks=4, return_lse=True)
    assert (y.float() - z.float()).abs().max() <= 2.0 ** -6 and (lse - lz).abs().max() <= 1e-4


def test_prefill_rows_without_tokens():
    """Sequences of no new tokens, and queries before position 0 (a length
    smaller than the number of queries): zeros, and -inf."""
    say("[prefill] empty rows")
    c = chunks("bf16", 2, 4, 64, 16, [0, 20, 0, 0], [40, 0, 0, 12], seed=5)
    c["lens"] = [30, 20, 0, 0]           # the first 10 queries of sequence 0 and all of sequence 3 see nothing
    c["pos"] = np.r_[np.arange(-10, 30), np.arange(-12, 0)]
    y, lse = run(c)
    assert torch.all(y[:10] == 0) and torch.all(y[40:] == 0) and torch.all(lse[:10] == float("-inf"))
    check(c, y, lse, label="empty rows")


@pytest.mark.parametrize("order", list(ORDERS))
def test_prefill_memory_orders(order):
    say(f"[prefill] cache order {order}")
    c = chunks("bf16", 3, 4, 64, 16, [10, 0], [90, 30], seed=6, order=order)
    y, lse = run(c)
    check(c, y, lse, label=order, most=20)


def test_prefill_strided_queries_and_output():
    say("[prefill] strided q and out")
    c = chunks("bf16", 2, 4, 128, 16, [0, 9], [50, 31], seed=7)
    wide = torch.zeros(81, 12, 128, dtype=torch.bfloat16, device=c["dev"])
    wide[:, 2:10] = c["q"].to(c["dev"])
    buf = torch.full((81, 10, 128), 7.0, dtype=torch.bfloat16, device=c["dev"])
    y, _ = run(c, q=wide[:, 2:10], out=buf[:, 1:9])
    plain, _ = run(c)
    assert torch.equal(y, plain) and torch.all(buf[:, 0] == 7) and torch.all(buf[:, 9] == 7)


@pytest.mark.parametrize("kind,past,new", [("bf16", [0, 300], [150, 70]), ("fp16", [2000], [9])])
def test_prefill_ignores_values_in_masked_places(kind, past, new):
    """Inf and NaN where no query sees them (past the end, between sinks and
    window): bit for bit the result of clean caches.  In the last token, which
    only the last query sees: every other row is unchanged, and the last one
    gets them."""
    say(f"[prefill] masked values, {kind} past {past} new {new}")
    window, sinks = 80, 3
    c = chunks(kind, 2, 4, 128, 16, past, new, seed=8)
    clean, lse = run(c, window, sinks)
    seen = np.zeros(c["f64"][0].shape[:2], bool)
    for s, n in enumerate(c["lens"]):
        for t in range(n):
            if t > past[s] - window or t < sinks:
                seen[c["tables"][s, t // 16], t % 16] = True
    hidden = torch.from_numpy(~seen).to(c["dev"])
    c["kd"][hidden] = float("nan")
    c["vd"][hidden] = float("inf")
    dirty, lse2 = run(c, window, sinks)
    assert torch.equal(clean, dirty) and torch.equal(lse, lse2)
    last = c["lens"][0] - 1
    at = (c["tables"][0, last // 16], last % 16)
    c["vd"][at[0], at[1], 0, 5] = float("-inf")
    c["vd"][at[0], at[1], 0, 6] = float("nan")
    c["kd"][at[0], at[1], 1, 3] = float("nan")
    y, _ = run(c, window, sinks)
    row = int(c["cu"][1]) - 1
    keep = [i for i in range(len(clean)) if i != row]
    assert torch.equal(y[keep], clean[keep])
    assert torch.all(y[row, :4, 5] == float("-inf")) and torch.isnan(y[row, :4, 6]).all()
    assert torch.equal(y[row, :4, :5], clean[row, :4, :5]) and torch.isnan(y[row, 4:]).all()


def test_prefill_invalid_pages_give_nan_and_no_access():
    say("[prefill] invalid pages")
    c = chunks("bf16", 2, 4, 128, 16, [60, 60, 60], [40, 40, 40], seed=9)
    good, _ = run(c)
    pages = c["kd"].shape[0]
    for bad in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        t = c["tables"].copy()
        t[1, 2] = bad
        t[2, 7] = bad                # past the end
        y, _ = run(c, tables=t)
        assert torch.isnan(y[40:80]).all() and torch.equal(y[:40], good[:40]) and torch.equal(y[80:], good[80:])
    y, _ = run(c, lens=[100, 2 ** 31 - 1, 100])
    assert torch.isnan(y[40:80]).all() and torch.equal(y[:40], good[:40]) and torch.equal(y[80:], good[80:])
    # trimmed pages before the window of every query
    t = c["tables"].copy()
    t[:, 1:2] = -1
    seen, _ = run(c, 29, 16)
    y, _ = run(c, 29, 16, tables=t)
    assert torch.equal(y, seen)
    # row counts that do not fit the rows: nothing outside is touched
    dev = c["dev"]
    for cu in ([0, 40, 200, 120], [0, -40, 80, 120], [5, 5, 5, 10 ** 9]):
        w4.attn_prefill(c["q"].to(dev), ints(cu, dev), c["kd"], c["vd"], ints(c["tables"], dev), ints(c["lens"], dev))
    torch.cuda.synchronize()


def test_prefill_nothing_to_do():
    dev = device()
    k = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=dev)
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=dev)
    y = w4.attn_prefill(q, ints([0, 0], dev), k, k, ints([[0, 1]], dev), ints([5], dev))
    assert y.shape == (0, 4, 64)


# Few queries per sequence go another way than many (and pages that are no
# multiple of 8 tokens always go the way of many): the cases below cross both.

@pytest.mark.parametrize("kind,kv,group,dim,page,past,new", [
    ("bf16", 2, 4, 128, 16, [3000, 7, 0], [4, 3, 1]),            # up to 16 rows
    ("fp16", 4, 7, 64, 32, [500, 2100], [4, 3]),                 # up to 32
    ("fp8", 2, 4, 128, 64, [5000, 0, 77], [9, 16, 0]),           # up to 64
    ("bf16", 1, 20, 256, 8, [300], [3]),
    ("fp8", 3, 1, 64, 16, [100, 900, 40], [40, 2, 1]),           # uneven: 40 rows in blocks of 16
    ("bf16", 2, 4, 128, 16, [4000, 3000], [40, 33]),             # many rows, the keys split
    ("fp16", 1, 8, 64, 16, [6000], [30]),
    ("fp8", 2, 7, 128, 32, [2500], [25]),
    ("bf16", 1, 4, 256, 16, [2000], [50]),
    ("bf16", 2, 4, 128, 11, [3000, 7], [4, 3]),
])
def test_prefill_few_and_split(kind, kv, group, dim, page, past, new):
    say(f"[prefill] few / split: {kind} {kv} x {group} heads of {dim}, page {page}, past {past}, new {new}")
    c = chunks(kind, kv, group, dim, page, past, new, seed=sum(past) + dim)
    for window, sinks in ((0, 0), (70, 5), (1500, 0)):
        y, lse = run(c, window, sinks)
        check(c, y, lse, window, sinks, label=f"window {window} sinks {sinks}", most=8)


@pytest.mark.parametrize("new", [[3, 2], [8, 8], [16, 12], [60, 50]])
def test_prefill_few_edges(new):
    """Rows that see nothing, pages that are missing, and values in masked places,
    for every way that few rows go."""
    say(f"[prefill] few, edges: new {new}")
    c = chunks("bf16", 2, 4, 128, 16, [600, 600], new, seed=sum(new))
    clean, lse = run(c, 90, 3)
    check(c, clean, lse, 90, 3, label="window", most=8)
    n0 = new[0]
    # a length below the number of queries
    lens = [2, c["lens"][1]]
    y, l2 = run(c, 90, 3, lens=lens)
    assert torch.all(y[:n0 - 2] == 0) and torch.all(l2[:n0 - 2] == float("-inf")) and torch.isfinite(y[n0 - 2:n0]).all()
    assert torch.equal(y[n0:], clean[n0:])
    # missing pages: of a seen token, and of one before every window
    t = c["tables"].copy()
    t[0, c["lens"][0] // 16 - 1] = -1
    t[1, 5:20] = c["kd"].shape[0]
    y, _ = run(c, 90, 3, tables=t)
    first = max(0, 16 * (c["lens"][0] // 16 - 1) - 600)          # the first query that sees a token of the missing page
    assert torch.isnan(y[first:n0]).all() and torch.equal(y[n0:], clean[n0:])
    # Inf and NaN in the last token's values: only the last query sees them
    last = c["lens"][0] - 1
    at = (c["tables"][0, last // 16], last % 16)
    c["vd"][at[0], at[1], 0, 5] = float("inf")
    c["vd"][at[0], at[1], 0, 6] = float("nan")
    c["kd"][at[0], at[1], 1, 3] = float("nan")
    y, _ = run(c, 90, 3)
    row = n0 - 1
    keep = [i for i in range(len(clean)) if i != row]
    assert torch.all(y[row, :4, 5] == float("inf")) and torch.isnan(y[row, :4, 6]).all() and torch.isnan(y[row, 4:]).all()
    assert torch.isfinite(y[keep]).all() and (y[keep].float() - clean[keep].float()).abs().max() <= 2.0 ** -6
    # uninitialised rows past the end
    held = -(-c["lens"][1] // 16) * 16
    if held > c["lens"][1]:
        c["vd"][c["tables"][1, held // 16 - 1], c["lens"][1] % 16:] = float("nan")
        z, _ = run(c, 90, 3)
        assert torch.equal(z, y) or torch.equal(torch.nan_to_num(z), torch.nan_to_num(y))


def test_prefill_row_counts_that_do_not_fit():
    """cu_seqlens that point outside the rows: nothing outside is touched."""
    say("[prefill] few rows, stray cu_seqlens")
    c = chunks("bf16", 2, 4, 128, 16, [60, 60, 60], [4, 4, 4], seed=9)
    dev = c["dev"]
    for cu in ([0, 4, 20, 12], [0, -4, 8, 12], [5, 5, 5, 10 ** 9], [7, 7, 7, 7]):
        w4.attn_prefill(c["q"].to(dev), ints(cu, dev), c["kd"], c["vd"], ints(c["tables"], dev), ints(c["lens"], dev))
    torch.cuda.synchronize()
