"""Rows into and out of the paged cache: rotated on the way (w4a4_kv_append_rope),
into a cache of 4 bits (w4a4_kv_append), and read back (w4a4_kv_read), against the
fp64 oracle.  Codes of 8 and 4 bits are those of the unrounded rotated values."""
import numpy as np
import pytest
import torch

import w4a4_block_scaled_amd as w4
from gpu_common import device, say
from kv_common import TYPES, as_f64, ints, on_device, table_of, values
from oracle import attention as A
from oracle import rotary as R
from rows_common import MOST, bytes_of, check_rotated, fp4_cache, fp4_tensor, freqs_of, on_gpu
from test_gpu_attn_decode import ORDERS

pytestmark = pytest.mark.gpu


def cache_of(kind, pages, page, heads, dim, gen, dev, order="page token head", gap=0):
    """(tensor on the device, its values in fp64 or, in 4 bits, its bytes)."""
    if kind == "fp4":
        t, _, _ = fp4_cache(pages, page, heads, dim, gen, gap)
        return on_gpu(t, dev), bytes_of(t).copy()
    x = values((pages, page, heads, dim), kind, gen)
    if kind == "fp8":
        return on_device(x.view(torch.uint8), ORDERS[order], dev).view(x.dtype), as_f64(x)
    return on_device(x, ORDERS[order], dev), as_f64(x)


CASES = [
    # cache, rows, kv heads, group, dim, rot, interleaved, page, past, new
    ("bf16", "bf16", 8, 4, 128, 128, False, 16, [0, 100, 5], [40, 1, 33]),
    ("fp16", "fp16", 2, 7, 64, 32, True, 11, [3, 0], [1, 64]),
    ("bf16", "bf16", 3, 5, 64, 20, False, 8, [7], [70]),
    ("fp8", "bf16", 4, 7, 128, 64, False, 24, [0, 30, 0, 1], [1, 2, 300, 5]),
    ("fp8", "fp16", 16, 1, 64, 16, True, 16, [1000, 0], [3, 50]),
    ("fp8", "bf16", 1, 4, 256, 250, False, 32, [20], [9]),
    ("fp4", "bf16", 4, 7, 128, 128, False, 32, [0, 100, 0], [130, 1, 65]),
    ("fp4", "fp16", 3, 5, 64, 64, True, 11, [5, 0], [40, 12]),
    ("fp4", "bf16", 16, 1, 64, 48, False, 16, [9] * 20, [1] * 20),
    ("fp4", "fp16", 1, 16, 256, 128, False, 64, [63, 64], [2, 200]),
    ("fp4", "bf16", 2, 2, 128, 6, False, 1, [3], [30]),
    ("fp4", "bf16", 1, 1, 128, 2, True, 128, [131000], [72]),
]


def expected(kind, before, new, tables, lens, cu, page, heads, dim, scale, high):
    """The cache after the rows `new` (fp64), from what it held."""
    after = before.copy()
    if kind == "fp4":
        R.append(after, new, tables, lens, cu, page, heads, dim, MOST[high])
        return after
    for s in range(len(lens)):
        for i in range(cu[s], cu[s + 1]):
            p = int(lens[s]) - int(cu[s + 1]) + i
            if p < 0 or p // page >= tables.shape[1] or not 0 <= tables[s, p // page] < len(after):
                continue
            after[tables[s, p // page], p % page] = new[i] if kind != "fp8" else A.e4m3_value(new[i] / scale[:, None])
    return after


@pytest.mark.parametrize("order", ["page token head", "page head token"])
@pytest.mark.parametrize("kind,high,kv,group,dim,rot,interleaved,page,past,new", CASES)
def test_append_rope_matches_the_oracle(kind, high, kv, group, dim, rot, interleaved, page, past, new, order):
    dev = device()
    say(f"[append_rope] {high} rows, {kind} cache, {kv} x {group} heads, {rot} of {dim}, page {page}, past {past}, new {new}")
    gen, rng = torch.Generator().manual_seed(dim + rot), np.random.default_rng(dim + page)
    lens = [a + b for a, b in zip(past, new)]
    cu = np.concatenate([[0], np.cumsum(new)])
    n = int(cu[-1])
    pages = sum(-(-x // page) for x in lens) + 2
    tables = table_of(lens, page, pages, max(-(-x // page) for x in lens) + 1, rng)
    (kd, kb), (vd, vb) = (cache_of(kind, pages, page, kv, dim, gen, dev, order, gap=group % 2) for _ in range(2))
    scale = [torch.rand(kv, generator=gen) + 0.5 if kind == "fp8" else None for _ in range(2)]
    rows = values((n, kv * (group + 2), dim), high, gen)
    q, k, v = rows.to(dev).split([kv * group, kv, kv], dim=1)
    f, factor = freqs_of(rot, 500000.0), 1.25
    pos = np.concatenate([np.arange(b) + a for a, b in zip(past, new)])
    out = w4.kv_append_rope(q, k, v, kd, vd, ints(tables, dev), ints(lens, dev), torch.from_numpy(f).to(dev),
                            cu_seqlens=ints(cu, dev), interleaved=interleaved, factor=factor,
                            **({"k_scale": scale[0].to(dev), "v_scale": scale[1].to(dev)} if kind == "fp8" else {}))
    q, k, v = rows.split([kv * group, kv, kv], dim=1)
    check_rotated(out, q, pos, f, high, interleaved, False, factor, "q")
    turned = R.rotate(as_f64(k), pos, f, interleaved, False, factor)
    s64 = [None if s is None else as_f64(s) for s in scale]
    if kind == "fp4":
        for name, got, want in (("k", kd, expected(kind, kb, turned, tables, lens, cu, page, kv, dim, None, high)),
                                ("v", vd, expected(kind, vb, as_f64(v), tables, lens, cu, page, kv, dim, None, high))):
            bad = (bytes_of(got) != want).sum()
            assert bad == 0, f"{name}: {bad} bytes differ"
        return
    want = expected(kind, vb, as_f64(v), tables, lens, cu, page, kv, dim, s64[1], high)
    assert np.array_equal(as_f64(vd), want)
    want = expected(kind, kb, turned, tables, lens, cu, page, kv, dim, s64[0], high)
    if kind == "fp8":
        assert np.array_equal(as_f64(kd), want)
        return
    at = [tables[s, p // page] for s, p in zip(np.repeat(np.arange(len(new)), new), pos)], pos % page
    check_rotated(kd[at[0], at[1]], k, pos, f, high, interleaved, False, factor, "k")
    got = as_f64(kd)
    want[at], got[at] = 0, 0
    assert np.array_equal(got, want)                     # every other row as it was


@pytest.mark.parametrize("case", [
    # calls of so many tokens that a workgroup takes queries, keys and values: one vector of a kind per
    # thread, several, more than are in flight at once; every way the pairs lie
    ("fp8", "fp16", 16, 1, 64, 16, True, 24, [10, 0, 3], [1000, 1, 99]),
    ("fp4", "bf16", 4, 7, 128, 128, False, 32, [0, 77], [1500, 1501]),
    ("bf16", "bf16", 2, 3, 256, 250, False, 16, [0], [2200]),
    ("fp8", "bf16", 1, 5, 128, 128, False, 64, [5, 0], [8000, 1300]),
    ("fp4", "fp16", 1, 1, 64, 34, False, 8, [0, 0], [9000, 8000]),
    ("fp16", "fp16", 3, 2, 128, 96, True, 11, [1], [2500])])
def test_append_rope_of_many_tokens(case):
    test_append_rope_matches_the_oracle(*case, "page token head")


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_rows_without_a_place(kind):
    """Rows of no sequence are left, rows at negative places and without a page are
    rotated and not stored; one row per sequence without cu; positions of one's own."""
    dev = device()
    say(f"[append_rope] rows without a place, {kind}")
    gen, f = torch.Generator().manual_seed(1), freqs_of(64)
    page, kv, dim, pages = 8, 2, 64, 6
    (kd, kb), (vd, vb) = (cache_of(kind, pages, page, kv, dim, gen, dev) for _ in range(2))
    rows = values((12, 8, dim), "bf16", gen)
    q, k, v = rows.to(dev).split([4, 2, 2], dim=1)
    tables = np.array([[0, 9], [1, -1], [2, 3]], np.int32)
    lens, cu = [10, 2, 17], [0, 4, 8, 10]                # rows 10, 11 belong to nobody
    q_out = torch.full((12, 4, dim), 9.0, dtype=torch.bfloat16, device=dev)
    out = w4.kv_append_rope(q, k, v, kd, vd, ints(tables, dev), ints(lens, dev), torch.from_numpy(f).to(dev),
                            cu_seqlens=ints(cu, dev), q_out=q_out)
    pos = np.array([6, 7, 8, 9, -2, -1, 0, 1, 15, 16])
    assert out is q_out and torch.all(q_out[10:] == 9)
    check_rotated(q_out[:10], rows[:10, :4], pos, f, "bf16")
    k64, v64 = R.rotate(as_f64(rows[:10, 4:6]), pos, f), as_f64(rows[:10, 6:])
    one = np.ones(kv)
    for got, before, new in ((kd, kb, k64), (vd, vb, v64)):
        want = expected(kind, before, new, tables, lens, cu, page, kv, dim, one, "bf16")
        if kind == "fp4":
            assert np.array_equal(bytes_of(got), want)
        elif kind == "fp8" or new is v64:
            assert np.array_equal(as_f64(got), want)
        else:
            assert np.abs(as_f64(got) - want).max() <= 2.0 ** -8 * 8     # a rounding of values below 8
    # own positions turn, the places store; without q; one row per sequence
    (kd, kb), (vd, vb) = (cache_of(kind, pages, page, kv, dim, gen, dev) for _ in range(2))
    pos = [70000, 5, -3]
    assert w4.kv_append_rope(None, k[:3], v[:3], kd, vd, ints(tables, dev), ints([8, 1, 16], dev), torch.from_numpy(f).to(dev),
                             positions=ints(pos, dev)) is None
    k64 = R.rotate(as_f64(rows[:3, 4:6]), pos, f)
    want = expected(kind, kb, k64, tables, [8, 1, 16], [0, 1, 2, 3], page, kv, dim, one, "bf16")
    if kind == "fp4":
        assert np.array_equal(bytes_of(kd), want)
    else:
        assert np.abs(as_f64(kd) - want).max() <= (0 if kind == "fp8" else 2.0 ** -8 * 8)


def test_queries_in_place_between_their_keys():
    dev = device()
    gen = torch.Generator().manual_seed(2)
    rows = values((50, 12, 128), "bf16", gen).to(dev)
    q, k, v = rows.split([8, 2, 2], dim=1)
    caches = [torch.zeros(9, 16, 2, 128, dtype=torch.bfloat16, device=dev) for _ in range(4)]
    tables, lens, cu = ints(np.arange(8).reshape(2, 4), dev), ints([30, 20], dev), ints([0, 30, 50], dev)
    f = torch.from_numpy(freqs_of(128)).to(dev)
    want = w4.kv_append_rope(q, k, v, *caches[:2], tables, lens, f, cu_seqlens=cu)
    keep = rows[:, 8:].clone()
    w4.kv_append_rope(q, k, v, *caches[2:], tables, lens, f, cu_seqlens=cu, q_out=q)
    assert torch.equal(q, want) and torch.equal(rows[:, 8:], keep)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("seqs", [63, 64, 65, 300])
@pytest.mark.parametrize("own", [False, True])
def test_many_sequences(kind, seqs, own):
    """More sequences than a wave has lanes, many without new tokens, with the tokens' places or positions
    of one's own; what was stored is read back."""
    dev = device()
    say(f"[append_rope] {seqs} sequences, {kind}, own positions {own}")
    gen, rng, f = torch.Generator().manual_seed(seqs), np.random.default_rng(seqs), freqs_of(64)
    page, kv, dim = 8, 1, 64
    new = rng.integers(0, 4, seqs)
    new[[0, 1, seqs - 1]] = 0
    past = rng.integers(0, 20, seqs)
    lens, cu = list(past + new), np.concatenate([[0], np.cumsum(new)])
    n, pages = int(cu[-1]), sum(-(-x // page) for x in lens) + 1
    tables = table_of(lens, page, pages, 4, rng)
    (kd, kb), (vd, vb) = (cache_of(kind, pages, page, kv, dim, gen, dev) for _ in range(2))
    rows = values((n, 4, dim), "bf16", gen)
    q, k, v = rows.to(dev).split([2, 1, 1], dim=1)
    place = np.concatenate([np.arange(b) + a for a, b in zip(past, new)])
    pos = rng.integers(0, 200000, n) if own else place
    out = w4.kv_append_rope(q, k, v, kd, vd, ints(tables, dev), ints(lens, dev), torch.from_numpy(f).to(dev),
                            cu_seqlens=ints(cu, dev), positions=ints(pos, dev) if own else None)
    check_rotated(out, rows[:, :2], pos, f, "bf16")
    k64, v64 = R.rotate(as_f64(rows[:, 2:3]), pos, f), as_f64(rows[:, 3:])
    read = w4.kv_read(kd, vd, ints(tables, dev), ints(lens, dev), ints(cu, dev), n)
    at = tables[np.repeat(np.arange(seqs), new), place // page], place % page
    for got, before, exact, back in ((kd, kb, k64, read[0]), (vd, vb, v64, read[1])):
        if kind == "fp4":
            want = expected(kind, before, exact, tables, lens, cu, page, kv, dim, None, "bf16")
            assert np.array_equal(bytes_of(got), want)
            rows_at = R.decode_blocks(*R.from_pages(want[:, :R.page_bytes(page, kv, dim)], page, kv, dim))[at]
            assert np.array_equal(as_f64(back), rows_at)
        else:
            assert torch.equal(got[at[0], at[1]], back)
    if kind == "bf16":
        check_rotated(read[0], rows[:, 2:3], pos, f, "bf16")
        assert torch.equal(read[1].cpu(), rows[:, 3:])


@pytest.mark.parametrize("high", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_ties_of_8_bits(high, interleaved):
    """Halfway between two 8-bit values, and the two neighbours of that in the rows' type: to the even one
    and to the nearer one, for keys at position 0 (which stay as they are) and for values.  With scale 0.75 the
    quotients are exact where the product 0.75 * value is."""
    dev = device()
    say(f"[append_rope] 8-bit ties, {high}")
    bits = torch.arange(0x08, 0x7e).to(torch.uint8)                       # normal values and their successors
    mid = (bits.view(torch.float8_e4m3fn).double() + (bits + 1).view(torch.float8_e4m3fn).double()) / 2
    assert torch.isfinite(mid).all()
    for unit in (1.0, 0.75, 2.0 ** -7):
        x = (mid * unit).to(TYPES[high])
        near = x.view(torch.int16)
        x = torch.cat([x, (near + 1).view(x.dtype), (near - 1).view(x.dtype)])
        x = torch.cat([x, -x, torch.zeros(-2 * len(x) % 64, dtype=x.dtype)]).view(-1, 1, 64)
        n = len(x)
        tables = np.arange(n, dtype=np.int32)[:, None]
        scale = torch.tensor([unit], device=dev)
        cache = torch.zeros(2, n, 1, 1, 64, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
        w4.kv_append_rope(None, x.to(dev), x.to(dev), *cache, ints(tables, dev), ints([1] * n, dev), torch.from_numpy(freqs_of(64)).to(dev),
                          interleaved=interleaved, k_scale=scale, v_scale=scale)
        want = A.e4m3_value(as_f64(x) / unit)
        for got in cache:
            assert np.array_equal(as_f64(got)[:, 0], want)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_of_zeros_inf_and_nan(kind, interleaved):
    """A pair with NaN or Inf spoils itself (in 4 bits its block), and no other; zeros stay zeros."""
    dev = device()
    say(f"[append_rope] zeros, Inf and NaN, {kind}, interleaved {interleaved}")
    page, kv, dim, n = 16, 2, 128, 20
    f, pos = freqs_of(128), np.arange(n) + 5
    rows = values((n, kv, dim), "bf16", torch.Generator().manual_seed(8))
    rows[3], rows[4, 0] = 0, -0.0
    at = [(6, 0, 5, float("nan")), (7, 1, 70, float("inf")), (8, 0, 127, -float("inf")), (9, 1, 0, float("nan"))]
    bad = np.zeros((n, kv, dim), bool)                      # of the turned keys
    clean = rows.clone()
    for t, h, d, x in at:
        rows[t, h, d] = x
        clean[t, h, d] = 0
        bad[t, h, [d, d ^ 1 if interleaved else d ^ 64]] = True
    tables, lens, cu = ints([[0, 1]], dev), ints([n + 5], dev), ints([0, n], dev)
    ours, other = ([w4.kv_cache_e2m1(3, page, kv, dim, device=dev) if kind == "fp4" else
                    torch.zeros(3, page, kv, dim, dtype=torch.bfloat16, device=dev).to(TYPES[kind]) for _ in range(2)] for _ in range(2))
    turn = torch.from_numpy(f).to(dev)
    w4.kv_append_rope(None, rows.to(dev), rows.to(dev), *ours, tables, lens, turn, cu_seqlens=cu, interleaved=interleaved)
    w4.kv_append_rope(None, clean.to(dev), clean.to(dev), *other, tables, lens, turn, cu_seqlens=cu, interleaved=interleaved)
    k, v = (as_f64(x) for x in w4.kv_read(*ours, tables, lens, cu, n))
    k2, v2 = (as_f64(x) for x in w4.kv_read(*other, tables, lens, cu, n))
    off = ~np.isfinite(as_f64(rows))
    if kind == "fp4":
        bad, off = (np.repeat(m.reshape(n, kv, -1, 32).any(-1), 32, -1).reshape(m.shape) for m in (bad, off))
        assert np.isnan(k[bad]).all() and np.isnan(v[off]).all()
    assert not np.isfinite(k[bad]).any() or kind == "fp8"  # (8 bits hold Inf as their largest value)
    assert np.isnan(k[6, 0, 5]) and np.isnan(k[9, 1, 0])
    assert np.array_equal(k[~bad], k2[~bad]) and np.array_equal(v[~off], v2[~off])
    assert not k[3].any() and not v[4, 0].any()


@pytest.mark.parametrize("factor", [2.0 ** -120, 1e-30, 3e20, 2.0 ** 100])
def test_factors_of_any_size_in_4_bits(factor):
    dev = device()
    say(f"[append_rope] 4 bit, factor {factor}")
    page, kv, dim, n = 16, 1, 128, 16
    f, pos = freqs_of(128), np.arange(n)
    rows = values((n, kv, dim), "bf16", torch.Generator().manual_seed(9))
    cache = w4.kv_cache_e2m1((2, 1), page, kv, dim, device=dev)
    before = bytes_of(cache[0]).copy()
    w4.kv_append_rope(None, rows.to(dev), rows.to(dev), *cache, ints([[0]], dev), ints([n], dev), torch.from_numpy(f).to(dev),
                      cu_seqlens=ints([0, n], dev), factor=factor)
    want = expected("fp4", before, R.rotate(as_f64(rows), pos, f, False, False, factor), np.array([[0]]), [n], [0, n], page, kv,
                    dim, None, "bf16")
    assert np.array_equal(bytes_of(cache[0]), want)


# ------------------------------------------------------------- 4-bit storing --

@pytest.mark.parametrize("high", ["bf16", "fp16"])
@pytest.mark.parametrize("kv,dim,page", [(2, 64, 8), (3, 128, 11), (1, 256, 16)])
def test_append_4_bit_is_the_quantizers_bits(high, kv, dim, page):
    """Blocks of every size the type has, zeros, ties, the largest exponent, Inf and NaN."""
    dev = device()
    say(f"[append] 4 bit, {high}, {kv} heads of {dim}, page {page}")
    gen, rng = torch.Generator().manual_seed(3), np.random.default_rng(3)
    n = 200
    low, top = (-130, 126) if high == "bf16" else (-22, 14)
    x = torch.randn(2, n, kv, dim // 32, 32, generator=gen) * torch.exp2(
        torch.randint(low, top, (2, n, kv, dim // 32, 1), generator=gen).float())
    x[:, 5] = 0.0
    x[0, 6, 0, 0, 3] = -0.0
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.5, -0.25, -5.0, 0.0, -0.0, 4.0, 4.0])
    x[:, 7] = torch.cat([grid, -grid])                      # ties, and values that saturate
    x[0, 8, 0, 0, 9], x[1, 9, 0, -1, 30], x[0, 10, -1, -1, 0] = float("nan"), float("inf"), -float("inf")
    x = x.flatten(-2).to(TYPES[high])
    x[1, 11] = torch.finfo(TYPES[high]).max
    x[1, 12] = torch.finfo(TYPES[high]).tiny
    lens, tables = [n], table_of([n], page, -(-n // page) + 1, -(-n // page), rng)
    (kd, kb), (vd, vb) = (cache_of("fp4", -(-n // page) + 1, page, kv, dim, gen, dev, gap=1) for _ in range(2))
    w4.kv_append(x[0].to(dev), x[1].to(dev), kd, vd, ints(tables, dev), ints(lens, dev), cu_seqlens=ints([0, n], dev))
    for got, before, new in ((kd, kb, x[0]), (vd, vb, x[1])):
        want = expected("fp4", before, as_f64(new), tables, lens, [0, n], page, kv, dim, None, high)
        assert np.array_equal(bytes_of(got), want)


@pytest.mark.parametrize("page", [16, 24, 11])
def test_forks_copies_and_compaction_of_4_bit_pages(page):
    """The bookkeeping moves a page's codes and scales together."""
    dev = device()
    say(f"[pages] 4 bit, page {page}")
    kv, dim, gen = 2, 64, torch.Generator().manual_seed(4)
    pool = w4.kv_cache_e2m1((2, 12), page, kv, dim, device=dev)
    tables, refs = torch.full((3, 4), -1, dtype=torch.int32, device=dev), torch.zeros(12, dtype=torch.int32, device=dev)
    lens = ints([page + 5, 3, 0], dev)
    w4.kv_reserve(tables, lens, refs, page)
    n = page + 8
    k, v = (values((n, kv, dim), "bf16", gen).to(dev) for _ in range(2))
    cu = ints([0, page + 5, n, n], dev)
    w4.kv_append(k, v, *pool, tables, lens, cu_seqlens=cu)
    want = w4.kv_read(*pool, tables, lens, cu, n)
    w4.kv_fork(pool, tables, lens, refs, ints([0], dev), ints([2], dev))
    both = ints([0, page + 5, n, n + page + 5], dev)
    got = w4.kv_read(*pool, tables, lens, both, n + page + 5)
    for g, w in zip(got, want):
        assert torch.equal(g[:n], w) and torch.equal(g[n:], w[:page + 5])
    w4.kv_free(tables, lens, refs, ints([1], dev))
    w4.kv_compact(pool, tables, refs)
    both = ints([0, page + 5, page + 5, 2 * page + 10], dev)
    got = w4.kv_read(*pool, tables, lens, both, 2 * page + 10)
    for g, w in zip(got, want):
        assert torch.equal(g[:page + 5], w[:page + 5]) and torch.equal(g[page + 5:], w[:page + 5])


# ------------------------------------------------------------------- reading --

def test_read_every_code_and_scale():
    """All 256 bytes of codes under all 256 scale bytes, in both types."""
    dev = device()
    page, kv, dim = 256, 8, 64
    codes = np.zeros((1, page, kv, dim), np.uint8)
    both = np.arange(256)
    # head h, token t: the bytes 32 h .. 32 h + 31 as pairs, every scale byte t
    pairs = np.stack([both & 15, both >> 4], -1).reshape(kv, dim)
    codes[0] = pairs[None]
    scales = np.broadcast_to(both[None, :, None, None], (1, page, kv, 2)).astype(np.uint8)
    t = on_gpu(fp4_tensor(R.to_pages(codes, scales), page, kv, dim), dev)
    want = R.decode_blocks(codes, scales)[0]
    for dtype in (torch.bfloat16, torch.float16):
        k, v = w4.kv_read(t, t, ints([[0]], dev), ints([page], dev), ints([0, page], dev), page, dtype=dtype)
        assert torch.equal(k.view(torch.int16), v.view(torch.int16))
        got = as_f64(k)
        e = both[:, None, None] - 127
        # within the type's range: BF16 from 2^-126 (0.5 * 2^-125) on, FP16 scales up to 13; and NaN
        fine = np.broadcast_to((e >= -125) & (e < 126) if dtype == torch.bfloat16 else (e >= -13) & (e <= 13), got.shape)
        assert np.array_equal(got[fine], want[fine])
        assert np.isnan(got[255]).all()
        if dtype == torch.float16:       # smaller ones to the type's steps of 2^-24
            low = np.broadcast_to(e < -13, got.shape)
            assert np.abs(got[low] - want[low]).max() <= 2.0 ** -25
        else:
            low = np.broadcast_to(e < -125, got.shape)
            assert np.abs(got[low] - want[low]).max() <= 2.0 ** -126
    assert not as_f64(k)[0].any()


@pytest.mark.parametrize("kind,high", [("bf16", "bf16"), ("fp16", "fp16"), ("fp8", "bf16"), ("fp8", "fp16"), ("fp4", "bf16"),
                                       ("fp4", "fp16")])
@pytest.mark.parametrize("kv,dim,page,past,new", [(2, 128, 16, [0, 50], [33, 1]), (3, 64, 11, [4], [40]), (1, 256, 8, [0, 0, 9], [5, 0, 300]),
                                                  (8, 128, 32, [30] * 40, [1] * 40)])
@pytest.mark.parametrize("order", ["page token head", "head page token"])
def test_read_matches_the_cache(kind, high, kv, dim, page, past, new, order):
    dev = device()
    say(f"[read] {kind} cache in {high}, {kv} heads of {dim}, page {page}, new {new[:3]}")
    gen, rng = torch.Generator().manual_seed(5), np.random.default_rng(5)
    lens, cu = [a + b for a, b in zip(past, new)], np.concatenate([[0], np.cumsum(new)])
    pages, n = sum(-(-x // page) for x in lens) + 2, int(cu[-1])
    tables = table_of(lens, page, pages, max(-(-x // page) for x in lens) + 1, rng)
    tables[-1, (lens[-1] - 1) // page] = pages + 3        # the last token's page is not to be had
    (kd, kb), (vd, vb) = (cache_of(kind, pages, page, kv, dim, gen, dev, order) for _ in range(2))
    scale = [torch.rand(kv, generator=gen) + 0.5 if kind == "fp8" else None for _ in range(2)]
    more = {"k_scale": scale[0].to(dev), "v_scale": scale[1].to(dev)} if kind == "fp8" else {}
    out = [torch.full((n + 2, kv + 1, dim), 3.0, dtype=TYPES[high], device=dev) for _ in range(2)]
    got = w4.kv_read(kd, vd, ints(tables, dev), ints(lens, dev), ints(cu, dev), n + 2, dtype=TYPES[high],
                     out=tuple(x[:, 1:] for x in out), **more)
    pos = np.concatenate([np.arange(b) + a for a, b in zip(past, new)])
    s = np.repeat(np.arange(len(new)), new)
    page_at = tables[s, pos // page]
    has = page_at < pages
    for x, whole, before, f in zip(got, out, (kb, vb), scale):
        assert torch.all(x[n:] == 3) and torch.all(whole[:, 0] == 3)
        x = as_f64(x[:n])
        assert np.isnan(x[~has]).all() and not has.all()
        rows = R.decode_blocks(*R.from_pages(before[:, :R.page_bytes(page, kv, dim)], page, kv, dim)) if kind == "fp4" else before
        want = rows[page_at[has], pos[has] % page]
        if f is None:
            assert np.array_equal(x[has], want)
        else:       # one rounding of an fp32 product
            want = want * as_f64(f)[:, None]
            u = 2.0 ** -8 if high == "bf16" else 2.0 ** -11
            assert np.all(np.abs(x[has] - want) <= (u + 2.0 ** -23) * np.abs(want) + 2.0 ** -25)


def test_append_and_read_in_a_graph():
    dev = device()
    gen = torch.Generator().manual_seed(6)
    page, kv, dim, group = 16, 2, 128, 3
    rows = values((20, kv * (group + 2), dim), "bf16", gen).to(dev)
    q, k, v = rows.split([kv * group, kv, kv], dim=1)
    pool = w4.kv_cache_e2m1((2, 2, 30), page, kv, dim, device=dev)
    tables, lens, cu = ints(np.arange(30).reshape(2, 15), dev), ints([12, 8], dev), ints([0, 12, 20], dev)
    f = torch.from_numpy(freqs_of(128)).to(dev)
    out, kv_out = torch.empty(20, kv * group, dim, dtype=torch.bfloat16, device=dev), torch.empty(2, 20, kv, dim, dtype=torch.bfloat16, device=dev)

    def step(i, q_out, pair):
        w4.kv_append_rope(q, k, v, *pool[i], tables, lens, f, cu_seqlens=cu, q_out=q_out)
        w4.kv_read(*pool[i], tables, lens, cu, 20, out=tuple(pair))
    step(0, out, kv_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0, out, kv_out)
    for i in range(4):
        rows.copy_(values(rows.shape, "bf16", torch.Generator().manual_seed(10 + i)))
        lens += 20
        a, b = torch.empty_like(out), torch.empty_like(kv_out)
        step(1, a, b)
        out.zero_(), kv_out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(b, kv_out), f"replay {i}"
        (a[:, 0] @ a[:, 1].t().contiguous()).sum().item()


def test_two_streams():
    """Calls of two streams at once, each on its own rows and caches, give what they give alone."""
    dev = device()
    say("[rows] two streams")
    page, kv, dim, group, n = 16, 4, 128, 4, 2000
    gen = torch.Generator().manual_seed(11)
    f = torch.from_numpy(freqs_of(dim)).to(dev)
    tables, lens, cu = ints(np.arange(126)[None], dev), ints([n], dev), ints([0, n], dev)
    sets = []
    for _ in range(2):
        rows = values((n, kv * (group + 2), dim), "bf16", gen).to(dev)
        sets.append((rows.split([kv * group, kv, kv], dim=1), w4.kv_cache_e2m1((2, 126), page, kv, dim, device=dev)))

    def call(part):
        (q, k, v), cache = part
        q = w4.kv_append_rope(q, k, v, *cache, tables, lens, f, cu_seqlens=cu)
        return [q, *w4.kv_read(*cache, tables, lens, cu, n), w4.attn_prefill(q, cu, *cache, tables, lens),
                w4.attn_decode(q[-1:], *cache, tables, lens), w4.rope(q, cu.new_zeros(n), f)]
    alone = [[t.clone() for t in call(part)] for part in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = []
        for s, part in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(call(part))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
