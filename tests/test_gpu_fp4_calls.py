"""Calls of rotary positions and of the 4-bit cache at the ends of what they take: more sequences than
a wave has lanes with a few tokens each, pages of up to 65536, many heads, tables and rows that are slices, masks
beyond every length, rows of no sequence."""
import numpy as np
import pytest
import torch

import w4a4_block_scaled_amd as w4
from gpu_common import device, say
from kv_common import as_f64, check_attention, ints, values
from oracle import rotary as R
from rows_common import bytes_of, check_rotated, chunks_fp4, freqs_of, make_fp4
from test_gpu_attn_decode import check as check_decode
from test_gpu_attn_fp4 import way_of
from test_gpu_kv_rows import cache_of, expected

pytestmark = pytest.mark.gpu


def prefill(c, window=0, sinks=0, **more):
    dev = c["dev"]
    return w4.attn_prefill(c["q"].to(dev), ints(c["cu"], dev), c["kd"], c["vd"], ints(c["tables"], dev), ints(c["lens"], dev),
                           window=window, sinks=sinks, return_lse=True, **more)


def check(c, y, lse, page, window, sinks, rows, label):
    dim = c["q"].shape[2]
    check_attention(y, lse.cpu(), c["q"], c["f64"], c["tables"], c["lens"], c["pos"], c["seqs"], c["high"], dim ** -0.5, window,
                    sinks, "once" if way_of(c, page) == "whole" else "two", label, rows)


@pytest.mark.parametrize("dim,most", [(64, 4), (128, 4), (128, 12), (256, 3), (128, 40)])
@pytest.mark.parametrize("seqs", [65, 130, 200])
def test_a_few_tokens_of_many_sequences(seqs, dim, most):
    """Some without new tokens, one with many; masks from one token to more than there are."""
    say(f"[few4] {seqs} sequences, up to {most} new tokens, D = {dim}")
    rng = np.random.default_rng(seqs + dim)
    new = rng.integers(0, most + 1, seqs)
    new[[0, 1, seqs - 1]] = 0, most, 0
    new[seqs // 2] = 3 * most
    past = rng.integers(0, 200, seqs)
    past[3] = 1500
    c = chunks_fp4(1, 4, dim, 8, list(past), list(new), seed=seqs, dev=device())
    n, picked = len(c["q"]), int(c["cu"][seqs // 2])
    for window, sinks in ((0, 0), (1, 0), (50, 300), (2 ** 31 - 1, 2 ** 31 - 1), (30, 2 ** 31 - 1)):
        y, lse = prefill(c, window, sinks)
        check(c, y, lse, 8, window, sinks, sorted({0, 1, n - 1, picked, picked + most, picked + 3 * most - 1, n // 3}), f"window {window}, sinks {sinks}")


@pytest.mark.parametrize("dim,page", [(64, 65536), (128, 8192), (256, 8192)])
def test_large_pages(dim, page):
    say(f"[page4] pages of {page}, D = {dim}")
    kv, dev, gen = 1 if page == 65536 else 2, device(), torch.Generator().manual_seed(dim)
    c = make_fp4(kv, 4, dim, page, [page + 1, 700], seed=dim, dev=dev, spare=0)
    y, lse = w4.attn_decode(c["q"].to(dev), c["kd"], c["vd"], ints(c["tables"], dev), ints(c["lens"], dev), window=900, sinks=3, return_lse=True)
    check_decode(c, y, lse, 900, 3)
    for new in ([3, 2], [90, 60]):
        p = chunks_fp4(kv, 4, dim, page, [page - 36, 600], new, seed=dim, dev=dev, spare=0)
        y, lse = prefill(p, 900, 3)
        check(p, y, lse, page, 900, 3, [0, 1, new[0] - 1, new[0]], f"new {new}")
    # rows across the border of two pages
    before = [bytes_of(x).copy() for x in (c["kd"], c["vd"])]
    rows, f = values((90, 2 + 2 * kv, dim), "bf16", gen), freqs_of(dim)
    q, k, v = rows.to(dev).split([2, kv, kv], dim=1)
    lens, cu = [page + 44, 1], [0, 90, 90]
    out = w4.kv_append_rope(q, k, v, c["kd"], c["vd"], ints(c["tables"], dev), ints(lens, dev), torch.from_numpy(f).to(dev), cu_seqlens=ints(cu, dev))
    pos = np.arange(page - 46, page + 44)
    check_rotated(out, rows[:, :2], pos, f, "bf16")
    for got, old, x in ((c["kd"], before[0], R.rotate(as_f64(rows[:, 2:2 + kv]), pos, f)), (c["vd"], before[1], as_f64(rows[:, 2 + kv:]))):
        assert np.array_equal(bytes_of(got), expected("fp4", old, x, c["tables"], lens, cu, page, kv, dim, None, "bf16"))


@pytest.mark.parametrize("way,past,new", [("few", [900, 40], [3, 2]), ("few", [900, 40], [1, 1]), ("whole", [700, 40], [150, 60]), ("split", [3000, 40], [30, 20])])
@pytest.mark.parametrize("kv,group,dim", [(1, 48, 64), (20, 1, 128), (1, 130, 128)])
def test_heads_strides_and_rows_of_no_sequence(way, past, new, kv, group, dim):
    """One kv head of many, many of one; queries, outputs and tables that are slices of larger tensors;
    rows behind the last sequence and before the first one are left."""
    page, dev = 16, device()
    c = chunks_fp4(kv, group, dim, page, past, new, seed=kv + dim, dev=dev)
    say(f"[strides4] {way_of(c, page)}, {kv} x {group} heads of {dim}")
    n, heads = len(c["q"]), kv * group
    want, lse = prefill(c)
    check(c, want, lse, page, 0, 0, [0, n - 1], "as it is")
    big = torch.zeros(n + 5, heads + 2, dim, dtype=torch.bfloat16, device=dev)
    big[2:2 + n, 1:1 + heads] = c["q"].to(dev)
    tables = torch.full((2, c["tables"].shape[1] + 3), 7, dtype=torch.int32, device=dev)
    tables[:, 3:] = ints(c["tables"], dev)
    out = torch.full((heads + 1, n + 5, dim), 5.0, dtype=torch.bfloat16, device=dev)
    got, lse = w4.attn_prefill(big[:, 1:1 + heads], ints(c["cu"] + 2, dev), c["kd"], c["vd"], tables[:, 3:], ints(c["lens"], dev),
                               out=out[1:].transpose(0, 1), return_lse=True)
    # which way a call goes follows from its number of rows
    if way_of({**c, "q": big[:, 1:1 + heads]}, page) == way_of(c, page):
        check(c, got[2:2 + n], lse[2:2 + n], page, 0, 0, [0, n - 1], "slices")
    assert torch.all(out[0] == 5) and torch.all(got[:2] == 5) and torch.all(got[2 + n:] == 5)


@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 65536, 8, 8), (2, 40000, 16, 6), (70001, 1, 8, 4), (3, 300, 512, 512)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_of_many_heads_and_tokens(tokens, heads, dim, rot, interleaved):
    say(f"[rope] {tokens} x {heads} heads of {dim}, {rot} turned")
    dev, x = device(), values((tokens, heads, dim), "fp16", torch.Generator().manual_seed(tokens))
    pos = np.arange(tokens) * 7
    y = w4.rope(x.to(dev), ints(pos, dev), torch.from_numpy(freqs_of(rot)).to(dev), interleaved=interleaved)
    check_rotated(y, x, pos, freqs_of(rot), "fp16", interleaved)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("kv,q_heads,n", [(300, 1, 3), (1, 700, 2), (37, 0, 90)])
def test_append_of_many_heads(kind, kv, q_heads, n):
    say(f"[append_rope] {kv} kv heads, {q_heads} query heads, {n} tokens, {kind}")
    dev, gen, page, dim = device(), torch.Generator().manual_seed(kv), 8, 64
    f, lens, cu = freqs_of(dim), [5, n + 4], [0, 0, n]
    tables = np.concatenate([[[1, -1], [3, 0]], np.arange(4, 24).reshape(2, 10)], 1).astype(np.int32)
    (kd, kb), (vd, vb) = (cache_of(kind, 24, page, kv, dim, gen, dev) for _ in range(2))
    q, k, v = (values((n, h, dim), "bf16", gen) for h in (q_heads, kv, kv))
    out = w4.kv_append_rope(q.to(dev), k.to(dev), v.to(dev), kd, vd, ints(tables, dev), ints(lens, dev), torch.from_numpy(f).to(dev),
                            cu_seqlens=ints(cu, dev))
    pos, one = np.arange(4, 4 + n), np.ones(kv)
    if q_heads:
        check_rotated(out, q, pos, f, "bf16")
    assert out.shape == q.shape
    turned = R.rotate(as_f64(k), pos, f)
    for got, old, x in ((kd, kb, turned), (vd, vb, as_f64(v))):
        want = expected(kind, old, x, tables, lens, cu, page, kv, dim, one, "bf16")
        if kind == "fp4":
            assert np.array_equal(bytes_of(got), want)
        elif kind == "fp8" or x is not turned:
            assert np.array_equal(as_f64(got), want)
        else:
            assert np.all(np.abs(as_f64(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17)
