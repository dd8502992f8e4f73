"""Attention over a cache held in 4 bits at the ends of its range: scales whose values
leave BF16's, in places that some rows do not see; queries near the smallest normal number; values
that FP16 holds as subnormals."""
import numpy as np
import pytest
import torch

import w4a4_block_scaled_amd as w4
from gpu_common import device, say
from kv_common import UNIT, as_f64, check_attention, ints
from oracle import attention as A
from oracle import rotary as R
from rows_common import chunks_fp4
from test_gpu_attn_edges import attend
from test_gpu_attn_fp4 import WAYS

pytestmark = pytest.mark.gpu
PREFILL = [w for w in WAYS if not w.startswith("decode")]


def parts_of(x, page, heads, dim):
    """(codes [pages, heads, page, dim / 2], scale bytes [pages, heads, dim / 32, page]) of a 4-bit cache's tensor."""
    raw, size = x.as_strided((x.shape[0], x.stride(0)), (x.stride(0), 1)), page * heads * dim // 2
    scales = raw[:, size:size + heads * (dim // 32) * page].unflatten(1, (heads, dim // 32, page))
    return raw[:, :size].unflatten(1, (heads, page, dim // 2)), scales


@pytest.mark.parametrize("way", PREFILL)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("high", ["bf16", "fp16"])
@pytest.mark.parametrize("byte,code", [(254, 0x77), (254, 0xff), (253, 0x66), (253, 0x11)])
def test_values_past_the_range_stay_with_the_rows_that_see_them(way, dim, high, byte, code):
    """A token's values of 6 * 2^127 and the like: the rows that do not see it, since their windows begin
    later or they come before it, keep every bit."""
    if way == "few, three blocks" and dim == 256:
        pytest.skip("these go as row tiles")
    say(f"[range4] {way}, D = {dim}, {high}, scale byte {byte}, codes {code:#x}")
    past, new, page = WAYS[way]
    window, sinks = 200, 3
    c = chunks_fp4(2, 4, dim, page, past, new, seed=dim, high=high, dev=device())
    clean, lse = attend(c, way, window, sinks)
    codes, scales = parts_of(c["vd"], page, 2, dim)
    kept = codes.clone(), scales.clone()
    # seen by the first row alone, and by the last one alone
    for token, others in ((past[0] - window + 1, slice(1, None)), (c["lens"][0] - 1, slice(0, new[0] - 1))):
        at = int(c["tables"][0, token // page])
        codes[at, :, token % page], scales[at, :, :, token % page] = code, byte
        y, l2 = attend(c, way, window, sinks)
        assert torch.equal(y[others], clean[others]) and torch.equal(l2, lse)
        assert torch.equal(y[new[0]:], clean[new[0]:])
        codes.copy_(kept[0])
        scales.copy_(kept[1])


@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("shift", [0, 100, 110, 118])
def test_small_queries(way, dim, shift):
    """Queries of 2^-shift, one value of each block of 32 2^11 times the others and its keys zero. The others
    are promised to within 2^-19 of their block's largest value or 2^-126 if that is more, and the scale of
    the softmax makes up for the shift, so they count as they do without it."""
    if way == "few, three blocks" and dim == 256:
        pytest.skip("these go as row tiles")
    say(f"[small4] {way}, D = {dim}, queries of 2^-{shift}")
    past, new, page = WAYS[way]
    c = chunks_fp4(2, 4, dim, page, past, new, seed=dim + shift, dev=device())
    q = c["q"].clone()
    q[..., 7::32] = torch.sign(q[..., 7::32]) * 3000
    c["q"] = (q.float() * 2.0 ** -shift).to(torch.bfloat16)
    codes, _ = parts_of(c["kd"], page, 2, dim)
    codes[..., 3::16] &= 15                                # the upper half of a byte each
    k64 = c["f64"][0].copy()
    k64[..., 7::32] = 0
    scale, dev = dim ** -0.5 * 2.0 ** shift, c["dev"]
    cache = c["kd"], c["vd"], ints(c["tables"], dev), ints(c["lens"], dev)
    if way.startswith("decode"):
        y, lse = w4.attn_decode(c["q"].to(dev), *cache, scale=scale, return_lse=True)
    else:
        y, lse = w4.attn_prefill(c["q"].to(dev), ints(c["cu"], dev), *cache, scale=scale, return_lse=True)
    got, lse, q64, u = as_f64(y), lse.cpu().numpy().astype(np.float64), as_f64(c["q"]), UNIT["bf16"]
    weights = u if way.startswith("whole") else 2.0 ** -15
    for i in sorted({0, 1, len(q) - 1, int(c["cu"][1]) - 1}):
        s = int(c["seqs"][i])
        for h in (0, 5, 7):
            o, ref, (a, big, size, n) = A.attend(q64[i, h], k64, c["f64"][1], c["tables"][s], c["lens"][s], int(c["pos"][i]),
                                                 h // 4, scale, 0, 0)
            keys = np.abs(A.rows(k64, c["tables"][s], range(n), h // 4)).reshape(n, -1, 32).sum(-1)
            off = np.maximum(np.abs(q64[i, h]).reshape(-1, 32).max(-1) * 2.0 ** -19, 2.0 ** -126)
            parts = (keys * off).sum(-1).max() * scale
            eta = (dim + 8) * 2.0 ** -23 * (size + parts) + 2.0 ** -22 + parts
            bound = u * np.abs(o) + (1 + u) * (weights + 2 * eta + n * 2.0 ** -22) * a + 2.0 ** -25
            err = np.abs(got[i, h] - o)
            assert np.all(err <= bound), f"row {i} head {h}: off by {err.max():.3e}, bound {bound[err.argmax()]:.3e}"
            assert abs(lse[i, h] - ref) <= eta + n * 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -22 * abs(ref)


@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("exponent", [-14, -18, -22, -24])
def test_small_values_with_fp16_queries(way, dim, exponent):
    """Values in steps of 2^(exponent - 1). Where they are widened to FP16 (row tiles) each is rounded to a
    multiple of 2^-24, by 2^-25 at most, and so is a weighted mean of them."""
    if way == "few, three blocks" and dim == 256:
        pytest.skip("these go as row tiles")
    say(f"[subnormal4] {way}, D = {dim}, values of 2^{exponent}")
    past, new, page = WAYS[way]
    c = chunks_fp4(2, 4, dim, page, past, new, seed=dim - exponent, high="fp16", dev=device())
    codes, scales = parts_of(c["vd"], page, 2, dim)
    scales.fill_(exponent + 127)
    size = page * 2 * dim // 2
    raw = c["vd"].as_strided((c["vd"].shape[0], c["vd"].stride(0)), (c["vd"].stride(0), 1))[:, :size + 2 * (dim // 32) * page]
    v64 = R.decode_blocks(*R.from_pages(raw.cpu().numpy(), page, 2, dim))
    y, _ = attend(c, way)
    got, q64, u, scale = as_f64(y), as_f64(c["q"]), UNIT["fp16"], dim ** -0.5
    tiles = way.startswith("whole") or way == "split"
    weights = u if way.startswith("whole") else 2.0 ** -20 if way == "split" else 2.0 ** -15
    for i in sorted({0, 1, len(q64) - 1, int(c["cu"][1]) - 1}):
        s = int(c["seqs"][i])
        for h in (0, 5, 7):
            o, _, (a, big, dots, n) = A.attend(q64[i, h], c["f64"][0], v64, c["tables"][s], c["lens"][s], int(c["pos"][i]),
                                               h // 4, scale, 0, 0)
            eta = (dim + 8) * 2.0 ** -23 * dots + 2.0 ** -22
            bound = u * np.abs(o) + (1 + u) * ((weights + 2 * eta + n * 2.0 ** -22) * a + n * 2.0 ** -24 * big) + 2.0 ** -25
            bound = bound + (2.0 ** -25 * (1 + u) * (1 + weights + 2 * eta) if tiles else 0)
            err = np.abs(got[i, h] - o)
            assert np.all(err <= bound), f"row {i} head {h}: off by {err.max():.3e}, bound {bound[err.argmax()]:.3e}"


@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("high", ["bf16", "fp16"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_inf_and_nan_among_queries(way, dim, high, value):
    """A head of a row of queries with Inf or NaN anywhere becomes NaN, and no other row or head changes."""
    if way == "few, three blocks" and dim == 256:
        pytest.skip("these go as row tiles")
    say(f"[odd queries4] {way}, D = {dim}, {high}, {value}")
    past, new, page = WAYS[way]
    c = chunks_fp4(2, 4, dim, page, past, new, seed=dim, high=high, dev=device())
    clean, lse = attend(c, way)
    odd = torch.zeros(clean.shape[:2], dtype=torch.bool)
    c["q"] = c["q"].clone()
    for row, head, d in ((0, 0, 5), (len(odd) - 1, 7, dim - 1), (len(odd) // 2, 3, dim // 2)):
        c["q"][row, head, d] = value
        odd[row, head] = True
    y, l2 = attend(c, way)
    odd = odd.to(y.device)
    assert torch.isnan(y[odd]).all() and torch.isnan(l2[odd]).all()
    assert torch.equal(y[~odd], clean[~odd]) and torch.equal(l2[~odd], lse[~odd])


@pytest.mark.parametrize("way", PREFILL)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("high", ["bf16", "fp16"])
@pytest.mark.parametrize("byte", [254, 255])
def test_keys_past_the_range_stay_with_the_rows_that_see_them(way, dim, high, byte):
    """A token's keys of 6 * 2^127 (a score past any other) or NaN: the rows that do not see it are as without
    it. With NaN bit for bit; a score that one row sees moves the references of the softmax of all rows
    in its wave, and with them which way their weights round, so there the other rows are compared with the
    64-bit values by the bound on every output, which holds for any reference."""
    if way == "few, three blocks" and dim == 256:
        pytest.skip("these go as row tiles")
    say(f"[range4] {way}, D = {dim}, {high}, keys with scale byte {byte}")
    past, new, page = WAYS[way]
    window, sinks = 200, 3
    c = chunks_fp4(2, 4, dim, page, past, new, seed=dim, high=high, dev=device())
    clean, lse = attend(c, way, window, sinks)
    codes, scales = parts_of(c["kd"], page, 2, dim)
    kept = codes.clone(), scales.clone()
    # few rows: weights in two parts of BF16, 2^-15 of them, which FP16's "once" (2^-11) covers
    weights = "two" if way == "split" or (high == "bf16" and way.startswith("few")) else "once"
    for token, others in ((past[0] - window + 1, slice(1, None)), (c["lens"][0] - 1, slice(0, new[0] - 1))):
        at = int(c["tables"][0, token // page])
        codes[at, :, token % page], scales[at, :, :, token % page] = 0x77, byte
        y, l2 = attend(c, way, window, sinks)
        assert torch.equal(y[new[0]:], clean[new[0]:])
        if byte == 254:
            near = [r for r in (0, 1, new[0] // 2, new[0] - 2, new[0] - 1) if r in range(*others.indices(new[0]))]
            check_attention(y, l2.cpu(), c["q"], c["f64"], c["tables"], c["lens"], c["pos"], c["seqs"], high, dim ** -0.5, window,
                            sinks, weights, "other rows", near)
        else:
            assert torch.equal(y[others], clean[others]) and torch.equal(l2[others], lse[others])
            own = 0 if others.start == 1 else new[0] - 1
            assert torch.isnan(y[own]).all() and torch.isnan(l2[own]).all()
        codes.copy_(kept[0])
        scales.copy_(kept[1])
