"""The oracle of rotary positions and of the 4-bit cache's pages, pinned by
exact rotations, by the plain formula in Python, and by torch and the weight
path's quantizer."""
import math

import numpy as np
import pytest
import torch

import oracle.quant as Q
from oracle import rotary as R
import w4a4_block_scaled_amd as w4


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_against_the_formula(interleaved):
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((4, 2, 12)), [0, 1, 77, -5]
    freqs = np.float32([1.0, 0.3, 0.01, 1e-4])
    y = R.rotate(x, pos, freqs, interleaved, factor=1.25)
    for t, p in enumerate(pos):
        for i, f in enumerate(freqs):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 4)
            z = complex(*x[t, 0, [a, b]]) * 1.25 * complex(math.cos(p * float(f)), math.sin(p * float(f)))
            assert abs(y[t, 0, a] - z.real) < 1e-14 and abs(y[t, 0, b] - z.imag) < 1e-14
    assert np.array_equal(y[..., 8:], x[..., 8:])


def test_rotations_add_and_come_back():
    rng = np.random.default_rng(1)
    x, freqs = rng.standard_normal((3, 2, 8)), np.float32([1.0, 0.5, 0.25, 0.125])
    once = R.rotate(R.rotate(x, [5] * 3, freqs), [7] * 3, freqs)
    assert np.abs(once - R.rotate(x, [12] * 3, freqs)).max() < 1e-14
    assert np.abs(R.rotate(R.rotate(x, [9, 1, 4], freqs), [9, 1, 4], freqs, inverse=True) - x).max() < 1e-14


def test_quarter_turns_are_exact_to_fp64():
    # 2^23 * float32(pi) / 2^22 radians: an angle whose sine is known from the float's own error
    f = np.float32(math.pi)
    y = R.rotate(np.array([[[1.0, 0.0]]]), [2 ** 20], [f])
    off = 2 ** 20 * (float(f) - math.pi)
    assert abs(y[0, 0, 0] - math.cos(off)) < 1e-9 and abs(y[0, 0, 1] - math.sin(off)) < 1e-9


def test_blocks_are_the_quantizers():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((64, 128)) * np.exp2(rng.integers(-20, 20, (64, 1)))).astype(np.float32)
    x[0] = 0
    codes, scales = R.encode_blocks(x)
    want, ws, _ = Q.quantize_rows(x, "mxfp4")
    assert np.array_equal(codes, want) and np.array_equal(scales, ws)
    assert np.array_equal(R.decode_blocks(codes, scales), Q.dequantize(Q.pack_nibbles(codes), scales, "mxfp4"))


def test_blocks_that_are_not_finite_and_the_largest_exponent():
    x = np.ones((3, 64))
    x[0, 5], x[1, 40] = np.nan, -np.inf
    x[2, :32] = 65504 * 1.4
    codes, scales = R.encode_blocks(x, most=13)
    assert scales.tolist() == [[255, 125], [125, 255], [140, 125]]
    assert not codes[0, :32].any() and (codes[2, :32] == 7).all()          # 6 * 2^13
    v = R.decode_blocks(codes, scales)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 1).all() and (v[2, :32] == 49152).all()


def test_pages_round_trip_and_append():
    rng = np.random.default_rng(3)
    page, heads, dim = 5, 3, 64
    codes, scales = rng.integers(0, 16, (4, page, heads, dim)).astype(np.uint8), rng.integers(0, 255, (4, page, heads, 2)).astype(np.uint8)
    raw = R.to_pages(codes, scales)
    assert raw.shape[1] == R.page_bytes(page, heads, dim) == w4.lib().w4a4_kv_page_bytes(page, heads, dim)
    c, s = R.from_pages(raw, page, heads, dim)
    assert np.array_equal(c, codes) and np.array_equal(s, scales)
    # token 6 of the second sequence: page 2, row 1
    new = rng.standard_normal((2, heads, dim))
    R.append(raw, new, np.array([[0, -1], [3, 2]]), [9, 7], [0, 1, 2], page, heads, dim)        # the first one has no page
    codes[2, 1], scales[2, 1] = R.encode_blocks(new[1])
    c, s = R.from_pages(raw, page, heads, dim)
    assert np.array_equal(c, codes) and np.array_equal(s, scales)


def test_kv_cache_e2m1_has_aligned_pages():
    for shape in ((7, 11, 3, 64), (1, 1, 1, 64), (2, 16, 8, 128), (3, 3, 1, 256)):
        t = w4.kv_cache_e2m1((2, shape[0]), *shape[1:], device="cpu")
        assert t.shape == (2, *shape[:3], shape[3] // 32 * 17) and t.stride(1) % 16 == 0
        assert 0 <= t.stride(1) - R.page_bytes(*shape[1:]) < 16
    with pytest.raises(w4.W4A4Error):
        w4.kv_cache_e2m1(4, 16, 2, 96, device="cpu")


# ------------------------------------------------------------- frequencies --

def test_frequencies():
    f, factor = w4.rope_freqs(8, 10000.0, device="cpu")
    assert factor == 1.0 and torch.equal(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64).float())
    g, factor = w4.rope_freqs(8, 10000.0, scaling="linear", scale=4.0, device="cpu")
    assert factor == 1.0 and torch.allclose(g * 4, f, rtol=1e-7, atol=0)
    # ntk: the fastest pair as it was, the slowest slower by the scale
    g, _ = w4.rope_freqs(8, 10000.0, scaling="ntk", scale=4.0, device="cpu")
    assert g[0] == 1 and abs(float(f[-1] / g[-1]) - 4) < 1e-5


def test_frequencies_by_bands():
    n, scale, low, high, rot = 8192, 8.0, 1.0, 4.0, 128
    f, _ = w4.rope_freqs(rot, 500000.0, device="cpu")
    g, factor = w4.rope_freqs(rot, 500000.0, scaling="bands", scale=scale, original=n, low=low, high=high, device="cpu")
    assert factor == 1.0
    kinds = set()
    for i in range(rot // 2):
        exact = 500000.0 ** (-2 * i / rot)
        turns = n * exact / (2 * math.pi)
        if turns > high:
            want, kind = exact, "kept"
        elif turns < low:
            want, kind = exact / scale, "divided"
        else:
            s = (turns - low) / (high - low)
            want, kind = (1 - s) * exact / scale + s * exact, "blended"
        kinds.add(kind)
        assert abs(float(g[i]) / want - 1) < 2 ** -23, (i, kind)
    assert kinds == {"kept", "divided", "blended"}


def test_frequencies_by_ramp():
    n, scale, rot, base = 4096, 16.0, 64, 10000.0
    g, factor = w4.rope_freqs(rot, base, scaling="yarn", scale=scale, original=n, device="cpu")
    assert abs(factor - (0.1 * math.log(16) + 1)) < 1e-12
    edge = [rot * math.log(n / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32.0, 1.0)]
    first, last = math.floor(edge[0]), math.ceil(edge[1])
    for i in range(rot // 2):
        exact = base ** (-2 * i / rot)
        r = min(max((i - first) / (last - first), 0.0), 1.0)
        assert abs(float(g[i]) / (exact * (1 - r) + exact / scale * r) - 1) < 2 ** -23, i


@pytest.mark.parametrize("more", [dict(scaling="other"), dict(scaling="bands"), dict(scaling="yarn"), dict(scale=0.0),
                                  dict(scaling="bands", original=100, low=4.0, high=4.0), dict(base=-1.0)])
def test_frequencies_refused(more):
    with pytest.raises(w4.W4A4Error):
        w4.rope_freqs(64, **{"base": 10000.0, "device": "cpu", **more})
    for rot in (0, 7, -2):
        with pytest.raises(w4.W4A4Error):
            w4.rope_freqs(rot, device="cpu")
