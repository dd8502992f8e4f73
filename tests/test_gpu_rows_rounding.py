"""Codes of rotated keys where fp32 cannot tell them: results beside a tie by less than its steps
(angles next to quarter turns), pairs of zeros, values beside the ends of a block's exponent."""
import numpy as np
import pytest
import torch

import w4a4_block_scaled_amd as w4
from gpu_common import device, say
from kv_common import TYPES, as_f64, ints
from oracle import attention as A
from oracle import rotary as R
from rows_common import MOST, bytes_of
from test_gpu_kv_rows import expected

pytestmark = pytest.mark.gpu

# halfway between two codes, upward and downward ties, of E4M3 and E2M1
TIES = {"fp8": [1.0625, 1.1875, 1.3125, 1.4375, 1.5625, 1.6875, 1.8125, 1.9375], "fp4": [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]}


def store(kind, rows, pos, freqs, high, interleaved, factor=1.0, scale=None):
    """(the cache after storing those keys, what it should hold), one row per token; of the values too."""
    dev, (n, heads, dim), page = device(), rows.shape, 16
    pages = -(-n // page)
    tables = np.arange(pages, dtype=np.int32)[None]
    cache = (w4.kv_cache_e2m1((2, pages), page, heads, dim, device=dev) if kind == "fp4" else
             torch.zeros(2, pages, page, heads, dim, dtype=torch.uint8, device=dev).view(TYPES[kind]))
    before = bytes_of(cache[0]).copy() if kind == "fp4" else as_f64(cache[0])
    more = {} if scale is None else {"k_scale": scale.to(dev), "v_scale": scale.to(dev)}
    w4.kv_append_rope(None, rows.to(dev), rows.to(dev), *cache, ints(tables, dev), ints([n], dev), torch.from_numpy(freqs).to(dev),
                      cu_seqlens=ints([0, n], dev), positions=ints(pos, dev), interleaved=interleaved, factor=factor, **more)
    new = R.rotate(as_f64(rows), pos, freqs, interleaved, False, float(np.float32(factor)))
    s64 = np.ones(heads) if scale is None else as_f64(scale)
    for got, x in zip(cache, (new, as_f64(rows))):
        want = expected(kind, before, x, tables, [n], [0, n], page, heads, dim, s64, high)
        have = bytes_of(got) if kind == "fp4" else as_f64(got)
        bad = have != want
        assert not bad.any(), f"{bad.sum()} of {bad.size} differ"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("high", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("rot", [64, 24])
def test_beside_a_tie(kind, high, interleaved, rot):
    """Ties turned by nearly a whole number of quarter turns: cos or sin is 1 - 2^-40 or so, which fp32 rounds to 1,
    and the other one 2^-20 or so times a partner of any size."""
    say(f"[append_rope] beside ties, {kind}, {high}, rot {rot}, interleaved {interleaved}")
    rng, n, dim, pairs = np.random.default_rng(rot), 600, 64, rot // 2
    pos = rng.integers(1, 1 << 17, n)
    # every frequency is met by some positions in a nearly whole number of quarter turns
    base = rng.integers(1, 1 << 17, pairs)
    freqs = (np.pi / 2 * rng.integers(1, 4096, pairs) / base).astype(np.float32)
    pos[:pairs * 8] = np.repeat(base, 8)
    x = rng.choice(TIES[kind], (n, 3, dim)) * rng.choice([-1.0, 1.0], (n, 3, dim))
    x[rng.random(x.shape) < 0.4] = 0.0
    x[:, 2] *= 2.0 ** rng.integers(-3, 4, (n, 1))
    if kind == "fp4":
        x[..., ::32] = 6.0                               # so that a block's exponent is 0
    store(kind, torch.from_numpy(x).to(TYPES[high]), pos, freqs, high, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("high", ["bf16", "fp16"])
def test_ends_of_a_blocks_exponent(high, interleaved):
    """Largest values turned to within 2^-40 of a power of two, below and above."""
    say(f"[append_rope] exponents, {high}, interleaved {interleaved}")
    rng, n, dim = np.random.default_rng(5), 512, 64
    base = rng.integers(1, 1 << 17, 32)
    freqs = (np.pi / 2 * rng.integers(1, 4096, 32) / base).astype(np.float32)
    pos = base[rng.integers(0, 32, n)]
    x = np.where(rng.random((n, 2, dim)) < 0.7, 0.0, rng.choice([-4.0, 4.0, -8.0, 8.0], (n, 2, dim)))
    x[:, 1] *= rng.choice([1.0, 2.0 ** -13, 2.0 ** 9], (n, 1))
    store("fp4", torch.from_numpy(x).to(TYPES[high]), pos, freqs, high, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("high", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("factor", [1.0, 1.37])
def test_zeros_and_scales(kind, high, interleaved, factor):
    """Rows, heads, pairs and single values of zero, of both signs, padding at the end; scales that are powers of
    two (where quotients of 16-bit values are often ties), none, and others."""
    say(f"[append_rope] zeros, {kind}, {high}, interleaved {interleaved}, factor {factor}")
    rng, n, heads, dim = np.random.default_rng(7), 300, 4, 64
    pos, freqs = rng.integers(0, 131072, n), (10000.0 ** (-np.arange(0, 32, 2) / 32)).astype(np.float32)
    x = torch.from_numpy(rng.standard_normal((n, heads, dim))).to(TYPES[high])
    x[rng.random(x.shape) < 0.2] = 0.0
    x[rng.random(x.shape) < 0.05] = -0.0
    x[:, 1, :16] = 0.0
    x[40:60] = 0.0
    x[60:80, 2] = -0.0
    x[200:] = 0.0
    for scale in ([None, [1.0, 0.5, 2.0 ** -7, 4.0], [0.8371, 1.0, 3.0, 0.1]] if kind == "fp8" else [None]):
        store(kind, x, pos, freqs, high, interleaved, factor, None if scale is None else torch.tensor(scale))
