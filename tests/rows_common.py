"""Shared helpers of the rotary and 4-bit cache tests.

Bound of a rotated 16-bit value y against the 64-bit one o, from the pair (a, b) and
the unit roundoff u of the type: cos and sin are fp64 rounded to fp32 (2^-24 of each
product), each product is rounded once and so is their sum, whose size is at most
that of the products: 3 * 2^-24 (|a| + |b|) factor; the angle's own error, 2^-48 and
less for positions below 2^24, is covered by a fourth; then one rounding to the type,
half a step: u |o|, and where the type is subnormal 2^-134 (BF16) or 2^-25 (FP16).
"""
import numpy as np
import torch

from kv_common import UNIT, as_f64, ints, table_of, values
from oracle import rotary as R
import w4a4_block_scaled_amd as w4

SMALL = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}
MOST = {"bf16": 127, "fp16": 13}          # largest exponent of a 4-bit block


def check_rotated(y, x, positions, freqs, kind, interleaved=False, inverse=False, factor=1.0, label=""):
    """y [tokens, heads, dim] (tensor) against the oracle's rotation of x (tensor)."""
    x, got, rot = as_f64(x), as_f64(y), 2 * len(freqs)
    want = R.rotate(x, positions, freqs, interleaved, inverse, factor)
    size = np.zeros_like(x)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * factor
    u = UNIT[kind]
    bound = u * np.abs(want) + (1 + u) * 4 * 2.0 ** -24 * size + SMALL[kind]
    err = np.abs(got - want)
    bad = err > bound
    assert not bad.any(), f"{label}: {bad.sum()} values off, {err[bad].max():.3e} against {bound[bad][err[bad].argmax()]:.3e}"
    assert np.array_equal(got[..., rot:], x[..., rot:]), label


def freqs_of(rot, base=10000.0):
    return (base ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)


def fp4_cache(pages, page, heads, dim, gen, gap=0):
    """A 4-bit cache on the CPU: (uint8 tensor as the binding takes it, codes, scales) of normal values."""
    codes, scales = R.encode_blocks(torch.randn(pages, page, heads, dim, generator=gen).numpy())
    raw = R.to_pages(codes, scales)
    return fp4_tensor(raw, page, heads, dim, gap), codes, scales


def fp4_tensor(raw, page, heads, dim, gap=0):
    """The tensor of pages' bytes, `gap` more units of 16 bytes between pages."""
    n, size = raw.shape
    stride = -(-size // 16) * 16 + 16 * gap
    store = torch.full((n, stride), 0x5a, dtype=torch.uint8)
    store[:, :size] = torch.from_numpy(raw)
    width = dim // 32 * 17
    return store.as_strided((n, page, heads, width), (stride, heads * width, width, 1))


def on_gpu(t, dev):
    """A 4-bit cache's tensor on the device, with its gaps."""
    n, stride = t.shape[0], t.stride(0)
    store = t.as_strided((n, stride), (stride, 1)).to(dev)
    return store.as_strided(t.shape, t.stride())


def bytes_of(t):
    """Bytes of the pages of a 4-bit cache, with the gaps, as an array [pages, stride]."""
    n, stride = t.shape[0], t.stride(0)
    return t.as_strided((n, stride), (stride, 1)).cpu().numpy()


def make_fp4(kv, group, dim, page, lens, seed, high="bf16", dev=None, spare=2, gap=0):
    """A decoding case over a 4-bit cache, as test_gpu_attn_decode's make()."""
    rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    width = max(1, -(-max(lens) // page)) + 1
    pages = sum(-(-n // page) for n in lens) + spare
    tables = table_of(lens, page, pages, width, rng)
    q = values((len(lens), kv * group, dim), high, gen)
    parts = [fp4_cache(pages, page, kv, dim, gen, gap) for _ in range(2)]
    f64 = [R.decode_blocks(c, s) for _, c, s in parts]
    kd, vd = (on_gpu(t, dev) for t, _, _ in parts)
    return {"q": q, "kd": kd, "vd": vd, "f64": f64, "tables": tables, "lens": lens, "high": high, "scales": [None, None],
            "dev": dev}


def chunks_fp4(kv, group, dim, page, past, new, seed, **more):
    """`new` tokens of each sequence after `past` earlier ones, as test_gpu_attn_prefill's chunks()."""
    c = make_fp4(kv, group, dim, page, [a + b for a, b in zip(past, new)], seed, **more)
    c["cu"] = np.concatenate([[0], np.cumsum(new)])
    c["q"] = values((int(c["cu"][-1]), kv * group, dim), c["high"], torch.Generator().manual_seed(seed + 1))
    c["seqs"] = np.repeat(np.arange(len(new)), new)
    c["pos"] = np.concatenate([np.arange(b) + a for a, b in zip(past, new)])
    return c
