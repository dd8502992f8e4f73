"""Rotary positions and the pages of the 4-bit cache, in fp64 on the CPU, from
the definitions (nothing shared with the GPU path)."""
from __future__ import annotations

import numpy as np

from . import formats as F


def rotate(x, positions, freqs, interleaved=False, inverse=False, factor=1.0):
    """Rows x [tokens, heads, dim] (any float type) rotated by position * freqs
    (float32 [rot / 2]) over their first `rot` values."""
    y = np.array(x, np.float64)
    rot = 2 * len(freqs)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(freqs, np.float32).astype(np.float64)
    # long double where it is wider: far positions' angles to all their bits
    c, s = (f(angle.astype(np.longdouble)).astype(np.float64)[:, None] * float(np.float32(factor)) for f in (np.cos, np.sin))
    s = -s if inverse else s
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    p, q = y[..., a].copy(), y[..., b].copy()
    y[..., a] = p * c - q * s
    y[..., b] = p * s + q * c
    return y


def encode_blocks(x, most=127):
    """(codes [..., dim], scale bytes [..., dim / 32]) of MXFP4 rows; `most`: the largest exponent."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    top = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1))
    e = np.where(top > 0, np.clip(np.frexp(top)[1] - 3, -127, most), -127)
    codes = F.e2m1_encode(np.where(bad[..., None], 0.0, b), np.ldexp(1.0, e)[..., None])
    codes = np.where(bad[..., None], 0, codes)
    return codes.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def decode_blocks(codes, scales):
    """Values of codes [..., dim] with scale bytes [..., dim / 32]; NaN where a byte is 255."""
    e = scales.astype(np.int64)
    unit = np.where(e == 255, np.nan, np.ldexp(1.0, e - 127))
    v = F.e2m1_value(codes).reshape(*codes.shape[:-1], -1, 32) * unit[..., None]
    return v.reshape(codes.shape)


def page_bytes(page, heads, dim):
    return page * heads * (dim // 2 + dim // 32)


def to_pages(codes, scales):
    """Bytes [pages, page * heads * dim * 17 / 32] of codes [pages, page, heads, dim] and scales
    [pages, page, heads, dim / 32]."""
    n = codes.shape[0]
    by_head = codes.transpose(0, 2, 1, 3)
    packed = by_head[..., ::2] | by_head[..., 1::2] << 4
    return np.concatenate([packed.reshape(n, -1), scales.transpose(0, 2, 3, 1).reshape(n, -1)], 1).astype(np.uint8)


def from_pages(raw, page, heads, dim):
    """(codes, scales) of to_pages's bytes."""
    n, size = raw.shape[0], page * heads * dim // 2
    packed = raw[:, :size].reshape(n, heads, page, dim // 2)
    codes = np.stack([packed & 15, packed >> 4], -1).reshape(n, heads, page, dim)
    scales = raw[:, size:].reshape(n, heads, dim // 32, page)
    return codes.transpose(0, 2, 1, 3), scales.transpose(0, 3, 1, 2)


def append(raw, new, tables, lens, cu, page, heads, dim, most=127):
    """Store the rows cu[s] .. cu[s + 1] - 1 of `new` [tokens, heads, dim] (fp64) at the end of sequence s, in place."""
    size = page * heads * dim // 2
    codes, scales = encode_blocks(new, most)
    for s in range(len(lens)):
        for i in range(cu[s], cu[s + 1]):
            p = int(lens[s]) - int(cu[s + 1]) + i
            if p < 0 or p // page >= tables.shape[1] or not 0 <= tables[s, p // page] < len(raw):
                continue
            to = raw[tables[s, p // page]]
            r = p % page
            to[:size].reshape(heads, page, dim // 2)[:, r] = codes[i][:, ::2] | codes[i][:, 1::2] << 4
            to[size:size + heads * page * (dim // 32)].reshape(heads, dim // 32, page)[:, :, r] = scales[i]
