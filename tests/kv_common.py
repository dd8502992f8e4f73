"""Shared helpers of the paged-cache and attention tests: caches and tables of
any layout, the oracle's values for a batch, and the bound on an output.

Bound of an attention output y (type with unit roundoff u: BF16 2^-8, FP16
2^-11) against the 64-bit value o, from the roundings the kernels make:

    |y - o| <= u |o| + (1 + u) (c + 2 eta + n 2^-22) A + n tiny V + 2^-25

A is the weighted mean of |V|, V its largest value, n the visible tokens.  eta
bounds the error of a score in the exponent: an fp32 dot product of D terms,
its scaling and the subtraction of the maximum ((D + 8) 2^-23 of sum_d |q_d
K_d| * scale) and the exp2 itself (2^-22).  n 2^-22 covers the fp32 sums and
their joins.  c is the rounding of the weights: u where they are rounded once
(prefill), 2^-15 (BF16) / 2^-20 (FP16) where they enter as two parts (decode).
tiny is FP16's absolute rounding of small weights, 2^-24 (0 for BF16).
"""
import numpy as np
import torch

from oracle import attention as A

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def table_of(lens, page, pages, width, rng, rows=None):
    """Block tables over shuffled pages, -1 past each sequence's end."""
    order = rng.permutation(pages)
    tables = np.full((rows or len(lens), width), -1, np.int32)
    at = 0
    for s, n in enumerate(lens):
        held = -(-n // page)
        tables[s, :held] = order[at:at + held]
        at += held
    assert at <= pages
    return tables


def ints(a, dev):
    return torch.tensor(np.asarray(a, np.int32), device=dev)


def values(shape, kind, gen):
    """Values of the type, on the CPU."""
    x = torch.randn(shape, generator=gen)
    return x.to(TYPES[kind])


def as_f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().float().numpy().astype(np.float64)


def on_device(t: torch.Tensor, order, dev) -> torch.Tensor:
    """t on the device with its first three axes in the given memory order."""
    back = [order.index(i) for i in range(3)]
    return t.permute(*order, 3).contiguous().to(dev).permute(*back, 3)


def check_attention(y, lse, q, kv, tables, lens, positions, seqs, kind, scale, window, sinks, weight_rounding, label,
                    rows=None):
    """Output rows (all, or `rows`) of y [n, q_heads, dim] against the oracle.  kv: fp64 (K, V) as
    they stand for; positions[i], seqs[i]: of row i."""
    u = UNIT[kind]
    tiny = 2.0 ** -24 if kind == "fp16" else 0.0
    k, v = kv
    group = q.shape[1] // k.shape[2]
    got, q = as_f64(y), as_f64(q)
    for i in range(len(q)) if rows is None else rows:
        s = seqs[i]
        for h in range(q.shape[1]):
            o, ref_lse, (a, big, size, n) = A.attend(q[i, h], k, v, tables[s], int(lens[s]), int(positions[i]),
                                                     h // group, scale, window, sinks)
            where = f"{label}: row {i} (sequence {s}, position {positions[i]}) head {h}"
            if n == 0:
                assert np.all(got[i, h] == 0), where
                assert lse is None or lse[i, h].item() == -np.inf, where
                continue
            eta = (q.shape[2] + 8) * 2.0 ** -23 * size + 2.0 ** -22
            c = u if weight_rounding == "once" else 2.0 ** -15 if kind == "bf16" else 2.0 ** -20
            bound = u * np.abs(o) + (1 + u) * (c + 2 * eta + n * 2.0 ** -22) * a + n * tiny * big + 2.0 ** -25
            err = np.abs(got[i, h] - o)
            assert np.all(err <= bound), f"{where}: off by {err.max():.3e}, bound {bound[err.argmax()]:.3e}"
            if lse is not None:
                # ln of an fp32 sum of n weights, plus the maximum's own error
                tol = eta + n * 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -22 * abs(ref_lse)
                assert abs(lse[i, h].item() - ref_lse) <= tol, f"{where}: lse {lse[i, h].item()} against {ref_lse}"
