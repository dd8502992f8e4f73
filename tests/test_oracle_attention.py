"""Pins of the attention oracle (oracle/attention.py): brute force with exact
rationals for the softmax's ingredients, torch's own attention and E4M3 cast,
and hand-made page states."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as A


@pytest.mark.parametrize("position,window,sinks,want", [
    (3, 0, 0, [0, 1, 2, 3]), (3, 2, 0, [2, 3]), (5, 2, 1, [0, 4, 5]), (5, 2, 9, [0, 1, 2, 3, 4, 5]), (0, 1, 0, [0]),
    (-1, 0, 4, []), (-3, 2, 4, []), (4, 100, 0, [0, 1, 2, 3, 4])])
def test_visible(position, window, sinks, want):
    assert np.flatnonzero(A.visible(position, 7, window, sinks)).tolist() == want


@pytest.mark.parametrize("length,window,sinks", [(1, 0, 0), (37, 0, 0), (37, 9, 0), (37, 9, 3), (37, 40, 5)])
def test_attend_against_torch(length, window, sinks):
    rng = np.random.default_rng(length + window)
    page, dim = 5, 16
    k, v = rng.standard_normal((12, page, 2, dim)), rng.standard_normal((12, page, 2, dim))
    table = rng.permutation(12)
    q = rng.standard_normal(dim)
    for head in range(2):
        out, lse, (a, big, size, n) = A.attend(q, k, v, table, length, length - 1, head, 0.3, window, sinks)
        at = [(table[t // page], t % page) for t in range(length)]
        kk = torch.tensor(np.stack([k[p, i, head] for p, i in at]))
        vv = torch.tensor(np.stack([v[p, i, head] for p, i in at]))
        mask = torch.tensor([not window or t > length - 1 - window or t < sinks for t in range(length)])
        want = torch.nn.functional.scaled_dot_product_attention(torch.tensor(q)[None, None], kk[None], vv[None],
                                                                mask[None, None], scale=0.3)[0, 0].numpy()
        assert np.allclose(out, want, rtol=1e-12, atol=1e-13)
        scores = [0.3 * float(kk[t] @ torch.tensor(q)) for t in range(length) if mask[t]]
        assert abs(lse - math.log(sum(math.exp(s) for s in scores))) < 1e-12
        assert n == len(scores) and np.all(np.abs(out) <= a + 1e-12) and np.all(a <= big + 1e-12) and size >= max(map(abs, scores)) - 1e-12


def test_attend_without_tokens():
    k = np.ones((1, 2, 1, 4))
    out, lse, _ = A.attend(np.ones(4), k, k, [0], 0, -1, 0, 1.0, 0, 0)
    assert np.all(out == 0) and lse == -np.inf


def test_e4m3_against_torch():
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.float16).float()
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(A.e4m3_value(x.numpy()), want, equal_nan=True)


def test_append_places_rows():
    cache = np.zeros((4, 2, 1, 1))
    new = np.arange(1.0, 7.0).reshape(6, 1, 1)
    A.append(cache, new, np.array([[3, 1], [0, -1]]), [4, 2], [0, 3, 6])
    assert cache[:, :, 0, 0].tolist() == [[5, 6], [2, 3], [0, 0], [0, 1]]


def test_pages_by_hand():
    data = np.arange(6.0)[:, None].copy()
    p = A.Pages([[4, 2, -1], [-1, -1, -1], [5, -1, -1]], [3, 0, 2], [0, 0, 1, 0, 1, 1], 2, data)
    p.fork([0], [1])                     # page 4 shared, page 2 (half full) copied to page 0
    assert p.tables[1].tolist() == [4, 0, -1] and p.lens[1] == 3 and p.refs.tolist() == [1, 0, 1, 0, 2, 1]
    assert data[:, 0].tolist() == [2, 1, 2, 3, 4, 5]
    p.lens[:] = [5, 4, 2]
    p.reserve()
    assert p.tables[0].tolist() == [4, 2, 1] and p.lacking == 0
    p.trim([0], 2, 0)                    # tokens 0 .. 3 lie before the window of the next token, 4 does not
    assert p.tables[0].tolist() == [-1, -1, 1] and p.refs.tolist() == [1, 1, 0, 0, 1, 1]
    remap = p.compact()
    assert remap.tolist() == [0, 1, -1, -1, 2, 3]
    assert p.tables.tolist() == [[-1, -1, 1], [2, 0, -1], [3, -1, -1]] and data[2:4, 0].tolist() == [4, 5]
    p.free([0, 1, 2])
    assert p.refs.tolist() == [0] * 6 and p.lens.tolist() == [0, 0, 0]
