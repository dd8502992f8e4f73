"""Rotary positions (w4a4_rope) against the fp64 oracle: pairings, parts of the
head, widths, strides, positions of any size, in place, gradients, graphs."""
import numpy as np
import pytest
import torch

import w4a4_block_scaled_amd as w4
from gpu_common import device, say
from kv_common import as_f64, values
from oracle import rotary as R
from rows_common import check_rotated, freqs_of

pytestmark = pytest.mark.gpu
TYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}


def rotate(x, pos, f, **more):
    dev = device()
    return w4.rope(x.to(dev) if not x.is_cuda else x, torch.tensor(pos, dtype=torch.int32, device=dev),
                   torch.from_numpy(f).to(dev), **more)


SHAPES = [
    # dim, rot
    (128, 128), (128, 64), (128, 32), (128, 2), (64, 64), (64, 20), (64, 16), (256, 256), (256, 96), (80, 80), (80, 32),
    (96, 94), (8, 8), (8, 4), (8, 2), (24, 6), (512, 512), (512, 34), (136, 128)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,rot", SHAPES)
def test_matches_the_oracle(dim, rot, kind, interleaved):
    for tokens, heads in ((1, 1), (3, 5), (17, 40), (1500, 2)):
        say(f"[rope] {kind}, {rot} of {dim}, {'pairs' if interleaved else 'halves'}, {tokens} x {heads}")
        gen = torch.Generator().manual_seed(dim + rot + tokens)
        x = values((tokens, heads, dim), kind, gen)
        pos = torch.randint(0, 131072, (tokens,), generator=gen).tolist()
        y = rotate(x, pos, freqs_of(rot, 500000.0), interleaved=interleaved, factor=1.1)
        check_rotated(y, x, pos, freqs_of(rot, 500000.0), kind, interleaved, False, float(np.float32(1.1)), f"{tokens} x {heads}")


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_of_any_size(interleaved):
    pos = [0, 1, -1, 65535, 131071, 1 << 20, 2 ** 24 + 1, -(2 ** 24)]
    f = freqs_of(64)
    x = values((len(pos), 3, 64), "fp16", torch.Generator().manual_seed(1))
    check_rotated(rotate(x, pos, f, interleaved=interleaved), x, pos, f, "fp16", interleaved, label="positions")
    # the ends of the type: the angle is right to 2^31 * 2^-53 radians, far below fp32's 2^-24
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 7]
    x = values((3, 3, 64), "fp16", torch.Generator().manual_seed(2))
    check_rotated(rotate(x, pos, f, interleaved=interleaved), x, pos, f, "fp16", interleaved, label="ends")


def test_position_zero_keeps_the_bits():
    x = values((5, 4, 128), "bf16", torch.Generator().manual_seed(3))
    assert torch.equal(rotate(x, [0] * 5, freqs_of(128)).cpu(), x)


@pytest.mark.parametrize("dim,rot,interleaved", [(128, 128, False), (128, 128, True), (64, 20, False), (96, 48, False), (256, 256, False)])
def test_strides_and_in_place(dim, rot, interleaved):
    dev = device()
    tokens, heads = 300, 7
    gen = torch.Generator().manual_seed(4)
    f, pos = freqs_of(rot), list(range(100, 100 + tokens))
    rows = values((tokens, heads + 3, dim), "bf16", gen).to(dev)
    want = rotate(rows[:, 1:1 + heads].contiguous(), pos, f, interleaved=interleaved)
    check_rotated(want, rows[:, 1:1 + heads], pos, f, "bf16", interleaved)
    # a slice of fused rows, head by head in memory, and into such
    assert torch.equal(rotate(rows[:, 1:1 + heads], pos, f, interleaved=interleaved), want)
    by_head = rows[:, 1:1 + heads].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.full((heads, tokens, dim), 7.0, dtype=torch.bfloat16, device=dev).transpose(0, 1)
    assert rotate(by_head, pos, f, interleaved=interleaved, out=out) is out and torch.equal(out, want)
    # one row for all tokens, one head for all
    one = rows[:1, 1:1 + heads].expand(tokens, heads, dim)
    assert torch.equal(rotate(one, pos, f, interleaved=interleaved), rotate(one.contiguous(), pos, f, interleaved=interleaved))
    # in place, the rest of the rows as it was
    before = rows.clone()
    view = rows[:, 1:1 + heads]
    rotate(view, pos, f, interleaved=interleaved, out=view)
    assert torch.equal(rows[:, 1:1 + heads], want)
    assert torch.equal(rows[:, :1], before[:, :1]) and torch.equal(rows[:, 1 + heads:], before[:, 1 + heads:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 20), (128, 64)])
def test_inverse_is_the_gradient(dim, rot, interleaved):
    """Against autograd through the formula in 64 bits, and against differences: the
    rotation is linear, so <g, R(x + d) - R(x)> = <R^T g, d> up to roundings."""
    tokens, heads = 6, 2
    gen = torch.Generator().manual_seed(5)
    f, pos = freqs_of(rot), [0, 3, 900, 12, 77777, 131071]
    g = values((tokens, heads, dim), "fp16", gen)
    x = torch.zeros(tokens, heads, dim, dtype=torch.float64, requires_grad=True)
    t = torch.tensor(pos, dtype=torch.float64)[:, None] * torch.from_numpy(f).double()
    c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = torch.cat([1.5 * (a * c - b * s), 1.5 * (a * s + b * c)], -1)
    back = g.double()
    ga, gb = (back[..., :rot:2], back[..., 1:rot:2]) if interleaved else (back[..., :rot // 2], back[..., rot // 2:rot])
    ((y * torch.cat([ga, gb], -1)).sum() + (x[..., rot:] * back[..., rot:]).sum()).backward()
    grad = rotate(g, pos, f, interleaved=interleaved, inverse=True, factor=1.5)
    assert np.abs(as_f64(grad) - x.grad.numpy()).max() <= 2.0 ** -11 * 1.5 * 6 + 4 * 2.0 ** -24 * 20
    check_rotated(grad, g, pos, f, "fp16", interleaved, True, 1.5)
    d = values((tokens, heads, dim), "fp16", gen)
    one = as_f64(rotate(d, pos, f, interleaved=interleaved, factor=1.5))
    n = d.numel()
    # both inner products: n terms, each off by half a step of a value of at most 1.5 * (6 + 6)
    assert abs((as_f64(g) * one).sum() - (as_f64(grad) * as_f64(d)).sum()) <= 2 * n * 2.0 ** -11 * 18


@pytest.mark.parametrize("dim,rot,interleaved", [(128, 128, False), (64, 16, True), (64, 20, False)])
def test_inf_and_nan_stay_in_their_pairs(dim, rot, interleaved):
    x = values((4, 2, dim), "bf16", torch.Generator().manual_seed(6))
    clean = rotate(x, [3] * 4, freqs_of(rot), interleaved=interleaved).cpu()
    x[1, 0, 1], x[2, 1, dim - 1] = float("nan"), float("inf")
    y = rotate(x, [3] * 4, freqs_of(rot), interleaved=interleaved).cpu()
    mate = 0 if interleaved else 1 + rot // 2
    assert torch.isnan(y[1, 0, [1, mate]]).all()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1, 0, [1, mate]] = False
    keep[2, 1, dim - 1] = False
    if rot == dim:
        keep[2, 1, dim - 2 if interleaved else dim // 2 - 1] = False
    assert torch.equal(y[keep], clean[keep])


def test_nothing_to_do():
    dev = device()
    x = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=dev)
    assert rotate(x, [], freqs_of(64)).shape == x.shape
    x = torch.zeros(3, 0, 64, dtype=torch.bfloat16, device=dev)
    assert rotate(x, [1, 2, 3], freqs_of(64)).shape == x.shape


def test_stream_and_graph():
    dev = device()
    f = torch.from_numpy(freqs_of(128)).to(dev)
    x = values((33, 6, 128), "bf16", torch.Generator().manual_seed(7)).to(dev)
    pos = torch.arange(33, dtype=torch.int32, device=dev)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w4.rope(x, pos, f, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.rope(x, pos, f, out=out)
    for i in range(4):
        x.copy_(values((33, 6, 128), "bf16", torch.Generator().manual_seed(8 + i)))
        pos += 1000
        want = w4.rope(x, pos, f)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"
        (want[:, 0] @ want[:, 1].t().contiguous()).sum().item()


def test_offsets_past_32_bits():
    """Rows 2^25 elements apart, up to 2^32 bytes and more in."""
    dev = device()
    tokens, stride = 70, 1 << 25
    x = torch.empty((tokens - 1) * stride + 256, dtype=torch.bfloat16, device=dev).as_strided((tokens, 2, 128), (stride, 128, 1))
    small = values((tokens, 2, 128), "bf16", torch.Generator().manual_seed(9))
    x.copy_(small)
    pos = list(range(tokens))
    check_rotated(rotate(x, pos, freqs_of(128)), small, pos, freqs_of(128), "bf16")
    out = rotate(x, pos, freqs_of(128), out=x)
    check_rotated(out, small, pos, freqs_of(128), "bf16")
