"""Attention over a cache held in 4 bits at the ends of its range: scales whose values
leave BF16's, in places that some rows do not see."""
import pytest
import torch

from gpu_common import device, say
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
