"""The example that runs the cache, the attention and the quantized linears
together, with a 16-bit and an 8-bit cache."""
import os
import sys

import pytest
import torch

from gpu_common import device, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache_type", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("page,window", [(16, 128), (24, 60)])
def test_decoder_attention(cache_type, page, window):
    import decoder_attention
    device()
    say(f"[example] {cache_type}, page {page}, window {window}")
    decoder_attention.run(cache_type=cache_type, page=page, window=window, say=say)
