"""The example of a decoder layer's attention with its keys stored as they are, in
caches of 16, 8 and 4 bits."""
import os
import sys

import pytest
import torch

from gpu_common import device, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache_type", [torch.bfloat16, torch.float8_e4m3fn, torch.uint8])
@pytest.mark.parametrize("page,window", [(16, 128), (24, 60)])
def test_keys_without_rotation(cache_type, page, window, monkeypatch):
    """Its new rows go through kv_append, and through kv_append_rope where they are rotated."""
    import decoder_attention
    dev = device()
    calls = {"kv_append": 0, "kv_append_rope": 0}

    def counted(name):
        entry = getattr(decoder_attention.w4, name)

        def call(*a, **k):
            calls[name] += 1
            return entry(*a, **k)
        return call
    for name in calls:
        monkeypatch.setattr(decoder_attention.w4, name, counted(name))
    for rotary in (False, True):
        calls.update(dict.fromkeys(calls, 0))
        say(f"[example] {cache_type}, page {page}, window {window}, rotary {rotary}")
        decoder_attention.run(steps=10, cache_type=cache_type, page=page, window=window, device=dev, say=say, rotary=rotary)
        # the prompts and ten steps; the copied-out rows are stored by kv_append either way
        assert calls == ({"kv_append": 1, "kv_append_rope": 11} if rotary else {"kv_append": 12, "kv_append_rope": 0})
