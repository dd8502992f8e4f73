"""What the binding of the paged cache and its attention refuses beyond the C
ABI: tensors that are not on a GPU, index tensors and workspaces whose memory is
not what the kernels would take it for.  (On CPU tensors throughout: each
refusal comes before anything is enqueued.)"""
import pytest
import torch

import os

import w4a4_block_scaled_amd as w4

pytestmark = pytest.mark.skipif(not os.path.exists(w4.library_path()),
                                reason="libw4a4.so not built (python -m w4a4_block_scaled_amd.build)")


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def calls(**over):
    """Every entry point with tensors that fit each other; `over` replaces some."""
    t = {"rows": torch.zeros(3, 2, 64, dtype=torch.bfloat16), "q": torch.zeros(3, 4, 64, dtype=torch.bfloat16),
         "k": torch.zeros(6, 16, 2, 64, dtype=torch.bfloat16), "tables": ints(3, 4), "lens": ints(3), "refs": ints(6),
         "cu": ints(4), "a": ints(2), "b": ints(2), "lacking": ints(1), "workspace": None}
    t.update(over)
    v = t["k"].clone()
    cache, where = (t["k"], v), (t["tables"], t["lens"])
    return {
        "kv_append": lambda: w4.kv_append(t["rows"], t["rows"], *cache, *where, cu_seqlens=t["cu"]),
        "attn_decode": lambda: w4.attn_decode(t["q"], *cache, *where, workspace=t["workspace"]),
        "attn_prefill": lambda: w4.attn_prefill(t["q"], t["cu"], *cache, *where, workspace=t["workspace"]),
        "kv_copy_pages": lambda: w4.kv_copy_pages(cache, t["a"], t["b"]),
        "kv_reserve": lambda: w4.kv_reserve(*where, t["refs"], 16, lacking=t["lacking"]),
        "kv_fork": lambda: w4.kv_fork(cache, *where, t["refs"], t["a"], t["b"], lacking=t["lacking"]),
        "kv_free": lambda: w4.kv_free(*where, t["refs"], t["a"]),
        "kv_trim": lambda: w4.kv_trim(*where, t["refs"], 16, 5, 0, t["a"]),
        "kv_compact": lambda: w4.kv_compact(cache, t["tables"], t["refs"]),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_tensors_on_the_cpu(name, monkeypatch):
    """Their addresses mean nothing to a kernel, whatever GPU is current."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: pytest.fail("asked for a stream"), raising=False)
    with pytest.raises(w4.W4A4Error, match="GPU") as e:
        calls()[name]()
    assert e.value.status == 2


def spread(*shape):
    """int32, two-dimensional, its entries not side by side."""
    return torch.zeros(shape[0], shape[1] * 2, dtype=torch.int32)[:, ::2]


@pytest.mark.parametrize("name,over", [
    ("kv_append", dict(cu=spread(2, 2))), ("attn_prefill", dict(cu=spread(2, 2))),
    ("kv_reserve", dict(refs=spread(2, 3))), ("kv_fork", dict(refs=spread(2, 3))), ("kv_free", dict(refs=spread(2, 3))),
    ("kv_free", dict(a=spread(1, 2))), ("kv_trim", dict(a=spread(1, 2))), ("kv_trim", dict(refs=spread(2, 3))),
    ("kv_compact", dict(refs=spread(2, 3))), ("kv_copy_pages", dict(a=ints(2, 2)[:, 0]))])
def test_index_tensors_with_gaps(name, over):
    with pytest.raises(w4.W4A4Error, match="contiguous") as e:
        calls(**over)[name]()
    assert e.value.status == 2


@pytest.mark.parametrize("name", ["attn_decode", "attn_prefill"])
@pytest.mark.parametrize("workspace", [torch.zeros(1 << 12, 2, dtype=torch.float32)[:, 0], torch.zeros(1).expand(1 << 24),
                                       torch.empty(1 << 24, dtype=torch.uint8, device="meta")])
def test_workspaces(name, workspace):
    """A workspace with gaps is shorter than it says, one elsewhere is not the device's."""
    with pytest.raises(w4.W4A4Error, match="workspace") as e:
        calls(workspace=workspace)[name]()
    assert e.value.status == 2


BIG = [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 40 + 1, -2 ** 31 - 1]


@pytest.mark.parametrize("value", BIG)
@pytest.mark.parametrize("call", [
    lambda t, x: w4.attn_decode(t["q"], t["k"], t["k"].clone(), t["tables"], t["lens"], window=x),
    lambda t, x: w4.attn_decode(t["q"], t["k"], t["k"].clone(), t["tables"], t["lens"], window=5, sinks=x),
    lambda t, x: w4.attn_prefill(t["q"], t["cu"], t["k"], t["k"].clone(), t["tables"], t["lens"], window=x),
    lambda t, x: w4.kv_trim(t["tables"], t["lens"], t["refs"], 16, x),
    lambda t, x: w4.kv_trim(t["tables"], t["lens"], t["refs"], 16, 5, x),
    lambda t, x: w4.kv_trim(t["tables"], t["lens"], t["refs"], x, 5),
    lambda t, x: w4.kv_reserve(t["tables"], t["lens"], t["refs"], x)])
def test_numbers_past_32_bits(call, value):
    """A C int would take their low 32 bits: a window of 2^32 + 5 as one of 5."""
    t = {"q": torch.zeros(3, 4, 64, dtype=torch.bfloat16), "k": torch.zeros(6, 16, 2, 64, dtype=torch.bfloat16),
         "tables": ints(3, 4), "lens": ints(3), "refs": ints(6), "cu": ints(4)}
    with pytest.raises(w4.W4A4Error, match="32 bits") as e:
        call(t, value)
    assert e.value.status == 2
