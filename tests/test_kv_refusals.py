"""What the paged cache's and the attention's entry points refuse, on the host
and before anything is enqueued: the C ABI's statuses, and the binding's checks
of tensors."""
import ctypes
import os

import pytest
import torch

import w4a4_block_scaled_amd as w4

pytestmark = pytest.mark.skipif(not os.path.exists(w4.library_path()),
                                reason="libw4a4.so not built (python -m w4a4_block_scaled_amd.build)")

FAKE, MIS = 1 << 20, (1 << 20) + 8          # never dereferenced
NULL, SHAPE, ALIGN, FORMAT, WORKSPACE = 1, 2, 3, 4, 5


def cache(**over):
    f = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, page_stride=16 * 2 * 128, token_stride=256, head_stride=128,
             dtype=0, pages=9, page_size=16, heads=2, head_dim=128)
    f.update(over)
    return w4._KvCache(**f)


def seqs(**over):
    f = dict(tables=FAKE, lens=FAKE, table_stride=4, seqs=3, max_pages=4)
    f.update(over)
    return w4._KvSeqs(**f)


CACHES = [
    (dict(dtype=3), FORMAT), (dict(pages=0), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=65537), SHAPE),
    (dict(heads=0), SHAPE), (dict(head_dim=96), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=MIS), ALIGN),
    (dict(token_stride=-256), SHAPE), (dict(token_stride=252), ALIGN), (dict(head_stride=4), ALIGN),
    (dict(dtype=2, head_stride=136), ALIGN), (dict(dtype=2, k_scale=FAKE + 2), ALIGN),
]
SEQS = [(dict(seqs=-1), SHAPE), (dict(max_pages=0), SHAPE), (dict(table_stride=3), SHAPE), (dict(tables=None), NULL),
        (dict(lens=None), NULL), (dict(lens=FAKE + 2), ALIGN)]


def append(c=None, s=None, cu=FAKE, tokens=5, dtype=0, k=FAKE, row=256, head=128, v=FAKE):
    return w4.lib().w4a4_kv_append(c or cache(), s or seqs(), cu, tokens, dtype, k, row, head, v, row, head, None)


def decode(c=None, s=None, dtype=0, heads=8, q=FAKE, row=1024, head=128, scale=0.1, window=0, sinks=0, out=FAKE, lse=None,
           ws=FAKE, size=1 << 30):
    return w4.lib().w4a4_attn_decode(c or cache(), s or seqs(), dtype, heads, q, row, head, scale, window, sinks, out, row,
                                     head, lse, ws, size, None)


def prefill(c=None, s=None, cu=FAKE, tokens=7, dtype=0, heads=8, q=FAKE, row=1024, head=128, scale=0.1, window=0, sinks=0,
            out=FAKE, lse=None, ws=FAKE, size=1 << 30):
    return w4.lib().w4a4_attn_prefill(c or cache(), s or seqs(), cu, tokens, dtype, heads, q, row, head, scale, window,
                                      sinks, out, row, head, lse, ws, size, None)


@pytest.mark.parametrize("call", [append, decode, prefill])
def test_caches_and_sequences(call):
    for over, status in CACHES:
        assert call(c=cache(**over)) == status, over
        assert w4.lib().w4a4_last_error().decode()
    for over, status in SEQS:
        assert call(s=seqs(**over)) == status, over
    assert call(dtype=2) == FORMAT                      # rows are 16-bit
    assert call(dtype=1) == FORMAT                      # FP16 rows, BF16 cache


@pytest.mark.parametrize("args,status", [
    (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE), (dict(cu=None), SHAPE), (dict(cu=FAKE + 2), ALIGN),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=MIS), ALIGN), (dict(row=-8), SHAPE), (dict(row=260), ALIGN),
    (dict(head=129), ALIGN)])
def test_append(args, status):
    assert append(**args) == status


@pytest.mark.parametrize("args,status", [
    (dict(heads=7), SHAPE), (dict(heads=0), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(window=-1), SHAPE),
    (dict(sinks=-1), SHAPE), (dict(q=None), NULL), (dict(out=None), NULL), (dict(q=MIS), ALIGN), (dict(row=1028), ALIGN),
    (dict(lse=FAKE + 2), ALIGN), (dict(ws=None), WORKSPACE), (dict(size=64), WORKSPACE), (dict(ws=MIS), ALIGN)])
def test_attention(args, status):
    assert decode(**args) == status
    assert prefill(**args) == status
    assert w4.lib().w4a4_last_error().decode()


def test_prefill_rows():
    assert prefill(cu=None) == NULL and prefill(cu=FAKE + 2) == ALIGN
    assert prefill(tokens=-1) == SHAPE and prefill(tokens=1 << 30) == SHAPE
    assert prefill(s=seqs(seqs=0)) == SHAPE


def test_empty_calls_are_no_ops():
    none = seqs(seqs=0, tables=None, lens=None)
    assert append(s=none, tokens=0, cu=None, k=None, v=None) == 0
    assert append(tokens=0, k=None, v=None) == 0
    assert decode(s=none, q=None, out=None, ws=None, size=0) == 0
    assert prefill(tokens=0, cu=None, q=None, out=None, ws=None, size=0) == 0
    assert copy(pairs=0, src=None, dst=None) == 0 and copy(n=0) == 0
    assert w4.lib().w4a4_kv_free(seqs(), FAKE, 9, None, 0, None) == 0


def test_workspace_sizes():
    L = w4.lib()
    assert L.w4a4_attn_decode_workspace_bytes(cache(), 3, 8) > 0
    assert L.w4a4_attn_decode_workspace_bytes(cache(), 3, 7) == 0
    assert L.w4a4_attn_decode_workspace_bytes(cache(head_dim=80), 3, 8) == 0
    assert L.w4a4_attn_prefill_workspace_bytes(cache(), 3, 7, 8) > 0
    assert L.w4a4_attn_prefill_workspace_bytes(cache(), 3, 7, 9) == 0
    assert L.w4a4_kv_workspace_bytes(-1, 9) == 0 and L.w4a4_kv_workspace_bytes(1, 0) == 0
    assert L.w4a4_kv_workspace_bytes(100, 9) >= 100 * 8


def copy(n=2, arrays=(FAKE, FAKE), stride=4096, size=4096, pages=9, src=FAKE, dst=FAKE, pairs=3):
    a = None if arrays is None else (ctypes.c_void_p * max(1, len(arrays)))(*arrays)
    return w4.lib().w4a4_kv_copy_pages(n, a, stride, size, pages, src, dst, pairs, None)


@pytest.mark.parametrize("args,status", [
    (dict(n=-1), SHAPE), (dict(arrays=None), NULL), (dict(arrays=(FAKE, None)), NULL), (dict(arrays=(FAKE, MIS)), ALIGN),
    (dict(stride=4095), SHAPE), (dict(size=0), SHAPE), (dict(pages=0), SHAPE), (dict(src=None), NULL),
    (dict(dst=FAKE + 1), ALIGN), (dict(pairs=-1), SHAPE), (dict(pairs=1 << 31), SHAPE)])
def test_copy_pages(args, status):
    assert copy(**args) == status


def test_bookkeeping():
    L, a = w4.lib(), (ctypes.c_void_p * 1)(FAKE)
    big = 1 << 30
    assert L.w4a4_kv_reserve(seqs(), 0, FAKE, 9, None, FAKE, big, None) == SHAPE
    assert L.w4a4_kv_reserve(seqs(), 16, None, 9, None, FAKE, big, None) == NULL
    assert L.w4a4_kv_reserve(seqs(), 16, FAKE, 9, FAKE + 2, FAKE, big, None) == ALIGN
    assert L.w4a4_kv_reserve(seqs(), 16, FAKE, 9, None, FAKE, 8, None) == WORKSPACE
    assert L.w4a4_kv_reserve(seqs(), 16, FAKE, 9, None, MIS, big, None) == ALIGN
    assert L.w4a4_kv_fork(1, a, 64, 64, seqs(), 16, FAKE, 9, None, FAKE, 2, None, FAKE, big, None) == NULL
    assert L.w4a4_kv_fork(1, a, 64, 64, seqs(), 16, FAKE, 9, FAKE, FAKE, -1, None, FAKE, big, None) == SHAPE
    assert L.w4a4_kv_fork(1, a, 64, 64, seqs(), 16, FAKE, 9, FAKE, FAKE, 2, None, None, big, None) == WORKSPACE
    assert L.w4a4_kv_free(seqs(), FAKE, 9, None, 2, None) == SHAPE
    assert L.w4a4_kv_free(seqs(), None, 9, FAKE, 2, None) == NULL
    assert L.w4a4_kv_free(seqs(), FAKE, 9, FAKE + 2, 2, None) == ALIGN
    assert L.w4a4_kv_trim(seqs(), 16, FAKE, 9, FAKE, 2, 0, 0, None) == SHAPE
    assert L.w4a4_kv_trim(seqs(), 16, FAKE, 9, FAKE, 2, 5, -1, None) == SHAPE
    assert L.w4a4_kv_compact(1, a, 64, 64, seqs(), FAKE, 9, None, FAKE, big, None) == NULL
    assert L.w4a4_kv_compact(1, a, 64, 64, seqs(), FAKE, 9, FAKE, FAKE, 8, None) == WORKSPACE


# ----------------------------------------------------------------- binding --

def tensors():
    k = torch.zeros(6, 16, 2, 64, dtype=torch.bfloat16)
    return {"q": torch.zeros(3, 4, 64, dtype=torch.bfloat16), "k_cache": k, "v_cache": k.clone(),
            "tables": torch.zeros(3, 4, dtype=torch.int32), "lens": torch.zeros(3, dtype=torch.int32)}


@pytest.mark.parametrize("name,make,status", [
    ("k_cache", lambda t: t[:, :, :, ::2], 2),                      # last dimension not contiguous, another shape
    ("v_cache", lambda t: t.to(torch.float16), 2),                  # K and V of different types
    ("v_cache", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2), 2),
    ("tables", lambda t: t.long(), 2), ("lens", lambda t: t.long(), 2), ("lens", lambda t: t[:2], 2),
    ("tables", lambda t: t.t().contiguous().t(), 2), ("q", lambda t: t[:2], 2), ("q", lambda t: t[..., :32], 2),
    ("q", lambda t: t.float(), 4)])
def test_binding_refuses_tensors(name, make, status):
    t = tensors()
    t[name] = make(t[name])
    with pytest.raises(w4.W4A4Error) as e:
        w4.attn_decode(**t)
    assert e.value.status == status


def test_binding_refuses_scales_lists_and_pages():
    t = tensors()
    with pytest.raises(w4.W4A4Error, match="float8"):
        w4.attn_decode(**t, k_scale=torch.ones(2))
    q8 = dict(t, k_cache=t["k_cache"].to(torch.float8_e4m3fn), v_cache=t["v_cache"].to(torch.float8_e4m3fn))
    with pytest.raises(w4.W4A4Error, match="scales"):
        w4.attn_decode(**q8, k_scale=torch.ones(3))
    with pytest.raises(w4.W4A4Error, match="cu_seqlens"):
        w4.attn_prefill(t["q"], torch.zeros(3, dtype=torch.int32), *[t[n] for n in ("k_cache", "v_cache", "tables", "lens")])
    rows = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(w4.W4A4Error, match="k is"):
        w4.kv_append(rows, rows.half(), t["k_cache"], t["v_cache"], t["tables"], t["lens"])
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(w4.W4A4Error, match="densely"):
        w4.kv_copy_pages([t["k_cache"][:, :, :1]], i, i)
    with pytest.raises(w4.W4A4Error, match="alike"):
        w4.kv_copy_pages([t["k_cache"], t["k_cache"][:5]], i, i)
    with pytest.raises(w4.W4A4Error, match="no caches"):
        w4.kv_copy_pages([], i, i)
    with pytest.raises(w4.W4A4Error, match="entries"):
        w4.kv_copy_pages([t["k_cache"]], i, i[:1])
    with pytest.raises(w4.W4A4Error, match="refs"):
        w4.kv_fork([t["k_cache"]], t["tables"], t["lens"], torch.zeros(5, dtype=torch.int32), i[:1], i[:1])
