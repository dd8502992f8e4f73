"""What the entry points of rotary positions, of rows into and out of the cache,
and of the 4-bit cache refuse, on the CPU: the host checks alone run (every call
here is refused or has nothing to do)."""
import math

import pytest
import torch

import w4a4_block_scaled_amd as w4
from test_kv_refusals import ALIGN, FAKE, FORMAT, MIS, NULL, SHAPE, WORKSPACE, cache, seqs

BIG = 2 ** 31


def fp4(**over):
    f = dict(dtype=4, page_stride=16 * 2 * 68, token_stride=0, head_stride=0)
    f.update(over)
    return cache(**f)


def rotation(**over):
    f = dict(freqs=FAKE, rot_dim=128, interleaved=0, inverse=0, factor=1.0)
    f.update(over)
    return w4._Rotation(**f)


def rope(r=None, tokens=5, positions=FAKE, dtype=0, heads=4, dim=128, x=FAKE, row=512, head=128, out=2 * FAKE, o_row=512,
         o_head=128, none=False):
    return w4.lib().w4a4_rope(None if none else r or rotation(), tokens, positions, dtype, heads, dim, x, row, head, out,
                              o_row, o_head, None)


def append(c=None, s=None, cu=FAKE, tokens=5, dtype=0, r=None, positions=None, q_heads=4, q=FAKE, q_row=1024, q_head=128,
           out=2 * FAKE, o_row=512, o_head=128, k=FAKE, row=256, head=128, v=FAKE, none=False):
    return w4.lib().w4a4_kv_append_rope(c or cache(), s or seqs(), cu, tokens, dtype, None if none else r or rotation(),
                                        positions, q_heads, q, q_row, q_head, out, o_row, o_head, k, row, head, v, row,
                                        head, None)


def plain_append(c=None, s=None, cu=FAKE, tokens=5, dtype=0, k=FAKE, row=256, head=128, v=FAKE):
    return w4.lib().w4a4_kv_append(c or fp4(), s or seqs(), cu, tokens, dtype, k, row, head, v, row, head, None)


def read(c=None, s=None, cu=FAKE, tokens=5, dtype=0, k=FAKE, row=256, head=128, v=FAKE):
    return w4.lib().w4a4_kv_read(c or cache(), s or seqs(), cu, tokens, dtype, k, row, head, v, row, head, None)


ROTATIONS = [(dict(freqs=None), NULL), (dict(freqs=FAKE + 2), ALIGN), (dict(rot_dim=0), SHAPE), (dict(rot_dim=-2), SHAPE),
             (dict(rot_dim=3), SHAPE), (dict(rot_dim=130), SHAPE), (dict(interleaved=2), SHAPE), (dict(inverse=-1), SHAPE),
             (dict(factor=0.0), SHAPE), (dict(factor=-1.0), SHAPE), (dict(factor=math.inf), SHAPE), (dict(factor=math.nan), SHAPE)]


@pytest.mark.parametrize("over,status", ROTATIONS)
def test_rotations(over, status):
    assert rope(rotation(**over)) == status
    assert append(r=rotation(**over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(none=True), NULL), (dict(dtype=2), FORMAT), (dict(dtype=4), FORMAT), (dict(dtype=-1), FORMAT), (dict(tokens=-1), SHAPE),
    (dict(tokens=BIG), SHAPE), (dict(heads=-1), SHAPE), (dict(heads=65537), SHAPE), (dict(dim=100), SHAPE), (dict(dim=0), SHAPE),
    (dict(dim=520), SHAPE), (dict(positions=None), NULL), (dict(positions=FAKE + 2), ALIGN), (dict(x=None), NULL),
    (dict(out=None), NULL), (dict(x=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(row=510), ALIGN), (dict(o_head=4), ALIGN),
    (dict(row=-512), SHAPE), (dict(o_head=-128), SHAPE), (dict(out=FAKE, o_row=1024), SHAPE), (dict(out=FAKE, o_head=256), SHAPE),
    # more workgroups than a launch has threads for
    (dict(tokens=BIG - 1, dim=512), SHAPE), (dict(tokens=2 ** 29, dim=128), SHAPE)])
def test_rope(over, status):
    assert rope(**over) == status
    assert w4.lib().w4a4_last_error().decode().startswith("rope")


def test_nothing_to_do_is_ok():
    assert rope(tokens=0, positions=None, x=None, out=None) == 0
    assert rope(heads=0, positions=None, x=None, out=None) == 0
    assert append(tokens=0, q=None, k=None, v=None) == 0
    assert append(s=seqs(seqs=0, tables=None, lens=None)) == 0
    assert read(tokens=0, k=None, v=None) == 0
    assert plain_append(tokens=0, k=None, v=None) == 0
    assert w4.lib().w4a4_last_error() == b""


@pytest.mark.parametrize("call", [append, read, plain_append])
@pytest.mark.parametrize("over,status", [
    (dict(tokens=-1), SHAPE), (dict(tokens=BIG), SHAPE), (dict(cu=None, tokens=5), SHAPE), (dict(cu=FAKE + 2), ALIGN),
    (dict(dtype=2), FORMAT), (dict(dtype=4), FORMAT), (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=MIS), ALIGN),
    (dict(v=MIS), ALIGN), (dict(row=252), ALIGN), (dict(head=-128), SHAPE), (dict(tokens=BIG - 1), SHAPE)])
def test_rows(call, over, status):
    assert call(**over) == status


@pytest.mark.parametrize("call", [append, read])
def test_rows_of_another_type(call):
    assert call(c=cache(dtype=1), dtype=0) == FORMAT
    assert call(c=cache(dtype=0), dtype=1) == FORMAT
    assert call(c=cache(heads=65537, head_stride=0)) == SHAPE


@pytest.mark.parametrize("over,status", [
    (dict(none=True), NULL), (dict(q_heads=-1), SHAPE), (dict(q_heads=65537), SHAPE), (dict(q=None), NULL), (dict(out=None), NULL),
    (dict(q=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(q_row=4), ALIGN), (dict(o_head=-8), SHAPE), (dict(out=FAKE), SHAPE),
    (dict(positions=FAKE + 2), ALIGN)])
def test_append_rope(over, status):
    assert append(**over) == status


def attend(c, prefill=False, ws=FAKE, ws_bytes=1 << 40, **more):
    if prefill:
        return w4.lib().w4a4_attn_prefill(c, seqs(), FAKE, 7, 0, 8, FAKE, 1024, 128, 0.1, 0, 0, FAKE, 1024, 128, None, ws,
                                          ws_bytes, None)
    return w4.lib().w4a4_attn_decode(c, seqs(), 0, 8, FAKE, 1024, 128, 0.1, 0, 0, FAKE, 1024, 128, None, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [lambda c: append(c=c), lambda c: read(c=c), lambda c: plain_append(c=c), attend,
                                  lambda c: attend(c, True)])
@pytest.mark.parametrize("over,status", [
    (dict(page_stride=16 * 2 * 68 - 16), SHAPE), (dict(page_stride=0), SHAPE), (dict(token_stride=64), SHAPE),
    (dict(head_stride=64), SHAPE), (dict(page_stride=16 * 2 * 68 + 8), ALIGN), (dict(k_scale=FAKE), FORMAT),
    (dict(v_scale=FAKE), FORMAT), (dict(k=MIS), ALIGN), (dict(head_dim=96), SHAPE), (dict(dtype=3), FORMAT), (dict(dtype=5), FORMAT)])
def test_caches_of_4_bits(call, over, status):
    assert call(fp4(**over)) == status


def test_workspaces_and_sizes():
    L = w4.lib()
    need = L.w4a4_attn_decode_workspace_bytes(fp4(), 3, 8)
    assert need > 0 and attend(fp4(), ws_bytes=need - 1) == WORKSPACE and attend(fp4(), ws=None) == WORKSPACE
    assert L.w4a4_attn_prefill_workspace_bytes(fp4(), 3, 40, 8) > 0
    assert L.w4a4_kv_page_bytes(16, 8, 128) == 16 * 8 * 68
    for bad in ((0, 8, 128), (65537, 8, 128), (16, 0, 128), (16, 8, 96)):
        assert L.w4a4_kv_page_bytes(*bad) == 0


# ----------------------------------------------------------------- binding --

def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def tensors():
    c = w4.kv_cache_e2m1((2, 6), 16, 2, 64, device="cpu")
    rows = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    return {"q": torch.zeros(3, 4, 64, dtype=torch.bfloat16), "k": rows, "v": rows.clone(), "k_cache": c[0], "v_cache": c[1],
            "tables": torch.zeros(3, 4, dtype=torch.int32), "lens": ints(1, 1, 1), "freqs": torch.ones(32)}


@pytest.mark.parametrize("name,make,status", [
    ("q", lambda t: t.half(), 4), ("v", lambda t: t.half(), 4), ("q", lambda t: t[:2], 2), ("k", lambda t: t[..., :32], 2),
    ("k", lambda t: t[:, :1], 2), ("freqs", lambda t: t.double(), 2), ("freqs", lambda t: t[::2], 2), ("freqs", lambda t: t[None], 2),
    ("freqs", lambda t: torch.ones(33), 2), ("freqs", lambda t: t[:0], 2), ("k_cache", lambda t: t[..., :33], 2),
    ("k_cache", lambda t: t.transpose(1, 2), 2), ("v_cache", lambda t: t.contiguous()[:, :8], 2), ("lens", lambda t: t[:2], 2),
    ("tables", lambda t: t.long(), 2)])
def test_binding_refuses(name, make, status):
    t = tensors()
    t[name] = make(t[name])
    if name == "k_cache" and t[name].shape[-1] == 34:
        t["v_cache"] = make(t["v_cache"])
    with pytest.raises(w4.W4A4Error) as e:
        w4.kv_append_rope(**t)
    assert e.value.status == status


def test_binding_refuses_more():
    t = tensors()
    for more, text in ((dict(k_scale=torch.ones(2)), "float8"), (dict(positions=ints(1, 2)), "positions"),
                       (dict(positions=torch.zeros(3)), "int32"), (dict(cu_seqlens=ints(0, 3)), "cu_seqlens"),
                       (dict(q_out=t["q"].half()), "q_out"), (dict(q_out=t["q"][:, :2]), "q_out"),
                       (dict(), "GPU")):
        with pytest.raises(w4.W4A4Error, match=text):
            w4.kv_append_rope(**t, **more)
    with pytest.raises(w4.W4A4Error, match="without q"):
        w4.kv_append_rope(**{**t, "q": None}, q_out=t["q"])
    x, pos, f = t["q"], ints(1, 2, 3), t["freqs"]
    for args, more, text in (((x[0], pos, f), {}, "tokens, heads"), ((x, pos[:2], f), {}, "positions"), ((x, pos.long(), f), {}, "int32"),
                             ((x.float(), pos, f), {}, "type"), ((x, pos, f), dict(out=x.half()), "out is"),
                             ((x, pos, f), dict(out=x[:, :3]), "out"), ((x[..., ::2], pos, f), {}, "x"), ((x, pos, f), {}, "GPU")):
        with pytest.raises(w4.W4A4Error, match=text):
            w4.rope(*args, **more)
    c = [t[n] for n in ("k_cache", "v_cache", "tables", "lens")]
    for args, more, text in (((*c, None, -1), {}, "tokens"), ((*c, ints(0, 3), 3), {}, "cu_seqlens"),
                             ((*c, None, 3), dict(dtype=torch.float32), "type"), ((*c, None, 3), dict(out=(t["k"], t["v"].half())), "out is"),
                             ((*c, None, 3), dict(out=(t["k"], t["q"])), "v"), ((*c, None, 3), {}, "GPU")):
        with pytest.raises(w4.W4A4Error, match=text):
            w4.kv_read(*args, **more)
    with pytest.raises(w4.W4A4Error, match="GPU"):
        w4.kv_append(t["k"], t["v"], *c)
    with pytest.raises(w4.W4A4Error, match="GPU"):
        w4.attn_decode(t["q"], *c)


def test_binding_refuses_what_a_c_type_does_not_hold():
    t = tensors()
    wide = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16).expand(1, BIG, 1, 64)
    with pytest.raises(w4.W4A4Error, match="does not fit"):
        w4.kv_append(t["k"], t["v"], wide, wide, t["tables"], t["lens"])
    wide = ints(0)[:, None].expand(BIG, 1)
    with pytest.raises(w4.W4A4Error, match="does not fit"):
        w4.kv_append(t["k"], t["v"], t["k_cache"], t["v_cache"], wide, None)


def test_calls_go_to_the_device_of_their_tensors(monkeypatch):
    """With another device current, that of the tensors is made so for the call, and the old one comes back."""
    state, seen = {"device": 0}, []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, state["device"] = state["device"], self.device

        def __exit__(self, *_):
            state["device"] = self.before
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["device"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    for device in (0, 1):
        w4._kv_call(device, lambda *a: seen.append((state["device"], *a)) or 0, "x")
    assert seen == [(0, "x", 1000), (1, "x", 1001)] and state["device"] == 0
    with pytest.raises(w4.W4A4Error) as e:
        w4._kv_call(1, lambda *a: 3)
    assert e.value.status == 3 and state["device"] == 0
    with pytest.raises(w4.W4A4Error, match="GPU"):
        w4._kv_call(-1, lambda *a: 0)
