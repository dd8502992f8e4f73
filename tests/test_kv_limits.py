"""Counts near 2^31 that the paged cache's and the attention's entry points
refuse on the host: the kernels count rows, sequences and list entries in 32
bits, a step past the last one included."""
import ctypes
import os

import pytest

import w4a4_block_scaled_amd as w4
from test_kv_refusals import FAKE, SHAPE, append, cache, copy, decode, prefill, seqs

pytestmark = pytest.mark.skipif(not os.path.exists(w4.library_path()),
                                reason="libw4a4.so not built (python -m w4a4_block_scaled_amd.build)")


@pytest.mark.parametrize("tokens,heads", [((1 << 31) // 8 - 1, 8), ((1 << 31) // 8 - 32, 8), ((1 << 31) - 1, 1)])
def test_rows_whose_last_tile_would_pass_32_bits(tokens, heads):
    one = cache(heads=1)
    assert prefill(c=one, heads=heads, tokens=tokens) == SHAPE
    assert prefill(c=one, heads=heads, tokens=tokens, s=seqs(seqs=1 << 28)) == SHAPE         # as few rows per sequence
    assert w4.lib().w4a4_attn_prefill_workspace_bytes(one, 3, tokens, heads) == 0


def test_sequences():
    many = seqs(seqs=(1 << 31) - 1)
    assert append(s=many, cu=FAKE) == SHAPE
    assert decode(s=many, heads=1, c=cache(heads=1)) == SHAPE
    assert prefill(s=many) == SHAPE
    L, a = w4.lib(), (ctypes.c_void_p * 1)(FAKE)
    assert L.w4a4_kv_reserve(many, 16, FAKE, 9, None, FAKE, 1 << 40, None) == SHAPE
    assert L.w4a4_kv_fork(1, a, 64, 64, many, 16, FAKE, 9, FAKE, FAKE, 2, None, FAKE, 1 << 40, None) == SHAPE
    assert L.w4a4_kv_free(many, FAKE, 9, FAKE, 2, None) == SHAPE
    assert L.w4a4_kv_compact(1, a, 64, 64, many, FAKE, 9, FAKE, FAKE, 1 << 40, None) == SHAPE


def test_row_tiles():
    """A row tile per sequence at least: more than one launch can have."""
    assert prefill(s=seqs(seqs=1 << 24), tokens=(1 << 28) + (1 << 24), heads=2) == SHAPE


def test_lists():
    a = (ctypes.c_void_p * 1)(FAKE)
    n = (1 << 31) - 1
    assert copy(pairs=n) == SHAPE
    assert w4.lib().w4a4_kv_fork(1, a, 64, 64, seqs(), 16, FAKE, 9, FAKE, FAKE, n, None, FAKE, 1 << 40, None) == SHAPE
