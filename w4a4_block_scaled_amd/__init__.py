"""Python binding of libw4a4 (the MI355X packed W4A4 block-scaled linear).

Argument marshalling only: every step of the path runs in the gfx950
kernels behind the C ABI declared in include/w4a4.h.  torch supplies device
memory and the current HIP stream.  The raw C functions are available on
``lib()`` under their C names; the wrappers below keep the same names
without the ``w4a4_`` prefix:

    codes, scales, t = quantize_act(x_bf16, c_fp32, "mxfp4")
    blob             = pack_weight(w_codes, w_scales, t_w, r, "mxfp4")
    y_bf16           = linear(codes, scales, t, blob, "mxfp4", N, K)

The paged key-value cache and the attention between the linears:

    q = kv_append_rope(q, k, v, k_cache, v_cache, tables, lens, freqs)
    out = attn_decode(q, k_cache, v_cache, tables, lens)

There is no fallback: if the library is missing or fails to load, the
functions raise.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
from typing import Optional, Tuple

import torch

__all__ = ["FORMATS", "lib", "library_path", "block_size", "scale_dtype", "quantize_act", "pack_weight",
           "unpack_weight", "linear", "linear_noalloc", "linear_workspace", "packed_weight_bytes", "W4A4Error",
           "attn_decode", "attn_prefill", "kv_append", "kv_copy_pages", "kv_reserve", "kv_fork", "kv_free", "kv_trim",
           "kv_compact", "kv_append_rope", "kv_read", "kv_cache_e2m1", "rope", "rope_freqs"]

FORMATS = {"mxfp4": 0, "nvfp4": 1, "mxint4": 2, "int4g64": 3, "mxfp8": 4, "mxint8": 5, "int8g128": 6}
_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None
_KV_LIB = None


class W4A4Error(RuntimeError):
    """A non-OK status from the C ABI (message from w4a4_last_error)."""

    def __init__(self, status: int, message: str):
        super().__init__(f"w4a4 status {status}: {message}")
        self.status = status


def library_path() -> str:
    """The in-tree libw4a4.so, or the file W4A4_LIBRARY names (a variant build
    of the same sources, e.g. the AddressSanitizer one)."""
    return os.environ.get("W4A4_LIBRARY") or os.path.join(_HERE, "libw4a4.so")


class _KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("dtype", ctypes.c_int32), ("pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _Rotation(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("factor", ctypes.c_float)]


class _KvSeqs(ctypes.Structure):
    _fields_ = [("tables", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


def lib() -> ctypes.CDLL:
    """Load libw4a4.so (built in-tree by build.py); raise if it is missing."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           f"`python -m w4a4_block_scaled_amd.build` (no fallback exists)")
    L = ctypes.CDLL(path)
    i64, sz, vp, i32 = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int
    L.w4a4_block_size.argtypes = [i32]
    L.w4a4_block_size.restype = i32
    for name in ("w4a4_act_codes_bytes", "w4a4_act_scales_bytes",
                 "w4a4_quantize_workspace_bytes", "w4a4_packed_weight_bytes"):
        getattr(L, name).argtypes = [i32, i64, i64]
        getattr(L, name).restype = sz
    L.w4a4_linear_workspace_bytes.argtypes = [i32, i64, i64, i64]
    L.w4a4_linear_workspace_bytes.restype = sz
    L.w4a4_quantize_act.argtypes = [i32, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.w4a4_quantize_act.restype = i32
    L.w4a4_quantize_act_multi.argtypes = [i32, i64, i64, vp, i32, vp, vp, vp, vp, vp, sz, vp]
    L.w4a4_quantize_act_multi.restype = i32
    L.w4a4_linear_grouped.argtypes = [i32, i32, i64, i64, vp, vp, vp, vp, vp, vp, vp]
    L.w4a4_linear_grouped.restype = i32
    L.w4a4_pack_weight.argtypes = [i32, i64, i64, vp, vp, vp, vp, vp, vp]
    L.w4a4_pack_weight.restype = i32
    L.w4a4_unpack_weight.argtypes = [i32, i64, i64, vp, vp, vp, vp, vp, vp]
    L.w4a4_unpack_weight.restype = i32
    L.w4a4_linear.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.w4a4_linear.restype = i32
    L.w4a4_linear_noalloc.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp, vp, vp]
    L.w4a4_linear_noalloc.restype = i32
    L.w4a4_dualquant_workspace_bytes.argtypes = [i32, i64, i64]
    L.w4a4_dualquant_workspace_bytes.restype = sz
    L.w4a4_dualquant_solve.argtypes = [i32, i64, i64, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.w4a4_dualquant_solve.restype = i32
    L.w4a4_probe_stream_read.argtypes = [vp, sz, vp, vp]
    L.w4a4_probe_stream_read.restype = i32
    L.w4a4_probe_empty.argtypes = [vp]
    L.w4a4_probe_empty.restype = i32
    L.w4a4_probe_mfma_fp4.argtypes = [vp, ctypes.c_int, ctypes.c_int, vp, vp]
    L.w4a4_probe_mfma_fp4.restype = i32
    _declare_kv(L, ctypes.POINTER(_KvCache), ctypes.POINTER(_KvSeqs), ctypes.POINTER(_Rotation))
    L.w4a4_last_error.argtypes = []
    L.w4a4_last_error.restype = ctypes.c_char_p
    L.w4a4_version.argtypes = []
    L.w4a4_version.restype = ctypes.c_char_p
    _LIB = L
    return L


def _declare_kv(L: ctypes.CDLL, cp, sp, rp) -> None:
    """The entry points of the cache, its attention and rotary positions; cp, sp, rp: how a cache, its
    sequences and a rotation are passed."""
    i64, sz, vp, i32, f32 = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.w4a4_kv_append.argtypes = [cp, sp, vp, i64, i32, vp, i64, i64, vp, i64, i64, vp]
    L.w4a4_attn_decode_workspace_bytes.argtypes = [cp, i64, i32]
    L.w4a4_attn_decode_workspace_bytes.restype = sz
    L.w4a4_attn_decode.argtypes = [cp, sp, i32, i32, vp, i64, i64, f32, i32, i32, vp, i64, i64, vp, vp, sz, vp]
    L.w4a4_attn_prefill_workspace_bytes.argtypes = [cp, i64, i64, i32]
    L.w4a4_attn_prefill_workspace_bytes.restype = sz
    L.w4a4_attn_prefill.argtypes = [cp, sp, vp, i64, i32, i32, vp, i64, i64, f32, i32, i32, vp, i64, i64, vp, vp, sz, vp]
    L.w4a4_kv_copy_pages.argtypes = [i32, vp, i64, i64, i32, vp, vp, i64, vp]
    L.w4a4_kv_workspace_bytes.argtypes = [i64, i64]
    L.w4a4_kv_workspace_bytes.restype = sz
    L.w4a4_kv_reserve.argtypes = [sp, i32, vp, i32, vp, vp, sz, vp]
    L.w4a4_kv_fork.argtypes = [i32, vp, i64, i64, sp, i32, vp, i32, vp, vp, i32, vp, vp, sz, vp]
    L.w4a4_kv_free.argtypes = [sp, vp, i32, vp, i32, vp]
    L.w4a4_kv_trim.argtypes = [sp, i32, vp, i32, vp, i32, i32, i32, vp]
    L.w4a4_kv_compact.argtypes = [i32, vp, i64, i64, sp, vp, i32, vp, vp, sz, vp]
    L.w4a4_kv_page_bytes.argtypes = [i32, i32, i32]
    L.w4a4_kv_page_bytes.restype = sz
    L.w4a4_rope.argtypes = [rp, i64, vp, i32, i32, i32, vp, i64, i64, vp, i64, i64, vp]
    L.w4a4_kv_append_rope.argtypes = [cp, sp, vp, i64, i32, rp, vp, i32, vp, i64, i64, vp, i64, i64, vp, i64, i64, vp,
                                      i64, i64, vp]
    L.w4a4_kv_read.argtypes = [cp, sp, vp, i64, i32, vp, i64, i64, vp, i64, i64, vp]
    for name in ("rope", "kv_append_rope", "kv_read", "kv_append", "attn_decode", "attn_prefill", "kv_copy_pages", "kv_reserve", "kv_fork", "kv_free",
                 "kv_trim", "kv_compact"):
        getattr(L, "w4a4_" + name).restype = i32


def _kv_lib() -> ctypes.CDLL:
    """lib() once more, with those structures passed as packed bytes: a third of a ctypes.Structure's
    cost per call."""
    global _KV_LIB
    if _KV_LIB is None:
        lib()
        L = ctypes.CDLL(library_path())
        _declare_kv(L, ctypes.c_char_p, ctypes.c_char_p, ctypes.c_char_p)
        _KV_LIB = L
    return _KV_LIB


_PACK_CACHE = struct.Struct("PPPPqqqiiiii").pack       # as _KvCache, _KvSeqs, _Rotation
_PACK_SEQS = struct.Struct("PPqii").pack
_PACK_ROTATION = struct.Struct("Piiif").pack


def _unfit(what: str, e: Exception) -> W4A4Error:
    return W4A4Error(2, f"{what}: an argument does not fit its C type ({e})")


def _fmt(fmt) -> int:
    if isinstance(fmt, str):
        return FORMATS[fmt]
    return int(fmt)


def _check(status: int) -> None:
    if status != 0:
        raise W4A4Error(status, lib().w4a4_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def scale_dtype(fmt) -> torch.dtype:
    """Element type of block scales: bytes (E8M0 / UE4M3), BF16 for INT4 G=64 and INT8 G=128."""
    return torch.bfloat16 if _fmt(fmt) in (FORMATS["int4g64"], FORMATS["int8g128"]) else torch.uint8


def code_cols(fmt, K: int) -> int:
    """Bytes of canonical codes per row of K elements (K/2; K for the 8-bit formats)."""
    return K if _fmt(fmt) in (FORMATS["mxfp8"], FORMATS["mxint8"], FORMATS["int8g128"]) else K // 2


def block_size(fmt) -> int:
    return lib().w4a4_block_size(_fmt(fmt))


def packed_weight_bytes(fmt, N: int, K: int) -> int:
    return lib().w4a4_packed_weight_bytes(_fmt(fmt), N, K)


def quantize_act(x: torch.Tensor, c: Optional[torch.Tensor], fmt,
                 out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None,
                 workspace: Optional[torch.Tensor] = None):
    """w4a4_quantize_act: x bf16 [M, K], c fp32 [K] or None -> (codes, scales, t).

    codes uint8 [M, K/2] ([M, K] for MXFP8 / MXINT8), scales [M, K/G] (uint8;
    bfloat16 for INT4 G=64),
    t fp32 [1] (NVFP4 tensor scale; unused for the other formats).
    """
    f = _fmt(fmt)
    L = lib()
    M, K = x.shape
    G = L.w4a4_block_size(f)
    if out is None:
        codes = torch.empty((M, code_cols(fmt, K)), dtype=torch.uint8, device=x.device)
        scales = torch.empty((M, K // G), dtype=scale_dtype(fmt), device=x.device)
        t = torch.ones(1, dtype=torch.float32, device=x.device)
    else:
        codes, scales, t = out
    ws_bytes = L.w4a4_quantize_workspace_bytes(f, M, K)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    _check(L.w4a4_quantize_act(f, M, K, _ptr(x), _ptr(c), _ptr(codes), _ptr(scales), _ptr(t),
                               _ptr(workspace), workspace.numel() if workspace is not None else 0,
                               _stream(x.device)))
    return codes, scales, t


def quantize_act_multi(x: torch.Tensor, cs, fmt, workspace: Optional[torch.Tensor] = None):
    """w4a4_quantize_act_multi: bf16 [M, K] and P column-scale vectors -> a list of
    (codes [M, K/2], scales [M, K/G], t [1] for NVFP4 else None), X read once."""
    f = _fmt(fmt)
    L = lib()
    M, K = x.shape
    P = len(cs)
    G = block_size(fmt)
    outs = [(torch.empty((M, K // 2), dtype=torch.uint8, device=x.device),
             torch.empty((M, K // G), dtype=torch.uint8, device=x.device),
             torch.ones(1, dtype=torch.float32, device=x.device) if f == FORMATS["nvfp4"] else None)
            for _ in range(P)]
    ws_bytes = P * L.w4a4_quantize_workspace_bytes(f, M, K)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    arr = ctypes.c_void_p * max(P, 1)
    c_arr = arr(*[_ptr(c) for c in cs])
    codes_arr = arr(*[_ptr(o[0]) for o in outs])
    scales_arr = arr(*[_ptr(o[1]) for o in outs])
    t_arr = arr(*[_ptr(o[2]) for o in outs])
    _check(L.w4a4_quantize_act_multi(f, M, K, _ptr(x), P, c_arr, codes_arr, scales_arr,
                                     t_arr if f == FORMATS["nvfp4"] else None, _ptr(workspace),
                                     workspace.numel() if workspace is not None else 0,
                                     _stream(x.device)))
    return outs


def pack_weight(codes: torch.Tensor, scales: torch.Tensor, t_w: Optional[torch.Tensor],
                r: torch.Tensor, fmt) -> torch.Tensor:
    """w4a4_pack_weight: canonical codes [N, K/2] ([N, K] for the 8-bit formats),
    scales, t_w [1] or None, r [N] -> blob."""
    f = _fmt(fmt)
    L = lib()
    N = codes.shape[0]
    K = codes.shape[1] * (1 if code_cols(fmt, 2) == 2 else 2)     # one byte or one nibble per code
    nbytes = L.w4a4_packed_weight_bytes(f, N, K)
    if nbytes == 0:
        raise W4A4Error(2, f"invalid packed weight shape N={N} K={K}")
    G = L.w4a4_block_size(f)
    if codes.dim() != 2 or tuple(scales.shape) != (N, K // G) or r.numel() != N:
        raise W4A4Error(2, f"pack_weight: codes {tuple(codes.shape)}, scales {tuple(scales.shape)} and "
                           f"r {tuple(r.shape)} do not describe one N={N} x K={K} weight")
    blob = torch.empty(nbytes, dtype=torch.uint8, device=codes.device)
    _check(L.w4a4_pack_weight(f, N, K, _ptr(codes), _ptr(scales), _ptr(t_w), _ptr(r), _ptr(blob),
                              _stream(codes.device)))
    return blob


def unpack_weight(blob: torch.Tensor, fmt, N: int, K: int):
    """w4a4_unpack_weight -> (codes [N, K/2], scales [N, K/G], r [N], t_w [1])."""
    f = _fmt(fmt)
    L = lib()
    G = L.w4a4_block_size(f)
    dev = blob.device
    codes = torch.empty((N, code_cols(fmt, K)), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, K // G), dtype=scale_dtype(fmt), device=dev)
    r = torch.empty(N, dtype=torch.float32, device=dev)
    t_w = torch.empty(1, dtype=torch.float32, device=dev)
    _check(L.w4a4_unpack_weight(f, N, K, _ptr(blob), _ptr(codes), _ptr(scales), _ptr(r), _ptr(t_w),
                                _stream(dev)))
    return codes, scales, r, t_w


_LINEAR_WS = {}


def linear_workspace(device, nbytes: int) -> torch.Tensor:
    """A cached, zero-filled linear workspace of `device`, at least `nbytes`
    long (needed by the MXFP4 split-K GEMM; its synchronization words start
    at zero and every call leaves them at zero, so the one buffer serves all
    calls issued in order on one stream)."""
    device = torch.device(device)
    ws = _LINEAR_WS.get(device)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 1), dtype=torch.uint8, device=device)
        _LINEAR_WS[device] = ws
    return ws


def linear(a_codes: torch.Tensor, a_scales: torch.Tensor, t_act: Optional[torch.Tensor],
           blob: torch.Tensor, fmt, N: int, K: int, out: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """w4a4_linear: quantized activations [M, K/2] x packed weight -> bf16 [M, N].

    Without `workspace`, shapes that need one use linear_workspace().
    """
    f = _fmt(fmt)
    L = lib()
    M = a_codes.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a_codes.device)
    ws_bytes = L.w4a4_linear_workspace_bytes(f, M, N, K)
    if ws_bytes and workspace is None:
        workspace = linear_workspace(a_codes.device, ws_bytes)
    _check(L.w4a4_linear(f, M, N, K, _ptr(a_codes), _ptr(a_scales), _ptr(t_act), _ptr(blob),
                         _ptr(out), _ptr(workspace),
                         workspace.numel() if workspace is not None else 0,
                         _stream(a_codes.device)))
    return out


def linear_noalloc(a_codes: torch.Tensor, a_scales: torch.Tensor, t_act: Optional[torch.Tensor],
                   blob: torch.Tensor, fmt, N: int, K: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """w4a4_linear_noalloc: as linear(), with the split-K workspace taken from
    the library's own per-device scratch array (nothing is allocated by the
    library; `out` is allocated here only when not given)."""
    f = _fmt(fmt)
    L = lib()
    M = a_codes.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a_codes.device)
    _check(L.w4a4_linear_noalloc(f, M, N, K, _ptr(a_codes), _ptr(a_scales), _ptr(t_act), _ptr(blob),
                                 _ptr(out), _stream(a_codes.device)))
    return out


def dualquant_solve(w: torch.Tensor, fmt, iters: int = 15, workspace: Optional[torch.Tensor] = None):
    """w4a4_dualquant_solve: fp32 weights [N, K] -> (r [N], c [K], codes [N, K/2],
    scales [N, K/G], t_w [1] for NVFP4 else None).

    The offline dual-scale solver; W ~ diag(r) Q diag(c) (x t_w for NVFP4).
    Without `workspace`, one of w4a4_dualquant_workspace_bytes() bytes is
    allocated here.
    """
    f = _fmt(fmt)
    L = lib()
    N, K = w.shape
    ws_bytes = L.w4a4_dualquant_workspace_bytes(f, N, K)
    if ws_bytes == 0:
        raise W4A4Error(2, f"dualquant_solve: unsupported format or shape N={N} K={K}")
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=w.device)
    r = torch.empty(N, dtype=torch.float32, device=w.device)
    c = torch.empty(K, dtype=torch.float32, device=w.device)
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((N, K // block_size(fmt)), dtype=torch.uint8, device=w.device)
    t_w = torch.ones(1, dtype=torch.float32, device=w.device) if f == FORMATS["nvfp4"] else None
    _check(L.w4a4_dualquant_solve(f, N, K, _ptr(w), int(iters), _ptr(r), _ptr(c), _ptr(codes),
                                  _ptr(scales), _ptr(t_w), _ptr(workspace), workspace.numel(),
                                  _stream(w.device)))
    return r, c, codes, scales, t_w


def linear_grouped(problems, fmt, K: int, outs=None):
    """w4a4_linear_grouped: problems = [(a_codes, a_scales, t_act, blob, N), ...]
    sharing M and K -> list of bf16 [M, N_p] outputs."""
    f = _fmt(fmt)
    L = lib()
    P = len(problems)
    M = problems[0][0].shape[0]
    dev = problems[0][0].device
    if outs is None:
        outs = [torch.empty((M, pr[4]), dtype=torch.bfloat16, device=dev) for pr in problems]
    arr = ctypes.c_void_p * P
    Ns = (ctypes.c_int64 * P)(*[int(pr[4]) for pr in problems])
    _check(L.w4a4_linear_grouped(f, P, M, K, Ns, arr(*[_ptr(pr[0]) for pr in problems]),
                                 arr(*[_ptr(pr[1]) for pr in problems]),
                                 arr(*[_ptr(pr[2]) for pr in problems]) if f == FORMATS["nvfp4"] else None,
                                 arr(*[_ptr(pr[3]) for pr in problems]), arr(*[_ptr(o) for o in outs]),
                                 _stream(dev)))
    return outs


def probe_stream_read(buf: torch.Tensor, sink: torch.Tensor) -> None:
    """w4a4_probe_stream_read: read all of `buf` (contiguous, its byte size a
    multiple of 16) once; `sink` a device buffer of at least 1 KiB."""
    _check(lib().w4a4_probe_stream_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                        _stream(buf.device)))


def probe_mfma_fp4(ops: torch.Tensor, iters: int, workgroups: int, sink: torch.Tensor) -> None:
    """w4a4_probe_mfma_fp4: `iters` rounds of 16 scaled FP4 MFMAs per wave on
    the 16 KiB of operand fragments in `ops`, over `workgroups` workgroups of
    4 waves; `sink` a device buffer of at least 1 KiB."""
    if ops.numel() * ops.element_size() < 16384:
        raise ValueError("probe_mfma_fp4: ops must hold 16 KiB")
    _check(lib().w4a4_probe_mfma_fp4(_ptr(ops), int(iters), int(workgroups), _ptr(sink), _stream(ops.device)))


def probe_empty(device) -> None:
    """w4a4_probe_empty: one empty kernel on the current stream of `device`."""
    _check(lib().w4a4_probe_empty(_stream(torch.device(device))))


# ---------------------------------------------------------------------------
# The paged key-value cache and its attention.  Everywhere:
#
#   k_cache, v_cache  [pages, page_size, heads, head_dim], the last dimension
#                     contiguous, the others in any order in memory (the same
#                     for both); bfloat16, float16 or float8_e4m3fn; or uint8, a
#                     cache in 4 bits: [pages, page_size, heads, head_dim * 17 / 32]
#                     bytes, pages laid out as W4A4_E2M1 says (see kv_cache_e2m1)
#   k_scale, v_scale  fp32 [heads] or None (1): a stored E4M3 value stands for
#                     value * scale
#   tables            int32 [seqs, max_pages]: page of the tokens page_size * j ..
#   lens              int32 [seqs]: tokens of each sequence, new ones included
#   refs              int32 [pages]: sequences on each page, 0 for a free one
#   caches            tensors of pages [..., pages, page_size, heads, head_dim], or
#                     one such tensor (leading dimensions: layers, K and V)

_KV_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2, torch.uint8: 4}


def _kv_type(t: torch.Tensor, what: str) -> int:
    f = _KV_TYPES.get(t.dtype)
    if f is None:
        raise W4A4Error(4, f"{what}: type {t.dtype} (bfloat16, float16, or of a cache float8_e4m3fn or uint8)")
    return f


_I32 = torch.int32


# `device` of the helpers below: a GPU's index, -1 for tensors elsewhere (get_device(), cheaper than
# comparing torch.device objects; _on_gpu refuses -1 before any call).

def _on(device: int) -> str:
    return "the cache's device" if device < 0 else f"cuda:{device}"


def _int32(what: str, device: int, *tensors) -> None:
    for t in tensors:
        if t is not None and (t.dtype is not _I32 or t.get_device() != device or not t.is_contiguous()):
            raise W4A4Error(2, f"{what}: index tensors are int32, on {_on(device)}, with contiguous entries")


def _c_ints(what: str, *numbers) -> None:
    """Refuses what a C int would cut to its low 32 bits."""
    for x in numbers:
        if not -2 ** 31 <= x < 2 ** 31:
            raise W4A4Error(2, f"{what}: {x} does not fit 32 bits")


def _kv_cache(what: str, k: torch.Tensor, v: torch.Tensor, k_scale, v_scale) -> Tuple[bytes, int, int, int, int]:
    """(w4a4_kv_cache packed, type, page_size, heads, head_dim)"""
    shape, stride, dtype = k.shape, k.stride(), k.dtype
    if len(shape) != 4 or shape != v.shape or stride != v.stride() or stride[3] != 1 or dtype != v.dtype or \
            k.get_device() != v.get_device():
        raise W4A4Error(2, f"{what}: caches {tuple(k.shape)} and {tuple(v.shape)} must be alike, [pages, page_size, "
                           "heads, head_dim] with a contiguous last dimension")
    f = _KV_TYPES.get(dtype)
    if f is None:
        _kv_type(k, what)
    ks = vs = 0
    if f == 2:
        for t in (k_scale, v_scale):
            if t is not None and (t.dtype != torch.float32 or t.numel() != shape[2] or not t.is_contiguous() or
                                  t.get_device() != k.get_device()):
                raise W4A4Error(2, f"{what}: scales are contiguous float32 [heads] on the cache's device")
        ks, vs = (0 if t is None else t.data_ptr() for t in (k_scale, v_scale))
    elif k_scale is not None or v_scale is not None:
        raise W4A4Error(4, f"{what}: scales belong to a float8_e4m3fn cache")
    pages, page, heads, dim = shape
    if f == 4:
        size = page * heads * dim
        if dim % 17 or (heads > 1 and stride[2] != dim) or (page > 1 and stride[1] != heads * dim):
            raise W4A4Error(2, f"{what}: a 4-bit cache is [pages, page_size, heads, head_dim * 17 / 32] bytes, each page "
                               f"contiguous, not {tuple(shape)} with strides {tuple(stride)}")
        dim = dim // 17 * 32
        at = (0, 0, stride[0] if pages > 1 else -(-size // 16) * 16, 0, 0)
    else:
        at = (ks, vs, *stride[:3])
    try:
        return _PACK_CACHE(k.data_ptr(), v.data_ptr(), *at, f, pages, page, heads, dim), f, page, heads, dim
    except (struct.error, OverflowError) as e:
        raise _unfit(what, e) from None


def _kv_seqs(what: str, tables: torch.Tensor, lens: Optional[torch.Tensor], device: int) -> Tuple[bytes, int]:
    """(w4a4_kv_seqs packed, their number)"""
    shape, stride = tables.shape, tables.stride()
    if len(shape) != 2 or (shape[1] > 1 and stride[1] != 1) or tables.dtype is not _I32 or \
            tables.get_device() != device or (lens is not None and (lens.dim() != 1 or lens.shape[0] != shape[0])):
        raise W4A4Error(2, f"{what}: tables {tuple(tables.shape)} must be int32 [seqs, max_pages] on {_on(device)} with "
                           "contiguous rows, lens [seqs]")
    if lens is not None and (lens.dtype is not _I32 or lens.get_device() != device or not lens.is_contiguous()):
        _int32(what, device, lens)
    seqs, width = shape
    try:
        return _PACK_SEQS(tables.data_ptr(), 0 if lens is None else lens.data_ptr(), stride[0] if seqs > 1 else width, seqs,
                          width), seqs
    except (struct.error, OverflowError) as e:
        raise _unfit(what, e) from None


def _kv_rows(what: str, x: torch.Tensor, rows: int, heads, dim: int, device: int) -> Tuple[int, int, int]:
    """(address, row stride, head stride) of rows x [rows, heads, dim]; heads None: any number."""
    shape, stride = x.shape, x.stride()
    if len(shape) != 3 or shape[0] != rows or shape[2] != dim or (heads is not None and shape[1] != heads) or \
            stride[2] != 1 or x.get_device() != device:
        raise W4A4Error(2, f"{what}: {tuple(x.shape)} (need [{rows}, {'heads' if heads is None else heads}, {dim}] with a "
                           f"contiguous last dimension, on {_on(device)})")
    return x.data_ptr(), stride[0], stride[1]


def _on_gpu(device: int) -> None:
    if device < 0:
        raise W4A4Error(2, "the cache and everything with it must be on a GPU")


def _kv_call(device: int, entry, *args) -> None:
    """entry(*args, the current stream of GPU `device`), with that as the current device: launches go there."""
    _on_gpu(device)
    if torch._C._cuda_getDevice() != device:
        with torch.cuda.device(device):
            status = entry(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        status = entry(*args, torch._C._cuda_getCurrentRawStream(device))
    if status:
        _check(status)


@functools.lru_cache(maxsize=4096)
def _attn_workspace_bytes(prefill: bool, dtype: int, page: int, heads: int, dim: int, seqs: int, tokens: int,
                          q_heads: int) -> int:
    """w4a4_attn_*_workspace_bytes: depends on these numbers alone."""
    stride = lib().w4a4_kv_page_bytes(page, heads, dim) + 15 & ~15 if dtype == 4 else 0
    c = _KvCache(16, 16, None, None, stride, 0, 0, dtype, 1, page, heads, dim)
    return (lib().w4a4_attn_prefill_workspace_bytes(c, seqs, tokens, q_heads) if prefill else
            lib().w4a4_attn_decode_workspace_bytes(c, seqs, q_heads))


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, tables: torch.Tensor,
              lens: torch.Tensor, *, cu_seqlens: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
              v_scale: Optional[torch.Tensor] = None) -> None:
    """w4a4_kv_append: store new keys and values [tokens, heads, head_dim] (any
    row and head strides) at the ends of their sequences.

    cu_seqlens int32 [seqs + 1]: sequence s has the rows cu[s] .. cu[s + 1] - 1,
    its last tokens; None: one row per sequence.
    """
    dev = k_cache.get_device()
    c, _, _, heads, dim = _kv_cache("kv_append", k_cache, v_cache, k_scale, v_scale)
    s, seqs = _kv_seqs("kv_append", tables, lens, dev)
    tokens = k.shape[0]
    rows = (*_kv_rows("kv_append: k", k, tokens, heads, dim, dev), *_kv_rows("kv_append: v", v, tokens, heads, dim, dev))
    if k.dtype != v.dtype:
        raise W4A4Error(4, f"kv_append: k is {k.dtype}, v is {v.dtype}")
    cu = None if cu_seqlens is None else _cu("kv_append", cu_seqlens, seqs, dev)
    _kv_call(dev, _kv_lib().w4a4_kv_append, c, s, cu, tokens, _kv_type(k, "kv_append"), *rows)


def kv_cache_e2m1(pages, page_size: int, heads: int, head_dim: int, device="cuda") -> torch.Tensor:
    """An empty 4-bit cache, uint8 [*pages, page_size, heads, head_dim * 17 / 32]; pages: their number, or a
    shape that ends with it, e.g. (layers, 2, pages) for K and V of all layers.  Pages
    begin at multiples of 16 bytes, so they may have gaps between them."""
    lead = (pages,) if isinstance(pages, int) else tuple(pages)
    size = lib().w4a4_kv_page_bytes(page_size, heads, head_dim)
    if size == 0:
        raise W4A4Error(2, f"kv_cache_e2m1: page_size={page_size} heads={heads} head_dim={head_dim}")
    store = torch.zeros((*lead, -(-size // 16) * 16), dtype=torch.uint8, device=device)
    width = head_dim // 32 * 17
    return store.as_strided((*lead, page_size, heads, width), (*store.stride()[:-1], heads * width, width, 1))


def rope_freqs(rot_dim: int, base: float = 10000.0, *, scaling: str = "none", scale: float = 1.0,
               original: int = 0, low: float = 1.0, high: float = 4.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
               device="cuda"):
    """(freqs float32 [rot_dim / 2], factor) of rotary positions: base^(-2 i / rot_dim) radians per position, and

    scaling "linear"  freqs / scale: positions compressed by `scale`
            "ntk"     base * scale^(rot_dim / (rot_dim - 2)): the slowest pair is stretched by `scale`, the
                      fastest not at all
            "bands"   by the turns that a pair makes over `original` positions: more than `high` as they are,
                      fewer than `low` divided by `scale`, between them a linear blend of the two
            "yarn"    between the pairs that make beta_fast and beta_slow turns over `original` positions a
                      linear ramp (over the pairs' numbers) from as they are to divided by `scale`; factor
                      0.1 ln(scale) + 1
    """
    if rot_dim < 2 or rot_dim % 2 or not base > 0 or not scale > 0:
        raise W4A4Error(2, f"rope_freqs: rot_dim={rot_dim} base={base} scale={scale}")
    if scaling in ("bands", "yarn") and original < 1:
        raise W4A4Error(2, f"rope_freqs: {scaling} needs the original number of positions, not {original}")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    if scaling == "ntk":
        if rot_dim < 4:
            raise W4A4Error(2, "rope_freqs: ntk needs two pairs")
        base = base * scale ** (rot_dim / (rot_dim - 2))
    f, factor = base ** (-i / rot_dim), 1.0
    if scaling == "linear":
        f = f / scale
    elif scaling == "bands":
        if not high > low:
            raise W4A4Error(2, f"rope_freqs: bands from {low} to {high} turns")
        keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / scale * (1 - keep)
    elif scaling == "yarn":
        if not beta_fast > beta_slow > 0 or not base > 1:
            raise W4A4Error(2, f"rope_freqs: beta_fast={beta_fast} beta_slow={beta_slow} base={base}")
        # the pair (as a real number) that makes n turns over the original positions
        at = [rot_dim * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (beta_fast, beta_slow)]
        first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot_dim - 1)
        ramp = ((i / 2 - first) / max(last - first, 1e-3)).clamp(0, 1)
        f, factor = f * (1 - ramp) + f / scale * ramp, 0.1 * math.log(scale) + 1.0 if scale > 1 else 1.0
    elif scaling not in ("none", "ntk"):
        raise W4A4Error(2, f"rope_freqs: scaling {scaling!r} (none, linear, ntk, bands or yarn)")
    return f.to(torch.float32).to(device), factor


def _rotation(what: str, freqs: torch.Tensor, interleaved, inverse, factor, device: int) -> bytes:
    if freqs.dtype is not torch.float32 or freqs.dim() != 1 or not freqs.is_contiguous() or freqs.get_device() != device:
        raise W4A4Error(2, f"{what}: freqs are contiguous float32 [rot_dim / 2] on {_on(device)}")
    try:
        return _PACK_ROTATION(freqs.data_ptr(), 2 * freqs.shape[0], bool(interleaved), bool(inverse), factor)
    except (struct.error, OverflowError) as e:
        raise _unfit(what, e) from None


def _positions(what: str, positions: Optional[torch.Tensor], tokens: int, device: int) -> Optional[int]:
    if positions is None:
        return None
    _int32(what, device, positions)
    if positions.numel() != tokens:
        raise W4A4Error(2, f"{what}: {positions.numel()} positions for {tokens} rows")
    return positions.data_ptr()


def _like_rows(what: str, out: Optional[torch.Tensor], x: torch.Tensor) -> torch.Tensor:
    if out is None:
        return x.new_empty(x.shape)
    if out.dtype != x.dtype:
        raise W4A4Error(4, f"{what} is {out.dtype}, its input {x.dtype}")
    return out


def rope(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, *, interleaved: bool = False,
         factor: float = 1.0, inverse: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """w4a4_rope: rows x [tokens, heads, head_dim] (any row and head strides) rotated by their positions
    (int32 [tokens]) over their first 2 * len(freqs) values; freqs and factor as from
    rope_freqs.  interleaved: pairs (2i, 2i + 1) instead of halves.  inverse: back, or a
    gradient.  out: x itself (in place), or other memory."""
    dev = x.get_device()
    r = _rotation("rope", freqs, interleaved, inverse, factor, dev)
    if x.dim() != 3:
        raise W4A4Error(2, f"rope: x {tuple(x.shape)} (need [tokens, heads, head_dim])")
    tokens, heads, dim = x.shape
    at = _positions("rope", positions, tokens, dev)
    out = _like_rows("rope: out", out, x)
    rows = (*_kv_rows("rope: x", x, tokens, None, dim, dev), *_kv_rows("rope: out", out, tokens, heads, dim, dev))
    _kv_call(dev, _kv_lib().w4a4_rope, r, tokens, at, _kv_type(x, "rope"), heads, dim, *rows)
    return out


def kv_append_rope(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, tables: torch.Tensor, lens: torch.Tensor, freqs: torch.Tensor, *,
                   cu_seqlens: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                   interleaved: bool = False, factor: float = 1.0, k_scale: Optional[torch.Tensor] = None,
                   v_scale: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None):
    """w4a4_kv_append_rope: kv_append of keys rotated as by rope(), with the queries [tokens, q_heads,
    head_dim] (or None) rotated into the result, q_out or a new tensor.

    positions int32 [tokens]: what is rotated by; None: the tokens' places in their sequences.
    """
    name, dev = "kv_append_rope", k_cache.get_device()
    c, _, _, kv_heads, dim = _kv_cache(name, k_cache, v_cache, k_scale, v_scale)
    s, seqs = _kv_seqs(name, tables, lens, dev)
    r = _rotation(name, freqs, interleaved, False, factor, dev)
    tokens = k.shape[0]
    rows = (*_kv_rows("kv_append_rope: k", k, tokens, kv_heads, dim, dev), *_kv_rows("kv_append_rope: v", v, tokens, kv_heads, dim, dev))
    if k.dtype != v.dtype or (q is not None and q.dtype != k.dtype):
        raise W4A4Error(4, f"{name}: k is {k.dtype}, v is {v.dtype}{'' if q is None else f', q is {q.dtype}'}")
    at = _positions(name, positions, tokens, dev)
    cu = None if cu_seqlens is None else _cu(name, cu_seqlens, seqs, dev)
    q_rows, heads, out = (None, 0, 0, None, 0, 0), 0, None
    if q is not None:
        q_at = _kv_rows(name + ": q", q, tokens, None, dim, dev)
        heads, out = q.shape[1], _like_rows(name + ": q_out", q_out, q)
        q_rows = (*q_at, *_kv_rows(name + ": q_out", out, tokens, heads, dim, dev))
    elif q_out is not None:
        raise W4A4Error(2, f"{name}: q_out without q")
    _kv_call(dev, _kv_lib().w4a4_kv_append_rope, c, s, cu, tokens, _kv_type(k, name), r, at, heads, *q_rows, *rows)
    return out


def kv_read(k_cache: torch.Tensor, v_cache: torch.Tensor, tables: torch.Tensor, lens: torch.Tensor,
            cu_seqlens: Optional[torch.Tensor], tokens: int, *, dtype: torch.dtype = torch.bfloat16,
            k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None, out=None):
    """w4a4_kv_read: (k, v) [tokens, heads, head_dim] of `dtype`: the rows that kv_append with the same
    cu_seqlens (tokens: its last entry; None: one row per sequence) stores, as the
    cache holds them.  out: (k, v) to write into; otherwise the two are halves of one allocation."""
    name, dev = "kv_read", k_cache.get_device()
    c, _, _, heads, dim = _kv_cache(name, k_cache, v_cache, k_scale, v_scale)
    s, seqs = _kv_seqs(name, tables, lens, dev)
    cu = None if cu_seqlens is None else _cu(name, cu_seqlens, seqs, dev)
    if tokens < 0:
        raise W4A4Error(2, f"{name}: {tokens} tokens")
    if out is None:
        out = torch.empty((2, tokens, heads, dim), dtype=dtype, device=k_cache.device).unbind()
    k, v = out
    if k.dtype != dtype or v.dtype != dtype:
        raise W4A4Error(4, f"{name}: out is {k.dtype} and {v.dtype}, not {dtype}")
    rows = (*_kv_rows("kv_read: k", k, tokens, heads, dim, dev), *_kv_rows("kv_read: v", v, tokens, heads, dim, dev))
    _kv_call(dev, _kv_lib().w4a4_kv_read, c, s, cu, tokens, _kv_type(k, name), *rows)
    return k, v


def _cu(what: str, cu: torch.Tensor, seqs: int, device: int) -> int:
    _int32(what, device, cu)
    if cu.numel() != seqs + 1:
        raise W4A4Error(2, f"{what}: cu_seqlens has {cu.numel()} entries for {seqs} sequences")
    return cu.data_ptr()


def _attn(name: str, q, cu, k_cache, v_cache, tables, lens, k_scale, v_scale, scale, window, sinks, out, return_lse,
          workspace):
    dev = k_cache.get_device()
    _c_ints(name, window, sinks)
    c, f, page, heads, dim = _kv_cache(name, k_cache, v_cache, k_scale, v_scale)
    s, seqs = _kv_seqs(name, tables, lens, dev)
    rows, q_heads = q.shape[0], q.shape[1]
    q_at = _kv_rows(name + ": q", q, seqs if cu is None else rows, None, dim, dev)
    if cu is not None:
        _cu(name, cu, seqs, dev)
    if out is None:
        out = q.new_empty((rows, q_heads, dim))
        out_at = (out.data_ptr(), q_heads * dim, dim)
    else:
        out_at = _kv_rows(name + ": out", out, rows, q_heads, dim, dev)
        if out.dtype != q.dtype:
            raise W4A4Error(4, f"{name}: out is {out.dtype}, q is {q.dtype}")
    lse = torch.empty((rows, q_heads), dtype=torch.float32, device=k_cache.device) if return_lse else None
    if workspace is None:
        size = _attn_workspace_bytes(cu is not None, f, page, heads, dim, seqs, rows, q_heads)
        if size:
            workspace = torch.empty(size, dtype=torch.uint8, device=k_cache.device)
    else:
        if workspace.device != k_cache.device or not workspace.is_contiguous():
            raise W4A4Error(2, f"{name}: the workspace must be contiguous, on {_on(dev)}")
        size = workspace.numel() * workspace.element_size()
    tail = (_kv_type(q, name), q_heads, *q_at, dim ** -0.5 if scale is None else scale, window, sinks, *out_at,
            None if lse is None else lse.data_ptr(), None if workspace is None else workspace.data_ptr(), size)
    if cu is None:
        _kv_call(dev, _kv_lib().w4a4_attn_decode, c, s, *tail)
    else:
        _kv_call(dev, _kv_lib().w4a4_attn_prefill, c, s, cu.data_ptr(), rows, *tail)
    return (out, lse) if return_lse else out


def attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, tables: torch.Tensor,
                lens: torch.Tensor, *, k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                scale: Optional[float] = None, window: int = 0, sinks: int = 0, out: Optional[torch.Tensor] = None,
                return_lse: bool = False, workspace: Optional[torch.Tensor] = None):
    """w4a4_attn_decode: one new token per sequence, q [seqs, q_heads, head_dim]
    -> out of the same shape and type (and lse fp32 [seqs, q_heads]).

    scale None: 1 / sqrt(head_dim).  window 0: every token is seen; otherwise
    the last `window` ones and the first `sinks`.
    """
    return _attn("attn_decode", q, None, k_cache, v_cache, tables, lens, k_scale, v_scale, scale, window, sinks, out,
                 return_lse, workspace)


def attn_prefill(q: torch.Tensor, cu_seqlens: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 tables: torch.Tensor, lens: torch.Tensor, *, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None, scale: Optional[float] = None, window: int = 0,
                 sinks: int = 0, out: Optional[torch.Tensor] = None, return_lse: bool = False,
                 workspace: Optional[torch.Tensor] = None):
    """w4a4_attn_prefill: the new tokens of every sequence, q [tokens, q_heads,
    head_dim], sequence s in the rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1, already
    stored in the cache; causal, with window and sinks as in attn_decode."""
    return _attn("attn_prefill", q, cu_seqlens, k_cache, v_cache, tables, lens, k_scale, v_scale, scale, window, sinks,
                 out, return_lse, workspace)


def _kv_page_layout(what: str, t: torch.Tensor):
    """(shape of pages, page stride in bytes, page bytes) of [..., pages, page_size, heads, head_dim]."""
    if t.dim() < 4:
        raise W4A4Error(2, f"{what}: a cache is [..., pages, page_size, heads, head_dim], got {tuple(t.shape)}")
    elt, size, stride = t.element_size(), t.shape[-4:], t.stride()[-4:]
    dense = 1
    for st, n in sorted(zip(stride[1:], size[1:])):
        if n > 1:
            if st != dense:
                raise W4A4Error(2, f"{what}: a page's {tuple(size[1:])} values must lie densely in memory")
            dense *= n
    return size, stride[0] * elt if size[0] > 1 else dense * elt, dense * elt


def _kv_arrays(what: str, caches):
    """(n, host array of base pointers, page stride, page bytes, pages, page_size, device)."""
    ptrs, first, dev = [], None, None
    for t in ((caches,) if isinstance(caches, torch.Tensor) else caches):
        layout = _kv_page_layout(what, t)
        if first is None:
            first, dev = layout, t.get_device()
        elif layout != first or t.get_device() != dev:
            raise W4A4Error(2, f"{what}: the caches must be alike")
        at, elt = [t.data_ptr()], t.element_size()
        for n, st in zip(t.shape[:-4], t.stride()[:-4]):
            at = [x + y for x in at for y in range(0, n * st * elt, st * elt)] if n > 1 and st > 0 else at * n
        ptrs += at
    if first is None:
        raise W4A4Error(2, f"{what}: no caches")
    size, stride, dense = first
    return len(ptrs), (ctypes.c_void_p * max(len(ptrs), 1))(*ptrs), stride, dense, size[0], size[1], dev


@functools.lru_cache(maxsize=4096)
def _kv_workspace_bytes(rows: int, pages: int) -> int:
    return lib().w4a4_kv_workspace_bytes(rows, pages)


def _kv_workspace(rows: int, pages: int, device: int) -> torch.Tensor:
    _on_gpu(device)
    return torch.empty(_kv_workspace_bytes(rows, pages), dtype=torch.uint8, device=device)


def _same_length(what: str, a: torch.Tensor, b: torch.Tensor) -> int:
    if a.dim() != 1 or a.shape != b.shape:
        raise W4A4Error(2, f"{what}: lists of {tuple(a.shape)} and {tuple(b.shape)} entries")
    return a.numel()


def kv_copy_pages(caches, src: torch.Tensor, dst: torch.Tensor) -> None:
    """w4a4_kv_copy_pages: page src[i] to page dst[i] (int32) in every cache."""
    n, arrays, stride, size, pages, _, dev = _kv_arrays("kv_copy_pages", caches)
    _int32("kv_copy_pages", dev, src, dst)
    pairs = _same_length("kv_copy_pages", src, dst)
    _kv_call(dev, lib().w4a4_kv_copy_pages, n, arrays, stride, size, pages, src.data_ptr(), dst.data_ptr(), pairs)


def kv_reserve(tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_size: int, *,
               lacking: Optional[torch.Tensor] = None) -> None:
    """w4a4_kv_reserve: pages for lens[s] tokens of every sequence, the lowest
    free ones first; lacking int32 [1]: the number that was not to be had."""
    _c_ints("kv_reserve", page_size)
    dev = refs.get_device()
    s, seqs = _kv_seqs("kv_reserve", tables, lens, dev)
    _int32("kv_reserve", dev, refs, lacking)
    ws = _kv_workspace(seqs, refs.numel(), dev)
    _kv_call(dev, _kv_lib().w4a4_kv_reserve, s, page_size, refs.data_ptr(), refs.numel(),
             None if lacking is None else lacking.data_ptr(), ws.data_ptr(), ws.numel())


def _check_pages(what: str, refs: torch.Tensor, pages: int) -> None:
    if refs.numel() != pages:
        raise W4A4Error(2, f"{what}: refs has {refs.numel()} entries for {pages} pages")


def kv_fork(caches, tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, parents: torch.Tensor,
            children: torch.Tensor, *, lacking: Optional[torch.Tensor] = None) -> None:
    """w4a4_kv_fork: sequence children[i] becomes a copy of parents[i] (int32):
    whole pages shared, a last page that is not full copied in every cache."""
    n, arrays, stride, size, pages, page, dev = _kv_arrays("kv_fork", caches)
    s, _ = _kv_seqs("kv_fork", tables, lens, dev)
    _int32("kv_fork", dev, refs, parents, children, lacking)
    _check_pages("kv_fork", refs, pages)
    count = _same_length("kv_fork", parents, children)
    ws = _kv_workspace(count, pages, dev)
    _kv_call(dev, _kv_lib().w4a4_kv_fork, n, arrays, stride, size, s, page, refs.data_ptr(), pages, parents.data_ptr(),
             children.data_ptr(), count, None if lacking is None else lacking.data_ptr(), ws.data_ptr(), ws.numel())


def kv_free(tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, seqs: Optional[torch.Tensor] = None) -> None:
    """w4a4_kv_free: let go of all pages of the sequences `seqs` (int32; None: all)."""
    s, all_seqs = _kv_seqs("kv_free", tables, lens, refs.get_device())
    _int32("kv_free", refs.get_device(), refs, seqs)
    _kv_call(refs.get_device(), _kv_lib().w4a4_kv_free, s, refs.data_ptr(), refs.numel(),
             None if seqs is None else seqs.data_ptr(), all_seqs if seqs is None else seqs.numel())


def kv_trim(tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_size: int, window: int, sinks: int = 0,
            seqs: Optional[torch.Tensor] = None) -> None:
    """w4a4_kv_trim: let go of the pages that no later token of the sequences
    `seqs` (None: all) sees under a window with sinks."""
    _c_ints("kv_trim", page_size, window, sinks)
    s, all_seqs = _kv_seqs("kv_trim", tables, lens, refs.get_device())
    _int32("kv_trim", refs.get_device(), refs, seqs)
    _kv_call(refs.get_device(), _kv_lib().w4a4_kv_trim, s, page_size, refs.data_ptr(), refs.numel(),
             None if seqs is None else seqs.data_ptr(), all_seqs if seqs is None else seqs.numel(), window, sinks)


def kv_compact(caches, tables: torch.Tensor, refs: torch.Tensor) -> torch.Tensor:
    """w4a4_kv_compact: move the pages in use to the front, in every cache, with
    tables and refs; returns remap int32 [pages]: new index, -1 for free pages."""
    n, arrays, stride, size, pages, _, dev = _kv_arrays("kv_compact", caches)
    s, _ = _kv_seqs("kv_compact", tables, None, dev)
    _int32("kv_compact", dev, refs)
    _check_pages("kv_compact", refs, pages)
    _on_gpu(dev)
    remap = torch.empty(pages, dtype=torch.int32, device=dev)
    ws = _kv_workspace(0, pages, dev)
    _kv_call(dev, _kv_lib().w4a4_kv_compact, n, arrays, stride, size, s, refs.data_ptr(), pages, remap.data_ptr(),
             ws.data_ptr(), ws.numel())
    return remap
