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

    kv_append(k, v, k_cache, v_cache, tables, lens)
    out = attn_decode(q, k_cache, v_cache, tables, lens)

There is no fallback: if the library is missing or fails to load, the
functions raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

__all__ = ["FORMATS", "lib", "library_path", "block_size", "scale_dtype", "quantize_act", "pack_weight",
           "unpack_weight", "linear", "linear_noalloc", "linear_workspace", "packed_weight_bytes", "W4A4Error",
           "attn_decode", "attn_prefill", "kv_append", "kv_copy_pages", "kv_reserve", "kv_fork", "kv_free", "kv_trim",
           "kv_compact"]

FORMATS = {"mxfp4": 0, "nvfp4": 1, "mxint4": 2, "int4g64": 3, "mxfp8": 4, "mxint8": 5, "int8g128": 6}
_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None


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
    cp, sp, f32 = ctypes.POINTER(_KvCache), ctypes.POINTER(_KvSeqs), ctypes.c_float
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
    for name in ("kv_append", "attn_decode", "attn_prefill", "kv_copy_pages", "kv_reserve", "kv_fork", "kv_free",
                 "kv_trim", "kv_compact"):
        getattr(L, "w4a4_" + name).restype = i32
    L.w4a4_last_error.argtypes = []
    L.w4a4_last_error.restype = ctypes.c_char_p
    L.w4a4_version.argtypes = []
    L.w4a4_version.restype = ctypes.c_char_p
    _LIB = L
    return L


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
#                     for both); bfloat16, float16 or float8_e4m3fn
#   k_scale, v_scale  fp32 [heads] or None (1): a stored E4M3 value stands for
#                     value * scale
#   tables            int32 [seqs, max_pages]: page of the tokens page_size * j ..
#   lens              int32 [seqs]: tokens of each sequence, new ones included
#   refs              int32 [pages]: sequences on each page, 0 for a free one
#   caches            tensors of pages [..., pages, page_size, heads, head_dim], or
#                     one such tensor (leading dimensions: layers, K and V)

_KV_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}


def _kv_type(t: torch.Tensor, what: str) -> int:
    f = _KV_TYPES.get(t.dtype)
    if f is None:
        raise W4A4Error(4, f"{what}: type {t.dtype} (bfloat16, float16 or float8_e4m3fn)")
    return f


def _int32(what: str, device, *tensors) -> None:
    for t in tensors:
        if t is not None and (t.dtype != torch.int32 or t.device != device or not t.is_contiguous()):
            raise W4A4Error(2, f"{what}: index tensors are int32, on {device}, with contiguous entries")


def _c_ints(what: str, *numbers) -> None:
    """Refuses what a C int would cut to its low 32 bits."""
    for x in numbers:
        if not -2 ** 31 <= x < 2 ** 31:
            raise W4A4Error(2, f"{what}: {x} does not fit 32 bits")


def _kv_cache(what: str, k: torch.Tensor, v: torch.Tensor, k_scale, v_scale) -> _KvCache:
    shape, stride = k.shape, k.stride()
    if len(shape) != 4 or shape != v.shape or stride != v.stride() or stride[3] != 1 or k.dtype != v.dtype or \
            k.device != v.device:
        raise W4A4Error(2, f"{what}: caches {tuple(k.shape)} and {tuple(v.shape)} must be alike, [pages, page_size, "
                           "heads, head_dim] with a contiguous last dimension")
    f = _kv_type(k, what)
    ks = vs = None
    if f == 2:
        for t in (k_scale, v_scale):
            if t is not None and (t.dtype != torch.float32 or t.numel() != shape[2] or not t.is_contiguous() or
                                  t.device != k.device):
                raise W4A4Error(2, f"{what}: scales are contiguous float32 [heads] on the cache's device")
        ks, vs = (None if t is None else t.data_ptr() for t in (k_scale, v_scale))
    elif k_scale is not None or v_scale is not None:
        raise W4A4Error(4, f"{what}: scales belong to a float8_e4m3fn cache")
    pages, page, heads, dim = shape
    return _KvCache(k.data_ptr(), v.data_ptr(), ks, vs, stride[0], stride[1], stride[2], f, pages, page, heads, dim)


def _kv_seqs(what: str, tables: torch.Tensor, lens: Optional[torch.Tensor], device) -> _KvSeqs:
    shape = tables.shape
    if len(shape) != 2 or (shape[1] > 1 and tables.stride(1) != 1) or tables.dtype != torch.int32 or \
            tables.device != device or (lens is not None and (lens.dim() != 1 or lens.shape[0] != shape[0])):
        raise W4A4Error(2, f"{what}: tables {tuple(tables.shape)} must be int32 [seqs, max_pages] on {device} with "
                           "contiguous rows, lens [seqs]")
    _int32(what, device, lens)
    seqs, width = shape
    return _KvSeqs(tables.data_ptr(), None if lens is None else lens.data_ptr(),
                   tables.stride(0) if seqs > 1 else width, seqs, width)


def _kv_rows(what: str, x: torch.Tensor, rows: int, heads, dim: int, device) -> Tuple[int, int, int]:
    """(address, row stride, head stride) of rows x [rows, heads, dim]; heads None: any number."""
    shape, stride = x.shape, x.stride()
    if len(shape) != 3 or shape[0] != rows or shape[2] != dim or (heads is not None and shape[1] != heads) or \
            stride[2] != 1 or x.device != device:
        raise W4A4Error(2, f"{what}: {tuple(x.shape)} (need [{rows}, {'heads' if heads is None else heads}, {dim}] with a "
                           f"contiguous last dimension, on {device})")
    return x.data_ptr(), stride[0], stride[1]


def _kv_stream(device: torch.device) -> int:
    """Handle of the current stream of `device`, which has to be a GPU (_stream without the torch.cuda.Stream object)."""
    if device.type != "cuda":
        raise W4A4Error(2, f"the cache and everything with it must be on a GPU, not on {device}")
    return torch._C._cuda_getCurrentRawStream(device.index)


@functools.lru_cache(maxsize=4096)
def _attn_workspace_bytes(prefill: bool, dtype: int, page: int, heads: int, dim: int, seqs: int, tokens: int,
                          q_heads: int) -> int:
    """w4a4_attn_*_workspace_bytes: depends on these numbers alone."""
    c = _KvCache(16, 16, None, None, 0, 0, 0, dtype, 1, page, heads, dim)
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
    dev = k_cache.device
    c = _kv_cache("kv_append", k_cache, v_cache, k_scale, v_scale)
    s = _kv_seqs("kv_append", tables, lens, dev)
    tokens = k.shape[0]
    rows = (*_kv_rows("kv_append: k", k, tokens, c.heads, c.head_dim, dev),
            *_kv_rows("kv_append: v", v, tokens, c.heads, c.head_dim, dev))
    if k.dtype != v.dtype:
        raise W4A4Error(4, f"kv_append: k is {k.dtype}, v is {v.dtype}")
    cu = None
    if cu_seqlens is not None:
        _int32("kv_append", dev, cu_seqlens)
        if cu_seqlens.numel() != s.seqs + 1:
            raise W4A4Error(2, f"kv_append: cu_seqlens has {cu_seqlens.numel()} entries for {s.seqs} sequences")
        cu = cu_seqlens.data_ptr()
    _check(lib().w4a4_kv_append(c, s, cu, tokens, _kv_type(k, "kv_append"), *rows, _kv_stream(dev)))


def _attn(name: str, q, cu, k_cache, v_cache, tables, lens, k_scale, v_scale, scale, window, sinks, out, return_lse,
          workspace):
    dev = k_cache.device
    _c_ints(name, window, sinks)
    c = _kv_cache(name, k_cache, v_cache, k_scale, v_scale)
    s = _kv_seqs(name, tables, lens, dev)
    rows, q_heads, dim = q.shape[0], q.shape[1], c.head_dim
    q_at = _kv_rows(name + ": q", q, s.seqs if cu is None else rows, None, dim, dev)
    if cu is not None:
        _int32(name, dev, cu)
        if cu.numel() != s.seqs + 1:
            raise W4A4Error(2, f"{name}: cu_seqlens has {cu.numel()} entries for {s.seqs} sequences")
    if out is None:
        out = torch.empty((rows, q_heads, dim), dtype=q.dtype, device=dev)
        out_at = (out.data_ptr(), q_heads * dim, dim)
    else:
        out_at = _kv_rows(name + ": out", out, rows, q_heads, dim, dev)
        if out.dtype != q.dtype:
            raise W4A4Error(4, f"{name}: out is {out.dtype}, q is {q.dtype}")
    lse = torch.empty((rows, q_heads), dtype=torch.float32, device=dev) if return_lse else None
    if workspace is None:
        size = _attn_workspace_bytes(cu is not None, c.dtype, c.page_size, c.heads, dim, s.seqs, rows, q_heads)
        if size:
            workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    else:
        if workspace.device != dev or not workspace.is_contiguous():
            raise W4A4Error(2, f"{name}: the workspace must be contiguous, on {dev}")
        size = workspace.numel() * workspace.element_size()
    tail = (_kv_type(q, name), q_heads, *q_at, dim ** -0.5 if scale is None else scale, window, sinks, *out_at,
            None if lse is None else lse.data_ptr(), None if workspace is None else workspace.data_ptr(), size,
            _kv_stream(dev))
    L = lib()
    _check(L.w4a4_attn_decode(c, s, *tail) if cu is None else L.w4a4_attn_prefill(c, s, cu.data_ptr(), rows, *tail))
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
            first, dev = layout, t.device
        elif layout != first or t.device != dev:
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


def _kv_workspace(rows: int, pages: int, device) -> torch.Tensor:
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
    _check(lib().w4a4_kv_copy_pages(n, arrays, stride, size, pages, src.data_ptr(), dst.data_ptr(), pairs, _kv_stream(dev)))


def kv_reserve(tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_size: int, *,
               lacking: Optional[torch.Tensor] = None) -> None:
    """w4a4_kv_reserve: pages for lens[s] tokens of every sequence, the lowest
    free ones first; lacking int32 [1]: the number that was not to be had."""
    _c_ints("kv_reserve", page_size)
    s = _kv_seqs("kv_reserve", tables, lens, refs.device)
    _int32("kv_reserve", refs.device, refs, lacking)
    ws = _kv_workspace(s.seqs, refs.numel(), refs.device)
    _check(lib().w4a4_kv_reserve(s, page_size, refs.data_ptr(), refs.numel(),
                                 None if lacking is None else lacking.data_ptr(), ws.data_ptr(), ws.numel(),
                                 _kv_stream(refs.device)))


def _check_pages(what: str, refs: torch.Tensor, pages: int) -> None:
    if refs.numel() != pages:
        raise W4A4Error(2, f"{what}: refs has {refs.numel()} entries for {pages} pages")


def kv_fork(caches, tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, parents: torch.Tensor,
            children: torch.Tensor, *, lacking: Optional[torch.Tensor] = None) -> None:
    """w4a4_kv_fork: sequence children[i] becomes a copy of parents[i] (int32):
    whole pages shared, a last page that is not full copied in every cache."""
    n, arrays, stride, size, pages, page, dev = _kv_arrays("kv_fork", caches)
    s = _kv_seqs("kv_fork", tables, lens, dev)
    _int32("kv_fork", dev, refs, parents, children, lacking)
    _check_pages("kv_fork", refs, pages)
    count = _same_length("kv_fork", parents, children)
    ws = _kv_workspace(count, pages, dev)
    _check(lib().w4a4_kv_fork(n, arrays, stride, size, s, page, refs.data_ptr(), pages, parents.data_ptr(),
                              children.data_ptr(), count, None if lacking is None else lacking.data_ptr(),
                              ws.data_ptr(), ws.numel(), _kv_stream(dev)))


def kv_free(tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, seqs: Optional[torch.Tensor] = None) -> None:
    """w4a4_kv_free: let go of all pages of the sequences `seqs` (int32; None: all)."""
    s = _kv_seqs("kv_free", tables, lens, refs.device)
    _int32("kv_free", refs.device, refs, seqs)
    _check(lib().w4a4_kv_free(s, refs.data_ptr(), refs.numel(), None if seqs is None else seqs.data_ptr(),
                              s.seqs if seqs is None else seqs.numel(), _kv_stream(refs.device)))


def kv_trim(tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_size: int, window: int, sinks: int = 0,
            seqs: Optional[torch.Tensor] = None) -> None:
    """w4a4_kv_trim: let go of the pages that no later token of the sequences
    `seqs` (None: all) sees under a window with sinks."""
    _c_ints("kv_trim", page_size, window, sinks)
    s = _kv_seqs("kv_trim", tables, lens, refs.device)
    _int32("kv_trim", refs.device, refs, seqs)
    _check(lib().w4a4_kv_trim(s, page_size, refs.data_ptr(), refs.numel(), None if seqs is None else seqs.data_ptr(),
                              s.seqs if seqs is None else seqs.numel(), window, sinks, _kv_stream(refs.device)))


def kv_compact(caches, tables: torch.Tensor, refs: torch.Tensor) -> torch.Tensor:
    """w4a4_kv_compact: move the pages in use to the front, in every cache, with
    tables and refs; returns remap int32 [pages]: new index, -1 for free pages."""
    n, arrays, stride, size, pages, _, dev = _kv_arrays("kv_compact", caches)
    s = _kv_seqs("kv_compact", tables, None, dev)
    _int32("kv_compact", dev, refs)
    _check_pages("kv_compact", refs, pages)
    remap = torch.empty(pages, dtype=torch.int32, device=dev)
    ws = _kv_workspace(0, pages, dev)
    _check(lib().w4a4_kv_compact(n, arrays, stride, size, s, refs.data_ptr(), pages, remap.data_ptr(), ws.data_ptr(),
                                 ws.numel(), _kv_stream(dev)))
    return remap
