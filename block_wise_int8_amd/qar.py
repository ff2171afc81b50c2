"""Binding of libqar (include/qar.h): argument marshalling only.

Every computation runs in libqar's HIP kernels; this module turns torch
tensors into device pointers, HIP streams into handles, allocates outputs
with torch when the caller passes none, and raises ``QarError`` on a
non-OK status.  The AllReduce's calls go through ctypes, the serving calls,
where the host's part counts, through an extension (csrc/qar_torch.cpp).  A
missing library raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import operator
import os
import re
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libqar.so")
EXTENSION = os.path.join(HERE, "_qar_torch.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "qar.h")

QAR_OK, QAR_ERR_INVALID_ARG, QAR_ERR_MISALIGNED, QAR_ERR_UNSUPPORTED, QAR_ERR_HIP, QAR_ERR_CAPACITY = range(6)
QAR_BF16, QAR_F32 = 0, 1
QAR_SCHEDULE_ONE_SHOT, QAR_SCHEDULE_RING = 0, 1
QAR_MAX_RANKS = 32
QAR_MAX_STREAMS = 16
QAR_STATIC_WORKSPACE_BYTES = 64 << 20
QAR_CHUNK_RUN_ELEMS = 1 << 18
BLOCK_SIZES = (64, 128, 256)
QAR_MX4_BLOCK = 32
QAR_KV8_PAGE = 64
QAR_KV8_MAX_SEQUENCES = 4096
QAR_ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
QAR_ROTATE_NORM, QAR_ROTATE_NEIGHBOURS, QAR_ROTATE_EACH_TOKEN = 1, 2, 4

_vp, _sz, _u32, _int = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32, ctypes.c_int

_SIGNATURES = {
    "qar_quantize_blocks": [_vp, _int, _sz, _u32, _vp, _vp, _vp],
    "qar_reduce_quantized": [_vp, _vp, _u32, _sz, _u32, _vp, _vp, _vp, _int, _vp],
    "qar_quantize_reduce": [_vp, _int, _u32, _vp, _vp, _u32, _sz, _u32, _vp, _vp, _vp, _int, _vp],
    "qar_reduce_quantized_pipelined": [_vp, _vp, _u32, _sz, _u32, _vp, _vp, _vp, _int, _u32, _vp, _u32, _vp],
    "qar_reduce_quantized_chunked": [_vp, _vp, _u32, _sz, _u32, _vp, _vp, _vp, _int, _u32, _vp, _u32],
    "qar_ring_step": [_vp, _vp, _vp, _int, _sz, _u32, _vp, _vp, _vp],
    "qar_dequantize": [_vp, _vp, _sz, _u32, _vp, _int, _vp],
    "qar_reduce_unquantized": [_vp, _u32, _sz, _int, _vp, _vp],
    "qar_quantize_rows": [_vp, _int, _sz, _sz, _u32, _vp, _vp, _vp],
    "qar_reduce_quantized_rows": [_vp, _vp, _u32, _sz, _sz, _u32, _vp, _vp, _vp, _int, _vp],
    "qar_ring_step_rows": [_vp, _vp, _vp, _int, _sz, _sz, _u32, _vp, _vp, _vp],
    "qar_dequantize_rows": [_vp, _vp, _sz, _sz, _u32, _vp, _int, _vp],
    "qar_allreduce_simulated": [_vp, _int, _u32, _sz, _u32, _int, _vp, _vp, _vp, _u32, _vp, _u32, _vp],
    "qar_allreduce_simulated_static": [_vp, _int, _u32, _sz, _u32, _int, _vp, _u32, _vp],
    "qar_quantize_blocks_e4m3": [_vp, _int, _sz, _u32, _vp, _vp, _vp],
    "qar_reduce_quantized_e4m3": [_vp, _vp, _u32, _sz, _u32, _vp, _vp, _vp, _int, _vp],
    "qar_quantize_reduce_e4m3": [_vp, _int, _u32, _vp, _vp, _u32, _sz, _u32, _vp, _vp, _vp, _int, _vp],
    "qar_ring_step_e4m3": [_vp, _vp, _vp, _int, _sz, _u32, _vp, _vp, _vp],
    "qar_dequantize_e4m3": [_vp, _vp, _sz, _u32, _vp, _int, _vp],
    "qar_quantize_blocks_int4": [_vp, _int, _sz, _u32, _vp, _vp, _vp],
    "qar_reduce_quantized_int4": [_vp, _vp, _u32, _sz, _u32, _vp, _vp, _vp, _int, _vp],
    "qar_quantize_reduce_int4": [_vp, _int, _u32, _vp, _vp, _u32, _sz, _u32, _vp, _vp, _vp, _int, _vp],
    "qar_ring_step_int4": [_vp, _vp, _vp, _int, _sz, _u32, _vp, _vp, _vp],
    "qar_dequantize_int4": [_vp, _vp, _sz, _u32, _vp, _int, _vp],
    "qar_mx4_quantize": [_vp, _int, _sz, _sz, _vp, _vp, _vp],
    "qar_mx4_dequantize": [_vp, _vp, _sz, _sz, _vp, _int, _vp],
    "qar_mx4_linear_workspace_bytes": [_sz, _sz, _sz],
    "qar_mx4_linear": [_vp, _int, _sz, _sz, _vp, _vp, _sz, _vp, _int, _vp, _sz, _vp],
    "qar_mx4_linear_fused": [_vp, _int, _sz, _sz, _vp, _vp, _sz, _vp, _int, _vp, _vp, _int, _vp, _sz, _vp],
    "qar_kv8_append": [_vp, _vp, _vp, _vp, _int, _u32, _vp],
    "qar_kv8_read": [_vp, _vp, _u32, _vp, _vp, _int, _vp],
    "qar_kv8_attention_workspace_bytes": [_u32, _u32, _u32, _u32, _u32, _u32, _int, _int],
    "qar_kv8_attention": [_vp, _vp, _int, _u32, _u32, _vp, ctypes.c_float, _vp, _vp, _vp, _sz, _vp],
    "qar_kv8_attention_shared_workspace_bytes": [_u32, _u32, _u32, _u32, _u32, _u32, _u32],
    "qar_kv8_attention_shared": [_vp, _vp, _int, _u32, _u32, _vp, _vp, _u32, _vp, ctypes.c_float, _vp, _vp, _sz, _vp],
    "qar_kv8_evict": [_vp, _vp, _vp, _u32, _u32, _vp, _vp, _vp],
    "qar_norm_rotate": [_vp, _int, _sz, _sz, _u32, _u32, _u32, _vp, _vp, _u32, _vp, _vp, ctypes.c_float, _u32, _vp, _vp, _vp,
                        _vp],
    "qar_kv8_fork": [_vp, _vp, _vp, _vp, _vp],
    "qar_kv8_free": [_vp, _vp, _vp, _vp],
    "qar_kv8_reserve": [_vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "qar_kv8_compact": [_vp, _vp, _vp, _vp, _vp],
    "qar_kv8_copy": [_vp, _vp, _vp, _vp, _u32, _vp],
    "qar_status_string": [_int],
    "qar_last_error": [],
}


class QarError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        L = lib()
        text = L.qar_status_string(status).decode()
        detail = L.qar_last_error().decode() if status in (QAR_ERR_HIP, QAR_ERR_CAPACITY) else ""
        super().__init__(f"{where}: {text}" + (f" ({detail})" if detail else ""))


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libqar (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIBRARY):
            raise RuntimeError(f"libqar is not built: {LIBRARY} is missing "
                               "(build it with __graft_entry__.build() or block_wise_int8_amd/build.py)")
        L = ctypes.CDLL(LIBRARY)
        for name, args in _SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = (ctypes.c_char_p if name in ("qar_status_string", "qar_last_error")
                         else _sz if name.endswith("_workspace_bytes") else _int)
        _lib = L
    return _lib


def declared_functions(header: str = HEADER) -> list[str]:
    """Names of the functions include/qar.h declares."""
    text = open(header).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(qar_\w+)\s*\(", text, re.M)))


# ----------------------------------------------------------------------------
# marshalling helpers


def _stream(stream) -> int:
    if stream is None:
        # the handle of torch.cuda.current_stream(), without building the Stream object (2.8 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return QAR_BF16
    if dt == torch.float32:
        return QAR_F32
    raise TypeError(f"libqar handles bfloat16 and float32 data, not {dt}")


def _dev(t: torch.Tensor, what: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA (HIP) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


def _check(status: int, where: str) -> None:
    if status != QAR_OK:
        raise QarError(status, where)


def _ptrs(ts: list[torch.Tensor]):
    arr = (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])
    return arr


# The C ABI sees only pointers, so a tensor too small for the call would be
# read or written past its end.  Every tensor handed to the library is
# therefore checked here first: type, element count and device.
_CODE_DTYPES = (torch.int8, torch.uint8)     # any byte container holds codes
_DATA_DTYPES = (torch.bfloat16, torch.float32)


def _expect(t: torch.Tensor, what: str, numel: int, dtypes: tuple, device: torch.device) -> torch.Tensor:
    _dev(t, what)
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{what} must hold {numel} elements for this call, not {t.numel()}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the call's other tensors on {device}")
    return t


def _nblocks(n: int, block: int):
    """Scale count of a flat call, or None when the library will refuse
    (n % block != 0 or an unsupported block: nothing is then dereferenced)."""
    if block not in BLOCK_SIZES or n % block:
        return None
    return n // block


def _expect_scales(t, what, nb, device):
    if nb is None:
        return _dev(t, what)
    return _expect(t, what, nb, (torch.float32,), device)


# ----------------------------------------------------------------------------
# the calls


# code formats: the C function suffix and the torch dtype that holds the codes
_INT8 = ("", torch.int8, 1)
_E4M3 = ("_e4m3", torch.uint8, 1)
_INT4 = ("_int4", torch.uint8, 2)          # two codes per byte


def _quantize(fmt, x, block, codes, scales, stream):
    name = "qar_quantize_blocks" + fmt[0]
    _dev(x, "x")
    n, dev = x.numel(), x.device
    nb = _nblocks(n, block)
    if codes is None:
        codes = torch.empty(n // fmt[2], dtype=fmt[1], device=dev)
    if scales is None:
        scales = torch.empty(max(n // block, 1) if block else 1, dtype=torch.float32, device=dev)
    if n:
        _expect(codes, "codes", n // fmt[2], _CODE_DTYPES, dev)
        _expect_scales(scales, "scales", nb, dev)
    _check(getattr(lib(), name)(x.data_ptr(), _dtype_code(x.dtype), n, block, _dev(codes, "codes").data_ptr(),
                                _dev(scales, "scales").data_ptr(), _stream(stream)), name)
    return codes, scales


def qar_quantize_blocks(x: torch.Tensor, block: int, codes: torch.Tensor | None = None,
                        scales: torch.Tensor | None = None, stream=None):
    """x (bf16/fp32, any shape, contiguous) -> (codes int8[n], scales fp32[n/block])."""
    return _quantize(_INT8, x, block, codes, scales, stream)


def qar_quantize_blocks_e4m3(x: torch.Tensor, block: int, codes: torch.Tensor | None = None,
                             scales: torch.Tensor | None = None, stream=None):
    """x (bf16/fp32) -> (FP8 E4M3 codes uint8[n], scales fp32[n/block])."""
    return _quantize(_E4M3, x, block, codes, scales, stream)


def _out_args(out: torch.Tensor | None, n: int, device: torch.device):
    if out is None:
        return None, QAR_BF16
    if n:
        _expect(out, "out", n, _DATA_DTYPES, device)
    return _dev(out, "out").data_ptr(), _dtype_code(out.dtype)


def _expect_ranks(codes, scales, n, fmt, nb, device):
    """codes[r] / scales[r] of every rank: n elements' worth of codes and nb
    scales each, all on one device.  (A rank count above QAR_MAX_RANKS is
    left to the library, which refuses it before reading any pointer.)"""
    if len(codes) != len(scales) or not codes:
        raise ValueError("need one scales tensor per codes tensor, at least one rank")
    for r, (c, s) in enumerate(zip(codes, scales)):
        if n:
            _expect(c, f"codes[{r}]", n // fmt[2], _CODE_DTYPES, device)
            _expect_scales(s, f"scales[{r}]", nb, device)
        else:
            _dev(c, f"codes[{r}]"), _dev(s, f"scales[{r}]")


def _outputs(fmt, n, block, nb, codes_out, scales_out, dev):
    """codes_out / scales_out: allocated when not given, else checked."""
    if codes_out is None:
        codes_out = torch.empty(n // fmt[2], dtype=fmt[1], device=dev)
    elif n:
        _expect(codes_out, "codes_out", n // fmt[2], _CODE_DTYPES, dev)
    if scales_out is None:
        scales_out = torch.empty(max(n // block, 1) if block else 1, dtype=torch.float32, device=dev)
    elif n:
        _expect_scales(scales_out, "scales_out", nb, dev)
    return codes_out, scales_out


def _reduce(fmt, codes, scales, block, codes_out, scales_out, out, stream):
    name = "qar_reduce_quantized" + fmt[0]
    if len(codes) != len(scales) or not codes:
        raise ValueError("need one scales tensor per codes tensor, at least one rank")
    n = _dev(codes[0], "codes[0]").numel() * fmt[2]            # elements
    dev = codes[0].device
    nb = _nblocks(n, block)
    _expect_ranks(codes, scales, n, fmt, nb, dev)
    codes_out, scales_out = _outputs(fmt, n, block, nb, codes_out, scales_out, dev)
    optr, odt = _out_args(out, n, dev)
    cp, sp = _ptrs(codes), _ptrs(scales)
    _check(getattr(lib(), name)(ctypes.cast(cp, _vp), ctypes.cast(sp, _vp), len(codes), n, block,
                                _dev(codes_out, "codes_out").data_ptr(), _dev(scales_out, "scales_out").data_ptr(),
                                optr, odt, _stream(stream)), name)
    return codes_out, scales_out


def qar_reduce_quantized(codes: list[torch.Tensor], scales: list[torch.Tensor], block: int,
                         codes_out: torch.Tensor | None = None, scales_out: torch.Tensor | None = None,
                         out: torch.Tensor | None = None, stream=None):
    """One-shot N-way reduce of rank-ordered (codes, scales) -> (codes_out, scales_out);
    ``out`` (optional bf16/fp32 tensor) receives the dequantized result."""
    return _reduce(_INT8, codes, scales, block, codes_out, scales_out, out, stream)


def qar_quantize_blocks_int4(x: torch.Tensor, block: int, codes: torch.Tensor | None = None,
                             scales: torch.Tensor | None = None, stream=None):
    """x (bf16/fp32) -> (4-bit codes packed two per byte, uint8[n/2]; scales fp32[n/block])."""
    return _quantize(_INT4, x, block, codes, scales, stream)


def qar_reduce_quantized_e4m3(codes: list[torch.Tensor], scales: list[torch.Tensor], block: int,
                              codes_out: torch.Tensor | None = None, scales_out: torch.Tensor | None = None,
                              out: torch.Tensor | None = None, stream=None):
    """The one-shot reduce with FP8 E4M3 codes (uint8 tensors)."""
    return _reduce(_E4M3, codes, scales, block, codes_out, scales_out, out, stream)


def _quantize_reduce(fmt, x_own, own, codes, scales, block, codes_out, scales_out, out, stream):
    name = "qar_quantize_reduce" + fmt[0]
    _dev(x_own, "x_own")
    n = x_own.numel()
    dev = x_own.device
    nb = _nblocks(n, block)
    _expect_ranks(codes, scales, n, fmt, nb, dev)
    codes_out, scales_out = _outputs(fmt, n, block, nb, codes_out, scales_out, dev)
    optr, odt = _out_args(out, n, dev)
    cp, sp = _ptrs(codes), _ptrs(scales)
    _check(getattr(lib(), name)(x_own.data_ptr(), _dtype_code(x_own.dtype), own, ctypes.cast(cp, _vp),
                                ctypes.cast(sp, _vp), len(codes), n, block, _dev(codes_out, "codes_out").data_ptr(),
                                _dev(scales_out, "scales_out").data_ptr(), optr, odt, _stream(stream)), name)
    return codes_out, scales_out


def qar_quantize_reduce(x_own: torch.Tensor, own: int, codes: list[torch.Tensor], scales: list[torch.Tensor],
                        block: int, codes_out: torch.Tensor | None = None, scales_out: torch.Tensor | None = None,
                        out: torch.Tensor | None = None, stream=None):
    """Quantize x_own into codes[own]/scales[own] and reduce all ranks in the
    same pass -> (codes_out, scales_out); ``out`` gets the dequantized result."""
    return _quantize_reduce(_INT8, x_own, own, codes, scales, block, codes_out, scales_out, out, stream)


def qar_reduce_quantized_int4(codes: list[torch.Tensor], scales: list[torch.Tensor], block: int,
                              codes_out: torch.Tensor | None = None, scales_out: torch.Tensor | None = None,
                              out: torch.Tensor | None = None, stream=None):
    """The one-shot reduce with packed 4-bit codes (uint8 tensors of n/2 bytes)."""
    return _reduce(_INT4, codes, scales, block, codes_out, scales_out, out, stream)


def qar_quantize_reduce_e4m3(x_own: torch.Tensor, own: int, codes: list[torch.Tensor],
                             scales: list[torch.Tensor], block: int, codes_out: torch.Tensor | None = None,
                             scales_out: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    """The one-kernel step with FP8 E4M3 codes."""
    return _quantize_reduce(_E4M3, x_own, own, codes, scales, block, codes_out, scales_out, out, stream)


def qar_reduce_quantized_pipelined(codes: list[torch.Tensor], scales: list[torch.Tensor], block: int,
                                   nchunks: int, streams: list, codes_out: torch.Tensor | None = None,
                                   scales_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                                   stream=None):
    """The reduce cut into ``nchunks`` chunks enqueued round-robin on ``streams``."""
    if len(codes) != len(scales) or not codes:
        raise ValueError("need one scales tensor per codes tensor, at least one rank")
    n = _dev(codes[0], "codes[0]").numel()
    dev = codes[0].device
    nb = _nblocks(n, block)
    _expect_ranks(codes, scales, n, _INT8, nb, dev)
    codes_out, scales_out = _outputs(_INT8, n, block, nb, codes_out, scales_out, dev)
    optr, odt = _out_args(out, n, dev)
    cp, sp = _ptrs(codes), _ptrs(scales)
    sts = (ctypes.c_void_p * len(streams))(*[_stream(s) for s in streams])
    _check(lib().qar_reduce_quantized_pipelined(
        ctypes.cast(cp, _vp), ctypes.cast(sp, _vp), len(codes), n, block,
        _dev(codes_out, "codes_out").data_ptr(), _dev(scales_out, "scales_out").data_ptr(), optr, odt,
        nchunks, ctypes.cast(sts, _vp), len(streams), _stream(stream)), "qar_reduce_quantized_pipelined")
    return codes_out, scales_out


def qar_reduce_quantized_chunked(codes: list[torch.Tensor], scales: list[torch.Tensor], block: int, nchunks: int,
                                 streams: list, codes_out: torch.Tensor | None = None,
                                 scales_out: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """The reduce cut into ``nchunks`` chunks (chunk c takes the runs c,
    c + nchunks, ... of QAR_CHUNK_RUN_ELEMS elements), chunk c enqueued on
    ``streams[c % len(streams)]`` behind that stream's earlier work, with no
    event or wait: the caller orders the streams."""
    if len(codes) != len(scales) or not codes:
        raise ValueError("need one scales tensor per codes tensor, at least one rank")
    n = _dev(codes[0], "codes[0]").numel()
    dev = codes[0].device
    nb = _nblocks(n, block)
    _expect_ranks(codes, scales, n, _INT8, nb, dev)
    codes_out, scales_out = _outputs(_INT8, n, block, nb, codes_out, scales_out, dev)
    optr, odt = _out_args(out, n, dev)
    cp, sp = _ptrs(codes), _ptrs(scales)
    sts = (ctypes.c_void_p * len(streams))(*[_stream(s) for s in streams])
    _check(lib().qar_reduce_quantized_chunked(
        ctypes.cast(cp, _vp), ctypes.cast(sp, _vp), len(codes), n, block,
        _dev(codes_out, "codes_out").data_ptr(), _dev(scales_out, "scales_out").data_ptr(), optr, odt,
        nchunks, ctypes.cast(sts, _vp), len(streams)), "qar_reduce_quantized_chunked")
    return codes_out, scales_out


def _ring_step(fmt, codes_in, scales_in, local, block, codes_out, scales_out, stream):
    name = "qar_ring_step" + fmt[0]
    _dev(local, "local")
    n, dev = local.numel(), local.device
    nb = _nblocks(n, block)
    if n:
        _expect(codes_in, "codes_in", n // fmt[2], _CODE_DTYPES, dev)
        _expect_scales(scales_in, "scales_in", nb, dev)
    _dev(codes_in, "codes_in"), _dev(scales_in, "scales_in")
    codes_out, scales_out = _outputs(fmt, n, block, nb, codes_out, scales_out, dev)
    _check(getattr(lib(), name)(codes_in.data_ptr(), scales_in.data_ptr(), local.data_ptr(),
                                _dtype_code(local.dtype), n, block, _dev(codes_out, "codes_out").data_ptr(),
                                _dev(scales_out, "scales_out").data_ptr(), _stream(stream)), name)
    return codes_out, scales_out


def qar_ring_step(codes_in: torch.Tensor, scales_in: torch.Tensor, local: torch.Tensor, block: int,
                  codes_out: torch.Tensor | None = None, scales_out: torch.Tensor | None = None, stream=None):
    """quantize(dequantize(codes_in, scales_in) + local) -> (codes_out, scales_out).
    Pass codes_out=codes_in, scales_out=scales_in to work in place."""
    return _ring_step(_INT8, codes_in, scales_in, local, block, codes_out, scales_out, stream)


def qar_quantize_reduce_int4(x_own: torch.Tensor, own: int, codes: list[torch.Tensor],
                             scales: list[torch.Tensor], block: int, codes_out: torch.Tensor | None = None,
                             scales_out: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    """The one-kernel step with packed 4-bit codes."""
    return _quantize_reduce(_INT4, x_own, own, codes, scales, block, codes_out, scales_out, out, stream)


def qar_ring_step_e4m3(codes_in: torch.Tensor, scales_in: torch.Tensor, local: torch.Tensor, block: int,
                       codes_out: torch.Tensor | None = None, scales_out: torch.Tensor | None = None, stream=None):
    """The ring step with FP8 E4M3 codes."""
    return _ring_step(_E4M3, codes_in, scales_in, local, block, codes_out, scales_out, stream)


def _dequantize(fmt, codes, scales, block, out, out_dtype, stream):
    name = "qar_dequantize" + fmt[0]
    _dev(codes, "codes"), _dev(scales, "scales")
    n = codes.numel() * fmt[2]               # elements
    dev = codes.device
    if codes.dtype not in _CODE_DTYPES:
        raise TypeError(f"codes must be torch.int8 or torch.uint8, not {codes.dtype}")
    if n:
        _expect_scales(scales, "scales", _nblocks(n, block), dev)
    if out is None:
        out = torch.empty(n, dtype=out_dtype, device=dev)
    elif n:
        _expect(out, "out", n, _DATA_DTYPES, dev)
    _check(getattr(lib(), name)(codes.data_ptr(), scales.data_ptr(), n, block, _dev(out, "out").data_ptr(),
                                _dtype_code(out.dtype), _stream(stream)), name)
    return out


def qar_dequantize(codes: torch.Tensor, scales: torch.Tensor, block: int, out: torch.Tensor | None = None,
                   out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """codes, scales -> out (bf16 or fp32)."""
    return _dequantize(_INT8, codes, scales, block, out, out_dtype, stream)


def qar_ring_step_int4(codes_in: torch.Tensor, scales_in: torch.Tensor, local: torch.Tensor, block: int,
                       codes_out: torch.Tensor | None = None, scales_out: torch.Tensor | None = None, stream=None):
    """The ring step with packed 4-bit codes."""
    return _ring_step(_INT4, codes_in, scales_in, local, block, codes_out, scales_out, stream)


def qar_dequantize_e4m3(codes: torch.Tensor, scales: torch.Tensor, block: int, out: torch.Tensor | None = None,
                        out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """FP8 E4M3 codes (uint8), scales -> out (bf16 or fp32)."""
    return _dequantize(_E4M3, codes, scales, block, out, out_dtype, stream)


def qar_dequantize_int4(codes: torch.Tensor, scales: torch.Tensor, block: int, out: torch.Tensor | None = None,
                        out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """Packed 4-bit codes (uint8, n/2 bytes), scales -> out (bf16 or fp32)."""
    return _dequantize(_INT4, codes, scales, block, out, out_dtype, stream)


def qar_reduce_unquantized(xs: list[torch.Tensor], out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The unquantized comparator: rank-order fp32 sum of N bf16/fp32 buffers."""
    if not xs:
        raise ValueError("need at least one rank")
    n, dt, dev = _dev(xs[0], "x[0]").numel(), xs[0].dtype, xs[0].device
    for r, x in enumerate(xs):
        _expect(x, f"x[{r}]", n, (dt,), dev)
    if out is None:
        out = torch.empty(n, dtype=dt, device=dev)
    else:
        _expect(out, "out", n, (dt,), dev)
    ptrs = _ptrs(xs)
    _check(lib().qar_reduce_unquantized(ctypes.cast(ptrs, _vp), len(xs), n, _dtype_code(xs[0].dtype),
                                        _dev(out, "out").data_ptr(), _stream(stream)), "qar_reduce_unquantized")
    return out


def qar_allreduce_simulated(xs: list[torch.Tensor], block: int, schedule: str = "one_shot", nchunks: int = 1,
                            streams: list | None = None, out: torch.Tensor | None = None,
                            workspace: tuple | None = None, stream=None) -> torch.Tensor:
    """The whole quantized AllReduce of N rank buffers on one GPU ('one_shot'
    or 'ring'); returns the dequantized result every rank would hold.
    ``workspace`` = (codes list, scales list) is allocated with torch when
    not given."""
    if not xs:
        raise ValueError("need at least one rank")
    sched = {"one_shot": QAR_SCHEDULE_ONE_SHOT, "ring": QAR_SCHEDULE_RING}[schedule]
    n, dt, dev = _dev(xs[0], "x[0]").numel(), xs[0].dtype, xs[0].device
    for r, x in enumerate(xs):
        _expect(x, f"x[{r}]", n, (dt,), dev)
    nwork = len(xs) if sched == QAR_SCHEDULE_ONE_SHOT else 1
    nb = _nblocks(n, block)
    if workspace is None:
        workspace = ([torch.empty(n, dtype=torch.int8, device=dev) for _ in range(nwork)],
                     [torch.empty(max(n // block, 1) if block else 1, dtype=torch.float32, device=dev)
                      for _ in range(nwork)])
    wc, ws = workspace
    if len(wc) < nwork or len(ws) < nwork:
        raise ValueError(f"the {schedule} schedule needs {nwork} codes and scales workspaces")
    wc, ws = list(wc)[:nwork], list(ws)[:nwork]
    if n:
        for r in range(nwork):
            _expect(wc[r], f"workspace codes[{r}]", n, _CODE_DTYPES, dev)
            _expect_scales(ws[r], f"workspace scales[{r}]", nb, dev)
    if out is None:
        out = torch.empty(n, dtype=dt, device=dev)
    else:
        _expect(out, "out", n, (dt,), dev)
    if streams is None:
        streams = [torch.cuda.current_stream()]
    xp, cp, sp = _ptrs(xs), _ptrs(wc), _ptrs(ws)
    sts = (ctypes.c_void_p * len(streams))(*[_stream(s) for s in streams])
    _check(lib().qar_allreduce_simulated(ctypes.cast(xp, _vp), _dtype_code(xs[0].dtype), len(xs), n, block, sched,
                                         ctypes.cast(cp, _vp), ctypes.cast(sp, _vp), _dev(out, "out").data_ptr(),
                                         nchunks, ctypes.cast(sts, _vp), len(streams), _stream(stream)),
           "qar_allreduce_simulated")
    return out


def qar_allreduce_simulated_static(xs: list[torch.Tensor], block: int, schedule: str = "one_shot",
                                   nchunks: int = 1, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """qar_allreduce_simulated on one stream with its staging in libqar's
    static device workspace (the library allocates nothing; ``out`` is
    allocated here with torch when not given)."""
    if not xs:
        raise ValueError("need at least one rank")
    sched = {"one_shot": QAR_SCHEDULE_ONE_SHOT, "ring": QAR_SCHEDULE_RING}[schedule]
    n, dt, dev = _dev(xs[0], "x[0]").numel(), xs[0].dtype, xs[0].device
    for r, x in enumerate(xs):
        _expect(x, f"x[{r}]", n, (dt,), dev)
    if out is None:
        out = torch.empty(n, dtype=dt, device=dev)
    else:
        _expect(out, "out", n, (dt,), dev)
    xp = _ptrs(xs)
    _check(lib().qar_allreduce_simulated_static(ctypes.cast(xp, _vp), _dtype_code(dt), len(xs), n, block, sched,
                                                out.data_ptr(), nchunks, _stream(stream)),
           "qar_allreduce_simulated_static")
    return out


# ----------------------------------------------------------------------------
# row-bounded blocks ([rows, row_len] tensors; the block grid restarts per row)


def row_blocks(rows: int, row_len: int, block: int) -> int:
    return rows * (-(-row_len // block))


def _row_nblocks(rows: int, row_len: int, block: int):
    """Scale count of a row-bounded call, or None for a block size the
    library refuses."""
    return row_blocks(rows, row_len, block) if block in BLOCK_SIZES else None


def qar_quantize_rows(x: torch.Tensor, block: int, codes: torch.Tensor | None = None,
                      scales: torch.Tensor | None = None, stream=None):
    """x: [rows, row_len] bf16/fp32 -> (codes [rows*row_len], scales [rows*ceil(row_len/block)])."""
    _dev(x, "x")
    rows, row_len = x.shape
    dev = x.device
    nrb = _row_nblocks(rows, row_len, block)
    if codes is None:
        codes = torch.empty(rows * row_len, dtype=torch.int8, device=dev)
    elif rows * row_len:
        _expect(codes, "codes", rows * row_len, _CODE_DTYPES, dev)
    if scales is None:
        scales = torch.empty(max(nrb or 0, 1), dtype=torch.float32, device=dev)
    elif rows * row_len:
        _expect_scales(scales, "scales", nrb, dev)
    _check(lib().qar_quantize_rows(x.data_ptr(), _dtype_code(x.dtype), rows, row_len, block,
                                   _dev(codes, "codes").data_ptr(), _dev(scales, "scales").data_ptr(),
                                   _stream(stream)), "qar_quantize_rows")
    return codes, scales


def qar_reduce_quantized_rows(codes: list[torch.Tensor], scales: list[torch.Tensor], rows: int, row_len: int,
                              block: int, codes_out: torch.Tensor | None = None,
                              scales_out: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    if len(codes) != len(scales) or not codes:
        raise ValueError("need one scales tensor per codes tensor, at least one rank")
    n = rows * row_len
    dev = _dev(codes[0], "codes[0]").device
    nrb = _row_nblocks(rows, row_len, block)
    _expect_ranks(codes, scales, n, _INT8, nrb, dev)
    if codes_out is None:
        codes_out = torch.empty(n, dtype=torch.int8, device=dev)
    elif n:
        _expect(codes_out, "codes_out", n, _CODE_DTYPES, dev)
    if scales_out is None:
        scales_out = torch.empty(max(nrb or 0, 1), dtype=torch.float32, device=dev)
    elif n:
        _expect_scales(scales_out, "scales_out", nrb, dev)
    optr, odt = _out_args(out, n, dev)
    cp, sp = _ptrs(codes), _ptrs(scales)
    _check(lib().qar_reduce_quantized_rows(ctypes.cast(cp, _vp), ctypes.cast(sp, _vp), len(codes), rows, row_len,
                                           block, _dev(codes_out, "codes_out").data_ptr(),
                                           _dev(scales_out, "scales_out").data_ptr(), optr, odt, _stream(stream)),
           "qar_reduce_quantized_rows")
    return codes_out, scales_out


def qar_ring_step_rows(codes_in: torch.Tensor, scales_in: torch.Tensor, local: torch.Tensor, block: int,
                       codes_out: torch.Tensor | None = None, scales_out: torch.Tensor | None = None, stream=None):
    """local: [rows, row_len]; codes/scales in the row-bounded layout."""
    _dev(codes_in, "codes_in"), _dev(scales_in, "scales_in"), _dev(local, "local")
    rows, row_len = local.shape
    n, dev = rows * row_len, local.device
    nrb = _row_nblocks(rows, row_len, block)
    if n:
        _expect(codes_in, "codes_in", n, _CODE_DTYPES, dev)
        _expect_scales(scales_in, "scales_in", nrb, dev)
    if codes_out is None:
        codes_out = torch.empty(n, dtype=torch.int8, device=dev)
    elif n:
        _expect(codes_out, "codes_out", n, _CODE_DTYPES, dev)
    if scales_out is None:
        scales_out = torch.empty(max(nrb or 0, 1), dtype=torch.float32, device=dev)
    elif n:
        _expect_scales(scales_out, "scales_out", nrb, dev)
    _check(lib().qar_ring_step_rows(codes_in.data_ptr(), scales_in.data_ptr(), local.data_ptr(),
                                    _dtype_code(local.dtype), rows, row_len, block,
                                    _dev(codes_out, "codes_out").data_ptr(), _dev(scales_out, "scales_out").data_ptr(),
                                    _stream(stream)), "qar_ring_step_rows")
    return codes_out, scales_out


def qar_dequantize_rows(codes: torch.Tensor, scales: torch.Tensor, rows: int, row_len: int, block: int,
                        out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                        stream=None) -> torch.Tensor:
    _dev(codes, "codes"), _dev(scales, "scales")
    n, dev = rows * row_len, codes.device
    if n:
        _expect(codes, "codes", n, _CODE_DTYPES, dev)
        _expect_scales(scales, "scales", _row_nblocks(rows, row_len, block), dev)
    if out is None:
        out = torch.empty(rows, row_len, dtype=out_dtype, device=dev)
    elif n:
        _expect(out, "out", n, _DATA_DTYPES, dev)
    _check(lib().qar_dequantize_rows(codes.data_ptr(), scales.data_ptr(), rows, row_len, block,
                                     _dev(out, "out").data_ptr(), _dtype_code(out.dtype), _stream(stream)),
           "qar_dequantize_rows")
    return out


# ----------------------------------------------------------------------------
# serving: microscaled 4-bit floating point


# These calls are short enough for the host's part to count, so an extension
# (csrc/qar_torch.cpp) checks the arguments, allocates and calls the library.
# It returns None where something does not fit; `_why_*` then find out what and
# raise.

_extension = None


def _serve():
    """The loaded extension (raises if it has not been built)."""
    global _extension
    if _extension is None:
        lib()
        try:
            from . import _qar_torch
        except ImportError as e:
            raise RuntimeError(f"{EXTENSION} does not load (build it with __graft_entry__.build() or "
                               f"block_wise_int8_amd/build.py): {e}") from e
        _extension = _qar_torch
    return _extension


def _done(result, where):
    """What the extension returned: a status or the call's tensors."""
    if type(result) is int:
        _check(result, where)
        return None
    return result


def _on_current(index):
    device = torch.cuda.current_device()
    if index != device:
        raise ValueError(f"the tensors are on GPU {index}, the current device is {device}")


def _whole(v, what, lo, hi):
    try:
        n = None if isinstance(v, (bool, torch.Tensor)) else operator.index(v)
    except TypeError:
        n = None
    if n is None or not lo <= n < hi:
        raise ValueError(f"{what} must be a whole number of at least {lo} and below {hi}, not {v}")


def _as_current(stream):
    """A context in which ``stream`` (a Stream or a handle) is the current one.  A call on a stream
    other than the current one is made inside it, so that what it allocates (outputs, workspaces)
    belongs to that stream and is not handed out again while the call runs."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _matrix(t, what):
    _dev(t, what)
    if t.dim() != 2:
        raise ValueError(f"{what} must have 2 dimensions, not {t.dim()}")
    return t


def _mx4_blocks(cols):
    return (cols + QAR_MX4_BLOCK - 1) // QAR_MX4_BLOCK


def qar_mx4_quantize(x: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                     stream=None):
    """x [rows, cols] (bf16/fp32) -> (E2M1 codes, two per byte, uint8[rows, nb * 16];
    power-of-two scales uint8[rows, nb]) with nb = ceil(cols / 32)."""
    if stream is not None:
        with _as_current(stream):
            return qar_mx4_quantize(x, codes, scales)
    made = _serve().mx4_quantize(x, codes, scales)
    return _done(made, "qar_mx4_quantize") if made is not None else _why_mx4_quantize(x, codes, scales)


def _why_mx4_quantize(x, codes, scales):
    rows, cols = _matrix(x, "x").shape
    _dtype_code(x.dtype)
    _why_mx4(codes, scales, rows, _mx4_blocks(cols), x.device)
    _on_current(x.get_device())
    raise ValueError("qar_mx4_quantize: the arguments do not fit")


def _why_mx4(codes, scales, rows, nb, device):
    if codes is not None:
        _expect(codes, "codes", rows * nb * 16, (torch.uint8,), device)
    if scales is not None:
        _expect(scales, "scales", rows * nb, (torch.uint8,), device)


def qar_mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, cols: int, out: torch.Tensor | None = None,
                       out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """codes uint8[rows, nb * 16], scales uint8[rows, nb] -> out [rows, cols] (bf16 or fp32)."""
    if stream is not None:
        with _as_current(stream):
            return qar_mx4_dequantize(codes, scales, cols, out, out_dtype)
    made = _serve().mx4_dequantize(codes, scales, cols, out, out_dtype)
    return _done(made, "qar_mx4_dequantize") if made is not None else _why_mx4_dequantize(codes, scales, cols, out, out_dtype)


def _why_mx4_dequantize(codes, scales, cols, out, out_dtype):
    _whole(cols, "cols", 0, 1 << 63)
    rows = _matrix(codes, "codes").shape[0]
    _dev(scales, "scales")
    _why_mx4(codes, scales, rows, _mx4_blocks(cols), codes.device)
    _why_out(out, out_dtype, rows * cols, codes.device)
    _on_current(codes.get_device())
    raise ValueError("qar_mx4_dequantize: the arguments do not fit")


def _why_out(out, out_dtype, numel, device):
    if out is not None:
        _expect(out, "out", numel, _DATA_DTYPES, device)
    elif out_dtype is not None:
        _dtype_code(out_dtype)


def qar_mx4_linear(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor | None = None,
                   out_dtype: torch.dtype | None = None, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """x [rows, inner] (bf16/fp32), quantized on the way, times the transposed mx4
    weights codes uint8[cols, nb * 16], scales uint8[cols, nb] -> out [rows, cols]
    (x's type unless out or out_dtype says otherwise).  ``workspace`` (at least
    lib().qar_mx4_linear_workspace_bytes(rows, inner, cols) bytes) is allocated
    with torch when not given."""
    if stream is not None:
        with _as_current(stream):
            return qar_mx4_linear(x, codes, scales, out, out_dtype, workspace)
    made = _serve().mx4_linear(x, codes, scales, out, out_dtype, workspace)
    if made is not None:
        return _done(made, "qar_mx4_linear")
    return _why_mx4_linear(x, codes, scales, out, out_dtype, workspace)


def _why_mx4_linear(x, codes, scales, out, out_dtype, workspace, where="qar_mx4_linear"):
    rows, inner = _matrix(x, "x").shape
    cols = _matrix(codes, "codes").shape[0]
    _dev(scales, "scales")
    _why_mx4(codes, scales, cols, _mx4_blocks(inner), x.device)
    _dtype_code(x.dtype)
    _why_out(out, out_dtype, rows * cols, x.device)
    _why_workspace(workspace, x.device)
    _on_current(x.get_device())
    raise ValueError(f"{where}: the arguments do not fit")


def qar_mx4_linear_fused(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, bias: torch.Tensor | None = None,
                         activation: str | None = None, residual: torch.Tensor | None = None,
                         out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """residual + activation(the product of qar_mx4_linear + bias) -> out [rows, cols], rounded once.  ``bias`` [cols]
    and ``residual`` [rows, cols] are of out's type; ``activation`` is None, "relu", "silu", "gelu" or "gelu_tanh";
    ``out`` may be the residual itself."""
    if stream is not None:
        with _as_current(stream):
            return qar_mx4_linear_fused(x, codes, scales, bias, activation, residual, out, out_dtype, workspace)
    number = QAR_ACTIVATIONS.get(activation) if activation is None or isinstance(activation, str) else None
    made = _serve().mx4_linear_fused(x, codes, scales, bias, number, residual, out, out_dtype, workspace)
    if made is not None:
        return _done(made, "qar_mx4_linear_fused")
    return _why_mx4_linear_fused(x, codes, scales, bias, activation, residual, out, out_dtype, workspace)


def _why_mx4_linear_fused(x, codes, scales, bias, activation, residual, out, out_dtype, workspace):
    if activation is not None and not (isinstance(activation, str) and activation in QAR_ACTIVATIONS):
        raise ValueError(f"activation must be one of {', '.join(map(str, QAR_ACTIVATIONS))}, not {activation}")
    if isinstance(x, torch.Tensor) and isinstance(codes, torch.Tensor) and x.dim() == codes.dim() == 2:
        numel = x.shape[0] * codes.shape[0]
        dtype = out.dtype if isinstance(out, torch.Tensor) else x.dtype if out_dtype is None else out_dtype
        if bias is not None:
            _shaped(bias, "bias", (codes.shape[0],), (dtype,), x.device)
        if residual is not None:
            _expect(residual, "residual", numel, (dtype,), x.device)
    _why_mx4_linear(x, codes, scales, out, out_dtype, workspace, "qar_mx4_linear_fused")


def _why_workspace(workspace, device):
    if workspace is not None and _dev(workspace, "workspace").device != device:
        raise ValueError(f"workspace is on {workspace.device}, the call's other tensors on {device}")


# ----------------------------------------------------------------------------
# serving: the 8-bit paged cache


# qar_kv8_cache of include/qar.h as bytes: six pointers, five 32-bit numbers and
# the padding behind them
_KV_PACK = struct.Struct("=6Q5I4x").pack


class KvCache:
    """The tensors of a paged 8-bit cache (qar_kv8_cache in include/qar.h):
    k int8[pages, kv_heads, 64, dim], v int8[pages, kv_heads, dim, 64],
    k_scales and v_scales fp32[pages, kv_heads], page_table int32[batch, width],
    lengths int32[batch].  They stay the caller's; every call looks at them anew."""
    __slots__ = ("k", "k_scales", "v", "v_scales", "page_table", "lengths")

    def __init__(self, k, k_scales, v, v_scales, page_table, lengths):
        self.k, self.k_scales, self.v, self.v_scales = k, k_scales, v, v_scales
        self.page_table, self.lengths = page_table, lengths

    @classmethod
    def empty(cls, pages: int, kv_heads: int, dim: int, batch: int, table_width: int, device="cuda") -> "KvCache":
        """A pool of ``pages`` pages and a table without entries."""
        return cls(torch.zeros((pages, kv_heads, QAR_KV8_PAGE, dim), dtype=torch.int8, device=device),
                   torch.zeros((pages, kv_heads), dtype=torch.float32, device=device),
                   torch.zeros((pages, kv_heads, dim, QAR_KV8_PAGE), dtype=torch.int8, device=device),
                   torch.zeros((pages, kv_heads), dtype=torch.float32, device=device),
                   torch.full((batch, table_width), -1, dtype=torch.int32, device=device),
                   torch.zeros(batch, dtype=torch.int32, device=device))

    def forked(self, batch: int, table_width: int | None = None) -> "KvCache":
        """The same pool with a table and lengths of its own for ``batch`` sequences (not set: what
        qar_kv8_fork writes), as wide as this one's unless said otherwise."""
        width = self.page_table.shape[1] if table_width is None else table_width
        new = self.page_table.new_empty
        return KvCache(self.k, self.k_scales, self.v, self.v_scales, new((batch, width)), new((batch,)))

    def _struct(self, what="cache"):
        """(the C struct as bytes, for calls of lib() itself, GPU index, batch, kv_heads, dim, table_width)"""
        k, v, ks, vs, table, lengths = self.k, self.v, self.k_scales, self.v_scales, self.page_table, self.lengths
        for name in self.__slots__:
            if not isinstance(getattr(self, name), torch.Tensor):
                raise TypeError(f"{what}.{name} must be a CUDA (HIP) tensor")
        if k.dim() != 4 or k.shape[2] != QAR_KV8_PAGE or table.dim() != 2:
            raise ValueError(f"{what}.k must be [pages, kv_heads, {QAR_KV8_PAGE}, dim] and {what}.page_table [batch, width]")
        pages, heads, page, dim = k.shape
        batch, width = table.shape
        if tuple(v.shape) != (pages, heads, dim, page):
            raise ValueError(f"{what}.v must be {(pages, heads, dim, page)}, not {tuple(v.shape)}")
        for name, numel, dt in (("k", k.numel(), torch.int8), ("v", k.numel(), torch.int8),
                                ("k_scales", pages * heads, torch.float32), ("v_scales", pages * heads, torch.float32),
                                ("page_table", batch * width, torch.int32), ("lengths", batch, torch.int32)):
            _expect(getattr(self, name), f"{what}.{name}", numel, (dt,), k.device)
        return _KV_PACK(k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr(), table.data_ptr(), lengths.data_ptr(),
                        pages, heads, dim, batch, width), k.get_device(), batch, heads, dim, width


def _shaped(t, what, shape, dtypes, device):
    if tuple(_dev(t, what).shape) != shape:
        raise ValueError(f"{what} must be {list(shape)}, not {list(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the call's other tensors on {device}")
    return t


_INT32, _F32 = (torch.int32,), (torch.float32,)


def qar_kv8_append(cache: KvCache, starts: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
    """k_new, v_new [batch, tokens, kv_heads, dim] (bf16/fp32) enter the cache at
    positions starts[b] (int32[batch]) of every sequence.  ``cache.lengths`` stays as it is."""
    if stream is not None:
        with _as_current(stream):
            return qar_kv8_append(cache, starts, k_new, v_new)
    made = _serve().kv8_append(cache, starts, k_new, v_new)
    return _done(made, "qar_kv8_append") if made is not None else _why_kv8_append(cache, starts, k_new, v_new)


def _why_kv8_append(cache, starts, k_new, v_new):
    _, index, batch, heads, dim, _ = cache._struct()
    shape, dev = (batch, k_new.shape[1] if _dev(k_new, "k_new").dim() == 4 else -1, heads, dim), cache.k.device
    _shaped(k_new, "k_new", shape, _DATA_DTYPES, dev)
    _shaped(v_new, "v_new", shape, (k_new.dtype,), dev)
    _shaped(starts, "starts", (batch,), _INT32, dev)
    _on_current(index)
    raise ValueError("qar_kv8_append: the arguments do not fit")


def qar_kv8_read(cache: KvCache, starts: torch.Tensor, tokens: int, out_dtype: torch.dtype = torch.bfloat16,
                 out: tuple | None = None, stream=None):
    """Tokens starts[b] .. starts[b] + tokens - 1 of every sequence as values
    (k, v), each [batch, tokens, kv_heads, dim]; zeros behind its length.
    ``out`` = (k, v) receives them instead of new tensors."""
    if stream is not None:
        with _as_current(stream):
            return qar_kv8_read(cache, starts, tokens, out_dtype, out)
    if out is not None:
        out = tuple(out)
    made = _serve().kv8_read(cache, starts, tokens, out_dtype, out)
    return _done(made, "qar_kv8_read") if made is not None else _why_kv8_read(cache, starts, tokens, out_dtype, out)


def _why_kv8_read(cache, starts, tokens, out_dtype, out):
    _, index, batch, heads, dim, _ = cache._struct()
    _whole(tokens, "tokens", 0, 1 << 32)
    shape, dev = (batch, tokens, heads, dim), cache.k.device
    _shaped(starts, "starts", (batch,), _INT32, dev)
    if out is None:
        _dtype_code(out_dtype)
    else:
        _shaped(out[0], "out[0]", shape, _DATA_DTYPES, dev)
        _shaped(out[1], "out[1]", shape, (out[0].dtype,), dev)
    _on_current(index)
    raise ValueError("qar_kv8_read: the arguments do not fit")


def qar_kv8_attention(cache: KvCache, q: torch.Tensor, q_lens: torch.Tensor | None = None, scale: float | None = None,
                      weights: torch.Tensor | None = None, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of q [batch, queries, heads, dim] (bf16/fp32), the last
    q_lens[b] (default: all) tokens of every sequence, over the cache -> out like q.
    ``scale`` defaults to dim ** -0.5.  ``weights`` fp32[batch, kv_heads, width * 64],
    when given, has the weight that each token received added.  ``workspace`` (at
    least lib().qar_kv8_attention_workspace_bytes(...) bytes) is allocated with
    torch when not given."""
    if stream is not None:
        with _as_current(stream):
            return qar_kv8_attention(cache, q, q_lens, scale, weights, out, workspace)
    made = _serve().kv8_attention(cache, q, q_lens, scale, weights, out, workspace)
    if made is not None:
        return _done(made, "qar_kv8_attention")
    return _why_kv8_attention(cache, q, q_lens, scale, weights, out, workspace)


def _why_kv8_attention(cache, q, q_lens, scale, weights, out, workspace, where="qar_kv8_attention"):
    _, index, batch, kv_heads, dim, width = cache._struct()
    dev = cache.k.device
    if _dev(q, "q").dim() != 4:
        raise ValueError(f"q must be [batch, queries, heads, dim], not {list(q.shape)}")
    shape = (batch, q.shape[1], q.shape[2], dim)
    _shaped(q, "q", shape, _DATA_DTYPES, dev)
    if q_lens is not None:
        _shaped(q_lens, "q_lens", (batch,), _INT32, dev)
    if scale is not None:
        float(scale)
    if weights is not None:
        _shaped(weights, "weights", (batch, kv_heads, width * QAR_KV8_PAGE), _F32, dev)
    if out is not None:
        _shaped(out, "out", shape, (q.dtype,), dev)
    _why_workspace(workspace, dev)
    _on_current(index)
    raise ValueError(f"{where}: the arguments do not fit")


def qar_kv8_attention_shared(cache: KvCache, q: torch.Tensor, starts: torch.Tensor, prefix: torch.Tensor,
                             q_lens: torch.Tensor | None = None, scale: float | None = None,
                             out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                             stream=None) -> torch.Tensor:
    """qar_kv8_attention for sequences that share their first tokens' pages, which are read once for each group:
    sequences starts[g] .. starts[g + 1] - 1 (int32[groups + 1]) have their first prefix[g] (int32[groups]) tokens in
    common, as far as each has tokens.  ``workspace`` (at least lib().qar_kv8_attention_shared_workspace_bytes(...) bytes)
    is allocated with torch when not given."""
    if stream is not None:
        with _as_current(stream):
            return qar_kv8_attention_shared(cache, q, starts, prefix, q_lens, scale, out, workspace)
    made = _serve().kv8_attention_shared(cache, q, starts, prefix, q_lens, scale, out, workspace)
    if made is not None:
        return _done(made, "qar_kv8_attention_shared")
    return _why_kv8_attention_shared(cache, q, starts, prefix, q_lens, scale, out, workspace)


def _why_kv8_attention_shared(cache, q, starts, prefix, q_lens, scale, out, workspace):
    cache._struct()
    dev = cache.k.device
    if _dev(starts, "starts").dim() != 1 or starts.shape[0] < 2:
        raise ValueError(f"starts must be [groups + 1], not {list(starts.shape)}")
    _shaped(starts, "starts", tuple(starts.shape), _INT32, dev)
    _shaped(prefix, "prefix", (starts.shape[0] - 1,), _INT32, dev)
    _why_kv8_attention(cache, q, q_lens, scale, None, out, workspace, "qar_kv8_attention_shared")


def qar_kv8_evict(cache: KvCache, into: KvCache, weights: torch.Tensor, recent: int, keep: int,
                  kept: torch.Tensor | None = None, moved: torch.Tensor | None = None, stream=None):
    """``into`` receives, of every sequence and head, the last min(recent, keep)
    tokens of ``cache`` and the heaviest others, ``keep`` in all, and its lengths
    -> (kept positions int32[batch, kv_heads, keep], -1 behind them; their weights, 0 behind them)."""
    if stream is not None:
        with _as_current(stream):
            return qar_kv8_evict(cache, into, weights, recent, keep, kept, moved)
    made = _serve().kv8_evict(cache, into, weights, recent, keep, kept, moved)
    if made is not None:
        return _done(made, "qar_kv8_evict")
    return _why_kv8_evict(cache, into, weights, recent, keep, kept, moved)


def _why_kv8_evict(cache, into, weights, recent, keep, kept, moved):
    _, index, batch, heads, _, width = cache._struct()
    if into._struct("into")[1] != index:
        raise ValueError(f"into is on {into.k.device}, cache on {cache.k.device}")
    if not 0 <= recent < 1 << 32 or not 1 <= keep < 1 << 31:
        raise ValueError(f"recent must be at least 0 and keep at least 1, not {recent} and {keep}")
    _whole(recent, "recent", 0, 1 << 32)
    _whole(keep, "keep", 1, 1 << 31)
    shape, dev = (batch, heads, keep), cache.k.device
    _shaped(weights, "weights", (batch, heads, width * QAR_KV8_PAGE), _F32, dev)
    if kept is not None:
        _shaped(kept, "kept", shape, _INT32, dev)
    if moved is not None:
        _shaped(moved, "moved", shape, _F32, dev)
    _on_current(index)
    raise ValueError("qar_kv8_evict: the arguments do not fit")


# ----------------------------------------------------------------------------
# serving: owners of the cache's pages


def qar_kv8_fork(cache: KvCache, refs: torch.Tensor, parents: torch.Tensor, into: KvCache, stream=None) -> None:
    """Sequence b of ``into`` (the same pool, see KvCache.forked) goes on from sequence parents[b]
    (int32[into's batch]) of ``cache`` and shares its pages, whose owners refs (int32[pages]) counts;
    a parent outside the batch gives an empty sequence."""
    if stream is not None:
        with _as_current(stream):
            return qar_kv8_fork(cache, refs, parents, into)
    made = _serve().kv8_fork(cache, refs, parents, into)
    return _done(made, "qar_kv8_fork") if made is not None else _why_kv8_fork(cache, refs, parents, into)


def _why_owned(cache, refs):
    _, index, batch, _, _, _ = cache._struct()
    _shaped(refs, "refs", (cache.k.shape[0],), _INT32, cache.k.device)
    return index, batch, cache.k.device


def _why_kv8_fork(cache, refs, parents, into):
    index, _, dev = _why_owned(cache, refs)
    _, other, batch, _, _, _ = into._struct("into")
    if other != index:
        raise ValueError(f"into is on {into.k.device}, cache on {dev}")
    _shaped(parents, "parents", (batch,), _INT32, dev)
    _on_current(index)
    raise ValueError("qar_kv8_fork: the arguments do not fit")


def qar_kv8_free(cache: KvCache, refs: torch.Tensor, keep: torch.Tensor | None = None, stream=None) -> None:
    """Every sequence is cut to its first keep[b] (int32[batch]; default: no) tokens; the pages behind them are released.
    ``cache.lengths`` as ``keep`` releases only what was given ahead."""
    if stream is not None:
        with _as_current(stream):
            return qar_kv8_free(cache, refs, keep)
    made = _serve().kv8_free(cache, refs, keep)
    return _done(made, "qar_kv8_free") if made is not None else _why_kv8_free(cache, refs, keep)


def _why_kv8_free(cache, refs, keep):
    index, batch, dev = _why_owned(cache, refs)
    if keep is not None:
        _shaped(keep, "keep", (batch,), _INT32, dev)
    _on_current(index)
    raise ValueError("qar_kv8_free: the arguments do not fit")


def qar_kv8_reserve(cache: KvCache, refs: torch.Tensor, tokens: torch.Tensor, room: torch.Tensor | None = None,
                    source: torch.Tensor | None = None, target: torch.Tensor | None = None, stream=None):
    """Pages for tokens[b] (int32[batch]) more tokens of every sequence -> (room int32[batch]: for how many
    there is room now; source, target int32[batch]: pages that qar_kv8_copy has to copy before they are written, or -1)."""
    if stream is not None:
        with _as_current(stream):
            return qar_kv8_reserve(cache, refs, tokens, room, source, target)
    made = _serve().kv8_reserve(cache, refs, tokens, room, source, target)
    if made is not None:
        return _done(made, "qar_kv8_reserve")
    return _why_kv8_reserve(cache, refs, tokens, room, source, target)


def _why_kv8_reserve(cache, refs, tokens, room, source, target):
    index, batch, dev = _why_owned(cache, refs)
    _shaped(tokens, "tokens", (batch,), _INT32, dev)
    for t, what in ((room, "room"), (source, "source"), (target, "target")):
        if t is not None:
            _shaped(t, what, (batch,), _INT32, dev)
    _on_current(index)
    raise ValueError("qar_kv8_reserve: the arguments do not fit")


def qar_kv8_compact(cache: KvCache, refs: torch.Tensor, source: torch.Tensor | None = None,
                    target: torch.Tensor | None = None, stream=None):
    """The pages in use get the pool's lowest numbers -> (source, target int32[pages // 2]: the moves that
    qar_kv8_copy has to make, -1 behind them)."""
    if stream is not None:
        with _as_current(stream):
            return qar_kv8_compact(cache, refs, source, target)
    made = _serve().kv8_compact(cache, refs, source, target)
    return _done(made, "qar_kv8_compact") if made is not None else _why_kv8_compact(cache, refs, source, target)


def _why_kv8_compact(cache, refs, source, target):
    index, _, dev = _why_owned(cache, refs)
    for t, what in ((source, "source"), (target, "target")):
        if t is not None:
            _shaped(t, what, (cache.k.shape[0] // 2,), _INT32, dev)
    _on_current(index)
    raise ValueError("qar_kv8_compact: the arguments do not fit")


def qar_kv8_copy(cache: KvCache, source: torch.Tensor, target: torch.Tensor, into: KvCache | None = None,
                 stream=None) -> None:
    """Page target[i] of ``into`` (default: ``cache``) becomes page source[i] of ``cache``, for every i where both
    (int32) are pages of their pools."""
    if stream is not None:
        with _as_current(stream):
            return qar_kv8_copy(cache, source, target, into)
    if into is None:
        into = cache
    made = _serve().kv8_copy(cache, into, source, target)
    return _done(made, "qar_kv8_copy") if made is not None else _why_kv8_copy(cache, into, source, target)


def _why_kv8_copy(cache, into, source, target):
    index = cache._struct()[1]
    if into._struct("into")[1] != index:
        raise ValueError(f"into is on {into.k.device}, cache on {cache.k.device}")
    if _dev(source, "source").dim() != 1:
        raise ValueError(f"source must have 1 dimension, not {source.dim()}")
    _shaped(source, "source", tuple(source.shape), _INT32, cache.k.device)
    _shaped(target, "target", tuple(source.shape), _INT32, cache.k.device)
    _on_current(index)
    raise ValueError("qar_kv8_copy: the arguments do not fit")


# ----------------------------------------------------------------------------
# serving: head norms and rotary positions


def qar_norm_rotate(qkv: torch.Tensor, heads: int, kv_heads: int, positions: torch.Tensor,
                    frequencies: torch.Tensor | None = None, q_gain: torch.Tensor | None = None,
                    k_gain: torch.Tensor | None = None, eps: float | None = None, interleaved: bool = False,
                    out: tuple | None = None, stream=None):
    """qkv [batch, tokens, heads + 2 * kv_heads, dim] (bf16/fp32) -> (q, k, v), each [batch, tokens, its heads, dim].
    Queries and keys are divided by the root of their mean square + ``eps`` and multiplied by their gain [dim]
    (where ``eps`` is given), then rotated by position * frequencies (fp32[pairs]): the pairs are channels j and
    j + pairs, or 2 j and 2 j + 1 where ``interleaved``.  ``positions`` int32[batch] are the first tokens',
    int32[batch, tokens] every token's.  ``out`` = (q, k, v) receives them instead of new tensors."""
    if stream is not None:
        with _as_current(stream):
            return qar_norm_rotate(qkv, heads, kv_heads, positions, frequencies, q_gain, k_gain, eps, interleaved, out)
    if out is not None:
        out = tuple(out)
    made = _serve().norm_rotate(qkv, heads, kv_heads, positions, frequencies, q_gain, k_gain, eps, interleaved, out)
    if made is not None:
        return _done(made, "qar_norm_rotate")
    return _why_norm_rotate(qkv, heads, kv_heads, positions, frequencies, q_gain, k_gain, eps, interleaved, out)


def _why_norm_rotate(qkv, heads, kv_heads, positions, frequencies, q_gain, k_gain, eps, interleaved, out):
    _whole(heads, "heads", 1, 1 << 32)
    _whole(kv_heads, "kv_heads", 1, 1 << 32)
    if _dev(qkv, "qkv").dim() != 4 or qkv.shape[2] != heads + 2 * kv_heads:
        raise ValueError(f"qkv must be [batch, tokens, {heads + 2 * kv_heads}, dim], not {list(qkv.shape)}")
    _dtype_code(qkv.dtype)
    (batch, tokens, _, dim), dev = qkv.shape, qkv.device
    each = isinstance(positions, torch.Tensor) and positions.dim() == 2
    _shaped(positions, "positions", (batch, tokens) if each else (batch,), _INT32, dev)
    if frequencies is not None:
        if _dev(frequencies, "frequencies").dim() != 1:
            raise ValueError(f"frequencies must have 1 dimension, not {frequencies.dim()}")
        _shaped(frequencies, "frequencies", tuple(frequencies.shape), _F32, dev)
    for t, what in ((q_gain, "q_gain"), (k_gain, "k_gain")):
        if t is not None:
            _shaped(t, what, (dim,), (qkv.dtype,), dev)
    if eps is not None:
        float(eps)
    if not isinstance(interleaved, bool):
        raise TypeError(f"interleaved must be True or False, not {interleaved}")
    if out is not None:
        if len(out) != 3:
            raise ValueError(f"out must be (q, k, v), not {len(out)} tensors")
        for t, what, n in zip(out, ("out[0]", "out[1]", "out[2]"), (heads, kv_heads, kv_heads)):
            _shaped(t, what, (batch, tokens, n, dim), (qkv.dtype,), dev)
    _on_current(qkv.get_device())
    raise ValueError("qar_norm_rotate: the arguments do not fit")
