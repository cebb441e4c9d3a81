"""ctypes binding of libsmla.so: argument marshalling only.

Names follow the C ABI (``include/smla.h``): ``decode`` -> ``smla_decode_ex``,
``combine`` -> ``smla_combine``, ``debug_gather`` -> ``smla_debug_gather``,
``workspace_bytes`` -> ``smla_workspace_bytes_ex``, ``read_error`` ->
``smla_read_error``, and ``read_kv``, ``span_keys``, ``span_scores``,
``select_spans``, ``decode_spans`` -> the entry points of the same names.  Tensors must already be on the current CUDA device, dense
and of the documented dtype; nothing is copied or converted here.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

from . import build as _build

SMLA_FLAG_BAD_PAGE = 0x1
SMLA_FLAG_TIMEOUT = 0x2
SMLA_FLAG_SMEM = 0x4
SMLA_DEBUG_SKIP_FIRST_COMMIT = 0x1
HEADS = 64
DIM = 512
PAGE_BYTES = 149504
SPAN_TOKENS = 64
PAGE_SPANS = 4
MAX_NSEL = 1024

_ERRORS = {-1: "invalid argument", -2: "unsupported device (needs sm_100)", -3: "CUDA runtime error",
           -4: "kernel launch failed"}


class SmlaError(RuntimeError):
    pass


class _Options(ctypes.Structure):
    _fields_ = [("nsplit", ctypes.c_int), ("out_bf16", ctypes.c_int), ("wait_timeout_ns", ctypes.c_uint64),
                ("debug_flags", ctypes.c_uint32), ("reserved1", ctypes.c_uint32)]


_lock = threading.Lock()
_lib = None


def library():
    """Load libsmla.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_build.LIB):
                raise SmlaError(f"{_build.LIB} is missing: build it with sparse_mla_decode_fp8_b200.build.build()")
            lib = ctypes.CDLL(_build.LIB)
            P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            lib.smla_decode.argtypes = [P, P, P, P, P, ctypes.c_float, P, P, I, I, I, I, I, P, Z, P]
            lib.smla_decode.restype = I
            lib.smla_decode_ex.argtypes = [P, P, P, P, P, ctypes.c_float, P, P, I, I, I, I, I, P, Z,
                                           ctypes.POINTER(_Options), P]
            lib.smla_decode_ex.restype = I
            lib.smla_combine.argtypes = [P, P, I, P, P, I, I, P]
            lib.smla_combine.restype = I
            lib.smla_num_splits.argtypes = [I, I, I]
            lib.smla_num_splits.restype = I
            lib.smla_workspace_bytes.argtypes = [I, I, I]
            lib.smla_workspace_bytes.restype = Z
            lib.smla_workspace_bytes_ex.argtypes = [I, I, I, I]
            lib.smla_workspace_bytes_ex.restype = Z
            lib.smla_read_error.argtypes = [P, P, ctypes.POINTER(ctypes.c_uint32)]
            lib.smla_read_error.restype = I
            lib.smla_debug_gather.argtypes = [P, P, P, P, I, I, I, I, P, P, P, Z, P]
            lib.smla_debug_gather.restype = I
            lib.smla_write_kv.argtypes = [P, I, I, P, P, P, I, I, I, P, P, P]
            lib.smla_write_kv.restype = I
            lib.smla_read_kv.argtypes = [P, P, P, I, P, I, I, I, P, I, P, P]
            lib.smla_read_kv.restype = I
            lib.smla_span_keys.argtypes = [P, P, P, P, P, I, I, I, I, P, P, P]
            lib.smla_span_keys.restype = I
            lib.smla_select_spans.argtypes = [P, I, P, I, I, I, P, P, I, P]
            lib.smla_select_spans.restype = I
            lib.smla_decode_spans.argtypes = [P, P, P, P, I, P, ctypes.c_float, P, P, I, I, I, I, P, Z,
                                              ctypes.POINTER(_Options), P]
            lib.smla_decode_spans.restype = I
            lib.smla_decode_spans_workspace_bytes.argtypes = [I]
            lib.smla_decode_spans_workspace_bytes.restype = Z
            lib.smla_span_scores.argtypes = [P, P, P, P, ctypes.c_float, P, I, I, I, I, P, Z, ctypes.POINTER(_Options), P]
            lib.smla_span_scores.restype = I
            lib.smla_span_scores_workspace_bytes.argtypes = [I, I]
            lib.smla_span_scores_workspace_bytes.restype = Z
            lib.smla_version.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise SmlaError(f"{what}: {_ERRORS.get(rc, rc)}")


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor, dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SmlaError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise SmlaError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise SmlaError(f"{name} must be contiguous")
    return t.data_ptr()


def version() -> str:
    return library().smla_version().decode()


def num_splits(B: int, topk: int) -> int:
    n = library().smla_num_splits(B, HEADS, topk)
    _check(min(n, 0), "smla_num_splits")
    return n


def workspace_bytes(B: int, topk: int, nsplit: int = 0) -> int:
    lib = library()
    n = lib.smla_workspace_bytes_ex(B, HEADS, topk, nsplit) if nsplit else lib.smla_workspace_bytes(B, HEADS, topk)
    if n == 0:
        raise SmlaError("smla_workspace_bytes: invalid sizes")
    return int(n)


def new_workspace(B: int, topk: int, nsplit: int = 0, device=None) -> torch.Tensor:
    """A zeroed uint8 workspace of the required size (the first 4 bytes are the error word)."""
    n = workspace_bytes(B, topk, nsplit)
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def decode(q, kv_cache, block_table, topk_idx, seq_lens, sm_scale, out=None, lse=None, workspace=None,
           nsplit: int = 0, wait_timeout_ns: int = 0, debug_flags: int = 0, stream=None, out_dtype=None):
    """smla_decode_ex: returns (out [B,64,512], lse fp32 [B,64]).  out is fp32, or bf16 when
    ``out_dtype`` is torch.bfloat16 or a bf16 ``out`` tensor is given."""
    B, H, D = q.shape
    topk = topk_idx.shape[1]
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.float32
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise SmlaError("out must be float32 or bfloat16")
    if out is None:
        out = torch.empty((B, H, D), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(B, topk, nsplit, q.device)
    opts = _Options(nsplit, 1 if out_dtype == torch.bfloat16 else 0, wait_timeout_ns, debug_flags, 0)
    rc = library().smla_decode_ex(
        _dev(q, torch.bfloat16, "q"), _dev(kv_cache, torch.uint8, "kv_cache"),
        _dev(block_table, torch.int32, "block_table"), _dev(topk_idx, torch.int32, "topk_idx"),
        _dev(seq_lens, torch.int32, "seq_lens"), float(sm_scale), _dev(out, out_dtype, "out"),
        _dev(lse, torch.float32, "lse"), B, H, topk, block_table.shape[1], kv_cache.shape[0],
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), ctypes.byref(opts), _stream(stream))
    _check(rc, "smla_decode")
    return out, lse


def combine(part_o, part_lse, out=None, lse=None, stream=None):
    """smla_combine: merge [B,H,nsplit,512] partials by their log-sum-exp."""
    B, H, ns, D = part_o.shape
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.float32, device=part_o.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=part_o.device)
    rc = library().smla_combine(_dev(part_o, torch.float32, "part_o"), _dev(part_lse, torch.float32, "part_lse"), ns,
                                _dev(out, torch.float32, "out"), _dev(lse, torch.float32, "lse"), B, H,
                                _stream(stream))
    _check(rc, "smla_combine")
    return out, lse


def read_error(workspace, stream=None) -> int:
    """smla_read_error: synchronise, return and clear the device error word."""
    v = ctypes.c_uint32(0)
    _check(library().smla_read_error(_dev(workspace, torch.uint8, "workspace"), _stream(stream), ctypes.byref(v)),
           "smla_read_error")
    return int(v.value)


def debug_gather(kv_cache, block_table, topk_idx, seq_lens, workspace=None, stream=None):
    """smla_debug_gather: (latents fp32 [B,topk,512], page_slot int32 [B,topk,2])."""
    B, topk = topk_idx.shape
    lat = torch.empty((B, topk, DIM), dtype=torch.float32, device=kv_cache.device)
    ps = torch.empty((B, topk, 2), dtype=torch.int32, device=kv_cache.device)
    if workspace is None:
        workspace = torch.zeros(256, dtype=torch.uint8, device=kv_cache.device)
    rc = library().smla_debug_gather(
        _dev(kv_cache, torch.uint8, "kv_cache"), _dev(block_table, torch.int32, "block_table"),
        _dev(topk_idx, torch.int32, "topk_idx"), _dev(seq_lens, torch.int32, "seq_lens"), B, topk,
        block_table.shape[1], kv_cache.shape[0], _dev(lat, torch.float32, "latents"),
        _dev(ps, torch.int32, "page_slot"), _dev(workspace, torch.uint8, "workspace"), workspace.numel(),
        _stream(stream))
    _check(rc, "smla_debug_gather")
    return lat, ps


def write_kv(latents, req, pos, block_table, kv_cache, err=None, stream=None) -> None:
    """smla_write_kv: quantise latents [n,512] (fp32 or bf16) into ``kv_cache`` at position
    pos[i] of request req[i]; ``err`` (a uint32 CUDA tensor of one element, or None)
    receives SMLA_FLAG_BAD_PAGE when a token's destination is out of range."""
    if latents.dtype not in (torch.float32, torch.bfloat16):
        raise SmlaError("latents must be float32 or bfloat16")
    n = latents.shape[0] if latents.dim() == 2 else 0
    if latents.dim() != 2 or latents.shape[1] != DIM:
        raise SmlaError("latents must be [n, 512]")
    if req.shape != (n,) or pos.shape != (n,):
        raise SmlaError("req and pos must be [n]")
    ep = None
    if err is not None:
        if err.dtype not in (torch.int32, torch.uint32) or err.numel() < 1 or not err.is_cuda:
            raise SmlaError("err must be a CUDA int32/uint32 tensor")
        ep = err.data_ptr()
    rc = library().smla_write_kv(
        _dev(latents, latents.dtype, "latents"), 1 if latents.dtype == torch.bfloat16 else 0, n,
        _dev(req, torch.int32, "req"), _dev(pos, torch.int32, "pos"), _dev(block_table, torch.int32, "block_table"),
        block_table.shape[0], block_table.shape[1], kv_cache.shape[0], _dev(kv_cache, torch.uint8, "kv_cache"), ep,
        _stream(stream))
    _check(rc, "smla_write_kv")


# ---------------------------------------------------------------- long contexts: spans and reading back
# These calls take a few microseconds of GPU time at small sizes, so what the binding checks it checks
# cheaply: one comparison of dtype, device index, shape and density per tensor.
_INT_MAX = (1 << 31) - 1
_U8, _I32, _U32, _F32, _BF16 = torch.uint8, torch.int32, torch.uint32, torch.float32, torch.bfloat16


def _current(t, name) -> int:
    """The device index of ``t``, which must be the current CUDA device: the library launches there."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SmlaError(f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise SmlaError(f"{name} must be on the current CUDA device, got {t.device}")
    return dev


def _ptr(t, dtype, dev: int, shape, name) -> int:
    """Device pointer of a dense tensor of this dtype, device and shape (None: any size there)."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            got = t.shape
            if got == shape or (len(got) == len(shape) and all(a is None or a == b for a, b in zip(shape, got))):
                return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SmlaError(f"{name} must be a CUDA tensor")
    raise SmlaError(f"{name} must be a contiguous {dtype} {list(shape)} on device {dev}, got {t.dtype} {list(t.shape)} on {t.device}")


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _size(t, dims: int, name) -> torch.Size:
    if not isinstance(t, torch.Tensor):
        raise SmlaError(f"{name} must be a tensor of {dims} dimensions")
    shape = t.shape
    # ctypes would pass a size modulo 2^32 (sizes between the first and the last are fixed ones, which _ptr checks)
    if len(shape) != dims or shape[0] > _INT_MAX or shape[-1] > _INT_MAX:
        raise SmlaError(f"{name} must be a tensor of {dims} dimensions below 2^31, got {list(shape)}")
    return shape


def _options(out_bf16: int, wait_timeout_ns: int, debug_flags: int):
    """smla_options for a call, or None for the defaults."""
    if not wait_timeout_ns and not debug_flags:
        return None
    if not 0 <= wait_timeout_ns < 1 << 64 or not 0 <= debug_flags < 1 << 32:
        raise SmlaError("wait_timeout_ns must lie in [0, 2^64) and debug_flags must lie in [0, 2^32)")
    return ctypes.byref(_Options(0, out_bf16, wait_timeout_ns, debug_flags, 0))


@functools.lru_cache(maxsize=None)
def _device(dev: int) -> torch.device:
    return torch.device("cuda", dev)


def _as_stream(stream, dev: int) -> torch.cuda.Stream:
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(_stream(stream), device=dev)


def _new(stream, shape, dtype, dev: int) -> torch.Tensor:
    """A dense tensor allocated on the stream that will write it (by its strides: half the time of torch.empty)."""
    strides = (1,) if len(shape) == 1 else (shape[1], 1) if len(shape) == 2 else (shape[1] * shape[2], shape[2], 1)
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=_device(dev))
    with torch.cuda.stream(_as_stream(stream, dev)):
        return torch.empty_strided(shape, strides, dtype=dtype, device=_device(dev))


def _scratch(nbytes: int, dev: int, stream) -> torch.Tensor:
    """A workspace for one call: only the error word has to start at zero."""
    ws = _new(stream, (nbytes,), _U8, dev)
    if stream is None:
        ws[:4].zero_()
    else:
        with torch.cuda.stream(_as_stream(stream, dev)):
            ws[:4].zero_()
    return ws


def _workspace(ws, dev: int) -> int:
    if not isinstance(ws, torch.Tensor) or ws.dtype is not _U8 or ws.get_device() != dev or not ws.is_contiguous():
        raise SmlaError(f"workspace must be a contiguous uint8 tensor on device {dev}")
    return ws.data_ptr()


def _err(err, dev: int):
    if err is None:
        return None
    if not isinstance(err, torch.Tensor) or err.dtype not in (_I32, _U32) or err.numel() < 1 or err.get_device() != dev:
        raise SmlaError("err must be a CUDA int32/uint32 tensor")
    return err.data_ptr()


def read_kv(kv_cache, req, pos, block_table, out=None, out_dtype=None, err=None, stream=None):
    """smla_read_kv: the cached tokens at position pos[i] of request req[i] as latents [n,512],
    bf16 (the default) or fp32; rows of tokens out of range are zeros, and ``err`` receives
    SMLA_FLAG_BAD_PAGE."""
    dev = _current(kv_cache, "kv_cache")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else _BF16
    if out_dtype is not _F32 and out_dtype is not _BF16:
        raise SmlaError("out must be float32 or bfloat16")
    (n,) = _size(req, 1, "req")
    B, blocks = _size(block_table, 2, "block_table")
    pages = _size(kv_cache, 2, "kv_cache")[0]
    if out is None:
        out = _new(stream, (n, DIM), out_dtype, dev)
    rc = library().smla_read_kv(
        _ptr(kv_cache, _U8, dev, (pages, PAGE_BYTES), "kv_cache"), _ptr(req, _I32, dev, (n,), "req"),
        _ptr(pos, _I32, dev, (n,), "pos"), n, _ptr(block_table, _I32, dev, (B, blocks), "block_table"), B, blocks, pages,
        _ptr(out, out_dtype, dev, (n, DIM), "out"), 1 if out_dtype is _BF16 else 0, _err(err, dev), _raw_stream(stream, dev))
    _check(rc, "smla_read_kv")
    return out


def span_keys(kv_cache, block_table, seq_lens, req, span, keys, err=None, stream=None):
    """smla_span_keys: recomputes the keys of span[i] of request req[i] in ``keys``
    (bf16 [num_pages,4,512], returned); ``err`` receives SMLA_FLAG_BAD_PAGE when a span is
    skipped."""
    dev = _current(kv_cache, "kv_cache")
    (n,) = _size(req, 1, "req")
    B, blocks = _size(block_table, 2, "block_table")
    pages = _size(kv_cache, 2, "kv_cache")[0]
    rc = library().smla_span_keys(
        _ptr(kv_cache, _U8, dev, (pages, PAGE_BYTES), "kv_cache"), _ptr(block_table, _I32, dev, (B, blocks), "block_table"),
        _ptr(seq_lens, _I32, dev, (B,), "seq_lens"), _ptr(req, _I32, dev, (n,), "req"), _ptr(span, _I32, dev, (n,), "span"),
        n, B, blocks, pages, _ptr(keys, _BF16, dev, (pages, PAGE_SPANS, DIM), "keys"), _err(err, dev),
        _raw_stream(stream, dev))
    _check(rc, "smla_span_keys")
    return keys


def span_scores_workspace_bytes(B: int, max_blocks: int) -> int:
    n = library().smla_span_scores_workspace_bytes(B, max_blocks)
    if n == 0:
        raise SmlaError("smla_span_scores_workspace_bytes: invalid sizes")
    return int(n)


def span_scores(q, keys, block_table, seq_lens, sm_scale, scores=None, workspace=None, wait_timeout_ns: int = 0,
                debug_flags: int = 0, stream=None):
    """smla_span_scores: fp32 [B,4 max_blocks], the attention each span of a request should get
    by its key, summed over the heads.  Without a ``workspace`` one is allocated for the call
    (and its error word is lost)."""
    dev = _current(q, "q")
    opts = _options(0, wait_timeout_ns, debug_flags)
    B, blocks = _size(block_table, 2, "block_table")
    pages = _size(keys, 3, "keys")[0]
    if scores is None:
        scores = _new(stream, (B, blocks * PAGE_SPANS), _F32, dev)
    if workspace is None:
        workspace = _scratch(span_scores_workspace_bytes(B, blocks), dev, stream)
    rc = library().smla_span_scores(
        _ptr(q, _BF16, dev, (B, HEADS, DIM), "q"), _ptr(keys, _BF16, dev, (pages, PAGE_SPANS, DIM), "keys"),
        _ptr(block_table, _I32, dev, (B, blocks), "block_table"), _ptr(seq_lens, _I32, dev, (B,), "seq_lens"), float(sm_scale),
        _ptr(scores, _F32, dev, (B, blocks * PAGE_SPANS), "scores"), B, HEADS, blocks, pages, _workspace(workspace, dev),
        workspace.numel(), opts, _raw_stream(stream, dev))
    _check(rc, "smla_span_scores")
    return scores


def select_spans(scores, seq_lens, nsel: int, keep_first: int = 0, keep_last: int = 0, spans=None, topk_idx=None,
                 tokens: bool = True, stream=None):
    """smla_select_spans: (spans int32 [B,nsel], topk_idx int32 [B,64 nsel]), the second None
    when ``tokens`` is false."""
    dev = _current(scores, "scores")
    B, width = _size(scores, 2, "scores")
    if not 1 <= nsel <= MAX_NSEL:
        raise SmlaError(f"nsel must lie in [1, {MAX_NSEL}]")
    if keep_first < 0 or keep_last < 0 or keep_first + keep_last > nsel:
        raise SmlaError("keep_first and keep_last must not be negative and must not add up to more than nsel")
    if spans is None:
        spans = _new(stream, (B, nsel), _I32, dev)
    if topk_idx is None and tokens:
        topk_idx = _new(stream, (B, nsel * SPAN_TOKENS), _I32, dev)
    rc = library().smla_select_spans(
        _ptr(scores, _F32, dev, (B, width), "scores"), width, _ptr(seq_lens, _I32, dev, (B,), "seq_lens"), nsel, keep_first,
        keep_last, _ptr(spans, _I32, dev, (B, nsel), "spans"),
        None if topk_idx is None else _ptr(topk_idx, _I32, dev, (B, nsel * SPAN_TOKENS), "topk_idx"), B, _raw_stream(stream, dev))
    _check(rc, "smla_select_spans")
    return spans, topk_idx


def decode_spans_workspace_bytes(B: int) -> int:
    n = library().smla_decode_spans_workspace_bytes(B)
    if n == 0:
        raise SmlaError("smla_decode_spans_workspace_bytes: invalid B or no sm_100 device")
    return int(n)


def decode_spans(q, kv_cache, block_table, seq_lens, sm_scale, spans=None, out=None, lse=None, workspace=None,
                 wait_timeout_ns: int = 0, debug_flags: int = 0, stream=None):
    """smla_decode_spans: (out bf16 [B,64,512], lse fp32 [B,64]) over the whole sequences, or
    over ``spans`` (int32 [B,nsel]) of them.  Without a ``workspace`` one is allocated for the
    call (and its error word is lost)."""
    dev = _current(q, "q")
    opts = _options(1, wait_timeout_ns, debug_flags)
    B, blocks = _size(block_table, 2, "block_table")
    pages = _size(kv_cache, 2, "kv_cache")[0]
    nsel, listed = 0, None
    if spans is not None:
        nsel = _size(spans, 2, "spans")[1]
        if not 1 <= nsel <= MAX_NSEL:  # an empty list is not "every span"
            raise SmlaError(f"spans must be [B, nsel] with nsel in [1, {MAX_NSEL}]")
        listed = _ptr(spans, _I32, dev, (B, nsel), "spans")
    if out is None:
        out = _new(stream, (B, HEADS, DIM), _BF16, dev)
    if lse is None:
        lse = _new(stream, (B, HEADS), _F32, dev)
    if workspace is None:
        workspace = _scratch(decode_spans_workspace_bytes(B), dev, stream)
    rc = library().smla_decode_spans(
        _ptr(q, _BF16, dev, (B, HEADS, DIM), "q"), _ptr(kv_cache, _U8, dev, (pages, PAGE_BYTES), "kv_cache"),
        _ptr(block_table, _I32, dev, (B, blocks), "block_table"), listed, nsel, _ptr(seq_lens, _I32, dev, (B,), "seq_lens"),
        float(sm_scale), _ptr(out, _BF16, dev, (B, HEADS, DIM), "out"), _ptr(lse, _F32, dev, (B, HEADS), "lse"), B, HEADS, blocks,
        pages, _workspace(workspace, dev), workspace.numel(), opts, _raw_stream(stream, dev))
    _check(rc, "smla_decode_spans")
    return out, lse
