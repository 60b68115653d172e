"""Thin Python binding over the C ABI of ``libdet.so`` (see ``include/det.h``).

Argument marshalling only: tensors become raw device pointers and sizes, the
current torch stream becomes the ``stream`` argument, and a workspace of the
size the library asks for is taken from torch's allocator when the caller
does not pass one.  Every step of every operation runs in the library's CUDA
kernels; there is no fallback.  If ``libdet.so`` is missing or cannot be
loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdet.so")

F32, F64 = 0, 1
BF16, F16 = 2, 3        # the language-model operators' 16-bit types (include/det_model.h)
MAX_TOP_K, MAX_BOUNDS = 32, 2047
OK = 0
ERR_CUDA = 6   # DET_ERR_CUDA: a CUDA call or launch failed (detail: det_last_cuda_error)
SCAN_INCLUSIVE, SCAN_EXCLUSIVE, SCAN_REVERSE = 0, 1, 2
SCAN_SEGMENT_RESTART = 4   # det_segmented_scan: each segment scanned as det_scan of the segment alone
SCAN_LANE_ELEMS = {torch.float32: 32, torch.float64: 16}
SCAN_CHUNK = {torch.float32: 32768, torch.float64: 16384}

_lock = threading.Lock()
_lib = None

_i64, _sz, _vp, _int, _flt = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_SIGNATURES = {
    "det_sum_workspace_bytes": (_sz, [_i64, _int]),
    "det_sum": (_int, [_vp, _i64, _int, _vp, _vp, _sz, _int, _vp]),
    "det_sum_noalloc": (_int, [_vp, _i64, _int, _vp, _int, _vp]),
    "det_scatter_add_workspace_bytes": (_sz, [_i64, _i64, _int]),
    "det_scatter_add": (_int, [_vp, _i64, _vp, _vp, _i64, _int, _vp, _vp, _vp, _sz, _int, _vp]),
    "det_scatter_add_rows_workspace_bytes": (_sz, [_i64, _i64, _i64, _int]),
    "det_scatter_add_rows": (_int, [_vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _int, _vp, _sz, _int, _vp]),
    "det_scan_workspace_bytes": (_sz, [_i64, _int]),
    "det_scan": (_int, [_vp, _vp, _i64, _int, _int, _vp, _vp, _sz, _int, _vp]),
    "det_segmented_scan_workspace_bytes": (_sz, [_i64, _i64, _int]),
    "det_segmented_scan": (_int, [_vp, _vp, _i64, _vp, _i64, _int, _int, _vp, _sz, _int, _vp]),
    "det_scatter_add_rows_ordered": (_int, [_vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _int, _vp, _sz, _int, _vp]),
    "det_scatter_add_vec_workspace_bytes": (_sz, [_i64, _i64, _i64, _int]),
    "det_scatter_add_vec": (_int, [_vp, _i64, _i64, _vp, _vp, _i64, _int, _vp, _sz, _int, _vp]),
    "det_gather_rows": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _i64, _int, _int, _vp]),
    "det_scatter_sub": (_int, [_vp, _i64, _vp, _vp, _i64, _int, _vp, _vp, _vp, _sz, _int, _vp]),
    "det_scatter_minmax_workspace_bytes": (_sz, [_i64, _int]),
    "det_scatter_min": (_int, [_vp, _i64, _vp, _vp, _i64, _int, _vp, _sz, _int, _vp]),
    "det_scatter_max": (_int, [_vp, _i64, _vp, _vp, _i64, _int, _vp, _sz, _int, _vp]),
    "det_scan_i32_workspace_bytes": (_sz, [_i64]),
    "det_scan_i32": (_int, [_vp, _vp, _i64, _int, _vp, _vp, _sz, _int, _vp]),
    "det_slot_alloc_workspace_bytes": (_sz, [_i64, _i64]),
    "det_slot_alloc": (_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _sz, _int, _vp]),
    "det_token_logprobs": (_int, [_vp, _i64, _i64, _i64, _vp, _int, _vp, _vp, _vp, _int, _vp, _vp, _vp]),
    "det_token_logprobs_backward": (_int, [_vp, _i64, _i64, _i64, _vp, _int, _vp, _vp, _vp, _vp, _vp, _i64, _vp]),
    "det_relative_bias": (_int, [_vp, _int, _i64, _vp, _i64, _int, _i64, _i64, _i64, _vp, _int, _vp]),
    "det_relative_bias_backward_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _i64, _int]),
    "det_relative_bias_backward": (_int, [_vp, _int, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _int, _i64,
                                          _vp, _int, _vp, _sz, _vp]),
    "det_paged_attention_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "det_paged_attention": (_int, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _vp,
                                   _i64, _i64, _vp, _i64, _i64, _i64, _i64, _int, _flt, _vp, _int, _vp, _i64, _i64,
                                   _vp, _vp, _vp, _sz, _vp]),
    "det_read_status": (_int, [_vp, _vp, ctypes.POINTER(_int)]),
    "det_status_string": (ctypes.c_char_p, [_int]),
    "det_last_cuda_error": (ctypes.c_char_p, []),
    "det_profile_set_events": (_int, [_vp, _int]),
    "det_profile_event_count": (_int, []),
    "det_profile_event_name": (ctypes.c_char_p, [_int]),
    "det_launch_count": (ctypes.c_ulonglong, []),
    "det_test_scan_withhold": (_int, [_i64, ctypes.c_uint64]),
    "det_profile_add_rate_probe": (_int, [_int, _int, _vp, _vp, ctypes.POINTER(ctypes.c_ulonglong)]),
    "det_atomic_sum": (_int, [_vp, _i64, _int, _vp, _vp]),
    "det_atomic_scatter_add": (_int, [_vp, _i64, _vp, _vp, _i64, _int, _vp]),
    "det_atomic_scatter_add_rows": (_int, [_vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _int, _vp]),
    "det_atomic_slot_alloc": (_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp]),
    "det_dlb_scan_workspace_bytes": (_sz, [_i64, _int]),
    "det_dlb_scan": (_int, [_vp, _vp, _i64, _int, _vp, _sz, _vp]),
}


class DetError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        detail = ""
        if code == ERR_CUDA:
            try:
                detail = " [" + lib().det_last_cuda_error().decode() + "]"
            except Exception:  # pragma: no cover - only when the library is absent
                pass
        super().__init__(f"{what}: {status_string(code)} (code {code}){detail}")


def lib():
    """The loaded ``libdet.so``; raises if it has not been built."""
    global _lib
    if _lib is not None:   # loaded: no lock on the per-call path
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                                   "(python -c 'import __graft_entry__ as g; g.build()')")
            handle = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(handle, name, None)
                if fn is None:
                    continue
                fn.restype = res
                fn.argtypes = args
            _lib = handle
    return _lib


def exported_symbols():
    h = lib()
    return {name for name in _SIGNATURES if getattr(h, name, None) is not None}


def status_string(code: int) -> str:
    try:
        return lib().det_status_string(int(code)).decode()
    except Exception:  # pragma: no cover - only when the library is absent
        return "unknown"


def _code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.float64:
        return F64
    raise TypeError(f"det supports float32 and float64 tensors, got {t.dtype}")


def _dev(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


# the current stream's handle without the Stream object around it (0.1 us instead of 3)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device=None) -> int:
    if stream is None:
        if device is not None and _raw_stream is not None:
            return _raw_stream(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def workspace(nbytes: int, device) -> torch.Tensor:
    """A device byte buffer with a 256-byte aligned start of at least nbytes."""
    buf = torch.empty(int(nbytes) + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + int(nbytes)]


def _ws(ws, nbytes, device):
    if ws is None:
        ws = workspace(nbytes, device)
    if ws.numel() < nbytes:
        raise DetError(4, "workspace")
    return ws


def _check(rc: int, what: str):
    if rc != OK:
        raise DetError(rc, what)


def read_status(ws: torch.Tensor, stream=None) -> int:
    st = _int(0)
    _check(lib().det_read_status(_ptr(ws), _stream(stream), ctypes.byref(st)), "det_read_status")
    return int(st.value)


# ---------------------------------------------------------------------------


def det_sum(x: torch.Tensor, out: torch.Tensor | None = None, *, block_threads: int = 0,
            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[0] = pairwise tree sum of x (see det.h)."""
    _dev(x, "x")
    code = _code(x)
    if out is None:
        out = torch.empty(1, dtype=x.dtype, device=x.device)
    n = x.numel()
    nbytes = lib().det_sum_workspace_bytes(n, code)
    ws = _ws(workspace, nbytes, x.device)
    _check(lib().det_sum(_ptr(x), n, code, _ptr(out), _ptr(ws), ws.numel(), block_threads,
                         _stream(stream)), "det_sum")
    return out


def det_scatter_add(out: torch.Tensor, bins: torch.Tensor, values: torch.Tensor, *,
                    perm_out: torch.Tensor | None = None, seg_offsets_out: torch.Tensor | None = None,
                    block_threads: int = 0, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """out[bins[i]] += values[i], in a fixed order (see det.h); returns out."""
    _dev(out, "out"), _dev(bins, "bins"), _dev(values, "values")
    code = _code(values)
    if out.dtype != values.dtype or bins.dtype != torch.int32:
        raise TypeError("out must match values' dtype and bins must be int32")
    n, m = values.numel(), out.numel()
    if bins.numel() != n:
        raise ValueError("bins and values differ in length")
    nbytes = lib().det_scatter_add_workspace_bytes(n, m, code)
    ws = _ws(workspace, nbytes, values.device)
    _check(lib().det_scatter_add(_ptr(out), m, _ptr(bins), _ptr(values), n, code, _ptr(perm_out),
                                 _ptr(seg_offsets_out), _ptr(ws), ws.numel(), block_threads,
                                 _stream(stream)), "det_scatter_add")
    return out


def det_gather_rows(src: torch.Tensor, idx: torch.Tensor, out: torch.Tensor | None = None, *, row_offset: int = 0,
                    block_threads: int = 0, stream=None) -> torch.Tensor:
    """out[i] = src[idx[i] + row_offset] (zeros outside src); src is 1-D (scalars) or 2-D (rows)."""
    _dev(src, "src"), _dev(idx, "idx")
    code = _code(src)
    if idx.dtype != torch.int32:
        raise TypeError("idx must be int32")
    W = 1 if src.dim() == 1 else src.shape[1]
    n = idx.numel()
    if out is None:
        out = torch.empty((n,) if src.dim() == 1 else (n, W), dtype=src.dtype, device=src.device)
    _check(lib().det_gather_rows(_ptr(out), _ptr(src), src.shape[0], W, _ptr(idx), int(row_offset), n, code,
                                 block_threads, _stream(stream)), "det_gather_rows")
    return out


def det_scatter_sub(out: torch.Tensor, bins: torch.Tensor, values: torch.Tensor, *,
                    perm_out: torch.Tensor | None = None, seg_offsets_out: torch.Tensor | None = None,
                    block_threads: int = 0, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """out[bins[i]] -= values[i]: the values negated and added in det_scatter_add's order; returns out."""
    _dev(out, "out"), _dev(bins, "bins"), _dev(values, "values")
    code = _code(values)
    if out.dtype != values.dtype or bins.dtype != torch.int32:
        raise TypeError("out must match values' dtype and bins must be int32")
    n, m = values.numel(), out.numel()
    if bins.numel() != n:
        raise ValueError("bins and values differ in length")
    nbytes = lib().det_scatter_add_workspace_bytes(n, m, code)
    ws = _ws(workspace, nbytes, values.device)
    _check(lib().det_scatter_sub(_ptr(out), m, _ptr(bins), _ptr(values), n, code, _ptr(perm_out),
                                 _ptr(seg_offsets_out), _ptr(ws), ws.numel(), block_threads,
                                 _stream(stream)), "det_scatter_sub")
    return out


def _scatter_minmax(fn, out, bins, values, block_threads, workspace, stream):
    _dev(out, "out"), _dev(bins, "bins"), _dev(values, "values")
    code = _code(values)
    if out.dtype != values.dtype or bins.dtype != torch.int32:
        raise TypeError("out must match values' dtype and bins must be int32")
    n, m = values.numel(), out.numel()
    if bins.numel() != n:
        raise ValueError("bins and values differ in length")
    ws = _ws(workspace, lib().det_scatter_minmax_workspace_bytes(m, code), values.device)
    _check(getattr(lib(), fn)(_ptr(out), m, _ptr(bins), _ptr(values), n, code, _ptr(ws), ws.numel(),
                              block_threads, _stream(stream)), fn)
    return out


def det_scatter_min(out: torch.Tensor, bins: torch.Tensor, values: torch.Tensor, *, block_threads: int = 0,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[b] = IEEE minimum of out[b] and the values aimed at b (see det.h); returns out."""
    return _scatter_minmax("det_scatter_min", out, bins, values, block_threads, workspace, stream)


def det_scatter_max(out: torch.Tensor, bins: torch.Tensor, values: torch.Tensor, *, block_threads: int = 0,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[b] = IEEE maximum of out[b] and the values aimed at b (see det.h); returns out."""
    return _scatter_minmax("det_scatter_max", out, bins, values, block_threads, workspace, stream)


def det_scan_i32(x: torch.Tensor, y: torch.Tensor | None = None, *, exclusive: bool = False,
                 total_out: torch.Tensor | None = None, block_threads: int = 0,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """int32 prefix sum modulo 2^32 (see det.h); y may be x; returns y."""
    _dev(x, "x")
    if x.dtype != torch.int32 or (y is not None and y.dtype != torch.int32):
        raise TypeError("det_scan_i32 takes int32 tensors")
    if total_out is not None and (total_out.dtype != torch.int32 or total_out.numel() < 1):
        raise TypeError("total_out must hold one int32")
    if y is None:
        y = torch.empty_like(x)
    n = x.numel()
    ws = _ws(workspace, lib().det_scan_i32_workspace_bytes(n), x.device)
    _check(lib().det_scan_i32(_ptr(x), _ptr(y), n, SCAN_EXCLUSIVE if exclusive else SCAN_INCLUSIVE, _ptr(total_out),
                              _ptr(ws), ws.numel(), block_threads, _stream(stream)), "det_scan_i32")
    return y


def det_slot_alloc(counter: torch.Tensor, index: torch.Tensor, *, count: torch.Tensor | None = None,
                   slot_out: torch.Tensor | None = None, index_offset: int = 0, block_threads: int = 0,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """slot = atomic_add(counter, index[i], count[i]) in thread order (see det.h); returns the slots."""
    _dev(counter, "counter"), _dev(index, "index")
    if counter.dtype != torch.int32 or index.dtype != torch.int32 or (count is not None and count.dtype != torch.int32):
        raise TypeError("det_slot_alloc takes int32 tensors")
    n = index.numel()
    if count is not None and count.numel() != n:
        raise ValueError("count must have one entry per record")
    if slot_out is None:
        slot_out = torch.empty(n, dtype=torch.int32, device=index.device)
    ws = _ws(workspace, lib().det_slot_alloc_workspace_bytes(n, counter.numel()), index.device)
    _check(lib().det_slot_alloc(_ptr(counter), counter.numel(), _ptr(index), int(index_offset), _ptr(count), n,
                                _ptr(slot_out), _ptr(ws), ws.numel(), block_threads, _stream(stream)),
           "det_slot_alloc")
    return slot_out


def det_scatter_add_rows(dst: torch.Tensor, idx: torch.Tensor, src: torch.Tensor, *, row_offset: int = 0,
                         prev_out: torch.Tensor | None = None, block_threads: int = 0,
                         workspace: torch.Tensor | None = None, stream=None, ordered: bool = False) -> torch.Tensor:
    """dst[idx[s] + row_offset] += src[s] row by row, in a fixed order; returns dst.

    ordered=False: per destination the rows are added by the pairwise tree and
    every contributor's prev is the row before the call.  ordered=True: the
    rows are applied one at a time in ascending s and prev is the running value
    (det_scatter_add_rows_ordered)."""
    _dev(dst, "dst"), _dev(idx, "idx"), _dev(src, "src")
    code = _code(src)
    if dst.dim() != 2 or src.dim() != 2 or dst.shape[1] != src.shape[1] or dst.dtype != src.dtype:
        raise ValueError("dst and src must be 2-D of one dtype with equal row length")
    if idx.dtype != torch.int32 or idx.numel() != src.shape[0]:
        raise ValueError("idx must be int32 with one entry per source row")
    R, W = dst.shape
    M = src.shape[0]
    nbytes = lib().det_scatter_add_rows_workspace_bytes(M, R, W, code)
    ws = _ws(workspace, nbytes, src.device)
    fn = "det_scatter_add_rows_ordered" if ordered else "det_scatter_add_rows"
    _check(getattr(lib(), fn)(_ptr(dst), R, W, _ptr(idx), int(row_offset), _ptr(src), M, _ptr(prev_out), code,
                              _ptr(ws), ws.numel(), block_threads, _stream(stream)), fn)
    return dst


def det_scatter_add_vec(out: torch.Tensor, bins: torch.Tensor, values: torch.Tensor, *, block_threads: int = 0,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[bins[i], :] += values[i, :] for composite values, component-wise in a fixed order; returns out."""
    _dev(out, "out"), _dev(bins, "bins"), _dev(values, "values")
    code = _code(values)
    if out.dim() != 2 or values.dim() != 2 or out.shape[1] != values.shape[1] or out.dtype != values.dtype:
        raise ValueError("out and values must be 2-D of one dtype with equal width")
    if bins.dtype != torch.int32 or bins.numel() != values.shape[0]:
        raise ValueError("bins must be int32 with one entry per record")
    m, width = out.shape
    n = values.shape[0]
    ws = _ws(workspace, lib().det_scatter_add_vec_workspace_bytes(n, m, width, code), values.device)
    _check(lib().det_scatter_add_vec(_ptr(out), m, width, _ptr(bins), _ptr(values), n, code, _ptr(ws), ws.numel(),
                                     block_threads, _stream(stream)), "det_scatter_add_vec")
    return out


def det_scan(x: torch.Tensor, y: torch.Tensor | None = None, *, flags: int = SCAN_INCLUSIVE,
             total_out: torch.Tensor | None = None, block_threads: int = 0,
             workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Anchored look-back prefix sum (see det.h); y may be x; returns y."""
    _dev(x, "x")
    code = _code(x)
    if y is None:
        y = torch.empty_like(x)
    n = x.numel()
    nbytes = lib().det_scan_workspace_bytes(n, code)
    ws = _ws(workspace, nbytes, x.device)
    _check(lib().det_scan(_ptr(x), _ptr(y), n, code, int(flags), _ptr(total_out), _ptr(ws), ws.numel(),
                          block_threads, _stream(stream)), "det_scan")
    return y


def det_segmented_scan(x: torch.Tensor, seg_offsets: torch.Tensor, y: torch.Tensor | None = None, *,
                       flags: int = SCAN_INCLUSIVE, block_threads: int = 0,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Segmented anchored look-back prefix sum over int64 CSR offsets."""
    _dev(x, "x"), _dev(seg_offsets, "seg_offsets")
    code = _code(x)
    if seg_offsets.dtype != torch.int64:
        raise TypeError("seg_offsets must be int64")
    if y is None:
        y = torch.empty_like(x)
    n, S = x.numel(), seg_offsets.numel() - 1
    nbytes = lib().det_segmented_scan_workspace_bytes(n, S, code)
    ws = _ws(workspace, nbytes, x.device)
    _check(lib().det_segmented_scan(_ptr(x), _ptr(y), n, _ptr(seg_offsets), S, code, int(flags), _ptr(ws),
                                    ws.numel(), block_threads, _stream(stream)), "det_segmented_scan")
    return y


# ---------------------------------------------------------------------------
# operators of language models (include/det_model.h)

_MODEL_CODES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_CACHE_CODES = {torch.bfloat16: BF16, torch.float16: F16}
_MOST_TOKENS = (1 << 31) - 2048


def _model_code(t: torch.Tensor, name: str, codes=_MODEL_CODES) -> int:
    code = codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be one of {[str(d) for d in codes]}, got {t.dtype}")
    return code


def _on(device, dtype, name: str, t: torch.Tensor, shape=None, contiguous: bool = True) -> torch.Tensor:
    """t, checked to be a tensor of this device, dtype and shape (each unless None)."""
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a CUDA tensor on one device with the others")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _unit_stride(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    return t


# torch.cuda.current_device() without its check that CUDA is initialized, which it is where there are CUDA tensors
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(device, fn, args):
    """fn(*args), a call of the library, with the tensors' device as the current one: kernels are launched on that, whatever
    the stream, and the library asks it for the number of SMs."""
    if _current_device() == device.index:
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _stream_object(stream, device):
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device)


def _hold(stream, device, *tensors):
    """Keeps the memory of a call's inputs until the work enqueued on `stream` has read them, should the caller drop
    them before."""
    s = _stream_object(stream, device)
    for t in tensors:
        if t is not None:
            t.record_stream(s)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A tensor that the work enqueued on `stream` writes: taken from that stream's memory (so no earlier work of
    another stream still uses it), and kept from reuse while the caller's current stream works on it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    s = _stream_object(stream, device)
    with torch.cuda.stream(s):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _model_ws(ws, nbytes, device, stream):
    if ws is None:
        # the allocator's blocks are 512-byte aligned
        return _empty((max(int(nbytes), 256),), torch.uint8, device, stream)
    _on(device, torch.uint8, "workspace", ws)
    if ws.numel() < nbytes:
        raise DetError(4, "workspace")
    return ws


class TokenLogprobs(NamedTuple):
    logprob: Optional[torch.Tensor]
    entropy: torch.Tensor
    lse: torch.Tensor
    top_logprob: Optional[torch.Tensor]
    top_index: Optional[torch.Tensor]


def _logit_rows(logits: torch.Tensor):
    """(rows, vocab, elements from one row to the next) of [..., vocab] logits."""
    _on(None, None, "logits", logits, contiguous=False)
    shape = logits.shape
    if len(shape) < 1:
        raise ValueError("logits must have at least one dimension")
    vocab = shape[-1]
    _unit_stride(logits, "logits")
    if len(shape) == 2:
        return shape[0], vocab, logits.stride(0)
    rows = shape[:-1].numel()   # without a vocabulary too: such rows have results
    if logits.is_contiguous():
        return rows, vocab, vocab
    stride = _row_stride(logits)
    if stride is None:
        raise ValueError("logits of other than two dimensions must have one stride from each row to the next")
    return rows, vocab, stride


def _row_stride(logits: torch.Tensor) -> Optional[int]:
    """The elements from each row of [..., vocab] logits to the next, or None if they differ (logits[:, :-1])."""
    stride = None
    for n, step in zip(reversed(logits.shape[:-1]), reversed(logits.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride, after = step, step * n
        elif step != after:
            return None
        else:
            after *= n
    return logits.shape[-1] if stride is None else stride


def det_token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *, top_k: int = 0,
                       stream=None) -> TokenLogprobs:
    """Log probabilities of the tokens under softmax(logits), entropy, log-sum-exp and the top_k
    alternatives of every row (see det_model.h).

    logits is [..., vocab] (float32, bfloat16 or float16) with any one stride from each row to the next, tokens
    int32 of the leading shape, or None for the other results alone.  Results are float32 of the leading shape
    (top_*: with top_k appended; top_index int32)."""
    rows, vocab, stride = _logit_rows(logits)
    code = _MODEL_CODES.get(logits.dtype)
    if code is None:
        _model_code(logits, "logits")
    dev, lead = logits.device, logits.shape[:-1]
    f32 = torch.float32
    logprob = token_ptr = logprob_ptr = top_logprob = top_index = top_lp_ptr = top_ix_ptr = None
    if tokens is not None:
        _on(dev, torch.int32, "tokens", tokens, lead)
        logprob = _empty(lead, f32, dev, stream)
        token_ptr, logprob_ptr = tokens.data_ptr(), logprob.data_ptr()
    entropy = _empty(lead, f32, dev, stream)
    lse = _empty(lead, f32, dev, stream)
    if top_k:
        if not 0 < top_k <= min(vocab, MAX_TOP_K):
            raise ValueError(f"top_k must be at most {MAX_TOP_K} and the vocabulary, got {top_k}")
        top_shape = (*lead, top_k)
        top_logprob = _empty(top_shape, f32, dev, stream)
        top_index = _empty(top_shape, torch.int32, dev, stream)
        top_lp_ptr, top_ix_ptr = top_logprob.data_ptr(), top_index.data_ptr()
    rc = _run(dev, lib().det_token_logprobs, (logits.data_ptr(), rows, vocab, stride, token_ptr, code, logprob_ptr,
                                              entropy.data_ptr(), lse.data_ptr(), top_k, top_lp_ptr, top_ix_ptr,
                                              _stream(stream, dev)))
    if rc:
        raise DetError(rc, "det_token_logprobs")
    if stream is not None:
        _hold(stream, dev, logits, tokens)
    return TokenLogprobs(logprob, entropy, lse, top_logprob, top_index)


def det_token_logprobs_backward(logits: torch.Tensor, tokens: Optional[torch.Tensor], lse: torch.Tensor,
                                entropy: Optional[torch.Tensor] = None, *,
                                grad_logprob: Optional[torch.Tensor] = None,
                                grad_entropy: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """The gradient for the logits of sum(grad_logprob * logprob + grad_entropy * entropy) (see det_model.h);
    lse and entropy are det_token_logprobs' results.  Has the logits' dtype and shape."""
    rows, vocab, stride = _logit_rows(logits)
    code = _model_code(logits, "logits")
    dev, lead = logits.device, logits.shape[:-1]
    _on(dev, torch.float32, "lse", lse, lead)
    for name, t in (("entropy", entropy), ("grad_logprob", grad_logprob), ("grad_entropy", grad_entropy)):
        if t is not None:
            _on(dev, torch.float32, name, t, lead)
    if grad_logprob is not None and tokens is None:
        raise ValueError("grad_logprob needs the tokens")
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs the entropy")
    if tokens is not None:
        _on(dev, torch.int32, "tokens", tokens, lead)
    if out is None:
        out = _empty(logits.shape, logits.dtype, dev, stream)
    else:
        _on(dev, logits.dtype, "out", out, logits.shape, contiguous=out.dim() != 2)
    _, _, out_stride = _logit_rows(out)
    _check(_run(dev, lib().det_token_logprobs_backward,
                (_ptr(logits), rows, vocab, stride, _ptr(tokens), code, _ptr(lse), _ptr(entropy), _ptr(grad_logprob),
                 _ptr(grad_entropy), _ptr(out), out_stride, _stream(stream, dev))), "det_token_logprobs_backward")
    if stream is not None:
        _hold(stream, dev, logits, tokens, lse, entropy, grad_logprob, grad_entropy, out)
    return out


def det_relative_bounds(num_buckets: int, max_distance: int, *, bidirectional: bool = False,
                        device="cuda") -> torch.Tensor:
    """The bounds of the usual logarithmic buckets, for det_relative_bias: of the buckets of one direction the first
    half (rounded down) hold one distance each, the others are logarithmic steps up to max_distance, and the
    last one takes every distance from there.  Computed from the integers alone, so no distance moves between
    buckets by a rounded logarithm."""
    if num_buckets < 2 or (bidirectional and num_buckets % 2):
        raise ValueError("num_buckets must be at least 2, and even when bidirectional")
    n = num_buckets // 2 if bidirectional else num_buckets
    exact = max(n // 2, 1)
    if max_distance <= exact:
        raise ValueError(f"max_distance must be above {exact}")
    steps = n - exact
    bounds = list(range(1, exact + 1))[:n - 1]
    for j in range(1, steps):
        # least d with log(d / exact) / log(max_distance / exact) * steps >= j
        goal = max_distance ** j * exact ** (steps - j)
        lo, hi = bounds[-1], max_distance
        while lo < hi:
            mid = (lo + hi) // 2
            if mid ** steps >= goal:
                hi = mid
            else:
                lo = mid + 1
        bounds.append(lo)
    return torch.tensor(bounds, dtype=torch.int32, device=device)


def _bounds(bounds: torch.Tensor, device, bidirectional: bool):
    """(number of bounds, number of buckets)"""
    _on(device, torch.int32, "bounds", bounds)
    if bounds.dim() != 1:
        raise ValueError("bounds must have one dimension")
    n = bounds.numel()
    return n, (n + 1) * (2 if bidirectional else 1)


def det_relative_bias(table: torch.Tensor, bounds: torch.Tensor, q_len: int, k_len: int, *, q_offset: int = 0,
                      bidirectional: bool = False, dtype: Optional[torch.dtype] = None,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[h, i, j] = table[bucket(j - i - q_offset), h], [heads, q_len, k_len] (see det_model.h).

    table is [buckets, heads]; bounds int32, the least distance of each bucket after the first, in rising order
    (det_relative_bounds); the result has the table's dtype unless dtype or out says otherwise."""
    _on(None, None, "table", table)
    if table.dim() != 2:
        raise ValueError("table must be [buckets, heads]")
    n, buckets = _bounds(bounds, table.device, bidirectional)
    heads = table.shape[1]
    if table.shape[0] != buckets:
        raise ValueError(f"the table must have {buckets} rows for {n} bounds, got {table.shape[0]}")
    table_code = _model_code(table, "table")
    if out is None:
        out = _empty((heads, q_len, k_len), dtype or table.dtype, table.device, stream)
    else:
        _on(table.device, dtype, "out", out, (heads, q_len, k_len))
    dev = table.device
    _check(_run(dev, lib().det_relative_bias,
                (table.data_ptr(), table_code, heads, bounds.data_ptr(), n, bool(bidirectional), q_len, k_len, q_offset,
                 out.data_ptr(), _model_code(out, "out"), _stream(stream, dev))), "det_relative_bias")
    if stream is not None:
        _hold(stream, dev, table, bounds, out)
    return out


def det_relative_bias_backward(grad: torch.Tensor, bounds: torch.Tensor, *, q_offset: int = 0,
                               bidirectional: bool = False, dtype: torch.dtype = torch.float32,
                               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient for det_relative_bias' table, [buckets, heads] of dtype: grad ([heads, q_len, k_len], or with a
    batch in front over which the bias was broadcast) summed over the pairs of each bucket (see det_model.h).  grad
    may have any strides but along the keys."""
    _on(None, None, "grad", grad, contiguous=False)
    if grad.dim() not in (3, 4):
        raise ValueError("grad must be [heads, q_len, k_len] or [batch, heads, q_len, k_len]")
    _unit_stride(grad, "grad")
    n, buckets = _bounds(bounds, grad.device, bidirectional)
    code = _model_code(grad, "grad")
    batch, (heads, q_len, k_len) = (grad.shape[0] if grad.dim() == 4 else 1), grad.shape[-3:]
    stride_b = grad.stride(0) if grad.dim() == 4 else 0
    out = _empty((buckets, heads), dtype, grad.device, stream)
    nbytes = lib().det_relative_bias_backward_workspace_bytes(batch, heads, q_len, k_len, n, int(bidirectional))
    ws = _model_ws(workspace, nbytes, grad.device, stream)
    dev = grad.device
    _check(_run(dev, lib().det_relative_bias_backward,
                (_ptr(grad), code, batch, heads, q_len, k_len, stride_b, grad.stride(-3), grad.stride(-2), _ptr(bounds), n,
                 int(bidirectional), int(q_offset), _ptr(out), _model_code(out, "dtype"), _ptr(ws), ws.numel(),
                 _stream(stream, dev))), "det_relative_bias_backward")
    if stream is not None:
        _hold(stream, dev, grad, bounds, workspace)
    return out


def _cache(device, dtype, name: str, t: torch.Tensor, shape):
    """(pointer, strides of pages, tokens and heads) of a key or value cache."""
    _on(device, dtype, name, t, shape, False)
    s_page, s_token, s_head, s_dim = t.stride()
    ptr = t.data_ptr()
    if s_dim != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if (ptr | (s_page | s_token | s_head) * 2) & 15:
        raise ValueError(f"{name} must be 16-byte aligned with strides that are multiples of 8 elements")
    return ptr, s_page, s_token, s_head


class PagedAttention(NamedTuple):
    out: torch.Tensor
    lse: torch.Tensor


def det_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                        lengths: torch.Tensor, *, scale: Optional[float] = None, max_len: Optional[int] = None,
                        bias_table: Optional[torch.Tensor] = None, bias_bounds: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> PagedAttention:
    """Attention of the last token of each sequence over its paged key-value cache (see det_model.h).

    q is [batch, heads, head_dim] (bfloat16 or float16, head_dim 64, 128 or 256); the caches are [pages, page_size,
    kv_heads, head_dim] views of any strides that are multiples of 8 elements; block_table is int32 [batch,
    max_pages], lengths int32 [batch].  scale defaults to head_dim ** -0.5.  max_len, a bound on the lengths that
    the host knows, saves launching for the whole table; longer sequences are cut at it.  bias_table
    ([buckets, heads], with bias_bounds as in det_relative_bias) adds the learned relative position bias.
    Returns the output, [batch, heads, head_dim] of q's dtype, and the scores' log-sum-exp, float32 [batch, heads]."""
    dev, dtype = q.device, q.dtype
    _on(None, None, "q", q, None, False)
    code = _CACHE_CODES.get(dtype)
    if code is None:
        _model_code(q, "q", _CACHE_CODES)
    cache_shape = k_cache.shape
    if q.dim() != 3 or len(cache_shape) != 4:
        raise ValueError("q must be [batch, heads, head_dim] and the caches [pages, page_size, kv_heads, head_dim]")
    batch, heads, dim = q.shape
    pages, page_size, kv_heads, cache_dim = cache_shape
    q_batch, q_head, q_dim = q.stride()
    if dim not in (64, 128, 256) or cache_dim != dim:
        raise ValueError(f"head_dim must be 64, 128 or 256 and the caches', got {dim} and {cache_dim}")
    if page_size < 1 or kv_heads < 1 or heads % kv_heads:
        raise ValueError("page_size must be positive and heads a multiple of kv_heads")
    if q_dim != 1:
        raise ValueError("q must be contiguous along its last dimension")
    k_ptr, k_page, k_token, k_head = _cache(dev, dtype, "k_cache", k_cache, None)
    v_ptr, v_page, v_token, v_head = _cache(dev, dtype, "v_cache", v_cache, cache_shape)
    _on(dev, torch.int32, "block_table", block_table, None, False)
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError("block_table must be [batch, max_pages]")
    max_pages = block_table.shape[1]
    table_stride, table_unit = block_table.stride()
    if table_unit != 1 and max_pages > 1:
        raise ValueError("block_table must be contiguous along its last dimension")
    _on(dev, torch.int32, "lengths", lengths, (batch,))
    bias_ptr = bounds_ptr = None
    bias_code = n_bounds = 0
    if bias_table is not None:
        if bias_bounds is None:
            raise ValueError("bias_table needs bias_bounds")
        n_bounds, buckets = _bounds(bias_bounds, dev, False)
        bias_code = _model_code(bias_table, "bias_table")
        _on(dev, None, "bias_table", bias_table)
        if bias_table.dim() != 2 or bias_table.shape[1] != heads or bias_table.shape[0] not in (buckets, 2 * buckets):
            raise ValueError(f"bias_table must be [{buckets} or {2 * buckets}, {heads}]")
        bias_ptr, bounds_ptr = bias_table.data_ptr(), bias_bounds.data_ptr()
    limit = min(max_pages * page_size, _MOST_TOKENS)
    if max_len is not None and max_len < limit:
        limit = int(max_len)
        if limit < 0:
            raise ValueError("max_len must not be negative")
    if out is None:
        out = _empty((batch, heads, dim), dtype, dev, stream)
    else:
        _on(dev, dtype, "out", out, (batch, heads, dim))
    lse = _empty((batch, heads), torch.float32, dev, stream)
    call = lib()
    ws = _model_ws(workspace, call.det_paged_attention_workspace_bytes(batch, heads, dim, limit), dev, stream)
    rc = _run(dev, call.det_paged_attention, (
        q.data_ptr(), q_batch, q_head, k_ptr, k_page, k_token, k_head, v_ptr, v_page, v_token, v_head, pages, page_size,
        block_table.data_ptr(), table_stride, max_pages, lengths.data_ptr(), batch, heads, kv_heads, dim, code,
        dim ** -0.5 if scale is None else scale, bias_ptr, bias_code, bounds_ptr, n_bounds, limit, out.data_ptr(),
        lse.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream, dev)))
    if rc:
        raise DetError(rc, "det_paged_attention")
    if stream is not None:
        _hold(stream, dev, q, k_cache, v_cache, block_table, lengths, bias_table, bias_bounds, out, workspace)
    return PagedAttention(out, lse)


# ---------------------------------------------------------------------------
# measurement hooks (include/det_profile.h)


class KernelTimer:
    """Records a CUDA event pair around each kernel the library launches
    while active; ``kernels()`` returns [(name, ms), ...] in launch order."""

    def __init__(self, capacity: int = 256):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * capacity)]
        for e in self.events:
            e.record()  # materialise the underlying cudaEvent_t
        torch.cuda.synchronize()
        self._arr = (ctypes.c_void_p * len(self.events))(*[e.cuda_event for e in self.events])
        self.capacity = capacity

    def __enter__(self):
        lib().det_profile_set_events(self._arr, self.capacity)
        return self

    def __exit__(self, *exc):
        self._count = lib().det_profile_event_count()
        self._names = [lib().det_profile_event_name(i).decode() for i in range(self._count)]
        lib().det_profile_set_events(None, 0)
        return False

    def kernels(self):
        torch.cuda.synchronize()
        return [(self._names[i], self.events[2 * i].elapsed_time(self.events[2 * i + 1]))
                for i in range(self._count)]


def launch_count() -> int:
    return int(lib().det_launch_count())


def add_rate_probe(dtype: torch.dtype, iters: int, sink: torch.Tensor, stream=None) -> int:
    """Enqueue the add-only probe launch; returns the additions it performs."""
    adds = ctypes.c_ulonglong(0)
    code = F32 if dtype == torch.float32 else F64
    _check(lib().det_profile_add_rate_probe(code, int(iters), _ptr(sink), _stream(stream), ctypes.byref(adds)),
           "det_profile_add_rate_probe")
    return int(adds.value)


# ---------------------------------------------------------------------------
# nondeterministic baselines (include/det_baselines.h): comparison only


def atomic_sum(x: torch.Tensor, out: torch.Tensor, stream=None) -> torch.Tensor:
    _check(lib().det_atomic_sum(_ptr(x), x.numel(), _code(x), _ptr(out), _stream(stream)), "det_atomic_sum")
    return out


def atomic_scatter_add(out: torch.Tensor, bins: torch.Tensor, values: torch.Tensor, stream=None) -> torch.Tensor:
    _check(lib().det_atomic_scatter_add(_ptr(out), out.numel(), _ptr(bins), _ptr(values), values.numel(),
                                        _code(values), _stream(stream)), "det_atomic_scatter_add")
    return out


def atomic_scatter_add_rows(dst, idx, src, prev_out=None, row_offset: int = 0, stream=None):
    R, W = dst.shape
    _check(lib().det_atomic_scatter_add_rows(_ptr(dst), R, W, _ptr(idx), int(row_offset), _ptr(src), src.shape[0],
                                             _ptr(prev_out), _code(src), _stream(stream)),
           "det_atomic_scatter_add_rows")
    return dst


def dlb_scan(x: torch.Tensor, y: torch.Tensor, workspace: torch.Tensor | None = None, stream=None):
    nbytes = lib().det_dlb_scan_workspace_bytes(x.numel(), _code(x))
    ws = _ws(workspace, nbytes, x.device)
    _check(lib().det_dlb_scan(_ptr(x), _ptr(y), x.numel(), _code(x), _ptr(ws), ws.numel(), _stream(stream)),
           "det_dlb_scan")
    return y


def atomic_slot_alloc(counter: torch.Tensor, index: torch.Tensor, slot_out: torch.Tensor, *,
                      count: torch.Tensor | None = None, index_offset: int = 0, stream=None) -> torch.Tensor:
    """Baseline: slot = atomicAdd(counter[index[i]], ...) in arrival order (see det_baselines.h)."""
    _check(lib().det_atomic_slot_alloc(_ptr(counter), counter.numel(), _ptr(index), int(index_offset), _ptr(count),
                                       index.numel(), _ptr(slot_out), _stream(stream)), "det_atomic_slot_alloc")
    return slot_out
