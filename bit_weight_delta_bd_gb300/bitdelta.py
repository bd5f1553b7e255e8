"""Thin ctypes binding of libbitdelta.so (include/bitdelta.h).

Argument marshalling only: every function here checks that its torch tensors
live on the current CUDA device with the expected dtype and layout, passes
their device pointers and the current CUDA stream to the C entry point of the
same name, and raises ``BitDeltaError`` on a non-OK status.  All arithmetic
runs in the library's sm_103a kernels; there is no fallback path, so a missing
or unloadable library raises instead of computing anything.

PyTorch is used for device memory and streams only.  bf16 buffers may be
passed as ``torch.bfloat16`` or as their ``torch.uint16``/``torch.int16`` bit
patterns.
"""
from __future__ import annotations

import array
import ctypes
import operator
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# BD_LIBRARY selects another build of the library (the bounds-checked one,
# libbitdelta_bounds.so, in its test)
LIB_PATH = os.environ.get("BD_LIBRARY") or os.path.join(_HERE, "libbitdelta.so")

BD_OK = 0
BD_ERR_INVALID_ARG = 1
BD_ERR_UNSUPPORTED_SHAPE = 2
BD_ERR_MISALIGNED = 3
BD_ERR_BAD_VARIANT = 4
BD_ERR_NONFINITE = 5
BD_ERR_CUDA = 6
BD_ERR_TIMEOUT = 7
BD_ERR_WORKSPACE = 8
BD_ERR_DEVICE = 9
BD_ERR_BOUNDS = 10
BD_ERR_BAD_INDEX = 11

BD_ALPHA_PER_MATRIX = 0
BD_ALPHA_PER_ROW = 1
BD_OUT_BF16 = 0
BD_OUT_F32 = 1
BD_OUT_E4M3 = 2
BD_KV_BF16 = 0
BD_KV_INT8 = 1
BD_KV_INT4 = 2
BD_MAX_AXES = 4
BD_MAX_VARIANTS = 64
BD_NOALLOC_MAX_ROWS = 262144

# Every symbol include/bitdelta.h declares.
EXPORTS = (
    "bd_version", "bd_status_string", "bd_last_cuda_error", "bd_cuda_error_string",
    "bd_compress_workspace_size", "bd_compress",
    "bd_linear_workspace_size", "bd_linear",
    "bd_linear_multi_workspace_size", "bd_linear_multi",
    "bd_route_workspace_size", "bd_route",
    "bd_debug_reconstruct", "bd_check_async", "bd_compress_noalloc", "bd_debug_bounds_check",
    "bd_debug_bounds_enabled",
    "bd_cache_create", "bd_cache_destroy", "bd_cache_set_source", "bd_cache_step", "bd_cache_release",
    "bd_cache_get_stats", "bd_cache_query", "bd_cache_debug_fail_load", "bd_materialize",
    "bd_monosoup_workspace_size", "bd_monosoup_merge",
    "bd_rms_norm_workspace_size", "bd_rms_norm",
    "bd_block_norm_workspace_size", "bd_block_norm",
    "bd_rope_append_workspace_size", "bd_rope_append",
    "bd_kv_read_workspace_size", "bd_kv_read",
    "bd_attention_workspace_size", "bd_attention",
)
BD_CACHE_SERVED = 0
BD_CACHE_BASE = 1
BD_CACHE_QUEUED = 2


class CacheStats(ctypes.Structure):
    """bd_cache_stats (include/bitdelta.h)."""
    _fields_ = [("steps", ctypes.c_int64), ("requests", ctypes.c_int64), ("hits", ctypes.c_int64),
                ("misses", ctypes.c_int64), ("queued", ctypes.c_int64), ("loads", ctypes.c_int64),
                ("evictions", ctypes.c_int64), ("bytes_loaded", ctypes.c_int64), ("slots", ctypes.c_int32),
                ("resident", ctypes.c_int32), ("pinned", ctypes.c_int32)]


class BitDeltaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        self.cuda_error = 0
        msg = f"{where}: {status_string(status)}"
        if self.status == BD_ERR_CUDA and _lib is not None:
            self.cuda_error = int(_lib.bd_last_cuda_error())
            msg += f" ({_lib.bd_cuda_error_string(self.cuda_error).decode()}, code {self.cuda_error})"
        super().__init__(msg)


_lib = None
_lock = threading.Lock()
_i64, _i32, _vp, _sz, _int = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libbitdelta.so (built by ``bit_weight_delta_bd_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"libbitdelta.so is not built ({path}); run __graft_entry__.build() first")
        lib = ctypes.CDLL(path)
        sig = {
            "bd_version": ([], _int),
            "bd_status_string": ([_int], ctypes.c_char_p),
            "bd_last_cuda_error": ([], _int),
            "bd_cuda_error_string": ([_int], ctypes.c_char_p),
            "bd_compress_workspace_size": ([_i64, _i64, _int], _sz),
            "bd_compress": ([_vp, _vp, _i64, _i64, _int, _vp, _vp, _vp, _sz, _vp], _int),
            "bd_linear_workspace_size": ([_i64, _i64, _i64], _sz),
            "bd_linear": ([_vp, _i64, _vp, _vp, _vp, _int, _i64, _i64, _vp, _int, _vp, _sz, _vp], _int),
            "bd_linear_multi_workspace_size": ([_i64, _i32, _i64, _i64], _sz),
            "bd_linear_multi": ([_vp, _i64, _vp, _i32, _vp, _vp, _int, _vp, _i64, _i64, _vp, _int, _vp, _sz, _vp],
                                _int),
            "bd_route_workspace_size": ([_i64, _i32], _sz),
            "bd_route": ([_vp, _i64, _i32, _vp, _vp, _vp, _sz, _vp], _int),
            "bd_debug_reconstruct": ([_vp, _vp, _vp, _int, _i64, _i64, _vp, _vp], _int),
            "bd_check_async": ([_vp, _vp], _int),
            "bd_debug_bounds_check": ([_vp], _int),
            "bd_debug_bounds_enabled": ([], _int),
            "bd_compress_noalloc": ([_vp, _vp, _i64, _i64, _int, _vp, _vp, _vp], _int),
            "bd_materialize": ([_vp, _vp, _vp, _int, _i64, _i64, _vp, _vp], _int),
            "bd_monosoup_workspace_size": ([_i64, _i64, _i32, _i32, _i32], _sz),
            "bd_monosoup_merge": ([_vp, _vp, _i32, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _int, _vp, _sz, _vp],
                                  _int),
            "bd_rms_norm_workspace_size": ([_i64, _i64], _sz),
            "bd_rms_norm": ([_vp, _vp, _i64, _i64, _vp, _vp, _i32, _vp, ctypes.c_float, _vp, _vp, _int, _vp, _vp, _sz,
                             _vp], _int),
            "bd_block_norm_workspace_size": ([_i64, _i64], _sz),
            "bd_block_norm": ([_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp, ctypes.c_float, ctypes.c_float, _vp, _vp,
                               _vp, _i32, ctypes.c_float, _vp, _vp, _int, _vp, _vp, _sz, _vp], _int),
            "bd_rope_append_workspace_size": ([_i64], _sz),
            "bd_rope_append": ([_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i32, _vp, _i32, _vp, _vp, _i64, _i32, _int,
                                _vp, _vp, _vp, _i64, _vp, _sz, _vp], _int),
            "bd_kv_read_workspace_size": ([_i64], _sz),
            "bd_kv_read": ([_vp, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _sz, _vp], _int),
            "bd_attention_workspace_size": ([_i64, _i64, _i32, _i32, _i32], _sz),
            "bd_attention": ([_vp, _i64, _vp, _i64, _i64, _i64, _i32, _vp, _vp, _i64, _vp, ctypes.c_float, _int, _vp,
                              _vp, _vp, _sz, _vp], _int),
            "bd_cache_create": ([_vp, _sz, _sz, _i32, ctypes.c_double, _vp, ctypes.POINTER(_vp)], _int),
            "bd_cache_destroy": ([_vp], None),
            "bd_cache_set_source": ([_vp, _i32, _vp, _sz], _int),
            "bd_cache_step": ([_vp, _vp, _i64, _vp, _vp, _vp], _int),
            "bd_cache_release": ([_vp, _vp], _int),
            "bd_cache_get_stats": ([_vp, ctypes.POINTER(CacheStats)], _int),
            "bd_cache_debug_fail_load": ([_vp, _i64], _int),
            "bd_cache_query": ([_vp, _i32, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                                ctypes.POINTER(ctypes.c_double)], _int),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def status_string(status: int) -> str:
    try:
        return load().bd_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def _check(status: int, where: str) -> None:
    if status != BD_OK:
        raise BitDeltaError(status, where)


_BF16_LIKE = (torch.bfloat16, torch.uint16, torch.int16)
_BF16_SET = frozenset(_BF16_LIKE)
_F32, _I32 = (torch.float32,), (torch.int32,)


def _ptr(t: torch.Tensor | None, name: str, dtypes=None, allow_none: bool = False, dev: int | None = None) -> int | None:
    # the usual case first: a call's checks cost more host time than a small
    # kernel takes (a CPU tensor's get_device() is -1)
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if (t.get_device() == (_device() if dev is None and t.is_cuda else dev) and (dtypes is None or t.dtype in dtypes)
            and t.is_contiguous()):
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not the current device")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    raise ValueError(f"{name} must be contiguous")


# torch's own short ways to the current device and stream (the public ones
# check the initialisation and build a Stream object on every call: 3 us)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream(stream, dev: int | None = None) -> int:
    return _raw_stream(_device() if dev is None else dev) if stream is None else stream.cuda_stream


def _ws(ws: torch.Tensor, dev: int | None = None) -> tuple[int, int]:
    if ws.dtype != torch.uint8:
        raise ValueError("workspace must be a torch.uint8 tensor")
    return _ptr(ws, "ws", None, False, dev), ws.numel()


def new_workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-filled workspace (the library requires zeros before first use)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


# ------------------------------------------------------------------------------- sizes

def bd_version() -> int:
    return int(load().bd_version())


def bd_compress_workspace_size(d_out: int, d_in: int, alpha_mode: int) -> int:
    return int(load().bd_compress_workspace_size(d_out, d_in, alpha_mode))


def bd_linear_workspace_size(T: int, d_out: int, d_in: int) -> int:
    return int(load().bd_linear_workspace_size(T, d_out, d_in))


def bd_linear_multi_workspace_size(T: int, V: int, d_out: int, d_in: int) -> int:
    return int(load().bd_linear_multi_workspace_size(T, V, d_out, d_in))


def bd_route_workspace_size(T: int, V: int) -> int:
    return int(load().bd_route_workspace_size(T, V))


# ------------------------------------------------------------------------------- calls

def bd_compress(w_base, w_ft, alpha_mode, signs, alpha, ws, stream=None) -> None:
    d_out, d_in = w_base.shape
    if tuple(w_ft.shape) != (d_out, d_in):
        raise ValueError("w_ft shape differs from w_base")
    wsp, wsn = _ws(ws)
    _check(load().bd_compress(_ptr(w_base, "w_base", _BF16_LIKE), _ptr(w_ft, "w_ft", _BF16_LIKE), d_out, d_in,
                              int(alpha_mode), _ptr(signs, "signs", (torch.int32, torch.uint32)),
                              _ptr(alpha, "alpha", (torch.float32,)), wsp, wsn, _stream(stream)), "bd_compress")


def bd_compress_noalloc(w_base, w_ft, alpha_mode, signs, alpha, stream=None) -> None:
    """bd_compress without a workspace, for callers that cannot allocate
    device memory; the library keeps the scratch in a fixed device array
    (at most BD_NOALLOC_MAX_ROWS rows; calls that overlap on the GPU race)."""
    d_out, d_in = w_base.shape
    if tuple(w_ft.shape) != (d_out, d_in):
        raise ValueError("w_ft shape differs from w_base")
    _check(load().bd_compress_noalloc(_ptr(w_base, "w_base", _BF16_LIKE), _ptr(w_ft, "w_ft", _BF16_LIKE), d_out,
                                      d_in, int(alpha_mode), _ptr(signs, "signs", (torch.int32, torch.uint32)),
                                      _ptr(alpha, "alpha", (torch.float32,)), _stream(stream)),
           "bd_compress_noalloc")


def bd_linear(x, w_base, signs, alpha, alpha_mode, y, ws, stream=None) -> None:
    T, d_in = x.shape
    d_out = w_base.shape[0]
    out_dtype = BD_OUT_F32 if y.dtype == torch.float32 else BD_OUT_BF16
    wsp, wsn = _ws(ws)
    _check(load().bd_linear(_ptr(x, "x", _BF16_LIKE), T, _ptr(w_base, "w_base", _BF16_LIKE),
                            _ptr(signs, "signs", (torch.int32, torch.uint32)), _ptr(alpha, "alpha", (torch.float32,)),
                            int(alpha_mode), d_out, d_in, _ptr(y, "y", (torch.float32, torch.bfloat16)), out_dtype,
                            wsp, wsn, _stream(stream)), "bd_linear")


def bd_linear_multi(x, vid, signs_list, alpha_list, alpha_mode, w_base, y, ws, stream=None) -> None:
    T, d_in = x.shape
    d_out = w_base.shape[0]
    V = len(signs_list)
    if len(alpha_list) != V:
        raise ValueError("signs_list and alpha_list differ in length")
    s_tab = (ctypes.c_void_p * max(V, 1))(*[_ptr(s, "signs", (torch.int32, torch.uint32)) for s in signs_list])
    a_tab = (ctypes.c_void_p * max(V, 1))(*[_ptr(a, "alpha", (torch.float32,)) for a in alpha_list])
    out_dtype = BD_OUT_F32 if y.dtype == torch.float32 else BD_OUT_BF16
    wsp, wsn = _ws(ws)
    _check(load().bd_linear_multi(_ptr(x, "x", _BF16_LIKE), T, _ptr(vid, "vid", (torch.int32,)), V,
                                  ctypes.addressof(s_tab), ctypes.addressof(a_tab), int(alpha_mode),
                                  _ptr(w_base, "w_base", _BF16_LIKE), d_out, d_in,
                                  _ptr(y, "y", (torch.float32, torch.bfloat16)), out_dtype, wsp, wsn,
                                  _stream(stream)), "bd_linear_multi")


def bd_materialize(w_base, signs, alpha, alpha_mode, w_eff, stream=None) -> None:
    d_out, d_in = w_base.shape
    _check(load().bd_materialize(_ptr(w_base, "w_base", _BF16_LIKE), _ptr(signs, "signs", (torch.int32, torch.uint32)),
                                 _ptr(alpha, "alpha", (torch.float32,)), int(alpha_mode), d_out, d_in,
                                 _ptr(w_eff, "w_eff", _BF16_LIKE), _stream(stream)), "bd_materialize")


def bd_monosoup_workspace_size(d_out: int, d_in: int, k: int, rank: int, l: int) -> int:
    return int(load().bd_monosoup_workspace_size(d_out, d_in, k, rank, l))


def bd_monosoup_merge(w_base, w_ft_list, rank, l, power_iters, omega, w_merged, ws, stream=None) -> None:
    """W_merged = W_base + (1/k) sum_i truncated_SVD_rank(W_i - W_base); omega [d_in][l] fp32 Gaussian."""
    d_out, d_in = w_base.shape
    k = len(w_ft_list)
    tab = (ctypes.c_void_p * max(k, 1))(*[_ptr(w, "w_ft", _BF16_LIKE) for w in w_ft_list])
    out_dtype = BD_OUT_F32 if w_merged.dtype == torch.float32 else BD_OUT_BF16
    wsp, wsn = _ws(ws)
    _check(load().bd_monosoup_merge(_ptr(w_base, "w_base", _BF16_LIKE), ctypes.addressof(tab), k, d_out, d_in,
                                    int(rank), int(l), int(power_iters),
                                    _ptr(omega, "omega", (torch.float32,), allow_none=True),
                                    _ptr(w_merged, "w_merged", _BF16_LIKE + (torch.float32,)), out_dtype, wsp, wsn,
                                    _stream(stream)), "bd_monosoup_merge")


def bd_rms_norm_workspace_size(T: int, d: int) -> int:
    return int(load().bd_rms_norm_workspace_size(T, d))


_dtype_of = operator.attrgetter("dtype")


def _row_ptrs(rows, n: int, name: str, dev: int) -> array.array:
    """Pointers of contiguous bf16 tensors of n elements.  (Checked a property at a time: a loop over 14 gains costs
    twice the time of the norm's kernel.)"""
    Tensor = torch.Tensor
    if not (set(map(Tensor.get_device, rows)) <= {dev} and set(map(Tensor.numel, rows)) <= {n}
            and set(map(_dtype_of, rows)) <= _BF16_SET and all(map(Tensor.is_contiguous, rows))):
        for t in rows:
            if t.numel() != n:
                raise ValueError(f"every {name} must have the shape [{n}]")
            _ptr(t, name, _BF16_LIKE, False, dev)
    return array.array("Q", map(Tensor.data_ptr, rows))


def bd_rms_norm(x, gain, eps, out, ws, residual=None, residual_out=None, scale=None, vid=None, gain_list=(),
                stream=None) -> None:
    """out = norm(x + residual) * gain (the gain of token t's variant, vid[t], out of gain_list); out bf16, fp32, or
    e4m3 with scale [T]; residual_out (which may be residual itself) receives x + residual."""
    shape = x.shape
    T, d = shape
    dev = _device()
    if gain.shape != (d,) or out.shape != shape:
        raise ValueError("gain must have the shape [d] and out that of x")
    if (residual is not None and residual.shape != shape) or (
            residual_out is not None and residual_out.shape != shape):
        raise ValueError("the residual's shape differs from x")
    if scale is not None and scale.numel() != T:
        raise ValueError("scale must have one value per row")
    if vid is not None and vid.numel() != T:
        raise ValueError("vid must have one id per row")
    tab, V = None, 0
    if vid is not None:
        V = len(gain_list)
        table = _row_ptrs(gain_list, d, "gain", dev)
        tab = table.buffer_info()[0] if V else None
    out_dtype = _OUT_DTYPES.get(out.dtype)
    if out_dtype is None:
        raise ValueError(f"out has dtype {out.dtype}, expected bfloat16, float32 or float8_e4m3fn")
    wsp, wsn = _ws(ws, dev)
    _check(load().bd_rms_norm(_ptr(x, "x", _BF16_LIKE, False, dev), _ptr(residual, "residual", _BF16_LIKE, True, dev),
                              T, d, _ptr(gain, "gain", _BF16_LIKE, False, dev), _ptr(vid, "vid", _I32, True, dev), V,
                              tab, eps, _ptr(residual_out, "residual_out", _BF16_LIKE, True, dev),
                              _ptr(out, "out", None, False, dev), out_dtype, _ptr(scale, "scale", _F32, True, dev),
                              wsp, wsn, _stream(stream, dev)), "bd_rms_norm")


def bd_block_norm_workspace_size(T: int, d: int) -> int:
    return int(load().bd_block_norm_workspace_size(T, d))


def bd_block_norm(x, residual, gain, eps, out, ws, residual_out=None, post_gain=None, gate=None, gate_idx=None,
                  block_scale: float = 1.0, residual_scale: float = 1.0, scale=None, vid=None, gain_list=(),
                  post_gain_list=(), stream=None) -> None:
    """The norms around a block that gave x: h = residual_scale * residual + block_scale * gate * norm(x) * post_gain,
    out = norm(h) * gain; residual_out (which may be residual itself) receives h.  post_gain None: x enters as it is.
    gate: [d] or [rows][d], one row for all tokens, a row for each, or row gate_idx[t] for token t.  Token t takes the
    gains of its variant, vid[t], out of gain_list and post_gain_list; out bf16, fp32, or e4m3 with scale [T]."""
    shape = x.shape
    T, d = shape
    dev = _device()
    if gain.shape != (d,) or out.shape != shape or residual.shape != shape:
        raise ValueError("gain must have the shape [d], out and residual that of x")
    if residual_out is not None and residual_out.shape != shape:
        raise ValueError("residual_out's shape differs from x")
    if post_gain is not None and post_gain.shape != (d,):
        raise ValueError("post_gain must have the shape [d]")
    if scale is not None and scale.numel() != T:
        raise ValueError("scale must have one value per row")
    if vid is not None and vid.numel() != T:
        raise ValueError("vid must have one id per row")
    gate_rows = 0
    if gate is not None:
        if gate.dim() not in (1, 2) or gate.shape[-1] != d:
            raise ValueError("gate must have the shape [d] or [rows][d]")
        gate_rows = gate.shape[0] if gate.dim() == 2 else 1
    if gate_idx is not None and (gate is None or gate_idx.numel() != T):
        raise ValueError("gate_idx must have one row of gate per token")
    tab = post_tab = None
    V = 0
    if vid is not None:
        V = len(gain_list)
        if post_gain is not None and len(post_gain_list) != V:
            raise ValueError("gain_list and post_gain_list differ in length")
        table = _row_ptrs(gain_list if post_gain is None else [*gain_list, *post_gain_list], d, "gain", dev)
        if V:
            tab = table.buffer_info()[0]
            post_tab = None if post_gain is None else tab + 8 * V
    out_dtype = _OUT_DTYPES.get(out.dtype)
    if out_dtype is None:
        raise ValueError(f"out has dtype {out.dtype}, expected bfloat16, float32 or float8_e4m3fn")
    wsp, wsn = _ws(ws, dev)
    _check(load().bd_block_norm(_ptr(x, "x", _BF16_LIKE, False, dev), _ptr(residual, "residual", _BF16_LIKE, False, dev),
                                T, d, _ptr(post_gain, "post_gain", _BF16_LIKE, True, dev), post_tab,
                                _ptr(gate, "gate", _BF16_LIKE, True, dev), gate_rows,
                                _ptr(gate_idx, "gate_idx", _I32, True, dev), block_scale, residual_scale,
                                _ptr(gain, "gain", _BF16_LIKE, False, dev), tab, _ptr(vid, "vid", _I32, True, dev), V,
                                eps, _ptr(residual_out, "residual_out", _BF16_LIKE, True, dev),
                                _ptr(out, "out", None, False, dev), out_dtype, _ptr(scale, "scale", _F32, True, dev),
                                wsp, wsn, _stream(stream, dev)), "bd_block_norm")


_OUT_DTYPES = {torch.bfloat16: BD_OUT_BF16, torch.float32: BD_OUT_F32, torch.float8_e4m3fn: BD_OUT_E4M3}


class _KvPages(ctypes.Structure):
    """bd_kv_pages (include/bitdelta.h)."""
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("n_pages", _i64), ("page_size", _i32),
                ("n_kv", _i32), ("head_dim", _i32), ("dtype", _i32)]


class KvPages:
    """One layer's paged KV cache: ``k`` and ``v`` [n_pages][n_kv][page_size][head_dim] as torch.bfloat16 or, with
    ``k_scale`` and ``v_scale`` [n_pages][n_kv][page_size] fp32, as torch.int8 codes, or [..][head_dim / 2] as
    torch.uint8, two 4-bit codes a byte, with scales [n_pages][n_kv][page_size][head_dim / 32][2] bf16: (scale, lowest
    value) of each group of 32 elements.  Keeps the tensors referenced."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be [n_pages][n_kv][page_size][head_dim] of one dtype")
        int8, int4 = k.dtype == torch.int8, k.dtype == torch.uint8
        if (int8 or int4) != (k_scale is not None) or (int8 or int4) != (v_scale is not None):
            raise ValueError("scales belong to an int8 or a 4-bit cache, and to them alone")
        dt = (k.dtype,) if int8 or int4 else _BF16_LIKE
        self.n_pages, self.n_kv, self.page_size, self.head_dim = (int(n) for n in k.shape)
        per, st = tuple(k.shape[:3]), _F32
        if int4:
            self.head_dim *= 2
            per, st = (*per, self.head_dim // 32, 2), _BF16_LIKE
        for t in (k_scale, v_scale):
            if t is not None and tuple(t.shape) != per:
                raise ValueError("scales must be [n_pages][n_kv][page_size], of 4-bit codes [..][head_dim / 32][2]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self._c = _KvPages(_ptr(k, "k", dt), _ptr(v, "v", dt), _ptr(k_scale, "k_scale", st, True),
                           _ptr(v_scale, "v_scale", st, True), self.n_pages, self.page_size, self.n_kv,
                           self.head_dim, BD_KV_INT8 if int8 else BD_KV_INT4 if int4 else BD_KV_BF16)
        self._addr = ctypes.addressof(self._c)
        self._dev = k.get_device()

    def _on(self, dev: int) -> int:
        """The address of the handle for a call on device dev, which the tensors have to be on."""
        if self._dev != dev:
            raise ValueError(f"cache is on cuda:{self._dev}, not the current device")
        return self._addr


def _heads(t, name: str, dim: int, dev: int) -> tuple[int, int]:
    """(pointer, row stride) of a bf16 [T][heads][dim] tensor whose rows may be apart."""
    s0, s1, s2 = t.stride()
    if s1 == dim and s2 == 1 and s0 > dim and t.get_device() == dev and t.dtype in _BF16_LIKE:
        return t.data_ptr(), s0
    T, heads, d = t.shape
    if d != dim or s2 != 1 or (heads > 1 and s1 != dim):
        raise ValueError(f"{name} must be [T][heads][{dim}] with contiguous rows")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    if t.dtype not in _BF16_LIKE:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {_BF16_LIKE}")
    return t.data_ptr(), (s0 if T > 1 else heads * dim)


def bd_rope_append_workspace_size(T: int) -> int:
    return int(load().bd_rope_append_workspace_size(T))


def rope_table(n_pos: int, rot_dim: int, theta: float, device=None) -> torch.Tensor:
    """[n_pos][rot_dim/2][2] fp32 (cos, sin) of p * theta^(-2i/rot_dim), formed in fp64."""
    freq = theta ** (-torch.arange(rot_dim // 2, dtype=torch.float64) / (rot_dim // 2))
    angle = torch.arange(n_pos, dtype=torch.float64)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], -1).float().contiguous().to(device or "cuda")


def bd_rope_append(q, k, v, pos, rope_table, slot, cache: KvPages, q_out, ws, axis_of_pair=None,
                   interleaved: bool = False, stream=None) -> None:
    """Turns q -> q_out and k by their positions and writes k and v at ``slot`` of the cache.  q, k, v: [T][heads][dim],
    rows may be apart (slices of one packed product); q = None skips q.  pos: [T] or [T][axes]; axis_of_pair: a host
    sequence of rot_dim/2 axis numbers."""
    T, n_kv, dim = k.shape
    dev = _device()
    if n_kv != cache.n_kv or v.shape != k.shape or dim != cache.head_dim:
        raise ValueError("k and v must be [T][n_kv][head_dim] of the cache")
    kp, ks = _heads(k, "k", dim, dev)
    vp, vs = _heads(v, "v", dim, dev)
    qp = qs = op = os_ = n_q = 0
    if q is not None:
        n_q = q.shape[1]
        if q.shape != (T, n_q, dim) or q_out.shape != q.shape:
            raise ValueError("q and q_out must have T rows of the same heads")
        qp, qs = _heads(q, "q", dim, dev)
        op, os_ = _heads(q_out, "q_out", dim, dev)
    n_axes = pos.shape[1] if pos is not None and pos.dim() == 2 else 1
    if (pos is not None and pos.shape[0] != T) or slot.numel() != T:
        raise ValueError("pos and slot must have one row per token")
    n_pos = pairs = 0
    if rope_table is not None:
        if rope_table.dim() != 3 or rope_table.shape[2] != 2:
            raise ValueError("rope_table must be [n_pos][rot_dim/2][2]")
        n_pos, pairs, _ = rope_table.shape
    axes = None
    if axis_of_pair is not None:
        if len(axis_of_pair) != pairs:
            raise ValueError("axis_of_pair must have rot_dim/2 entries")
        axes = bytes(axis_of_pair)
    wsp, wsn = _ws(ws, dev)
    _check(load().bd_rope_append(qp, qs, kp, ks, vp, vs, T, n_q, _ptr(pos, "pos", _I32, True, dev), n_axes, axes,
                                 _ptr(rope_table, "rope_table", _F32, True, dev), n_pos, 2 * pairs, interleaved,
                                 _ptr(slot, "slot", _I32, False, dev), cache._on(dev), op, os_, wsp, wsn,
                                 _stream(stream, dev)), "bd_rope_append")


def bd_kv_read_workspace_size(rows: int) -> int:
    return int(load().bd_kv_read_workspace_size(rows))


def bd_kv_read(cache: KvPages, page_table, kv_off, k_out, v_out, ws, stream=None) -> None:
    """Gathers the sequences' tokens out of the pages into k_out, v_out [rows][n_kv][head_dim] bf16."""
    n_seq, max_pages = page_table.shape
    rows, heads, dim = k_out.shape
    dev = _device()
    if heads != cache.n_kv or dim != cache.head_dim or v_out.shape != k_out.shape:
        raise ValueError("k_out and v_out must be [rows][n_kv][head_dim]")
    if kv_off.numel() != n_seq + 1:
        raise ValueError("kv_off must have n_seq + 1 entries")
    wsp, wsn = _ws(ws, dev)
    _check(load().bd_kv_read(cache._on(dev), _ptr(page_table, "page_table", _I32, False, dev), max_pages,
                             _ptr(kv_off, "kv_off", _I32, False, dev), n_seq, rows,
                             _ptr(k_out, "k_out", _BF16_LIKE, False, dev), _ptr(v_out, "v_out", _BF16_LIKE, False, dev),
                             wsp, wsn, _stream(stream, dev)), "bd_kv_read")


def bd_attention_workspace_size(T: int, n_seq: int, n_q: int, n_kv: int, head_dim: int) -> int:
    return int(load().bd_attention_workspace_size(T, n_seq, n_q, n_kv, head_dim))


def bd_attention(q, q_off, cache: KvPages, page_table, kv_len, scale, max_new, out, ws, causal: bool = True, lse=None,
                 stream=None) -> None:
    """Attention of the new tokens q [T][n_q][head_dim] (rows may be apart) of n_seq sequences over the paged cache."""
    T, n_q, dim = q.shape
    n_seq, max_pages = page_table.shape
    dev = _device()
    if dim != cache.head_dim or out.shape != q.shape:
        raise ValueError("q and out must be [T][n_q][head_dim] of the cache")
    if q_off.numel() != n_seq + 1 or kv_len.numel() != n_seq:
        raise ValueError("q_off must have n_seq + 1 entries and kv_len n_seq")
    if lse is not None and lse.shape != (T, n_q):
        raise ValueError("lse must be [T][n_q]")
    qp, qs = _heads(q, "q", dim, dev)
    wsp, wsn = _ws(ws, dev)
    _check(load().bd_attention(qp, qs, _ptr(q_off, "q_off", _I32, False, dev), T, n_seq, max_new, n_q, cache._on(dev),
                               _ptr(page_table, "page_table", _I32, False, dev), max_pages,
                               _ptr(kv_len, "kv_len", _I32, False, dev), scale, causal,
                               _ptr(out, "out", _BF16_LIKE, False, dev), _ptr(lse, "lse", _F32, True, dev), wsp, wsn,
                               _stream(stream, dev)), "bd_attention")


def bd_route(vid, V, perm, seg_off, ws, stream=None) -> None:
    T = vid.numel()
    wsp, wsn = _ws(ws)
    _check(load().bd_route(_ptr(vid, "vid", (torch.int32,)), T, int(V), _ptr(perm, "perm", (torch.int32,)),
                           _ptr(seg_off, "seg_off", (torch.int32,)), wsp, wsn, _stream(stream)), "bd_route")


def bd_debug_reconstruct(w_base, signs, alpha, alpha_mode, w_eff, stream=None) -> None:
    d_out, d_in = w_base.shape
    _check(load().bd_debug_reconstruct(_ptr(w_base, "w_base", _BF16_LIKE),
                                       _ptr(signs, "signs", (torch.int32, torch.uint32)),
                                       _ptr(alpha, "alpha", (torch.float32,)), int(alpha_mode), d_out, d_in,
                                       _ptr(w_eff, "w_eff", (torch.float32,)), _stream(stream)),
           "bd_debug_reconstruct")


def bd_debug_bounds_check() -> tuple[int, int]:
    """(status, kernel bits): BD_ERR_BOUNDS if a kernel of a bounds-checked
    build met an index outside its buffer since the last call; synchronises
    the device."""
    bits = ctypes.c_uint32(0)
    st = int(load().bd_debug_bounds_check(ctypes.byref(bits)))
    return st, int(bits.value)


def bd_debug_bounds_enabled() -> bool:
    return bool(load().bd_debug_bounds_enabled())


def bd_check_async(ws, stream=None) -> int:
    """Waits for the stream and returns (and clears) the asynchronous status."""
    wsp, _ = _ws(ws)
    return int(load().bd_check_async(wsp, _stream(stream)))


class DeltaCache:
    """The bd_cache_* entry points (delta cache of section "Altyapı ayrıntıları").

    ``arena`` is a torch.uint8 CUDA tensor the cache divides into slots of
    ``slot_bytes``; ``arena=None`` with ``n_slots`` runs the policy without
    any CUDA call (steps then report slot offsets).  Host sources are CPU
    tensors (page-locked for asynchronous copies); they are kept referenced
    here for as long as the cache lives."""

    def __init__(self, arena, slot_bytes: int, n_pinned: int, rate_decay: float = 1.0, copy_stream=None,
                 n_slots: int | None = None):
        lib = load()
        if arena is None:
            if n_slots is None:
                raise ValueError("a dry-run cache needs n_slots")
            ptr, nbytes, cs = None, int(n_slots) * int(slot_bytes), None
        else:
            if arena.dtype != torch.uint8:
                raise ValueError("arena must be a torch.uint8 tensor")
            ptr, nbytes = _ptr(arena, "arena"), arena.numel()
            cs = (copy_stream or torch.cuda.current_stream()).cuda_stream
        h = _vp()
        _check(lib.bd_cache_create(ptr, nbytes, int(slot_bytes), int(n_pinned), float(rate_decay), cs,
                                   ctypes.byref(h)), "bd_cache_create")
        self._h, self._lib, self.dry = h, lib, arena is None
        self._arena, self._sources = arena, {}

    def set_source(self, variant: int, host: torch.Tensor) -> None:
        if host.is_cuda or not host.is_contiguous():
            raise ValueError("a source is a contiguous CPU tensor")
        _check(self._lib.bd_cache_set_source(self._h, int(variant), host.data_ptr(),
                                             host.numel() * host.element_size()), "bd_cache_set_source")
        self._sources[int(variant)] = host

    def step(self, vids, stream=None):
        """Per request: (device address or slot offset, or None; state)."""
        import numpy as np

        v = np.ascontiguousarray(np.asarray(vids, dtype=np.int32))
        n = v.size
        delta = (_vp * max(n, 1))()
        state = np.zeros(max(n, 1), np.int32)
        st = None if self.dry else _stream(stream)
        _check(self._lib.bd_cache_step(self._h, v.ctypes.data, n, st, delta, state.ctypes.data), "bd_cache_step")
        # a served request's slot offset 0 (dry run) reads back from ctypes as None
        return [(delta[i] or 0) if state[i] == BD_CACHE_SERVED else None for i in range(n)], state[:n].copy()

    def release(self, stream=None) -> None:
        _check(self._lib.bd_cache_release(self._h, None if self.dry else _stream(stream)), "bd_cache_release")

    def stats(self) -> dict:
        out = CacheStats()
        _check(self._lib.bd_cache_get_stats(self._h, ctypes.byref(out)), "bd_cache_get_stats")
        return {name: getattr(out, name) for name, _ in CacheStats._fields_}

    def query(self, variant: int):
        r, pn, rate = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_double()
        _check(self._lib.bd_cache_query(self._h, int(variant), ctypes.byref(r), ctypes.byref(pn), ctypes.byref(rate)),
               "bd_cache_query")
        return bool(r.value), bool(pn.value), rate.value

    def debug_fail_load(self, n: int) -> None:
        """Test aid: the n-th load from now fails like a failed copy (bd_cache_debug_fail_load)."""
        _check(self._lib.bd_cache_debug_fail_load(self._h, int(n)), "bd_cache_debug_fail_load")

    def close(self) -> None:
        if self._h:
            self._lib.bd_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
