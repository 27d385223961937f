"""Python binding of libnq.so, the groupwise-quantized small-T GEMV library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI of ``include/nq.h``.  PyTorch is used for device
memory and streams (tensors pass their ``data_ptr()``, streams their
``cuda_stream`` handle).  The library must have been built (``build()`` below
or ``python quantized_weight_decode_gb300/buildlib.py``); importing works without
it, but every call raises if it is missing -- there is no fallback path.

Names follow the C ABI: ``gemv`` is ``nq_gemv``, ``pack`` is ``nq_pack`` ...
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import numpy as np

__all__ = [
    "NQError", "ROUTE_AUTO", "ROUTE_MMA", "ROUTE_FFMA", "lib", "lib_path", "build",
    "packed_bytes", "pack", "pack_gate_up", "unpack", "pack_device", "quantize_rtn", "quantize_search", "gemv", "gemv_swiglu", "mlp", "mlp_one_launch_ok", "interleave_gate_up", "gemv_head",
    "head_workspace_bytes", "gemv_head_noalloc", "gemv_head_topk", "head_topk_workspace_bytes",
    "dequant",
    "last_device_error", "plan", "selftest_wait_timeout", "status_string", "layout_version",
    "QuantizedWeight", "EXPORTED",
    "ROPE_HALF", "ROPE_INTERLEAVED", "ROPE_SCALINGS", "CACHE_PAGE", "rope_steps", "rope", "KVCache",
    "AttentionPlan",
]

ROUTE_AUTO, ROUTE_MMA, ROUTE_FFMA = 0, 1, 2
# x placement of a plan (nq_x_place)
X_PLACES = ("smem", "regs", "regs2", "hybrid")
OK, EINVAL, EALIGN, ERANGE, ECUDA, ETIMEOUT, EUNSUPPORTED = 0, -1, -2, -3, -4, -5, -6

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libnq.so")
_lib = None
_lock = threading.Lock()

# Every symbol declared in include/nq.h, with its ctypes signature.
_i64, _i32, _vp, _szp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)
_ip = ctypes.POINTER(ctypes.c_int)
_f32 = ctypes.c_float
_SIGS = {
    "nq_packed_bytes": (_i32, [_i64, _i64, _i32, _szp, _szp]),
    "nq_pack": (_i32, [_vp, _vp, _i64, _i64, _i32, _vp, _vp]),
    "nq_pack_gate_up": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp]),
    "nq_unpack": (_i32, [_vp, _vp, _i64, _i64, _i32, _vp, _vp]),
    "nq_pack_device": (_i32, [_vp, _vp, _i64, _i64, _i32, _vp, _vp, _vp]),
    "nq_quantize_rtn": (_i32, [_vp, _i64, _i64, _i32, _vp, _vp, _vp]),
    "nq_quantize_search": (_i32, [_vp, _vp, _i64, _i64, _i32, _vp, _vp, _vp]),
    "nq_gemv": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp]),
    "nq_gemv_ex": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _i32, _i32, _vp]),
    "nq_gemv_swiglu": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp]),
    "nq_mlp": (_i32, [_vp, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp]),
    "nq_mlp_ex": (_i32, [_vp, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _i32,
                         _vp]),
    "nq_mlp_one_launch_ok": (_i32, [_i64, _i64, _i64, _i32, _i32, _i32, _ip]),
    "nq_gemv_head": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp,
                            ctypes.c_size_t, _vp]),
    "nq_head_workspace_bytes": (_i32, [_szp]),
    "nq_gemv_head_topk": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _vp,
                                 _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "nq_head_topk_workspace_bytes": (_i32, [_szp]),
    "nq_gemv_head_noalloc": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp,
                                    _vp]),
    "nq_rope_steps": (_i32, [_i32, ctypes.c_double, _i32, ctypes.c_double, ctypes.c_double, _vp, _vp]),
    "nq_rope": (_i32, [_vp, _vp, _i32, _i64, _i32, _i32, _i32, _i64, _i64, _i64, _i64, _vp, _vp,
                       _i32, _f32, _i32, _vp]),
    "nq_cache_append": (_i32, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _vp,
                               _i32, _i64, _i64, _i64, _i64, _vp, _vp, _i32, _i32, _f32, _vp]),
    "nq_cache_read": (_i32, [_vp, _vp, _i64, _vp, _vp, _i32, _vp]),
    "nq_tree_attention": (_i32, [_vp, _vp, _i64, _i64, _i64, _i32, _vp, _i64, _i32, _vp, _vp, _vp,
                                 _i32, _i32, _i64, _f32, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "nq_tree_attention_workspace_bytes": (_i32, [_i32, _i32, _i64, _i32, _i32, _i32, _i64, _szp]),
    "nq_dequant": (_i32, [_vp, _vp, _vp, _i64, _i64, _i32, _vp]),
    "nq_last_device_error": (_i32, [_vp]),
    "nq_gemv_plan": (_i32, [_i64, _i64, _i32, _i32, _i32, _i32, _ip, _ip, _ip, _ip, _ip]),
    "nq_gemv_plan_x": (_i32, [_i64, _i64, _i32, _i32, _i32, _i32, _ip]),
    "nq_selftest_wait_timeout": (_i32, [_i32, _vp]),
    "nq_status_string": (ctypes.c_char_p, [_i32]),
    "nq_layout_version": (_i32, []),
}
EXPORTED = tuple(_SIGS)


class NQError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


def lib_path() -> str:
    return _LIB_PATH


def build(force: bool = False) -> str:
    """Compile libnq.so for sm_103a in-tree (needs nvcc)."""
    from . import buildlib as _b
    return _b.build(force=force)


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"{_LIB_PATH} is missing: build it with quantized_weight_decode_gb300.build() "
                    "(there is no fallback implementation)")
            h = ctypes.CDLL(_LIB_PATH)
            for name, (res, args) in _SIGS.items():
                f = getattr(h, name)
                f.restype = res
                f.argtypes = args
            _lib = h
    return _lib


def status_string(code: int) -> str:
    return lib().nq_status_string(int(code)).decode()


def layout_version() -> int:
    return int(lib().nq_layout_version())


def _check(rc: int, where: str) -> None:
    if rc != OK:
        raise NQError(rc, where)


_raw_stream = None


def _current_stream_handle() -> int | None:
    """The current device's current stream (by its handle where torch gives it
    directly: a tenth of the host time of a Stream object, which counts for
    calls of a few microseconds)."""
    global _raw_stream
    import torch
    if _raw_stream is None:
        get, dev = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        torch.cuda.current_stream()                    # (initialises CUDA)
        _raw_stream = ((lambda: get(dev())) if get and dev
                       else (lambda: torch.cuda.current_stream().cuda_stream))
    return _raw_stream() or None


def _stream_handle(stream) -> int | None:
    if stream is None:
        return _current_stream_handle()
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _stream_object(stream):
    """torch's object of a stream given as None (the current one), a handle or an object."""
    import torch
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return stream


def _empty(shape, dtype, device, stream):
    """Memory for a call's result or scratch.  For a call on another stream than the
    current one it is taken for that stream (a piece that the current stream's
    pending work still uses would be written too early), and it is not handed out
    again before what the current stream has read of it by its release."""
    import torch
    if stream is None or _stream_handle(stream) == _current_stream_handle():
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream()
    with torch.cuda.stream(_stream_object(stream)):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _dptr(t):
    return None if t is None else int(t.data_ptr())


# ---------------------------------------------------------------- host side
def packed_bytes(K: int, N: int, bits: int) -> tuple[int, int]:
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().nq_packed_bytes(K, N, bits, ctypes.byref(cb), ctypes.byref(sb)), "nq_packed_bytes")
    return cb.value, sb.value


def pack(codes: np.ndarray, scales: np.ndarray, bits: int) -> tuple[np.ndarray, np.ndarray]:
    """Host packer: int8 codes [N, K] and FP16 scale bits [N, K/64] -> packed
    codes (uint8) and packed scales (uint16), as numpy arrays."""
    codes = np.ascontiguousarray(codes, dtype=np.int8)
    scales = np.ascontiguousarray(scales).view(np.uint16)
    N, K = codes.shape
    cb, sb = packed_bytes(K, N, bits)
    out = np.empty(cb, dtype=np.uint8)
    sout = np.empty(sb // 2, dtype=np.uint16)
    _check(lib().nq_pack(codes.ctypes.data, scales.ctypes.data, K, N, bits,
                         out.ctypes.data, sout.ctypes.data), "nq_pack")
    return out, sout


def pack_gate_up(codes_gate: np.ndarray, scales_gate: np.ndarray, codes_up: np.ndarray,
                 scales_up: np.ndarray, bits: int) -> tuple[np.ndarray, np.ndarray]:
    """Host packer of a gate+up matrix in nq_gemv_swiglu's row order
    (nq_pack_gate_up): gate and up int8 codes [I, K], FP16 scale bits
    [I, K/64] -> packed codes and scales of the [2 I, K] matrix."""
    cg = np.ascontiguousarray(codes_gate, dtype=np.int8)
    cu = np.ascontiguousarray(codes_up, dtype=np.int8)
    sg = np.ascontiguousarray(scales_gate).view(np.uint16)
    su = np.ascontiguousarray(scales_up).view(np.uint16)
    I, K = cg.shape
    cb, sb = packed_bytes(K, 2 * I, bits)
    out = np.empty(cb, dtype=np.uint8)
    sout = np.empty(sb // 2, dtype=np.uint16)
    _check(lib().nq_pack_gate_up(cg.ctypes.data, sg.ctypes.data, cu.ctypes.data, su.ctypes.data,
                                 K, I, bits, out.ctypes.data, sout.ctypes.data), "nq_pack_gate_up")
    return out, sout


def unpack(packed: np.ndarray, scales_packed: np.ndarray, K: int, N: int,
           bits: int) -> tuple[np.ndarray, np.ndarray]:
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    scales_packed = np.ascontiguousarray(scales_packed).view(np.uint16)
    codes = np.empty((N, K), dtype=np.int8)
    scales = np.empty((N, K // 64), dtype=np.uint16)
    _check(lib().nq_unpack(packed.ctypes.data, scales_packed.ctypes.data, K, N, bits,
                           codes.ctypes.data, scales.ctypes.data), "nq_unpack")
    return codes, scales


# ---------------------------------------------------------------- device side
def pack_device(codes, scales, bits: int, packed=None, scales_packed=None, stream=None):
    """Device packer.  codes: int8 cuda [N, K]; scales: 16-bit cuda [N, K/64].
    Returns (packed uint8 tensor, packed scales int16 tensor)."""
    import torch
    N, K = codes.shape
    cb, sb = packed_bytes(K, N, bits)
    if packed is None:
        packed = _empty(cb, torch.uint8, codes.device, stream)
    if scales_packed is None:
        scales_packed = _empty(sb // 2, torch.int16, codes.device, stream)
    _check(lib().nq_pack_device(_dptr(codes), _dptr(scales), K, N, bits, _dptr(packed),
                                _dptr(scales_packed), _stream_handle(stream)), "nq_pack_device")
    return packed, scales_packed


def quantize_rtn(w, bits: int, codes=None, scales=None, stream=None):
    """Device round-to-nearest encoder: fp32 cuda w [N, K] -> (int8 codes [N, K],
    int16 FP16-scale bits [N, K/64])."""
    import torch
    N, K = w.shape
    if codes is None:
        codes = _empty((N, K), torch.int8, w.device, stream)
    if scales is None:
        scales = _empty((N, K // 64), torch.int16, w.device, stream)
    _check(lib().nq_quantize_rtn(_dptr(w), K, N, bits, _dptr(codes), _dptr(scales),
                                 _stream_handle(stream)), "nq_quantize_rtn")
    return codes, scales


def quantize_search(w, bits: int, imatrix=None, codes=None, scales=None, stream=None):
    """Searched encoder on the device: w fp32 [N, K] (device tensor), imatrix
    fp32 [K] or None -> (codes int8 [N, K], scales int16 FP16 bits [N, K/64])."""
    import torch
    N, K = w.shape
    if codes is None:
        codes = _empty((N, K), torch.int8, w.device, stream)
    if scales is None:
        scales = _empty((N, K // 64), torch.int16, w.device, stream)
    _check(lib().nq_quantize_search(_dptr(w), _dptr(imatrix), K, N, bits, _dptr(codes),
                                    _dptr(scales), _stream_handle(stream)), "nq_quantize_search")
    return codes, scales


def gemv(packed, scales, x, y, K: int, N: int, T: int, bits: int, route: int = ROUTE_AUTO,
         ksplit: int = 0, stream=None) -> None:
    """y[T, N] (fp32 cuda) = x[T, K] (bf16 cuda) @ dequant(W)^T, asynchronous."""
    if route == ROUTE_AUTO and ksplit == 0:
        rc = lib().nq_gemv(_dptr(packed), _dptr(scales), _dptr(x), _dptr(y), K, N, T, bits,
                           _stream_handle(stream))
    else:
        rc = lib().nq_gemv_ex(_dptr(packed), _dptr(scales), _dptr(x), _dptr(y), K, N, T, bits,
                              route, ksplit, _stream_handle(stream))
    _check(rc, "nq_gemv")


def interleave_gate_up(gate, up):
    """Rows of the gate+up matrix in the order nq_gemv_swiglu expects: row
    16 r + m = gate row 8 r + m, row 16 r + 8 + m = up row 8 r + m (m < 8).
    Works on numpy arrays or torch tensors [I, ...] (I a multiple of 8)."""
    i = gate.shape[0]
    rest = tuple(gate.shape[1:])
    g = gate.reshape((i // 8, 1, 8) + rest)
    u = up.reshape((i // 8, 1, 8) + rest)
    try:
        import torch
        if isinstance(gate, torch.Tensor):
            return torch.cat([g, u], dim=1).reshape((2 * i,) + rest)
    except ImportError:
        pass
    import numpy as np
    return np.concatenate([g, u], axis=1).reshape((2 * i,) + rest)


def gemv_swiglu(packed_gu, scales_gu, x, act, K: int, N: int, T: int, bits: int, stream=None):
    """act[T, N/2] (bf16 tensor) = silu(gate) * up from a gate+up matrix packed
    with interleave_gate_up's row order."""
    _check(lib().nq_gemv_swiglu(_dptr(packed_gu), _dptr(scales_gu), _dptr(x), _dptr(act), K, N, T,
                                bits, _stream_handle(stream)), "nq_gemv_swiglu")


def mlp(gu, down, x, act, y, T: int, launches: int = 0, stream=None):
    """The layer MLP: gu, down are QuantizedWeight (gu packed interleaved);
    act [T, I] bf16 scratch, y [T, H_out] fp32.  launches: 0 = the library's
    choice, 1 = one launch (nq_mlp_ex), 2 = two launches."""
    _check(lib().nq_mlp_ex(_dptr(gu.packed), _dptr(gu.scales), gu.bits, _dptr(down.packed),
                           _dptr(down.scales), down.bits, _dptr(x), _dptr(act), _dptr(y), gu.K,
                           gu.N // 2, down.N, T, launches, _stream_handle(stream)), "nq_mlp_ex")


def mlp_one_launch_ok(H: int, I: int, H_out: int, T: int, bits_gu: int, bits_down: int) -> bool:
    """Whether nq_mlp_ex(launches=1) supports this layer shape here."""
    v = ctypes.c_int()
    _check(lib().nq_mlp_one_launch_ok(H, I, H_out, T, bits_gu, bits_down, ctypes.byref(v)),
           "nq_mlp_one_launch_ok")
    return bool(v.value)


def head_workspace_bytes() -> int:
    """Workspace bytes nq_gemv_head needs on the current device."""
    v = ctypes.c_size_t()
    _check(lib().nq_head_workspace_bytes(ctypes.byref(v)), "nq_head_workspace_bytes")
    return int(v.value)


def gemv_head(packed, scales, x, K: int, N: int, T: int, bits: int, y=None, workspace=None,
              argmax=None, maxval=None, lse=None, stream=None):
    """Fused verify head: y = x W^T (stored if `y` is given) and, per token,
    the argmax, the maximum and the logsumexp of the N outputs.  Returns
    (argmax int32 [T], maxval fp32 [T], lse fp32 [T]) device tensors; the
    workspace is allocated here if not passed (torch memory)."""
    import torch
    dev = x.device
    if workspace is None:
        workspace = _empty(head_workspace_bytes(), torch.uint8, dev, stream)
    if argmax is None:
        argmax = _empty(T, torch.int32, dev, stream)
    if maxval is None:
        maxval = _empty(T, torch.float32, dev, stream)
    if lse is None:
        lse = _empty(T, torch.float32, dev, stream)
    _check(lib().nq_gemv_head(_dptr(packed), _dptr(scales), _dptr(x), _dptr(y), K, N, T, bits,
                              _dptr(argmax), _dptr(maxval), _dptr(lse), _dptr(workspace),
                              workspace.numel() * workspace.element_size(),
                              _stream_handle(stream)), "nq_gemv_head")
    return argmax, maxval, lse


def head_topk_workspace_bytes() -> int:
    """Workspace bytes nq_gemv_head_topk needs on the current device."""
    v = ctypes.c_size_t()
    _check(lib().nq_head_topk_workspace_bytes(ctypes.byref(v)), "nq_head_topk_workspace_bytes")
    return int(v.value)


def gemv_head_topk(packed, scales, x, K: int, N: int, T: int, bits: int, k: int, y=None,
                   workspace=None, topk_idx=None, topk_val=None, argmax=None, maxval=None,
                   lse=None, stream=None):
    """gemv_head plus the k largest logits of every token (larger value
    first, equal values by smaller index).  Returns (topk_idx int32 [T, k],
    topk_val fp32 [T, k], argmax, maxval, lse) device tensors; the workspace
    and outputs not passed are allocated here (torch memory)."""
    import torch
    dev = x.device
    if workspace is None:
        workspace = _empty(head_topk_workspace_bytes(), torch.uint8, dev, stream)
    kk = max(k, 1)          # a bad k is the library's to reject
    if topk_idx is None:
        topk_idx = _empty((T, kk), torch.int32, dev, stream)
    if topk_val is None:
        topk_val = _empty((T, kk), torch.float32, dev, stream)
    if argmax is None:
        argmax = _empty(T, torch.int32, dev, stream)
    if maxval is None:
        maxval = _empty(T, torch.float32, dev, stream)
    if lse is None:
        lse = _empty(T, torch.float32, dev, stream)
    _check(lib().nq_gemv_head_topk(_dptr(packed), _dptr(scales), _dptr(x), _dptr(y), K, N, T, bits,
                                   k, _dptr(topk_idx), _dptr(topk_val), _dptr(argmax),
                                   _dptr(maxval), _dptr(lse), _dptr(workspace),
                                   workspace.numel() * workspace.element_size(),
                                   _stream_handle(stream)), "nq_gemv_head_topk")
    return topk_idx, topk_val, argmax, maxval, lse


def gemv_head_noalloc(packed, scales, x, K: int, N: int, T: int, bits: int, y=None,
                      argmax=None, maxval=None, lse=None, stream=None):
    """gemv_head through the entry point that allocates nothing: the library
    uses its own fixed device scratch instead of a workspace.  Calls must not
    overlap on the GPU.  Returns (argmax, maxval, lse); output tensors the
    caller does not pass are created here (torch memory)."""
    import torch
    dev = x.device
    if argmax is None:
        argmax = _empty(T, torch.int32, dev, stream)
    if maxval is None:
        maxval = _empty(T, torch.float32, dev, stream)
    if lse is None:
        lse = _empty(T, torch.float32, dev, stream)
    _check(lib().nq_gemv_head_noalloc(_dptr(packed), _dptr(scales), _dptr(x), _dptr(y), K, N, T,
                                      bits, _dptr(argmax), _dptr(maxval), _dptr(lse),
                                      _stream_handle(stream)), "nq_gemv_head_noalloc")
    return argmax, maxval, lse


def dequant(packed, scales, K: int, N: int, bits: int, out=None, stream=None):
    import torch
    if out is None:
        out = _empty((N, K), torch.float32, packed.device, stream)
    _check(lib().nq_dequant(_dptr(packed), _dptr(scales), _dptr(out), K, N, bits,
                            _stream_handle(stream)), "nq_dequant")
    return out


def last_device_error(stream=None) -> int:
    """Synchronise the stream, return and clear the device status word."""
    return int(lib().nq_last_device_error(_stream_handle(stream)))


def plan(K: int, N: int, T: int, bits: int, route: int = ROUTE_AUTO, ksplit: int = 0) -> dict:
    vals = [ctypes.c_int() for _ in range(5)]
    _check(lib().nq_gemv_plan(K, N, T, bits, route, ksplit, *[ctypes.byref(v) for v in vals]),
           "nq_gemv_plan")
    keys = ("route", "ksplit", "clusters", "stages", "smem")
    out = {k: v.value for k, v in zip(keys, vals)}
    xp = ctypes.c_int()
    _check(lib().nq_gemv_plan_x(K, N, T, bits, route, ksplit, ctypes.byref(xp)), "nq_gemv_plan_x")
    out["x"] = X_PLACES[xp.value]
    return out


def selftest_wait_timeout(limit_us: int, stream=None) -> None:
    _check(lib().nq_selftest_wait_timeout(limit_us, _stream_handle(stream)),
           "nq_selftest_wait_timeout")


class QuantizedWeight:
    """A packed weight W[N, K] resident on the device, with its GEMV."""

    def __init__(self, packed, scales, K: int, N: int, bits: int):
        self.packed, self.scales, self.K, self.N, self.bits = packed, scales, K, N, bits

    @classmethod
    def from_fp32(cls, w, bits: int, stream=None) -> "QuantizedWeight":
        codes, scales = quantize_rtn(w, bits, stream=stream)
        packed, sp = pack_device(codes, scales, bits, stream=stream)
        N, K = w.shape
        return cls(packed, sp, K, N, bits)

    @property
    def nbytes(self) -> int:
        return self.packed.numel() + 2 * self.scales.numel()

    def gemv(self, x, y=None, route: int = ROUTE_AUTO, ksplit: int = 0, stream=None):
        import torch
        T = x.shape[0]
        if y is None:
            y = _empty((T, self.N), torch.float32, x.device, stream)
        gemv(self.packed, self.scales, x, y, self.K, self.N, T, self.bits, route, ksplit, stream)
        return y


# ---------------------------------------------------------------- rotary, cache, attention
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_SCALINGS = ("plain", "linear", "ntk", "yarn")
CACHE_PAGE = 64


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return 0
    if t.dtype == torch.bfloat16:
        return 1
    raise TypeError(f"float32 or bfloat16 expected, got {t.dtype}")


def _heads_last(t, where: str):
    """The strides of a [tokens, heads, head_dim] tensor, whose last dimension
    has to be contiguous."""
    st = t.stride()
    if len(st) != 3 or (st[2] != 1 and t.shape[2] > 1 and t.numel()):
        raise ValueError(f"{where}: [tokens, heads, head_dim] with a contiguous last dimension expected")
    return st


def _vector(t, dtype, n: int, where: str):
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{where}: a contiguous {dtype} tensor of {n} entries expected")
    return t


def _reachable(dev: int, where: str, *tensors) -> None:
    """Refuses tensors (None: not given) that are not in the memory of cuda device `dev`."""
    for t in tensors:
        if t is not None and t.get_device() != dev or dev < 0:
            raise ValueError(f"{where}: cuda tensors on one device expected")


def rope_steps(rotary_dim: int, base: float = 10000.0, scaling: str = "plain", scale_factor: float = 1.0,
               trained_context: float = 0.0, device="cuda"):
    """Rotary steps (nq_rope_steps): (int64 tensor [rotary_dim / 2] on `device`,
    the factor on cosine and sine)."""
    import torch
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling: one of {ROPE_SCALINGS}")
    steps = np.zeros(max(rotary_dim // 2, 1), dtype=np.uint64)
    factor = ctypes.c_float()
    _check(lib().nq_rope_steps(rotary_dim, base, ROPE_SCALINGS.index(scaling), scale_factor,
                               trained_context, steps.ctypes.data, ctypes.addressof(factor)),
           "nq_rope_steps")
    return torch.from_numpy(steps.view(np.int64)).to(device), factor.value


@functools.cache
def _rope_function():
    """rope as a function of torch's autograd: linear in x, its gradient is the adjoint."""
    import torch

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, positions, steps, layout, factor, adjoint, stream):
            ctx.save_for_backward(positions, steps)
            ctx.how = layout, factor, adjoint
            return rope(x.detach(), positions, steps, None, layout, factor, adjoint, stream)

        @staticmethod
        def backward(ctx, grad):
            positions, steps = ctx.saved_tensors
            layout, factor, adjoint = ctx.how
            if grad.data_ptr() % 16 or (grad.stride(2) != 1 and grad.shape[2] > 1):
                grad = grad.clone(memory_format=torch.contiguous_format)  # (a sum's gradient is one value with strides of 0)
            return (rope(grad, positions, steps, None, layout, factor, not adjoint),) + (None,) * 6

    return Rope


def rope(x, positions, steps, out=None, layout: int = ROPE_HALF, factor: float = 1.0,
         adjoint: bool = False, stream=None):
    """Rotated x [tokens, heads, head_dim] (fp32 or bf16 cuda; strides allowed in
    the first two dimensions): nq_rope.  positions: int32 [tokens]; steps: int64
    [rotary_dim / 2] (rope_steps).  adjoint: the transposed rotation, which
    takes the gradient of the result to that of x.  out may be x.  Where x
    requires a gradient (and gradients are on), so does the result, whose
    gradient is rotated back by the adjoint; out cannot be given then."""
    import torch
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("rope: no out for a tensor that requires a gradient")
        return _rope_function().apply(x, positions, steps, layout, factor, adjoint, stream)
    xs = _heads_last(x, "rope")
    tokens, heads, dim = x.shape
    if out is None:
        out = _empty((tokens, heads, dim), x.dtype, x.device, stream)
    elif out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("rope: out has another shape or type than x")
    os = _heads_last(out, "rope")
    _vector(positions, torch.int32, tokens, "rope: positions")
    half = steps.numel()
    _vector(steps, torch.int64, half, "rope: steps")
    code = _dtype_code(x)
    _reachable(x.get_device(), "rope", out, positions, steps)
    rc = lib().nq_rope(x.data_ptr(), out.data_ptr(), code, tokens, heads, dim, 2 * half,
                       xs[0], xs[1], os[0], os[1], positions.data_ptr(), steps.data_ptr(), layout,
                       factor, adjoint, _stream_handle(stream))
    if rc:
        _check(rc, "nq_rope")
    return out


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", _vp), ("k_scales", _vp), ("v_codes", _vp), ("v_scales", _vp),
                ("pages", _i64), ("kv_heads", _i32), ("head_dim", _i32), ("k_bits", _i32),
                ("v_bits", _i32)]


class AttentionPlan:
    """What calls of KVCache.attention over batches of one size share: the
    bounds it was made for, the workspace, and the outputs of calls that bring
    none of their own (torch memory, kept by the plan, and beyond it until the
    streams of its calls are done with it).  Calls sharing a plan must be ordered
    (one stream), and each overwrites the outputs of the one before.  `stream`:
    the stream of its calls, if that is not the current one.  A stream given by
    its handle has to outlive the plan."""

    def __init__(self, seqs: int, max_drafts: int, q_heads: int, kv_heads: int, head_dim: int,
                 max_context: int, device="cuda", stream=None):
        import torch
        v = ctypes.c_size_t()
        _check(lib().nq_tree_attention_workspace_bytes(seqs, max_drafts, seqs * max_drafts, q_heads,
                                                       kv_heads, head_dim, max_context,
                                                       ctypes.byref(v)),
               "nq_tree_attention_workspace_bytes")
        self.seqs, self.max_drafts, self.max_context = seqs, max_drafts, max_context
        self.bytes = int(v.value)
        self.workspace = _empty(self.bytes, torch.uint8, device, stream) if self.bytes else None
        self._workspace_ptr = _dptr(self.workspace)
        self._outputs = {}
        # the stream that the workspace was taken for
        self._home = _stream_handle(stream) if self.bytes else None

    def outputs(self, total: int, q_heads: int, head_dim: int, device, stream=None):
        """The plan's (out, lse) for `total` drafted tokens, for a call on `stream`."""
        got = self._outputs.get((total, q_heads, head_dim))
        handle = _stream_handle(stream)
        if got is None:
            import torch
            # one piece for the largest batch, of which every other one takes the
            # front: it stays where it is (a captured graph may hold it)
            most = max(total, self.seqs * self.max_drafts)
            got = self._outputs.get((most, q_heads, head_dim))
            if got is None:
                got = (_empty((most, q_heads, head_dim), torch.bfloat16, device, stream),
                       _empty((most, q_heads), torch.float32, device, stream), handle)
                self._outputs[(most, q_heads, head_dim)] = got
            got = got[0][:total], got[1][:total], got[2]
            self._outputs[(total, q_heads, head_dim)] = got
        if got[2] != handle:
            for t in got[:2]:
                t.record_stream(_stream_object(stream))
        return got


class KVCache:
    """A quantised KV cache (layout in include/nq.h): k_codes, v_codes uint8
    [pages, kv_heads, 64, head_dim * bits / 8], k_scales, v_scales float16
    [pages, kv_heads, 64, head_dim / 64], cuda, contiguous.  A token's slot is
    page * 64 + offset."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        import torch
        pages, heads, page, groups = k_scales.shape
        self.pages, self.kv_heads, self.head_dim = pages, heads, 64 * groups
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_bits, self.v_bits = (8 * c.shape[3] // self.head_dim for c in (k_codes, v_codes))
        for c, s, bits in ((k_codes, k_scales, self.k_bits), (v_codes, v_scales, self.v_bits)):
            if (c.dtype != torch.uint8 or s.dtype != torch.float16 or not c.is_contiguous()
                    or not s.is_contiguous() or tuple(s.shape) != (pages, heads, CACHE_PAGE, groups)
                    or tuple(c.shape) != (pages, heads, CACHE_PAGE, self.head_dim * bits // 8)):
                raise ValueError("KVCache: codes or scales of another type, shape or layout than documented")
        if len({t.device for t in (k_codes, k_scales, v_codes, v_scales)}) != 1:
            raise ValueError("KVCache: codes and scales on one device expected")
        self._struct = _CacheStruct(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                                    v_scales.data_ptr(), pages, heads, self.head_dim, self.k_bits,
                                    self.v_bits)
        self._ref = ctypes.addressof(self._struct)
        self._device = k_codes.get_device()

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, k_bits: int = 8, v_bits: int = 8,
              device="cuda") -> "KVCache":
        import torch
        parts = []
        for bits in (k_bits, v_bits):
            parts.append(torch.zeros((pages, kv_heads, CACHE_PAGE, head_dim * bits // 8),
                                     dtype=torch.uint8, device=device))
            parts.append(torch.zeros((pages, kv_heads, CACHE_PAGE, head_dim // 64),
                                     dtype=torch.float16, device=device))
        return cls(*parts)

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size()
                   for t in (self.k_codes, self.k_scales, self.v_codes, self.v_scales))

    def append(self, k, v, slots, q=None, q_out=None, positions=None, steps=None,
               layout: int = ROPE_HALF, factor: float = 1.0, stream=None):
        """Write k, v [tokens, kv_heads, head_dim] (fp32 or bf16) into slots
        (int32 [tokens]; negative: not written), k rotated by positions and
        steps if given; with q [tokens, q_heads, head_dim], also the rotated q
        in bf16, which is returned (nq_cache_append, one launch)."""
        import torch
        ks, vs = _heads_last(k, "append"), _heads_last(v, "append")
        tokens = k.shape[0]
        dtype = k.dtype
        if k.shape != (tokens, self.kv_heads, self.head_dim) or v.shape != k.shape or v.dtype != dtype:
            raise ValueError(f"append: k and v [tokens, {self.kv_heads}, {self.head_dim}] of one type expected")
        _vector(slots, torch.int32, tokens, "append: slots")
        heads, q_ptr, out_ptr, qs, os = 0, None, None, (0, 0), (0, 0)
        if q is not None:
            qs = _heads_last(q, "append")
            heads = q.shape[1]
            if q.shape != (tokens, heads, self.head_dim) or q.dtype != dtype:
                raise ValueError("append: q of another shape or type than k")
            if q_out is None:
                q_out = _empty((tokens, heads, self.head_dim), torch.bfloat16, q.device, stream)
            elif q_out.shape != q.shape or q_out.dtype != torch.bfloat16:
                raise ValueError("append: q_out of another shape than q, or not bfloat16")
            os = _heads_last(q_out, "append")
            q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
        half, pos_ptr, steps_ptr = 0, None, None
        if steps is not None:
            if positions is None:
                raise ValueError("append: steps without positions")
            _vector(positions, torch.int32, tokens, "append: positions")
            half = steps.numel()
            _vector(steps, torch.int64, half, "append: steps")
            pos_ptr, steps_ptr = positions.data_ptr(), steps.data_ptr()
        code = _dtype_code(k)
        _reachable(self._device, "append", k, v, slots, q, q_out, None if steps is None else positions, steps)
        rc = lib().nq_cache_append(self._ref, k.data_ptr(), v.data_ptr(), code, tokens, ks[0],
                                   ks[1], vs[0], vs[1], slots.data_ptr(), q_ptr, out_ptr, heads, qs[0],
                                   qs[1], os[0], os[1], pos_ptr, steps_ptr, 2 * half, layout, factor,
                                   _stream_handle(stream))
        if rc:
            _check(rc, "nq_cache_append")
        return q_out

    def read(self, slots, dtype=None, k_out=None, v_out=None, stream=None):
        """The values of the tokens in slots (int32 [n]): (k, v) [n, kv_heads,
        head_dim] of `dtype` (bf16 by default, or fp32): nq_cache_read."""
        import torch
        n = slots.numel()
        _vector(slots, torch.int32, n, "read: slots")
        dtype = dtype or (torch.bfloat16 if k_out is None else k_out.dtype)
        shape = (n, self.kv_heads, self.head_dim)
        if k_out is None:
            k_out = _empty(shape, dtype, slots.device, stream)
        if v_out is None:
            v_out = _empty(shape, dtype, slots.device, stream)
        for t in (k_out, v_out):
            if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
                raise ValueError(f"read: contiguous outputs of shape {shape} and type {dtype} expected")
        code = _dtype_code(k_out)
        _reachable(self._device, "read", slots, k_out, v_out)
        rc = lib().nq_cache_read(self._ref, slots.data_ptr(), n, k_out.data_ptr(), v_out.data_ptr(),
                                 code, _stream_handle(stream))
        if rc:
            _check(rc, "nq_cache_read")
        return k_out, v_out

    def attention_plan(self, seqs: int, max_drafts: int, q_heads: int, max_context: int) -> AttentionPlan:
        """The plan of attention() for batches of up to `seqs` sequences with up
        to `max_drafts` drafted tokens each over up to `max_context` committed ones."""
        return AttentionPlan(seqs, max_drafts, q_heads, self.kv_heads, self.head_dim, max_context,
                             self.k_codes.device)

    def attention(self, q, page_table, lengths, starts=None, tree=None, scale: float | None = None,
                  plan: AttentionPlan | None = None, out=None, lse=None, stream=None):
        """Attention of drafted tokens (nq_tree_attention): q bf16 [total, q_heads,
        head_dim]; page_table int32 [seqs, width]; lengths int32 [seqs]
        (committed tokens); starts int32 [seqs + 1], or None: total / seqs
        drafted tokens each; tree int64 [total] (bit b: sees drafted token b of
        its sequence), or None: a chain.  scale: head_dim ** -0.5 by default.
        plan: attention_plan() of at least these sizes (made here if None,
        with the page table's width as the context's bound).  Returns (out bf16
        [total, q_heads, head_dim], lse fp32 [total, q_heads]): the tensors
        given, else the plan's own, which its next call overwrites.  Rows of a
        sequence whose starts the kernel finds wrong (last_device_error) are not
        written: they hold what was there."""
        import torch
        qs = _heads_last(q, "attention")
        total, heads, dim = q.shape
        seqs, width = page_table.shape
        if q.dtype != torch.bfloat16 or dim != self.head_dim:
            raise ValueError(f"attention: bfloat16 q of head_dim {self.head_dim} expected")
        if page_table.dtype != torch.int32 or (width > 1 and page_table.stride(1) != 1):
            raise ValueError("attention: int32 page_table [seqs, width] with contiguous rows expected")
        _vector(lengths, torch.int32, seqs, "attention: lengths")
        if starts is not None:
            _vector(starts, torch.int32, seqs + 1, "attention: starts")
        if tree is not None:
            _vector(tree, torch.int64, total, "attention: tree")
        _reachable(self._device, "attention", q, page_table, lengths, starts, tree, out, lse)
        if seqs == 0:                        # an empty batch: nothing to launch
            if total:
                raise ValueError("attention: drafted tokens of no sequence")
            plan = None
        elif plan is None:
            drafts = min(64, total) if starts is not None else -(-total // seqs)
            plan = AttentionPlan(seqs, max(1, drafts), heads, self.kv_heads, self.head_dim, width * CACHE_PAGE,
                                 self.k_codes.device, stream)
        if out is None or lse is None:
            own = (plan.outputs(total, heads, dim, q.device, stream) if plan is not None
                   else (torch.empty_like(q), torch.empty((0, heads), dtype=torch.float32, device=q.device)))
        if out is None:
            out = own[0]
        elif out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous():
            raise ValueError("attention: out of another shape than q, not bfloat16 or not contiguous")
        if lse is None:
            lse = own[1]
        else:
            _vector(lse, torch.float32, total * heads, "attention: lse")
        if plan is None:
            return out, lse
        handle = _stream_handle(stream)
        if plan._home != handle and plan.bytes:              # keep the workspace until the call is done with it
            plan.workspace.record_stream(_stream_object(stream))
        rc = lib().nq_tree_attention(
            self._ref, q.data_ptr(), qs[0], qs[1], total, heads, page_table.data_ptr(),
            page_table.stride(0), width, lengths.data_ptr(), None if starts is None else starts.data_ptr(),
            None if tree is None else tree.data_ptr(), seqs, plan.max_drafts, plan.max_context,
            self.head_dim ** -0.5 if scale is None else scale, out.data_ptr(), lse.data_ptr(),
            plan._workspace_ptr, plan.bytes, handle)
        if rc:
            _check(rc, "nq_tree_attention")
        return out, lse
