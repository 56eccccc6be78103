"""Python binding of the C ABI in include/falcon.h (ctypes; argument marshalling only).

Every function here forwards to ``_build/libfalcon.so``; all arithmetic runs in
the library's CUDA kernels. There is no fallback: if the library has not been
built (``weight_linear_attention_gb300.build.build()``) or cannot be loaded,
every call raises.

PyTorch is used only to hand over device pointers and the current CUDA stream.
"""

from __future__ import annotations

import collections
import contextlib
import ctypes
import functools
import os
import struct
import threading

from . import build as _build

FALCON_1, FALCON_1A, FALCON_2, FALCON_2A, FALCON_3, FALCON_3A = 1, 2, 3, 4, 5, 6
FALCON_F32, FALCON_BF16 = 0, 1
FALCON_E4M3 = 2  # output of the root-mean-square norm only
FALCON_OK = 0
FALCON_ERR_INVALID_ARG = 1
FALCON_ERR_UNSUPPORTED = 2
FALCON_ERR_MISALIGNED = 3
FALCON_ERR_CUDA = 4
FALCON_ERR_DEVICE_TIMEOUT = 5

GLR_GATES = {"decay": 0, "sigmoid": 1, "mix": 2}
GN_ACTS = {"none": 0, "silu": 1, "gelu": 2, "sigmoid": 3}

VARIANTS = {"falcon1": FALCON_1, "falcon1a": FALCON_1A, "falcon2": FALCON_2, "falcon2a": FALCON_2A,
            "falcon3": FALCON_3, "falcon3a": FALCON_3A}


class FalconDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("heads", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("dk", ctypes.c_int64),
        ("dv", ctypes.c_int64),
        ("window", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("pos", ctypes.c_int64),
        ("eps", ctypes.c_float),
        ("eps_gamma", ctypes.c_float),
    ]


assert ctypes.sizeof(FalconDims) == 64


class FalconSeqDims(ctypes.Structure):
    """falcon_seq_dims_t: the sizes of the strided [B,H,T,d] operators."""

    _fields_ = [
        ("batch", ctypes.c_int64),
        ("heads", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("d", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


assert ctypes.sizeof(FalconSeqDims) == 40


class FalconGdrDims(ctypes.Structure):
    """falcon_gdr_dims_t: the sizes of the gated delta rule."""

    _fields_ = [
        ("batch", ctypes.c_int64),
        ("heads", ctypes.c_int64),
        ("qk_heads", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("dk", ctypes.c_int64),
        ("dv", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


assert ctypes.sizeof(FalconGdrDims) == 56


class FalconRmsDims(ctypes.Structure):
    """falcon_rms_dims_t: the sizes of the root-mean-square norm."""

    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("d", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
    ]


assert ctypes.sizeof(FalconRmsDims) == 32

_lock = threading.Lock()
_lib = None

EXPORTED = ("falcon_fwd", "falcon_workspace_bytes", "falcon_fwd_static", "falcon_tail_bytes",
            "falcon_status_string", "falcon_device_status", "falcon_kernel_for", "falcon_abi_version",
            "falcon_bwd", "falcon_bwd_workspace_bytes", "falcon_glr_fwd", "falcon_glr_bwd", "falcon_gn_fwd",
            "falcon_gn_bwd", "falcon_gn_bwd_workspace_bytes", "falcon_gdr_fwd", "falcon_gdr_bwd",
            "falcon_gdr_workspace_bytes", "falcon_rms_fwd", "falcon_rms_bwd", "falcon_rms_bwd_workspace_bytes")
STATIC_WORKSPACE_BYTES = 16 << 20


class FalconError(RuntimeError):
    def __init__(self, status: int, what: str = "falcon_fwd"):
        self.status = status
        super().__init__(f"{what} failed with status {status}: {status_string(status)}")


def lib_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Load the C-ABI library (raises if it is missing)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or _build.LIB
        if not os.path.exists(p):
            raise RuntimeError(f"CUDA library not built: {p} (run weight_linear_attention_gb300.build.build())")
        lib = ctypes.CDLL(p)
        vp = ctypes.c_void_p
        lib.falcon_fwd.restype = ctypes.c_int
        lib.falcon_fwd.argtypes = [ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                   ctypes.POINTER(FalconDims), ctypes.c_int, vp, ctypes.c_size_t, vp]
        lib.falcon_fwd_static.restype = ctypes.c_int
        lib.falcon_fwd_static.argtypes = [ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                          ctypes.POINTER(FalconDims), ctypes.c_int, vp]
        lib.falcon_workspace_bytes.restype = ctypes.c_size_t
        lib.falcon_workspace_bytes.argtypes = [ctypes.c_int, ctypes.POINTER(FalconDims), ctypes.c_int]
        lib.falcon_tail_bytes.restype = ctypes.c_size_t
        lib.falcon_tail_bytes.argtypes = [ctypes.POINTER(FalconDims)]
        lib.falcon_status_string.restype = ctypes.c_char_p
        lib.falcon_status_string.argtypes = [ctypes.c_int]
        lib.falcon_device_status.restype = ctypes.c_int
        lib.falcon_device_status.argtypes = [vp]
        lib.falcon_kernel_for.restype = ctypes.c_int
        lib.falcon_kernel_for.argtypes = [ctypes.c_int, ctypes.POINTER(FalconDims), ctypes.c_int]
        lib.falcon_abi_version.restype = ctypes.c_int
        lib.falcon_abi_version.argtypes = []
        lib.falcon_bwd.restype = ctypes.c_int
        lib.falcon_bwd.argtypes = [ctypes.c_int] + [vp] * 16 + [ctypes.POINTER(FalconDims), ctypes.c_int, vp,
                                                                ctypes.c_size_t, vp]
        lib.falcon_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.falcon_bwd_workspace_bytes.argtypes = [ctypes.c_int, ctypes.POINTER(FalconDims), ctypes.c_int]
        i32, f32 = ctypes.c_int, ctypes.c_float
        for name, args in (("falcon_glr_fwd", [i32] + [vp] * 6 + [vp, vp, vp]),
                           ("falcon_glr_bwd", [i32] + [vp] * 10 + [vp, vp, vp]),
                           ("falcon_gn_fwd", [i32] + [vp] * 6 + [vp, vp, f32, vp]),
                           ("falcon_gn_bwd", [i32] + [vp] * 10 + [vp, vp, f32, vp, ctypes.c_size_t, vp]),
                           ("falcon_gdr_fwd", [vp] * 11 + [f32, vp, ctypes.c_size_t, vp]),
                           ("falcon_gdr_bwd", [vp] * 17 + [f32, vp, ctypes.c_size_t, vp]),
                           ("falcon_rms_fwd", [vp] * 9 + [f32, vp]),
                           ("falcon_rms_bwd", [vp] * 9 + [f32, vp, ctypes.c_size_t, vp])):
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = args
        lib.falcon_gdr_workspace_bytes.restype = ctypes.c_size_t
        lib.falcon_gdr_workspace_bytes.argtypes = [vp, i32]
        lib.falcon_rms_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.falcon_rms_bwd_workspace_bytes.argtypes = [vp]
        lib.falcon_gn_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.falcon_gn_bwd_workspace_bytes.argtypes = [vp]
        if path is None:
            _lib = lib
        return lib


def make_dims(batch, heads, seqlen, dk, dv, *, window=1, dtype=FALCON_BF16, pos=0, eps=1e-6,
              eps_gamma=1e-6) -> FalconDims:
    return FalconDims(int(batch), int(heads), int(seqlen), int(dk), int(dv), int(window), int(dtype), int(pos),
                      float(eps), float(eps_gamma))


def status_string(status: int) -> str:
    return load().falcon_status_string(int(status)).decode()


def falcon_tail_bytes(dims: FalconDims) -> int:
    return int(load().falcon_tail_bytes(ctypes.byref(dims)))


def falcon_workspace_bytes(variant: int, dims: FalconDims, chunk: int) -> int:
    return int(load().falcon_workspace_bytes(int(variant), ctypes.byref(dims), int(chunk)))


def falcon_kernel_for(variant: int, dims: FalconDims, chunk: int) -> int:
    return int(load().falcon_kernel_for(int(variant), ctypes.byref(dims), int(chunk)))


def falcon_device_status(stream=None) -> int:
    return int(load().falcon_device_status(_stream_handle(stream)))


def falcon_abi_version() -> int:
    return int(load().falcon_abi_version())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream_handle(stream):
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _as_current(stream, device):
    """A context in which `stream` (a torch stream, an object with its handle, or the handle) is the current one. What a
    call allocates in it belongs to that stream: the allocator reuses a block behind the work of the stream that it
    belongs to, so a workspace from another stream's pool could be handed out again while the kernels still use it."""
    t = _t()
    handle = _handle(stream, device)
    if handle == 1:  # cudaStreamLegacy, the default stream's other name, which torch knows as 0
        handle = stream = 0
    if device.index is not None and t.current_device() == device.index and t.raw_stream(device.index) == handle:
        return contextlib.nullcontext()
    if not isinstance(stream, t.torch.cuda.Stream):
        stream = t.torch.cuda.ExternalStream(handle, device=device)
    return t.torch.cuda.stream(stream)


def _handle(stream, device):
    """The raw handle of a stream argument."""
    if isinstance(stream, int):
        return stream
    if isinstance(stream, _t().torch.cuda.Stream) and stream.device != device:
        raise ValueError(f"stream must be on {device}, got one on {stream.device}")
    return stream.cuda_stream


def falcon_fwd(variant, q, k, v, beta, lam, S0, tail, out, S_final, tail_out, dims: FalconDims, chunk: int,
               workspace=None, workspace_bytes=None, stream=None) -> int:
    """The C entry point with the same argument order; tensors or raw device pointers. Returns the status.

    ``workspace_bytes`` defaults to the size of a tensor workspace (0 for a raw pointer)."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None or isinstance(workspace, int) else \
            workspace.numel() * workspace.element_size()
    return int(load().falcon_fwd(int(variant), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(lam), _ptr(S0),
                                 _ptr(tail), _ptr(out), _ptr(S_final), _ptr(tail_out), ctypes.byref(dims),
                                 int(chunk), _ptr(workspace), int(workspace_bytes), _stream_handle(stream)))


def falcon_fwd_static(variant, q, k, v, beta, lam, S0, tail, out, S_final, tail_out, dims: FalconDims, chunk: int,
                      stream=None) -> int:
    """The no-allocation C entry point (the library's own fixed scratch); returns the status."""
    return int(load().falcon_fwd_static(int(variant), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(lam), _ptr(S0),
                                        _ptr(tail), _ptr(out), _ptr(S_final), _ptr(tail_out), ctypes.byref(dims),
                                        int(chunk), _stream_handle(stream)))


def falcon_bwd(variant, q, k, v, beta, lam, S0, tail, dout, dS_final, dq, dk, dv, dbeta, dlam, dS0, dtail,
               dims: FalconDims, chunk: int, workspace=None, workspace_bytes=None, stream=None) -> int:
    """The C entry point falcon_bwd with the same argument order; tensors or raw device pointers."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None or isinstance(workspace, int) else \
            workspace.numel() * workspace.element_size()
    return int(load().falcon_bwd(int(variant), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(lam), _ptr(S0),
                                 _ptr(tail), _ptr(dout), _ptr(dS_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta),
                                 _ptr(dlam), _ptr(dS0), _ptr(dtail), ctypes.byref(dims), int(chunk),
                                 _ptr(workspace), int(workspace_bytes), _stream_handle(stream)))


def falcon_bwd_workspace_bytes(variant: int, dims: FalconDims, chunk: int) -> int:
    return int(load().falcon_bwd_workspace_bytes(int(variant), ctypes.byref(dims), int(chunk)))


def backward(variant, q, k, v, beta, lam, dout, S0=None, dS_final=None, tail=None, *, pos=0, chunk=64, eps=1e-6,
             eps_gamma=1e-6, want_dS0=True, stream=None):
    """Allocate fp32 gradients and a workspace with torch on q's device and call falcon_bwd; raises
    FalconError on a nonzero status. Returns a dict dq, dk, dv, dbeta, dlam, dS0 (None unless
    want_dS0), dtail (None unless pos > 0). With `stream` (a torch stream or a raw handle) the whole call, its
    allocations too, is that stream's, as inside torch.cuda.stream(stream)."""
    import torch

    if stream is not None:
        with _as_current(stream, q.device):
            return backward(variant, q, k, v, beta, lam, dout, S0, dS_final, tail, pos=pos, chunk=chunk, eps=eps,
                            eps_gamma=eps_gamma, want_dS0=want_dS0)
    if isinstance(variant, str):
        variant = VARIANTS[variant]
    B, H, T, dk_ = q.shape
    dv_ = v.shape[-1]
    dt = FALCON_BF16 if q.dtype == torch.bfloat16 else FALCON_F32
    dims = make_dims(B, H, T, dk_, dv_, dtype=dt, pos=pos, eps=eps, eps_gamma=eps_gamma)
    f32 = dict(dtype=torch.float32, device=q.device)
    g = {"dq": torch.empty((B, H, T, dk_), **f32), "dk": torch.empty((B, H, T, dk_), **f32),
         "dv": torch.empty((B, H, T, dv_), **f32), "dbeta": torch.empty((B, H, T), **f32),
         "dlam": torch.empty((B, H, T), **f32),
         "dS0": torch.empty((B, H, dk_, dv_), **f32) if want_dS0 else None,
         "dtail": torch.empty((B, H, dk_), **f32) if pos > 0 else None}
    n = falcon_bwd_workspace_bytes(variant, dims, chunk)
    ws = torch.empty(n, dtype=torch.uint8, device=q.device) if n > 0 else None
    st = falcon_bwd(variant, q, k, v, beta, lam, S0, tail, dout, dS_final, g["dq"], g["dk"], g["dv"], g["dbeta"],
                    g["dlam"], g["dS0"], g["dtail"], dims, chunk, ws)
    if st != FALCON_OK:
        raise FalconError(st, "falcon_bwd")
    return g


def workspace_for(variant, dims: FalconDims, chunk: int, device):
    """A workspace tensor sized for falcon_fwd's split path, or None when no path needs one."""
    import torch

    n = falcon_workspace_bytes(variant, dims, chunk)
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def forward(variant, q, k, v, beta, lam, S0=None, tail=None, *, pos=0, window=1, chunk=64, eps=1e-6,
            eps_gamma=1e-6, want_state=True, want_tail=True, split=True, stream=None):
    """Allocate outputs with torch on q's device and call falcon_fwd; raises FalconError on a nonzero status.

    Returns (out, S_final or None, tail_out or None). tail/tail_out are flat byte-sized
    buffers in q's dtype, laid out per (b,h) as keys[window][dk] then vals[window-1][dv].
    ``split=True`` hands falcon_fwd a workspace whenever a path can use one; ``False`` runs the
    single-pass kernels. With `stream` (a torch stream or a raw handle) the whole call, its allocations too, is that
    stream's, as inside torch.cuda.stream(stream).
    """
    import torch

    if stream is not None:
        with _as_current(stream, q.device):
            return forward(variant, q, k, v, beta, lam, S0, tail, pos=pos, window=window, chunk=chunk, eps=eps,
                           eps_gamma=eps_gamma, want_state=want_state, want_tail=want_tail, split=split)
    if isinstance(variant, str):
        variant = VARIANTS[variant]
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = FALCON_BF16 if q.dtype == torch.bfloat16 else FALCON_F32
    dims = make_dims(B, H, T, dk, dv, window=window, dtype=dt, pos=pos, eps=eps, eps_gamma=eps_gamma)
    out = torch.empty((B, H, T, dv), dtype=q.dtype, device=q.device)
    S_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if want_state else None
    tail_out = None
    if want_tail:
        n = falcon_tail_bytes(dims) // q.element_size()
        tail_out = torch.empty(n, dtype=q.dtype, device=q.device)
    ws = workspace_for(variant, dims, chunk, q.device) if split else None
    st = falcon_fwd(variant, q, k, v, beta, lam, S0, tail, out, S_final, tail_out, dims, chunk, ws)
    if st != FALCON_OK:
        raise FalconError(st)
    return out, S_final, tail_out


def split_tail(tail_flat, B, H, W, dk, dv):
    """View a flat tail buffer as (keys [B,H,W,dk], vals [B,H,W-1,dv])."""
    per = W * dk + (W - 1) * dv
    t = tail_flat.view(B, H, per)
    return t[..., : W * dk].reshape(B, H, W, dk), t[..., W * dk:].reshape(B, H, W - 1, dv)


def join_tail(keys, vals):
    """Pack (keys [B,H,W,dk], vals [B,H,W-1,dv]) into the flat tail layout."""
    import torch

    B, H = keys.shape[:2]
    return torch.cat([keys.reshape(B, H, -1), vals.reshape(B, H, -1)], dim=-1).reshape(-1).contiguous()


# ---- the strided [B,H,T,d] operators: gated linear recurrence and head norm


def make_seq_dims(batch, heads, seqlen, d, *, dtype=FALCON_BF16) -> FalconSeqDims:
    return FalconSeqDims(int(batch), int(heads), int(seqlen), int(d), int(dtype), 0)


def _strides(strides):
    """A flat sequence of (batch, head, token) strides per tensor as an int64 array, or None (dense)."""
    return None if strides is None else (ctypes.c_int64 * len(strides))(*strides)


def falcon_glr_fwd(gate, x, g, h0, lengths, out, h_final, dims: FalconSeqDims, strides=None, stream=None) -> int:
    """The C entry point with the same argument order; tensors or raw device pointers, `strides` 9 values or
    None. Returns the status."""
    return int(load().falcon_glr_fwd(int(gate), _ptr(x), _ptr(g), _ptr(h0), _ptr(lengths), _ptr(out), _ptr(h_final),
                                     ctypes.byref(dims), _strides(strides), _stream_handle(stream)))


def falcon_glr_bwd(gate, x, g, out, h0, lengths, dout, dh_final, dx, dg, dh0, dims: FalconSeqDims, strides=None,
                   stream=None) -> int:
    """The C entry point (`strides` 18 values or None); returns the status."""
    return int(load().falcon_glr_bwd(int(gate), _ptr(x), _ptr(g), _ptr(out), _ptr(h0), _ptr(lengths), _ptr(dout),
                                     _ptr(dh_final), _ptr(dx), _ptr(dg), _ptr(dh0), ctypes.byref(dims),
                                     _strides(strides), _stream_handle(stream)))


def falcon_gn_fwd(act, x, z, weight, bias, lengths, y, dims: FalconSeqDims, strides=None, eps=1e-5,
                  stream=None) -> int:
    """The C entry point (`strides` 9 values or None); returns the status."""
    return int(load().falcon_gn_fwd(int(act), _ptr(x), _ptr(z), _ptr(weight), _ptr(bias), _ptr(lengths), _ptr(y),
                                    ctypes.byref(dims), _strides(strides), float(eps), _stream_handle(stream)))


def falcon_gn_bwd(act, x, z, weight, bias, lengths, dy, dx, dz, dweight, dbias, dims: FalconSeqDims, strides=None,
                  eps=1e-5, workspace=None, workspace_bytes=None, stream=None) -> int:
    """The C entry point (`strides` 15 values or None); returns the status."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None or isinstance(workspace, int) else \
            workspace.numel() * workspace.element_size()
    return int(load().falcon_gn_bwd(int(act), _ptr(x), _ptr(z), _ptr(weight), _ptr(bias), _ptr(lengths), _ptr(dy),
                                    _ptr(dx), _ptr(dz), _ptr(dweight), _ptr(dbias), ctypes.byref(dims),
                                    _strides(strides), float(eps), _ptr(workspace), int(workspace_bytes),
                                    _stream_handle(stream)))


def falcon_gn_bwd_workspace_bytes(dims: FalconSeqDims) -> int:
    return int(load().falcon_gn_bwd_workspace_bytes(ctypes.byref(dims)))


_PACK_DIMS = struct.Struct("=4q2i").pack
_PACK_STRIDES = {n: struct.Struct(f"={3 * n}q").pack for n in (3, 5, 6)}


_Torch = collections.namedtuple("_Torch", "torch float32 codes raw_stream current_device empty")


@functools.lru_cache(maxsize=None)
def _t():
    """What the calls below need of torch, looked up once: the module, the types' codes, and how to ask for the current
    stream's handle and the current device without building an object (0.1 us against 1.1 for
    torch.cuda.current_stream, of the 7 us that a call on small tensors takes)."""
    import torch

    return _Torch(torch, torch.float32, {torch.bfloat16: FALCON_BF16, torch.float32: FALCON_F32},
                  torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice, torch.empty)


def _seq_call(what, choice, x, views, arrays, shape, lengths, names, stream):
    """Checks the tensors of one call and marshals them. `views` (tensors or None) are [B,H,T,d] like x in x's type,
    `arrays` (tensors or None) contiguous fp32 of `shape`; `names` has the views' names, then the arrays'. Returns
    the library's function `what`, the pointers (views, arrays, lengths), the packed falcon_seq_dims_t and strides,
    and the stream's handle (the current one's where `stream` is None)."""
    torch, f32, codes, raw_stream, current_device, _ = _t()
    full, dtype, index = x.shape, x.dtype, x.get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    if choice is None:
        raise ValueError(f"{what}: no such gate or activation")
    if dtype not in codes:
        raise ValueError(f"unsupported dtype {dtype}: float32 or bfloat16")
    pointers, strides = [], []
    for t in views:
        if t is None:
            pointers.append(None)
            strides += (0, 0, 0)
            continue
        layout = t.stride()
        if t.shape != full or t.dtype is not dtype or t.get_device() != index or layout[3] != 1 and full[3] > 1:
            raise ValueError(f"{names[len(pointers)]} must be {tuple(full)} {dtype} on {x.device} with contiguous "
                             f"channels, got {tuple(t.shape)} {t.dtype} on {t.device} with strides {layout}")
        strides += layout[:3]
        pointers.append(t.data_ptr())
    for t in arrays:
        if t is None:
            pointers.append(None)
            continue
        if t.shape != shape or t.dtype is not f32 or t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"{names[len(pointers)]} must be contiguous {tuple(shape)} {f32} on {x.device}, got "
                             f"{tuple(t.shape)} {t.dtype} on {t.device}")
        pointers.append(t.data_ptr())
    if lengths is None:
        pointers.append(None)
    else:
        if lengths.shape != full[:1] or lengths.dtype is not torch.int32 or lengths.get_device() != index or \
                not lengths.is_contiguous():
            raise ValueError(f"lengths must be contiguous ({full[0]},) torch.int32 on {x.device}, got "
                             f"{tuple(lengths.shape)} {lengths.dtype} on {lengths.device}")
        pointers.append(lengths.data_ptr())
    fn = getattr(_lib or load(), what)
    if index != current_device():
        fn = _on_device(fn, index)
    return fn, pointers, _PACK_DIMS(*full, codes[dtype], 0), _PACK_STRIDES[len(views)](*strides), \
        raw_stream(index) if stream is None else _handle(stream, x.device)


def _on_device(fn, index):
    """fn with device `index` current."""

    def call(*args):
        with _t().torch.cuda.device(index):
            return fn(*args)

    return call


def _sizes(x):
    if x.dim() != 4:
        raise ValueError(f"x must be [B,H,T,d], got {tuple(x.shape)}")
    return x.shape


def _empty(x, shape, dtype, stream):
    """A tensor beside x whose memory belongs to `stream` (None: the current one)."""
    if stream is None:
        return _t().empty(shape, dtype=dtype, device=x.device)
    with _as_current(stream, x.device):
        return _t().empty(shape, dtype=dtype, device=x.device)


@functools.lru_cache(maxsize=256)
def _gn_bwd_bytes(dims):
    """falcon_gn_bwd_workspace_bytes of a packed falcon_seq_dims_t (a function of the sizes alone)."""
    return int(load().falcon_gn_bwd_workspace_bytes(dims))


def glr_forward(gate, x, g, h0=None, *, lengths=None, out=None, h_final=None, want_state=True, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t per channel; returns (out, h_final or None).

    gate: "decay" (a = exp(g), u = x), "sigmoid" (a = sigmoid(g), u = x) or "mix" (a = sigmoid(g),
    u = (1 - a) x). x, g: [B,H,T,d], float32 or bfloat16, any strides with contiguous channels (so
    `proj.view(B, T, H, d).transpose(1, 2)` and column blocks are passed as they are). h0: fp32 [B,H,d] or
    None (zero). lengths: int32 [B] or None; rows behind them come back as zeros. out (a [B,H,T,d] view) and
    h_final (may be h0: updated in place) are written where given, else allocated dense. With `stream` (a torch
    stream or a raw handle) the kernels run there and what is allocated belongs to it, as inside
    torch.cuda.stream(stream); where all outputs are given that costs nothing."""
    B, H, T, d = _sizes(x)
    if out is None:
        out = _empty(x, x.shape, x.dtype, stream)
    if h_final is None and want_state:
        h_final = _empty(x, (B, H, d), _t().float32, stream)
    code = GLR_GATES.get(gate)
    fn, pointers, dims, strides, handle = _seq_call(
        "falcon_glr_fwd", code, x, (x, g, out), (h0, h_final), (B, H, d), lengths, ("x", "g", "out", "h0", "h_final"),
        stream)
    p_x, p_g, p_out, p_h0, p_h_final, p_lengths = pointers
    st = fn(code, p_x, p_g, p_h0, p_lengths, p_out, p_h_final, dims, strides, handle)
    if st != FALCON_OK:
        raise FalconError(st, "falcon_glr_fwd")
    return out, h_final


def glr_backward(gate, x, g, out, dout, h0=None, dh_final=None, *, lengths=None, dx=None, dg=None, dh0=None,
                 stream=None):
    """Gradients of one glr_forward call, from its inputs, its output `out` and the adjoints of out and
    h_final. Returns a dict dx, dg (in x's dtype), dh0 (fp32); each is written where given, else allocated.
    stream: as for glr_forward."""
    B, H, T, d = _sizes(x)
    dx = _empty(x, x.shape, x.dtype, stream) if dx is None else dx
    dg = _empty(x, x.shape, x.dtype, stream) if dg is None else dg
    dh0 = _empty(x, (B, H, d), _t().float32, stream) if dh0 is None else dh0
    code = GLR_GATES.get(gate)
    fn, pointers, dims, strides, handle = _seq_call(
        "falcon_glr_bwd", code, x, (x, g, out, dout, dx, dg), (h0, dh_final, dh0), (B, H, d), lengths,
        ("x", "g", "out", "dout", "dx", "dg", "h0", "dh_final", "dh0"), stream)
    p_x, p_g, p_out, p_dout, p_dx, p_dg, p_h0, p_dh_final, p_dh0, p_lengths = pointers
    st = fn(code, p_x, p_g, p_out, p_h0, p_lengths, p_dout, p_dh_final, p_dx, p_dg, p_dh0, dims, strides, handle)
    if st != FALCON_OK:
        raise FalconError(st, "falcon_glr_bwd")
    return {"dx": dx, "dg": dg, "dh0": dh0}


def groupnorm_forward(x, weight=None, bias=None, z=None, *, act="none", eps=1e-5, lengths=None, y=None, stream=None):
    """Group norm of each token's head over its d channels: n = weight (x - mean) / sqrt(var + eps) + bias,
    y = act(n), or n * act(z) with a gate z.

    x, z: [B,H,T,d] views as for glr_forward; weight, bias: fp32 [H,d] or None; act: "none", "silu", "gelu"
    (erf) or "sigmoid". y is written where given, else allocated in the output projection's layout: a [B,H,T,d]
    view of a dense [B,T,H,d], so `y.transpose(1, 2).reshape(B, T, H * d)` is free. stream: as for glr_forward."""
    B, H, T, d = _sizes(x)
    if y is None:
        y = _empty(x, (B, T, H, d), x.dtype, stream).transpose(1, 2)
    code = GN_ACTS.get(act)
    fn, pointers, dims, strides, handle = _seq_call(
        "falcon_gn_fwd", code, x, (x, z, y), (weight, bias), (H, d), lengths, ("x", "z", "y", "weight", "bias"), stream)
    p_x, p_z, p_y, p_weight, p_bias, p_lengths = pointers
    st = fn(code, p_x, p_z, p_weight, p_bias, p_lengths, p_y, dims, strides, eps, handle)
    if st != FALCON_OK:
        raise FalconError(st, "falcon_gn_fwd")
    return y


def groupnorm_backward(x, dy, weight=None, bias=None, z=None, *, act="none", eps=1e-5, lengths=None, dx=None,
                       dz=None, dweight=None, dbias=None, workspace=None, want_params=True, stream=None):
    """Gradients of one groupnorm_forward call. Returns a dict dx, dz (None without a gate), dweight, dbias
    (fp32 [H,d]; None unless want_params or given). Each is written where given, else allocated dense; so is the
    workspace, uint8 of falcon_gn_bwd_workspace_bytes, which dweight and dbias need. stream: as for glr_forward."""
    B, H, T, d = _sizes(x)
    dx = _empty(x, x.shape, x.dtype, stream) if dx is None else dx
    if z is not None and dz is None:
        dz = _empty(x, x.shape, x.dtype, stream)
    if want_params:
        dweight = _empty(x, (H, d), _t().float32, stream) if dweight is None else dweight
        dbias = _empty(x, (H, d), _t().float32, stream) if dbias is None else dbias
    code = GN_ACTS.get(act)
    fn, pointers, dims, strides, handle = _seq_call(
        "falcon_gn_bwd", code, x, (x, z, dy, dx, dz), (weight, bias, dweight, dbias), (H, d), lengths,
        ("x", "z", "dy", "dx", "dz", "weight", "bias", "dweight", "dbias"), stream)
    size = 0
    if dweight is not None or dbias is not None:
        if workspace is None:
            size = _gn_bwd_bytes(dims)
            if size > 0:
                workspace = _empty(x, size, _t().torch.uint8, stream)
        else:
            if workspace.get_device() != x.get_device() or not workspace.is_contiguous():
                raise ValueError(f"workspace must be contiguous on {x.device}, got one on {workspace.device}")
            size = workspace.numel() * workspace.element_size()
    p_x, p_z, p_dy, p_dx, p_dz, p_weight, p_bias, p_dweight, p_dbias, p_lengths = pointers
    st = fn(code, p_x, p_z, p_weight, p_bias, p_lengths, p_dy, p_dx, p_dz, p_dweight, p_dbias, dims, strides, eps,
            _ptr(workspace), size, handle)
    if st != FALCON_OK:
        raise FalconError(st, "falcon_gn_bwd")
    return {"dx": dx, "dz": dz, "dweight": dweight, "dbias": dbias}


# ---- the block around the read: gated delta rule, root-mean-square norm


def make_gdr_dims(batch, heads, seqlen, dk, dv, *, qk_heads=None, dtype=FALCON_BF16) -> FalconGdrDims:
    return FalconGdrDims(int(batch), int(heads), int(heads if qk_heads is None else qk_heads), int(seqlen), int(dk),
                         int(dv), int(dtype), 0)


def make_rms_dims(batch, seqlen, d, *, dtype=FALCON_BF16, out_dtype=None) -> FalconRmsDims:
    return FalconRmsDims(int(batch), int(seqlen), int(d), int(dtype), int(dtype if out_dtype is None else out_dtype))


def _ws_bytes(workspace, workspace_bytes):
    if workspace_bytes is None:
        return 0 if workspace is None or isinstance(workspace, int) else workspace.numel() * workspace.element_size()
    return int(workspace_bytes)


def falcon_gdr_fwd(q, k, v, beta, g, S0, lengths, out, S_final, dims: FalconGdrDims, strides=None, scale=1.0,
                   workspace=None, workspace_bytes=None, stream=None) -> int:
    """The C entry point with the same argument order; tensors or raw device pointers, `strides` 18 values or None.
    Returns the status."""
    return int(load().falcon_gdr_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(S0), _ptr(lengths),
                                     _ptr(out), _ptr(S_final), ctypes.byref(dims), _strides(strides), float(scale),
                                     _ptr(workspace), _ws_bytes(workspace, workspace_bytes), _stream_handle(stream)))


def falcon_gdr_bwd(q, k, v, beta, g, S0, lengths, dout, dS_final, dq, dk, dv, dbeta, dg, dS0, dims: FalconGdrDims,
                   strides=None, scale=1.0, workspace=None, workspace_bytes=None, stream=None) -> int:
    """The C entry point (`strides` 33 values or None); returns the status."""
    return int(load().falcon_gdr_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(S0), _ptr(lengths),
                                     _ptr(dout), _ptr(dS_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(dg),
                                     _ptr(dS0), ctypes.byref(dims), _strides(strides), float(scale), _ptr(workspace),
                                     _ws_bytes(workspace, workspace_bytes), _stream_handle(stream)))


def falcon_gdr_workspace_bytes(dims: FalconGdrDims, backward: bool = False) -> int:
    return int(load().falcon_gdr_workspace_bytes(ctypes.byref(dims), int(backward)))


def falcon_rms_fwd(x, residual, weight, lengths, h, y, scales, dims: FalconRmsDims, strides=None, eps=1e-6,
                   stream=None) -> int:
    """The C entry point (`strides` 8 values or None); returns the status."""
    return int(load().falcon_rms_fwd(_ptr(x), _ptr(residual), _ptr(weight), _ptr(lengths), _ptr(h), _ptr(y),
                                     _ptr(scales), ctypes.byref(dims), _strides(strides), float(eps),
                                     _stream_handle(stream)))


def falcon_rms_bwd(h, weight, lengths, dy, dh, dx, dweight, dims: FalconRmsDims, strides=None, eps=1e-6,
                   workspace=None, workspace_bytes=None, stream=None) -> int:
    """The C entry point (`strides` 8 values or None); returns the status."""
    return int(load().falcon_rms_bwd(_ptr(h), _ptr(weight), _ptr(lengths), _ptr(dy), _ptr(dh), _ptr(dx),
                                     _ptr(dweight), ctypes.byref(dims), _strides(strides), float(eps),
                                     _ptr(workspace), _ws_bytes(workspace, workspace_bytes), _stream_handle(stream)))


def falcon_rms_bwd_workspace_bytes(dims: FalconRmsDims) -> int:
    return int(load().falcon_rms_bwd_workspace_bytes(ctypes.byref(dims)))


_PACK_GDR = struct.Struct("=6q2i").pack
_PACK_RMS = struct.Struct("=3q2i").pack
_PACK_8, _PACK_18, _PACK_33 = (struct.Struct(f"={n}q").pack for n in (8, 18, 33))


def _refuse(name, t, shape, dtype, device, what="contiguous channels"):
    raise ValueError(f"{name} must be {tuple(shape)} {dtype} on {device} with {what}, got {tuple(t.shape)} {t.dtype} on "
                     f"{t.device} with strides {t.stride()}")


def _views(names, tensors, shapes, dtype, index, x, pointers, strides):
    """Checks strided tensors (the last axis contiguous), None for one that is not there, and notes their pointers and
    their other axes' strides."""
    for name, t, shape in zip(names, tensors, shapes):
        if t is None:
            pointers.append(None)
            strides += (0,) * (len(shape) - 1)
            continue
        layout = t.stride()
        if t.shape != shape or t.dtype is not dtype or t.get_device() != index or layout[-1] != 1 and shape[-1] > 1:
            _refuse(name, t, shape, dtype, x.device)
        strides += layout[:-1]
        pointers.append(t.data_ptr())


def _gate_views(names, tensors, shape, index, x, pointers, strides):
    """The same for fp32 [B,H,T] tensors, whose tokens may lie apart."""
    f32 = _t().float32
    for name, t in zip(names, tensors):
        if t.shape != shape or t.dtype is not f32 or t.get_device() != index:
            _refuse(name, t, shape, f32, x.device, "any strides")
        strides += t.stride()
        pointers.append(t.data_ptr())


def _dense(name, t, shape, dtype, index, x):
    """The pointer of a contiguous array, None without one."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        _refuse(name, t, shape, dtype, x.device, "no gaps")
    return t.data_ptr()


def _launch(what, index, args):
    fn = getattr(_lib or load(), what)
    if index != _t().current_device():
        fn = _on_device(fn, index)
    st = fn(*args)
    if st != FALCON_OK:
        raise FalconError(st, what)


def _workspace(workspace, need, x, stream):
    """A workspace tensor of at least `need` bytes and its size; allocated beside x where none is given."""
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = _empty(x, need, _t().torch.uint8, stream)
    elif workspace.get_device() != x.get_device() or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {x.device}, got one on {workspace.device}")
    return workspace, workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=256)
def _gdr_bytes(dims, backward):
    return int(load().falcon_gdr_workspace_bytes(dims, backward))


@functools.lru_cache(maxsize=256)
def _rms_bytes(dims):
    return int(load().falcon_rms_bwd_workspace_bytes(dims))


def _gdr_sizes(q, v):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError(f"q and v must be [B,H,T,d], got {tuple(q.shape)} and {tuple(v.shape)}")
    index, dtype = q.get_device(), q.dtype
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    code = _t().codes.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}: float32 or bfloat16")
    B, Hk, T, dk = q.shape
    H, dv = v.shape[1], v.shape[3]
    if Hk != H and (Hk == 0 or H == 0 or H % Hk):
        raise ValueError(f"the heads of q and k must divide those of v, got {Hk} and {H}")
    if dk == 0 or dv == 0:
        raise ValueError(f"q and v must have channels, got {tuple(q.shape)} and {tuple(v.shape)}")
    return index, dtype, B, H, Hk, T, dk, dv, _PACK_GDR(B, H, Hk, T, dk, dv, code, 0)


def gdr_forward(q, k, v, beta, g, S0=None, *, scale=None, lengths=None, out=None, S_final=None, want_state=True,
                workspace=None, stream=None):
    """Gated delta rule: S_t = a_t S_{t-1} + k_t (beta_t (v_t - a_t S_{t-1}^T k_t))^T with a_t = exp(g_t),
    out_t = scale S_t^T q_t; returns (out, S_final or None).

    q, k: [B,Hk,T,dk], v: [B,H,T,dv], float32 or bfloat16, any strides with contiguous channels (column blocks of one
    projection are passed as they are); Hk divides H, and each head of q and k is shared by H / Hk heads of v that
    follow each other. dk, dv up to 128. beta (gain), g (log decay): fp32 [B,H,T], any strides. S0: fp32 [B,H,dk,dv]
    or None (zero). scale: dk ** -0.5 unless given. lengths: int32 [B] or None; rows behind them come back as zeros.
    out (a [B,H,T,dv] view) and S_final (may be S0: updated in place) are written where given; out is else allocated
    in the output projection's layout, a view of a dense [B,T,H,dv]. workspace: uint8 of falcon_gdr_workspace_bytes,
    allocated unless given (up to 32 tokens need none). stream: as for glr_forward."""
    index, dtype, B, H, Hk, T, dk, dv, dims = _gdr_sizes(q, v)
    t = _t()
    if out is None:
        out = _empty(v, (B, T, H, dv), dtype, stream).transpose(1, 2)
    if S_final is None and want_state:
        S_final = _empty(v, (B, H, dk, dv), t.float32, stream)
    pointers, strides = [], []
    of_qk, of_v = (B, Hk, T, dk), (B, H, T, dv)
    _views(("q", "k", "v"), (q, k, v), (of_qk, of_qk, of_v), dtype, index, q, pointers, strides)
    _gate_views(("beta", "g"), (beta, g), (B, H, T), index, q, pointers, strides)
    _views(("out",), (out,), (of_v,), dtype, index, q, pointers, strides)
    p_out = pointers.pop()
    state = (B, H, dk, dv)
    p_S0 = _dense("S0", S0, state, t.float32, index, q)
    p_last = _dense("S_final", S_final, state, t.float32, index, q)
    p_len = _dense("lengths", lengths, (B,), t.torch.int32, index, q)
    workspace, size = _workspace(workspace, _gdr_bytes(dims, 0), q, stream)
    _launch("falcon_gdr_fwd", index, (*pointers, p_S0, p_len, p_out, p_last, dims, _PACK_18(*strides),
                                      dk ** -0.5 if scale is None else scale, _ptr(workspace), size,
                                      t.raw_stream(index) if stream is None else _handle(stream, q.device)))
    return out, S_final


def gdr_backward(q, k, v, beta, g, dout, S0=None, dS_final=None, *, scale=None, lengths=None, dq=None, dk=None,
                 dv=None, dbeta=None, dg=None, dS0=None, workspace=None, stream=None):
    """Gradients of one gdr_forward call, from its inputs and the adjoints of out and S_final. Returns a dict dq, dk,
    dv (in q's type), dbeta, dg, dS0 (fp32); each is written where given, else allocated dense. workspace: as for
    gdr_forward, of falcon_gdr_workspace_bytes(dims, backward=True). stream: as for glr_forward."""
    index, dtype, B, H, Hk, T, n_k, n_v, dims = _gdr_sizes(q, v)
    t = _t()
    f32, state = t.float32, (B, H, n_k, n_v)
    dq = _empty(q, (B, Hk, T, n_k), dtype, stream) if dq is None else dq
    dk = _empty(q, (B, Hk, T, n_k), dtype, stream) if dk is None else dk
    dv = _empty(q, (B, H, T, n_v), dtype, stream) if dv is None else dv
    dbeta = _empty(q, (B, H, T), f32, stream) if dbeta is None else dbeta
    dg = _empty(q, (B, H, T), f32, stream) if dg is None else dg
    dS0 = _empty(q, state, f32, stream) if dS0 is None else dS0
    pointers, strides = [], []
    of_qk, of_v, of_t = (B, Hk, T, n_k), (B, H, T, n_v), (B, H, T)
    _views(("q", "k", "v"), (q, k, v), (of_qk, of_qk, of_v), dtype, index, q, pointers, strides)
    _gate_views(("beta", "g"), (beta, g), of_t, index, q, pointers, strides)
    _views(("dout", "dq", "dk", "dv"), (dout, dq, dk, dv), (of_v, of_qk, of_qk, of_v), dtype, index, q, pointers, strides)
    _gate_views(("dbeta", "dg"), (dbeta, dg), of_t, index, q, pointers, strides)
    p_S0 = _dense("S0", S0, state, f32, index, q)
    p_dS = _dense("dS_final", dS_final, state, f32, index, q)
    p_dS0 = _dense("dS0", dS0, state, f32, index, q)
    p_len = _dense("lengths", lengths, (B,), t.torch.int32, index, q)
    workspace, size = _workspace(workspace, _gdr_bytes(dims, 1), q, stream)
    _launch("falcon_gdr_bwd", index, (*pointers[:5], p_S0, p_len, pointers[5], p_dS, *pointers[6:], p_dS0, dims,
                                      _PACK_33(*strides), n_k ** -0.5 if scale is None else scale, _ptr(workspace),
                                      size, t.raw_stream(index) if stream is None else _handle(stream, q.device)))
    return {"dq": dq, "dk": dk, "dv": dv, "dbeta": dbeta, "dg": dg, "dS0": dS0}


def _rms_sizes(x):
    """[B,T,d], or [N,d] as one sequence of N tokens."""
    if x.dim() not in (2, 3):
        raise ValueError(f"x must be [B,T,d] or [N,d], got {tuple(x.shape)}")
    index = x.get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    code = _t().codes.get(x.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {x.dtype}: float32 or bfloat16")
    return index, code, (1, *x.shape) if x.dim() == 2 else tuple(x.shape)


def _row_strides(strides, flat):
    """(batch, token) strides per tensor from the tensors' own: flat tokens are one sequence."""
    if not flat:
        return strides
    out = [0] * (2 * len(strides))
    out[1::2] = strides
    return out


def rmsnorm_forward(x, weight=None, residual=None, *, eps=1e-6, lengths=None, y=None, h=None, scales=None,
                    out_dtype=None, stream=None):
    """Root-mean-square norm with the residual's addition, per token: h = x + residual, y = weight h /
    sqrt(mean h^2 + eps); returns (y, h, scales).

    x, residual: [B,T,d] or [N,d], float32 or bfloat16, any strides with contiguous channels; weight: fp32 [d] or None.
    h, in x's type, is what is normalised; it may be x or residual (updated in place), and without a residual it is x
    itself. out_dtype (or y's type): x's, or torch.float8_e4m3fn, with fp32 scales [B,T] (or [N]): a token's largest
    |y| / 448, of which y holds the multiples (else scales is None). lengths: int32 [B] or None; rows behind them come
    back as zeros. y, h and scales are written where given, else allocated dense. stream: as for glr_forward."""
    index, code, (B, T, d) = _rms_sizes(x)
    t = _t()
    torch = t.torch
    kind = y.dtype if y is not None else x.dtype if out_dtype is None else out_dtype
    if out_dtype is not None and kind is not out_dtype:
        raise ValueError(f"y must be {out_dtype}, got {kind}")
    eight = kind is torch.float8_e4m3fn
    if not eight and kind is not x.dtype:
        raise ValueError(f"y must be {x.dtype} or torch.float8_e4m3fn, got {kind}")
    if residual is None and h is not None:
        raise ValueError("h is written with a residual only: without one it is x")
    if scales is not None and not eight:
        raise ValueError("scales go with an output in 8 bits")
    y = _empty(x, x.shape, kind, stream) if y is None else y
    if residual is not None and h is None:
        h = _empty(x, x.shape, x.dtype, stream)
    if eight and scales is None:
        scales = _empty(x, x.shape[:-1], t.float32, stream)
    pointers, strides, shape = [], [], x.shape
    _views(("x", "residual", "h"), (x, residual, h), (shape, shape, shape), x.dtype, index, x, pointers, strides)
    _views(("y",), (y,), (shape,), kind, index, x, pointers, strides)
    p_x, p_r, p_h, p_y = pointers
    _launch("falcon_rms_fwd", index, (
        p_x, p_r, _dense("weight", weight, (d,), t.float32, index, x), _dense("lengths", lengths, (B,), torch.int32, index, x),
        p_h, p_y, _dense("scales", scales, x.shape[:-1], t.float32, index, x),
        _PACK_RMS(B, T, d, code, FALCON_E4M3 if eight else code), _PACK_8(*_row_strides(strides, len(shape) == 2)), eps,
        t.raw_stream(index) if stream is None else _handle(stream, x.device)))
    return y, x if residual is None else h, scales


def rmsnorm_backward(h, dy, weight=None, dh=None, *, eps=1e-6, lengths=None, dx=None, dweight=None, workspace=None,
                     want_params=True, stream=None):
    """Gradients of one rmsnorm_forward call, from what it normalised (its h, or x without a residual), the adjoint of y
    and that of h (None: nothing else reads it). Returns a dict dx, the gradient of x and of the residual alike (in h's
    type; may be dh, written in place), and dweight (fp32 [d]; None unless want_params or given). workspace: uint8 of
    falcon_rms_bwd_workspace_bytes, which dweight needs, allocated unless given. stream: as for glr_forward."""
    index, code, (B, T, d) = _rms_sizes(h)
    t = _t()
    dx = _empty(h, h.shape, h.dtype, stream) if dx is None else dx
    if want_params and dweight is None:
        dweight = _empty(h, (d,), t.float32, stream)
    pointers, strides, shape = [], [], h.shape
    _views(("h", "dy", "dh", "dx"), (h, dy, dh, dx), (shape, shape, shape, shape), h.dtype, index, h, pointers, strides)
    p_h, p_dy, p_dh, p_dx = pointers
    dims, size = _PACK_RMS(B, T, d, code, code), 0
    if dweight is not None:
        workspace, size = _workspace(workspace, _rms_bytes(dims), h, stream)
    _launch("falcon_rms_bwd", index, (
        p_h, _dense("weight", weight, (d,), t.float32, index, h),
        _dense("lengths", lengths, (B,), t.torch.int32, index, h), p_dy, p_dh, p_dx,
        _dense("dweight", dweight, (d,), t.float32, index, h), dims, _PACK_8(*_row_strides(strides, len(shape) == 2)),
        eps, _ptr(workspace), size,
        t.raw_stream(index) if stream is None else _handle(stream, h.device)))
    return {"dx": dx, "dweight": dweight}
