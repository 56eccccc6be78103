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

_lock = threading.Lock()
_lib = None

EXPORTED = ("falcon_fwd", "falcon_workspace_bytes", "falcon_fwd_static", "falcon_tail_bytes",
            "falcon_status_string", "falcon_device_status", "falcon_kernel_for", "falcon_abi_version",
            "falcon_bwd", "falcon_bwd_workspace_bytes", "falcon_glr_fwd", "falcon_glr_bwd", "falcon_gn_fwd",
            "falcon_gn_bwd", "falcon_gn_bwd_workspace_bytes")
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
                           ("falcon_gn_bwd", [i32] + [vp] * 10 + [vp, vp, f32, vp, ctypes.c_size_t, vp])):
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = args
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
