"""ctypes binding of libssd.so: argument marshalling only.

PyTorch provides device memory and the current stream; every step of the
computation runs in the library's HIP kernels. If the library has not been
built, every call raises -- there is no fallback implementation.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

__all__ = [
    "SSDError",
    "SSDDesc",
    "lib_path",
    "load_library",
    "make_desc",
    "status_string",
    "effective_chunk_size",
    "workspace_bytes",
    "workspace_bytes_varlen",
    "workspace_status",
    "workspace_status_varlen",
    "forward",
    "forward_noalloc",
    "chunk_cumsum",
    "chunk_state",
    "cumsum_chunk_state",
    "state_passing",
    "chunk_scan",
    "decode_step",
    "forward_varlen",
    "conv1d_split",
    "selective_scan",
    "selective_scan_varlen",
    "selective_scan_workspace_bytes",
    "selective_step",
    "conv1d",
    "conv1d_varlen",
    "conv1d_split_varlen",
    "conv1d_step",
    "conv1d_split_step",
    "group_norm",
    "EXPORTED_SYMBOLS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))

# Every symbol include/ssd.h declares.
EXPORTED_SYMBOLS = (
    "ssd_status_string",
    "ssd_effective_chunk_size",
    "ssd_workspace_bytes",
    "ssd_forward",
    "ssd_forward_fused",
    "ssd_forward_split",
    "ssd_workspace_status",
    "ssd_forward_noalloc",
    "ssd_chunk_cumsum",
    "ssd_chunk_state",
    "ssd_cumsum_chunk_state",
    "ssd_state_passing",
    "ssd_chunk_scan",
    "ssd_decode_step",
    "ssd_workspace_bytes_varlen",
    "ssd_forward_varlen",
    "ssd_workspace_status_varlen",
    "ssd_conv1d_split",
    "ssd_selective_scan_workspace_bytes",
    "ssd_selective_scan",
    "ssd_selective_scan_varlen",
    "ssd_selective_step",
    "ssd_conv1d",
    "ssd_conv1d_step",
    "ssd_group_norm",
)

SSD_DTYPE_F32 = 0
SSD_DTYPE_BF16 = 1


class SSDError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class SSDDesc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("nheads", ctypes.c_int64),
        ("headdim", ctypes.c_int64),
        ("dstate", ctypes.c_int64),
        ("ngroups", ctypes.c_int64),
        ("io_dtype", ctypes.c_int32),
        ("chunk_size", ctypes.c_int32),
        ("dt_bias", ctypes.c_void_p),
        ("dt_softplus", ctypes.c_int32),
        ("dt_clamp", ctypes.c_int32),
        ("dt_min", ctypes.c_float),
        ("dt_max", ctypes.c_float),
    ]


# (the C structs' pairs of strides, token and batch, are laid out flat here)
class SelectiveDesc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("channels", ctypes.c_int64),
        ("dstate", ctypes.c_int64),
        ("ngroups", ctypes.c_int64),
        ("io_dtype", ctypes.c_int32),
        ("dt_dtype", ctypes.c_int32),
        ("dt_bias", ctypes.c_void_p),
        ("dt_softplus", ctypes.c_int32),
        ("dt_clamp", ctypes.c_int32),
        ("dt_min", ctypes.c_float),
        ("dt_max", ctypes.c_float),
        ("x_token", ctypes.c_int64),
        ("x_batch", ctypes.c_int64),
        ("dt_token", ctypes.c_int64),
        ("dt_batch", ctypes.c_int64),
        ("z_token", ctypes.c_int64),
        ("z_batch", ctypes.c_int64),
        ("B_token", ctypes.c_int64),
        ("B_batch", ctypes.c_int64),
        ("C_token", ctypes.c_int64),
        ("C_batch", ctypes.c_int64),
    ]


class Conv1dDesc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("channels", ctypes.c_int64),
        ("out0", ctypes.c_int64),
        ("out1", ctypes.c_int64),
        ("out2", ctypes.c_int64),
        ("conv_width", ctypes.c_int32),
        ("silu", ctypes.c_int32),
        ("io_dtype", ctypes.c_int32),
        ("x_token", ctypes.c_int64),
        ("x_batch", ctypes.c_int64),
    ]


class GroupNormDesc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("rows", ctypes.c_int64),
        ("channels", ctypes.c_int64),
        ("ngroups", ctypes.c_int64),
        ("io_dtype", ctypes.c_int32),
        ("center", ctypes.c_int32),
        ("gate_first", ctypes.c_int32),
        ("silu", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("x_token", ctypes.c_int64),
        ("x_batch", ctypes.c_int64),
        ("z_token", ctypes.c_int64),
        ("z_batch", ctypes.c_int64),
    ]


def lib_path() -> str:
    return os.environ.get("SSD_LIB", os.path.join(_HERE, "libssd.so"))


_lib = None
_lock = threading.Lock()


def load_library():
    """Load libssd.so once. Raises if it is missing: build it first with
    ``python -m mamba_ssd_scan_fwd_amd.build``."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"libssd.so not found at {path}; build it with `python -m mamba_ssd_scan_fwd_amd.build`"
            )
        lib = ctypes.CDLL(path)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        dp = ctypes.POINTER(SSDDesc)
        lib.ssd_status_string.argtypes = [ctypes.c_int]
        lib.ssd_status_string.restype = ctypes.c_char_p
        lib.ssd_effective_chunk_size.argtypes = [dp, ctypes.POINTER(i32)]
        lib.ssd_effective_chunk_size.restype = ctypes.c_int
        lib.ssd_workspace_bytes.argtypes = [dp, ctypes.POINTER(sz)]
        lib.ssd_workspace_bytes.restype = ctypes.c_int
        lib.ssd_forward.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ssd_forward.restype = ctypes.c_int
        lib.ssd_forward_fused.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ssd_forward_fused.restype = ctypes.c_int
        lib.ssd_forward_split.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ssd_forward_split.restype = ctypes.c_int
        lib.ssd_workspace_status.argtypes = [dp, vp, sz, vp, ctypes.POINTER(ctypes.c_uint32),
                                             ctypes.POINTER(ctypes.c_uint32)]
        lib.ssd_workspace_status.restype = ctypes.c_int
        lib.ssd_workspace_status_varlen.argtypes = [dp, ctypes.c_int64, vp, sz, vp, ctypes.POINTER(ctypes.c_uint32),
                                                    ctypes.POINTER(ctypes.c_uint32)]
        lib.ssd_workspace_status_varlen.restype = ctypes.c_int
        lib.ssd_forward_noalloc.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.ssd_forward_noalloc.restype = ctypes.c_int
        lib.ssd_chunk_cumsum.argtypes = [dp, vp, vp, vp, vp, vp]
        lib.ssd_chunk_cumsum.restype = ctypes.c_int
        lib.ssd_chunk_state.argtypes = [dp, vp, vp, vp, vp, vp, vp]
        lib.ssd_chunk_state.restype = ctypes.c_int
        lib.ssd_cumsum_chunk_state.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.ssd_cumsum_chunk_state.restype = ctypes.c_int
        lib.ssd_state_passing.argtypes = [dp, vp, vp, vp, vp, vp]
        lib.ssd_state_passing.restype = ctypes.c_int
        lib.ssd_chunk_scan.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.ssd_chunk_scan.restype = ctypes.c_int
        lib.ssd_decode_step.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.ssd_decode_step.restype = ctypes.c_int
        lib.ssd_workspace_bytes_varlen.argtypes = [dp, ctypes.c_int64, ctypes.POINTER(sz)]
        lib.ssd_workspace_bytes_varlen.restype = ctypes.c_int
        lib.ssd_forward_varlen.argtypes = [dp, vp, ctypes.c_int64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ssd_forward_varlen.restype = ctypes.c_int
        lib.ssd_conv1d_split.argtypes = [dp, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp]
        lib.ssd_conv1d_split.restype = ctypes.c_int
        i64 = ctypes.c_int64
        sp, cp, gp = ctypes.POINTER(SelectiveDesc), ctypes.POINTER(Conv1dDesc), ctypes.POINTER(GroupNormDesc)
        lib.ssd_selective_scan_workspace_bytes.argtypes = [sp, i64, ctypes.POINTER(sz)]
        lib.ssd_selective_scan_workspace_bytes.restype = ctypes.c_int
        lib.ssd_selective_scan.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ssd_selective_scan.restype = ctypes.c_int
        lib.ssd_selective_scan_varlen.argtypes = [sp, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ssd_selective_scan_varlen.restype = ctypes.c_int
        lib.ssd_selective_step.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp]
        lib.ssd_selective_step.restype = ctypes.c_int
        lib.ssd_conv1d.argtypes = [cp, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.ssd_conv1d.restype = ctypes.c_int
        lib.ssd_conv1d_step.argtypes = [cp, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp]
        lib.ssd_conv1d_step.restype = ctypes.c_int
        lib.ssd_group_norm.argtypes = [gp, vp, vp, vp, vp, vp, vp]
        lib.ssd_group_norm.restype = ctypes.c_int
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load_library().ssd_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise SSDError(status, where)


def make_desc(batch, seqlen, nheads, headdim, dstate, ngroups, io_dtype, chunk_size=0, *,
              dt_bias=None, dt_softplus=False, dt_limit=None) -> SSDDesc:
    """The C descriptor. dt preprocessing: ``dt_bias`` (fp32 [H] device
    tensor) is added to dt, ``dt_softplus`` applies log(1 + e^z), and
    ``dt_limit = (lo, hi)`` clamps the result."""
    if isinstance(io_dtype, torch.dtype):
        io = {torch.float32: SSD_DTYPE_F32, torch.bfloat16: SSD_DTYPE_BF16}.get(io_dtype)
        if io is None:
            raise TypeError(f"unsupported io dtype {io_dtype}")
    elif io_dtype in ("fp32", "f32", "float32"):
        io = SSD_DTYPE_F32
    elif io_dtype in ("bf16", "bfloat16"):
        io = SSD_DTYPE_BF16
    else:
        io = int(io_dtype)
    d = SSDDesc(int(batch), int(seqlen), int(nheads), int(headdim), int(dstate), int(ngroups), io,
                int(chunk_size))
    if dt_bias is not None:
        d.dt_bias = dt_bias.data_ptr()
    d.dt_softplus = 1 if dt_softplus else 0
    if dt_limit is not None:
        d.dt_clamp = 1
        d.dt_min, d.dt_max = float(dt_limit[0]), float(dt_limit[1])
    return d


def effective_chunk_size(desc: SSDDesc) -> int:
    q = ctypes.c_int32(0)
    _check(load_library().ssd_effective_chunk_size(ctypes.byref(desc), ctypes.byref(q)),
           "ssd_effective_chunk_size")
    return int(q.value)


def workspace_bytes(desc: SSDDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_workspace_bytes(ctypes.byref(desc), ctypes.byref(n)), "ssd_workspace_bytes")
    return int(n.value)


def workspace_bytes_varlen(desc: SSDDesc, num_seqs: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_workspace_bytes_varlen(ctypes.byref(desc), ctypes.c_int64(num_seqs), ctypes.byref(n)),
           "ssd_workspace_bytes_varlen")
    return int(n.value)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtype=None, device=None, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _desc_from(x, B, chunk_size, dt_pre=None):
    bsz, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    return make_desc(bsz, L, H, P, N, G, x.dtype, chunk_size, **_dt_kw(dt_pre, H, x.device))


def _dt_kw(dt_pre, H, dev):
    """dt_pre: None or dict(bias=tensor|None, softplus=bool, limit=(lo, hi)|None)."""
    if not dt_pre:
        return {}
    bias = dt_pre.get("bias")
    if bias is not None:
        _need(bias, "dt bias", torch.float32, dev, (H,))
    return dict(dt_bias=bias, dt_softplus=bool(dt_pre.get("softplus", False)), dt_limit=dt_pre.get("limit"))


def forward(x, dt, A, B, C, D=None, init_state=None, *, chunk_size: int = 0,
            return_final_state: bool = True, y=None, final_state=None, workspace=None,
            library_workspace: bool = False, dt_pre=None, fused: bool = False, split: bool = False,
            stream=None):
    """SSD forward pass on the GPU. Returns (y, final_state or None).

    x [b, L, H, P] and B, C [b, L, G, N] in fp32 or bf16 (all the same);
    dt [b, L, H], A [H], D [H] (optional) and init_state [b, H, P, N]
    (optional) in fp32. ``final_state`` may be passed as ``init_state`` for an
    in-place state update. With ``library_workspace=True`` the library
    allocates its workspace itself, in stream order. ``dt_pre`` asks for the
    dt preprocessing: dict(bias=[H] fp32 tensor, softplus=True, limit=(lo, hi)).
    ``fused=True`` calls ssd_forward_fused (the one-pass kernel; raises where
    the shape is not supported by it) and ``split=True`` ssd_forward_split
    (always the separate steps) instead of ssd_forward, which picks one of
    the two paths by shape.
    """
    if fused and split:
        raise ValueError("fused and split exclude each other")
    dev = x.device
    _need(x, "x", device=dev)
    io = x.dtype
    bsz, L, H, P = x.shape
    _need(B, "B", io, dev)
    G, N = B.shape[2], B.shape[3]
    _need(C, "C", io, dev, B.shape)
    _need(dt, "dt", torch.float32, dev, (bsz, L, H))
    _need(A, "A", torch.float32, dev, (H,))
    if D is not None:
        _need(D, "D", torch.float32, dev, (H,))
    if init_state is not None:
        _need(init_state, "init_state", torch.float32, dev, (bsz, H, P, N))
    desc = _desc_from(x, B, chunk_size, dt_pre)
    if y is None:
        y = torch.empty_like(x)
    else:
        _need(y, "y", io, dev, x.shape)
    if final_state is None and return_final_state:
        final_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=dev)
    elif final_state is not None:
        _need(final_state, "final_state", torch.float32, dev, (bsz, H, P, N))
    nws = workspace_bytes(desc)
    if library_workspace:
        workspace, wsize = None, 0
    elif workspace is None:
        workspace = torch.empty(nws, dtype=torch.uint8, device=dev)
        wsize = nws
    else:
        wsize = workspace.numel() * workspace.element_size()
        if wsize < nws:
            raise ValueError(f"workspace needs {nws} bytes")
    name = "ssd_forward_fused" if fused else "ssd_forward_split" if split else "ssd_forward"
    st = getattr(load_library(), name)(
        ctypes.byref(desc), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_state),
        _ptr(y), _ptr(final_state), _ptr(workspace), ctypes.c_size_t(wsize), _stream(stream, dev))
    _check(st, name)
    return y, final_state


def forward_noalloc(x, dt, A, B, C, D=None, init_state=None, *, chunk_size: int = 0,
                    return_final_state: bool = True, y=None, final_state=None, dt_pre=None, stream=None):
    """ssd_forward_noalloc: the forward pass of ``forward`` with the
    workspace taken from the library's fixed per-GPU scratch (256 MiB); the
    library allocates nothing. ``y`` and ``final_state`` are allocated here
    when not given (pass them to keep the call allocation-free end to end).
    Returns (y, final_state or None)."""
    dev = x.device
    _need(x, "x", device=dev)
    io = x.dtype
    bsz, L, H, P = x.shape
    _need(B, "B", io, dev)
    G, N = B.shape[2], B.shape[3]
    _need(C, "C", io, dev, B.shape)
    _need(dt, "dt", torch.float32, dev, (bsz, L, H))
    _need(A, "A", torch.float32, dev, (H,))
    if D is not None:
        _need(D, "D", torch.float32, dev, (H,))
    if init_state is not None:
        _need(init_state, "init_state", torch.float32, dev, (bsz, H, P, N))
    desc = _desc_from(x, B, chunk_size, dt_pre)
    if y is None:
        y = torch.empty_like(x)
    else:
        _need(y, "y", io, dev, x.shape)
    if final_state is None and return_final_state:
        final_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=dev)
    elif final_state is not None:
        _need(final_state, "final_state", torch.float32, dev, (bsz, H, P, N))
    st = load_library().ssd_forward_noalloc(
        ctypes.byref(desc), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_state),
        _ptr(y), _ptr(final_state), _stream(stream, dev))
    _check(st, "ssd_forward_noalloc")
    return y, final_state


PATH_NAMES = {0: "none", 1: "split", 2: "split-segmented", 3: "one-pass"}
STATUS_WAIT_CUT_OFF_ONE_PASS = 1
STATUS_WAIT_CUT_OFF_SEGMENTED = 2
STATUS_CHAIN_INCOMPLETE = 4
STATUS_NO_RECORD = 8


def workspace_status(desc: SSDDesc, workspace, stream=None):
    """(path name, status bits) of the last whole-forward call that used
    ``workspace`` (a uint8 device tensor) with ``desc``; synchronises the
    stream. Status 0 means the call completed as designed."""
    path = ctypes.c_uint32(0)
    bits = ctypes.c_uint32(0)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load_library().ssd_workspace_status(ctypes.byref(desc), _ptr(workspace), ctypes.c_size_t(nbytes),
                                               _stream(stream, workspace.device), ctypes.byref(path),
                                               ctypes.byref(bits)), "ssd_workspace_status")
    return PATH_NAMES.get(int(path.value), str(path.value)), int(bits.value)


def workspace_status_varlen(desc: SSDDesc, num_seqs: int, workspace, stream=None):
    """workspace_status for the workspace of a forward_varlen call with
    ``desc`` and ``num_seqs`` sequences."""
    path = ctypes.c_uint32(0)
    bits = ctypes.c_uint32(0)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load_library().ssd_workspace_status_varlen(
        ctypes.byref(desc), ctypes.c_int64(num_seqs), _ptr(workspace), ctypes.c_size_t(nbytes),
        _stream(stream, workspace.device), ctypes.byref(path), ctypes.byref(bits)), "ssd_workspace_status_varlen")
    return PATH_NAMES.get(int(path.value), str(path.value)), int(bits.value)


def _chunk_shape(desc):
    q = effective_chunk_size(desc)
    nc = -(-desc.seqlen // q)
    return q, nc


def chunk_cumsum(dt, A, *, headdim, dstate, ngroups=1, io_dtype=torch.bfloat16, chunk_size=0, dt_pre=None,
                 stream=None):
    """Step 1 alone. Returns (dA_cumsum, dt_chunked), each [b, H, nc, Q] fp32."""
    dev = dt.device
    _need(dt, "dt", torch.float32, dev)
    bsz, L, H = dt.shape
    _need(A, "A", torch.float32, dev, (H,))
    desc = make_desc(bsz, L, H, headdim, dstate, ngroups, io_dtype, chunk_size, **_dt_kw(dt_pre, H, dev))
    q, nc = _chunk_shape(desc)
    cs = torch.empty((bsz, H, nc, q), dtype=torch.float32, device=dev)
    dtc = torch.empty_like(cs)
    _check(load_library().ssd_chunk_cumsum(ctypes.byref(desc), _ptr(dt), _ptr(A), _ptr(cs), _ptr(dtc),
                                           _stream(stream, dev)), "ssd_chunk_cumsum")
    return cs, dtc


def chunk_state(x, B, dA_cumsum, dt_chunked, *, chunk_size=0, stream=None):
    """Step 2 alone. Returns states [b, H, nc, P, N] in the io dtype."""
    dev = x.device
    _need(x, "x", device=dev)
    _need(B, "B", x.dtype, dev)
    desc = _desc_from(x, B, chunk_size)
    q, nc = _chunk_shape(desc)
    bsz, L, H, P = x.shape
    _need(dA_cumsum, "dA_cumsum", torch.float32, dev, (bsz, H, nc, q))
    _need(dt_chunked, "dt_chunked", torch.float32, dev, (bsz, H, nc, q))
    states = torch.empty((bsz, H, nc, P, B.shape[3]), dtype=x.dtype, device=dev)
    _check(load_library().ssd_chunk_state(ctypes.byref(desc), _ptr(x), _ptr(B), _ptr(dA_cumsum),
                                          _ptr(dt_chunked), _ptr(states), _stream(stream, dev)),
           "ssd_chunk_state")
    return states


def cumsum_chunk_state(x, B, dt, A, *, chunk_size=0, dt_pre=None, stream=None):
    """Steps 1 and 2 in one call. Returns (dA_cumsum, dt_chunked, states)."""
    dev = x.device
    _need(x, "x", device=dev)
    _need(B, "B", x.dtype, dev)
    desc = _desc_from(x, B, chunk_size, dt_pre)
    q, nc = _chunk_shape(desc)
    bsz, L, H, P = x.shape
    _need(dt, "dt", torch.float32, dev, (bsz, L, H))
    _need(A, "A", torch.float32, dev, (H,))
    cs = torch.empty((bsz, H, nc, q), dtype=torch.float32, device=dev)
    dtc = torch.empty_like(cs)
    states = torch.empty((bsz, H, nc, P, B.shape[3]), dtype=x.dtype, device=dev)
    _check(load_library().ssd_cumsum_chunk_state(ctypes.byref(desc), _ptr(x), _ptr(B), _ptr(dt), _ptr(A),
                                                 _ptr(cs), _ptr(dtc), _ptr(states), _stream(stream, dev)),
           "ssd_cumsum_chunk_state")
    return cs, dtc, states


def state_passing(states, dA_cumsum, init_state=None, *, seqlen, ngroups=1, chunk_size=0,
                  return_final_state=True, final_state=None, stream=None):
    """Step 3 alone, in place over ``states``. Returns (states, final_state)."""
    dev = states.device
    _need(states, "states", device=dev)
    bsz, H, nc, P, N = states.shape
    desc = make_desc(bsz, seqlen, H, P, N, ngroups, states.dtype, chunk_size)
    q, nc2 = _chunk_shape(desc)
    if nc2 != nc:
        raise ValueError("states does not match seqlen / chunk size")
    _need(dA_cumsum, "dA_cumsum", torch.float32, dev, (bsz, H, nc, q))
    if init_state is not None:
        _need(init_state, "init_state", torch.float32, dev, (bsz, H, P, N))
    if final_state is None and return_final_state:
        final_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=dev)
    _check(load_library().ssd_state_passing(ctypes.byref(desc), _ptr(states), _ptr(dA_cumsum),
                                            _ptr(init_state), _ptr(final_state), _stream(stream, dev)),
           "ssd_state_passing")
    return states, final_state


def chunk_scan(x, B, C, D, dA_cumsum, dt_chunked, states, *, chunk_size=0, y=None, stream=None):
    """Steps 4+5 alone. ``states`` holds the entering states. Returns y."""
    dev = x.device
    _need(x, "x", device=dev)
    _need(B, "B", x.dtype, dev)
    _need(C, "C", x.dtype, dev, B.shape)
    desc = _desc_from(x, B, chunk_size)
    q, nc = _chunk_shape(desc)
    bsz, L, H, P = x.shape
    _need(dA_cumsum, "dA_cumsum", torch.float32, dev, (bsz, H, nc, q))
    _need(dt_chunked, "dt_chunked", torch.float32, dev, (bsz, H, nc, q))
    _need(states, "states", x.dtype, dev, (bsz, H, nc, P, B.shape[3]))
    if D is not None:
        _need(D, "D", torch.float32, dev, (H,))
    if y is None:
        y = torch.empty_like(x)
    _check(load_library().ssd_chunk_scan(ctypes.byref(desc), _ptr(x), _ptr(B), _ptr(C), _ptr(D),
                                         _ptr(dA_cumsum), _ptr(dt_chunked), _ptr(states), _ptr(y),
                                         _stream(stream, dev)), "ssd_chunk_scan")
    return y


def decode_step(x, dt, A, B, C, D, state, *, y=None, dt_pre=None, stream=None):
    """One recurrent step: x [b, H, P], dt [b, H], B/C [b, G, N], state
    [b, H, P, N] fp32 updated in place. Returns y [b, H, P] (io dtype)."""
    dev = x.device
    _need(x, "x", device=dev)
    bsz, H, P = x.shape
    _need(dt, "dt", torch.float32, dev, (bsz, H))
    _need(A, "A", torch.float32, dev, (H,))
    _need(B, "B", x.dtype, dev)
    _need(C, "C", x.dtype, dev, tuple(B.shape))
    if D is not None:
        _need(D, "D", torch.float32, dev, (H,))
    G, N = B.shape[1], B.shape[2]
    _need(state, "state", torch.float32, dev, (bsz, H, P, N))
    io = "bf16" if x.dtype == torch.bfloat16 else "fp32"
    desc = make_desc(bsz, 1, H, P, N, G, io, 0, **_dt_kw(dt_pre, H, dev))
    if y is None:
        y = torch.empty_like(x)
    _check(load_library().ssd_decode_step(ctypes.byref(desc), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                                          _ptr(D), _ptr(state), _ptr(y), _stream(stream, dev)),
           "ssd_decode_step")
    return y


def forward_varlen(x, dt, A, B, C, D=None, *, cu_seqlens, init_states=None, chunk_size: int = 0,
                   return_final_states: bool = True, y=None, final_states=None, workspace=None,
                   dt_pre=None, stream=None):
    """Packed variable-length sequences: x [1, T, H, P], dt [1, T, H],
    B/C [1, T, G, N]; sequence s is tokens [cu_seqlens[s], cu_seqlens[s+1])
    (cu_seqlens: int32 device tensor [S+1]). Without init_states the packed
    stream is cut into fixed chunks (sequences may share a chunk); with them,
    into chunks per sequence. Returns (y, final_states [S, H, P, N] or None)."""
    dev = x.device
    _need(x, "x", device=dev)
    io = x.dtype
    one, T, H, P = x.shape
    if one != 1:
        raise ValueError("packed sequences: x must be [1, T, H, P]")
    _need(B, "B", io, dev)
    G, N = B.shape[2], B.shape[3]
    _need(C, "C", io, dev, B.shape)
    _need(dt, "dt", torch.float32, dev, (1, T, H))
    _need(A, "A", torch.float32, dev, (H,))
    if D is not None:
        _need(D, "D", torch.float32, dev, (H,))
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    S = cu_seqlens.numel() - 1
    if init_states is not None:
        _need(init_states, "init_states", torch.float32, dev, (S, H, P, N))
    desc = _desc_from(x, B, chunk_size, dt_pre)
    if y is None:
        y = torch.empty_like(x)
    if final_states is None and return_final_states:
        final_states = torch.empty((S, H, P, N), dtype=torch.float32, device=dev)
    lib = load_library()
    if workspace is None:
        workspace = torch.empty(workspace_bytes_varlen(desc, S), dtype=torch.uint8, device=dev)
    _check(lib.ssd_forward_varlen(ctypes.byref(desc), _ptr(cu_seqlens), ctypes.c_int64(S), _ptr(x), _ptr(dt),
                                  _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_states), _ptr(y),
                                  _ptr(final_states), _ptr(workspace),
                                  ctypes.c_size_t(workspace.numel() * workspace.element_size()),
                                  _stream(stream, dev)), "ssd_forward_varlen")
    return y, final_states


def conv1d_split(xbc, weight, bias=None, *, nheads, headdim, ngroups, dstate, silu=True, conv_state_in=None,
                 conv_state_out=None, stream=None):
    """Short causal depthwise convolution of the packed [x | B | C] channels,
    split into x [b, L, H, P], B and C [b, L, G, N]. weight [CH, K] fp32."""
    dev = xbc.device
    _need(xbc, "xbc", device=dev)
    bsz, L, CH = xbc.shape
    if CH != nheads * headdim + 2 * ngroups * dstate:
        raise ValueError("xbc channels must be H*P + 2*G*N")
    _need(weight, "weight", torch.float32, dev)
    K = weight.shape[1]
    if bias is not None:
        _need(bias, "bias", torch.float32, dev, (CH,))
    desc = make_desc(bsz, L, nheads, headdim, dstate, ngroups, xbc.dtype, 0)
    x = torch.empty((bsz, L, nheads, headdim), dtype=xbc.dtype, device=dev)
    B = torch.empty((bsz, L, ngroups, dstate), dtype=xbc.dtype, device=dev)
    C = torch.empty_like(B)
    _check(load_library().ssd_conv1d_split(ctypes.byref(desc), ctypes.c_int32(K), _ptr(xbc), _ptr(weight),
                                           _ptr(bias), ctypes.c_int32(1 if silu else 0), _ptr(conv_state_in),
                                           _ptr(conv_state_out), _ptr(x), _ptr(B), _ptr(C), _stream(stream, dev)),
           "ssd_conv1d_split")
    return x, B, C


# ---- the layer operators around the scan -------------------------------------
#
# Inputs may be views of wider buffers (rows of contiguous channels, any
# distance between tokens and batch rows). A call for one token takes a few
# microseconds on the GPU, so what the host does for it is kept short: one
# look at each tensor, one descriptor, the raw handle of the current stream.

_IO = {torch.float32: SSD_DTYPE_F32, torch.bfloat16: SSD_DTYPE_BF16}
_F32, _I32 = torch.float32, torch.int32


def _io(t, name):
    code = _IO.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported io dtype {t.dtype}")
    return code


def _dim(t, name, n):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {t.dim()}")


def _unlike(t, name, dtype, device, shape):
    """Raises for the first thing in which ``t`` is not as it has to be."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}, got {tuple(t.shape)}")


def _strides(t, name, dtype, device, shape, lead):
    """(token, batch) stride of a strided input of ``shape`` = (batch, tokens,
    channels..) with ``lead`` 2, or (batch, channels..) with ``lead`` 1; 0
    stands for dense."""
    if t.dtype != dtype or t.shape != shape or t.device != device:
        _unlike(t, name, dtype, device, shape)
    if t.is_contiguous():
        return 0, 0
    st = t.stride()
    width = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] != 1 and st[i] != width:
            raise ValueError(f"{name}: the channels of a token must be contiguous")
        width *= shape[i]
    rows = shape[1] if lead == 2 else 1
    token = st[1] if rows > 1 else width
    batch = st[0] if shape[0] > 1 else (rows - 1) * token + width
    if token < width or batch < width:
        raise ValueError(f"{name}: tokens must not overlap (an expanded dimension needs a copy)")
    return token, batch


def _dense(t, name, device, shape, dtype=_F32):
    """Address of a dense argument, None for one that is not given."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        _unlike(t, name, dtype, device, shape)
    return t.data_ptr()


def _out(t, name, like, shape):
    """The output given, or a new dense one of ``like``'s type and device."""
    if t is None:
        return like.new_empty(shape)
    _dense(t, name, like.device, shape, like.dtype)
    return t


def _offsets(cu_seqlens, device):
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must hold num_seqs + 1 offsets, num_seqs >= 1")
    return _dense(cu_seqlens, "cu_seqlens", device, cu_seqlens.shape, _I32), cu_seqlens.numel() - 1


class _On:
    """Makes a tensor's device and the given stream the current ones. Outputs
    and workspaces allocated inside then belong to that stream, so their
    memory is not handed out again before the kernels that use it have run."""

    def __init__(self, device, stream):
        self.guards = [torch.cuda.device(device)] + ([] if stream is None else [torch.cuda.stream(stream)])

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)
        return False


_HERE_ALREADY = contextlib.nullcontext()


def _on(device, stream):
    if stream is None and device.index == torch.cuda.current_device():
        return _HERE_ALREADY
    return _On(device, stream)


def _used_on(stream, device, *tensors):
    """After a call on ``stream``: inputs that belong to the caller's stream,
    and outputs that belong to this one, are in use on both."""
    here = torch.cuda.current_stream(device)
    if stream == here:
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
            t.record_stream(here)


def _current(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def _selective_desc(x, dt, A, B, C, z, dt_pre, lead):
    dev, io = x.device, x.dtype
    shape = x.shape
    E = shape[-1]
    _dim(A, "A", 2)
    _dim(B, "B", lead + 2)
    N, G = A.shape[1], B.shape[lead]
    bc = (*shape[:lead], G, N)
    ddt = dt.dtype
    if ddt is not _F32 and ddt is not io:
        raise TypeError(f"dt must be torch.float32 or {io}, got {ddt}")
    bias, softplus, clamp, lo, hi = None, 0, 0, 0.0, 0.0
    if dt_pre:
        bias = _dense(dt_pre.get("bias"), "dt bias", dev, (E,))
        softplus = 1 if dt_pre.get("softplus") else 0
        limit = dt_pre.get("limit")
        if limit is not None:
            clamp, lo, hi = 1, float(limit[0]), float(limit[1])
    xt, xb = _strides(x, "x", io, dev, shape, lead)
    dtt, dtb = _strides(dt, "dt", ddt, dev, shape, lead)
    zt, zb = (0, 0) if z is None else _strides(z, "z", io, dev, shape, lead)
    bt, bb = _strides(B, "B", io, dev, bc, lead)
    ct, cb = _strides(C, "C", io, dev, bc, lead)
    return SelectiveDesc(shape[0], shape[1] if lead == 2 else 1, E, N, G, _io(x, "x"), _IO[ddt], bias, softplus, clamp,
                         lo, hi, xt, xb, dtt, dtb, zt, zb, bt, bb, ct, cb)


def _data(t):
    return None if t is None else t.data_ptr()


def selective_scan_workspace_bytes(desc: SelectiveDesc, num_seqs: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_selective_scan_workspace_bytes(ctypes.byref(desc), num_seqs, ctypes.byref(n)),
           "ssd_selective_scan_workspace_bytes")
    return int(n.value)


def _selective_prompts(x, dt, A, B, C, D, z, cu_seqlens, init, y, final, want_final, workspace, dt_pre, stream):
    dev = x.device
    cu, S = (None, 0) if cu_seqlens is None else _offsets(cu_seqlens, dev)
    d = _selective_desc(x, dt, A, B, C, z, dt_pre, 2)
    E, N = d.channels, d.dstate
    states = (S if S else d.batch, E, N)
    Ap, Dp = _dense(A, "A", dev, (E, N)), _dense(D, "D", dev, (E,))
    ip = _dense(init, "init_states" if S else "init_state", dev, states)
    lib = load_library()
    need = selective_scan_workspace_bytes(d, S)
    with _on(dev, stream):
        y = _out(y, "y", x, x.shape)
        if final is not None or want_final:
            final = _out(final, "final_states" if S else "final_state", A, states)
        if workspace is None:
            if need:
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        elif not workspace.is_contiguous() or workspace.device != dev or workspace.nbytes < need:
            raise ValueError(f"workspace needs {need} contiguous bytes on {dev}")
        size = 0 if workspace is None else workspace.nbytes
        if S:
            st = lib.ssd_selective_scan_varlen(ctypes.byref(d), cu, S, x.data_ptr(), dt.data_ptr(), Ap, B.data_ptr(),
                                               C.data_ptr(), Dp, _data(z), ip, y.data_ptr(), _data(final),
                                               _data(workspace), size, _current(dev))
        else:
            st = lib.ssd_selective_scan(ctypes.byref(d), x.data_ptr(), dt.data_ptr(), Ap, B.data_ptr(), C.data_ptr(),
                                        Dp, _data(z), ip, y.data_ptr(), _data(final), _data(workspace), size,
                                        _current(dev))
    _check(st, "ssd_selective_scan_varlen" if S else "ssd_selective_scan")
    if stream is not None:
        _used_on(stream, dev, x, dt, A, B, C, D, z, init, y, final, workspace, cu_seqlens, (dt_pre or {}).get("bias"))
    return y, final


def selective_scan(x, dt, A, B, C, D=None, z=None, init_state=None, *, return_final_state: bool = True, y=None,
                   final_state=None, workspace=None, dt_pre=None, stream=None):
    """Selective scan over a batch of prompts (a decay for every channel and
    state). Returns (y [b, L, E], final_state [b, E, N] fp32 or None).

    x, z [b, L, E] and B, C [b, L, G, N] in fp32 or bf16 (all the same; z
    optional: y is multiplied by silu(z)); dt [b, L, E] in fp32 or the same;
    A [E, N], D [E] (optional) and init_state [b, E, N] (optional) in fp32.
    x, dt, z, B and C may be views of wider buffers. ``dt_pre`` as for
    ``forward``, its bias [E]. ``final_state`` may be ``init_state``.
    """
    _dim(x, "x", 3)
    return _selective_prompts(x, dt, A, B, C, D, z, None, init_state, y, final_state, return_final_state,
                              workspace, dt_pre, stream)


def _packed(x, cu_seqlens):
    _dim(x, "x", 3)
    if x.shape[0] != 1:
        raise ValueError("packed sequences: x must be [1, T, channels]")
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")


def selective_scan_varlen(x, dt, A, B, C, D=None, z=None, *, cu_seqlens, init_states=None,
                          return_final_states: bool = True, y=None, final_states=None, workspace=None, dt_pre=None,
                          stream=None):
    """``selective_scan`` over packed sequences: x, dt, z [1, T, E], B, C
    [1, T, G, N], sequence s being tokens [cu_seqlens[s], cu_seqlens[s+1])
    (int32 device tensor [S+1]). Returns (y, final_states [S, E, N] or None).
    Where cu_seqlens ends before T, y of the tokens behind it is not written."""
    _packed(x, cu_seqlens)
    return _selective_prompts(x, dt, A, B, C, D, z, cu_seqlens, init_states, y, final_states, return_final_states,
                              workspace, dt_pre, stream)


def selective_step(x, dt, A, B, C, D, z, state, *, state_slots=None, y=None, dt_pre=None, stream=None):
    """One token through the selective scan: x, dt, z [b, E], B, C [b, G, N],
    ``state`` [slots, E, N] fp32 updated in place. Row b's state is slot
    ``state_slots[b]`` (int32 [b]; slot b without it); a row with a slot
    outside the pool, or one that an earlier row has, is left alone. Returns
    y [b, E] (pass ``y`` to keep what such rows held)."""
    _dim(x, "x", 2)
    dev, shape = x.device, x.shape
    d = _selective_desc(x, dt, A, B, C, z, dt_pre, 1)
    _dim(state, "state", 3)
    E, N = A.shape
    n = state.shape[0]
    sp, Ap, Dp = _dense(state, "state", dev, (n, E, N)), _dense(A, "A", dev, (shape[1], N)), _dense(D, "D", dev, (E,))
    slots = _dense(state_slots, "state_slots", dev, shape[:1], _I32)
    with _on(dev, stream):
        y = _out(y, "y", x, shape)
        st = load_library().ssd_selective_step(ctypes.byref(d), x.data_ptr(), dt.data_ptr(), Ap, B.data_ptr(),
                                               C.data_ptr(), Dp, _data(z), sp, slots, n, y.data_ptr(), _current(dev))
    _check(st, "ssd_selective_step")
    if stream is not None:
        _used_on(stream, dev, x, dt, A, B, C, D, z, state, state_slots, y, (dt_pre or {}).get("bias"))
    return y


def _conv_desc(x, weight, widths, silu, lead):
    shape = x.shape
    _dim(weight, "weight", 2)
    CH, K = weight.shape
    if CH != shape[-1]:
        raise ValueError(f"weight must have shape ({shape[-1]}, K), got {tuple(weight.shape)}")
    return Conv1dDesc(shape[0], shape[1] if lead == 2 else 1, CH, *widths, K, 1 if silu else 0, _io(x, "x"),
                      *_strides(x, "x", x.dtype, x.device, shape, lead))


def _split_widths(CH, nheads, headdim, ngroups, dstate):
    if CH != nheads * headdim + 2 * ngroups * dstate:
        raise ValueError("xbc channels must be H*P + 2*G*N")
    return nheads * headdim, ngroups * dstate, ngroups * dstate


def _conv_prompts(x, weight, bias, widths, shapes, outs, cu_seqlens, state_in, state_out, silu, stream):
    dev = x.device
    cu, S = (None, 0) if cu_seqlens is None else _offsets(cu_seqlens, dev)
    d = _conv_desc(x, weight, widths, silu, 2)
    CH, K = weight.shape
    states = (S if S else x.shape[0], CH, K - 1)
    wp, bp = _dense(weight, "weight", dev, (CH, K)), _dense(bias, "bias", dev, (CH,))
    name = "conv_states" if S else "conv_state"
    ip, op = _dense(state_in, name + "_in", dev, states), _dense(state_out, name + "_out", dev, states)
    with _on(dev, stream):
        outs = [_out(o, "y", x, s) for o, s in zip(outs, shapes)]
        ptrs = [o.data_ptr() for o in outs] + [None] * (3 - len(outs))
        st = load_library().ssd_conv1d(ctypes.byref(d), cu, S, x.data_ptr(), wp, bp, ip, op, *ptrs, _current(dev))
    _check(st, "ssd_conv1d")
    if stream is not None:
        _used_on(stream, dev, x, weight, bias, state_in, state_out, cu_seqlens, *outs)
    return outs


def conv1d(x, weight, bias=None, *, silu=True, conv_state_in=None, conv_state_out=None, y=None, stream=None):
    """Short causal depthwise convolution of x [b, L, CH] (fp32 or bf16, a
    view of a wider buffer or dense), weight [CH, K] fp32, K in 1..4, with an
    optional SiLU. ``conv_state_in`` and ``conv_state_out`` [b, CH, K-1] fp32
    hold the inputs before the first token and the last ones. Returns y."""
    _dim(x, "x", 3)
    return _conv_prompts(x, weight, bias, (x.shape[2], 0, 0), [x.shape], [y], None, conv_state_in,
                         conv_state_out, silu, stream)[0]


def conv1d_varlen(x, weight, bias=None, *, cu_seqlens, silu=True, conv_states_in=None, conv_states_out=None, y=None,
                  stream=None):
    """``conv1d`` over packed sequences x [1, T, CH]: sequence s is tokens
    [cu_seqlens[s], cu_seqlens[s+1]) (int32 device tensor [S+1]), its states
    row s of ``conv_states_in`` and ``conv_states_out`` [S, CH, K-1]."""
    _packed(x, cu_seqlens)
    return _conv_prompts(x, weight, bias, (x.shape[2], 0, 0), [x.shape], [y], cu_seqlens, conv_states_in,
                         conv_states_out, silu, stream)[0]


def conv1d_split_varlen(xbc, weight, bias=None, *, cu_seqlens, nheads, headdim, ngroups, dstate, silu=True,
                        conv_states_in=None, conv_states_out=None, stream=None):
    """``conv1d_split`` over packed sequences: xbc [1, T, H*P + 2*G*N] into
    the x [1, T, H, P], B and C [1, T, G, N] that ``forward_varlen`` reads."""
    _packed(xbc, cu_seqlens)
    T = xbc.shape[1]
    widths = _split_widths(xbc.shape[2], nheads, headdim, ngroups, dstate)
    shapes = [(1, T, nheads, headdim), (1, T, ngroups, dstate), (1, T, ngroups, dstate)]
    return tuple(_conv_prompts(xbc, weight, bias, widths, shapes, [None] * 3, cu_seqlens, conv_states_in,
                               conv_states_out, silu, stream))


def _conv_token(x, weight, bias, widths, shapes, outs, conv_state, state_slots, silu, stream):
    dev = x.device
    d = _conv_desc(x, weight, widths, silu, 1)
    CH, K = weight.shape
    _dim(conv_state, "conv_state", 3)
    n = conv_state.shape[0]
    wp, bp = _dense(weight, "weight", dev, (CH, K)), _dense(bias, "bias", dev, (CH,))
    cp = _dense(conv_state, "conv_state", dev, (n, CH, K - 1))
    slots = _dense(state_slots, "state_slots", dev, x.shape[:1], _I32)
    with _on(dev, stream):
        outs = [_out(o, "y", x, s) for o, s in zip(outs, shapes)]
        ptrs = [o.data_ptr() for o in outs] + [None] * (3 - len(outs))
        st = load_library().ssd_conv1d_step(ctypes.byref(d), x.data_ptr(), wp, bp, cp, slots, n, *ptrs, _current(dev))
    _check(st, "ssd_conv1d_step")
    if stream is not None:
        _used_on(stream, dev, x, weight, bias, conv_state, state_slots, *outs)
    return outs


def conv1d_step(x, weight, bias, conv_state, *, silu=True, state_slots=None, y=None, stream=None):
    """``conv1d`` at one token: x [b, CH], ``conv_state`` [slots, CH, K-1]
    fp32 moved on in place. ``state_slots`` as for ``selective_step``.
    Returns y [b, CH]."""
    _dim(x, "x", 2)
    return _conv_token(x, weight, bias, (x.shape[1], 0, 0), [x.shape], [y], conv_state, state_slots, silu, stream)[0]


def conv1d_split_step(xbc, weight, bias, conv_state, *, nheads, headdim, ngroups, dstate, silu=True,
                      state_slots=None, stream=None):
    """``conv1d_split`` at one token: xbc [b, H*P + 2*G*N] into the x
    [b, H, P], B and C [b, G, N] that ``decode_step`` reads; ``conv_state`` and
    ``state_slots`` as for ``conv1d_step``."""
    _dim(xbc, "xbc", 2)
    b = xbc.shape[0]
    widths = _split_widths(xbc.shape[1], nheads, headdim, ngroups, dstate)
    shapes = [(b, nheads, headdim), (b, ngroups, dstate), (b, ngroups, dstate)]
    return tuple(_conv_token(xbc, weight, bias, widths, shapes, [None] * 3, conv_state, state_slots, silu, stream))


def group_norm(x, weight=None, bias=None, z=None, *, ngroups=1, eps=1e-5, center=True, gate_first=False, silu=False,
               out=None, stream=None):
    """Group norm over the channels of each token of x [.., C] (up to two
    leading dimensions, views allowed), weight and bias [C] fp32. ``center``
    False gives the root-mean-square form. ``z`` (like x) gates with silu(z),
    before the norm with ``gate_first``, else behind it; ``silu`` applies the
    SiLU to the result instead."""
    rank = x.dim()
    if not 1 <= rank <= 3:
        raise ValueError("x must have 1 to 3 dimensions")
    _dim(x, "x", rank)
    dev, io, shape = x.device, x.dtype, x.shape
    if z is not None and z.shape != shape:
        raise ValueError(f"z must have shape {tuple(shape)}, got {tuple(z.shape)}")
    x3, z3 = x, z
    if rank != 3:
        x3 = x.view((1,) * (3 - rank) + tuple(shape))
        z3 = None if z is None else z.view(x3.shape)
    b, rows, C = x3.shape
    d = GroupNormDesc(b, rows, C, int(ngroups), _io(x, "x"), 1 if center else 0, 1 if gate_first else 0,
                      1 if silu else 0, float(eps), *_strides(x3, "x", io, dev, x3.shape, 2),
                      *((0, 0) if z is None else _strides(z3, "z", io, dev, x3.shape, 2)))
    wp, bp = _dense(weight, "weight", dev, (C,)), _dense(bias, "bias", dev, (C,))
    with _on(dev, stream):
        out = _out(out, "out", x, shape)
        st = load_library().ssd_group_norm(ctypes.byref(d), x.data_ptr(), wp, bp, _data(z), out.data_ptr(),
                                           _current(dev))
    _check(st, "ssd_group_norm")
    if stream is not None:
        _used_on(stream, dev, x, weight, bias, z, out)
    return out
