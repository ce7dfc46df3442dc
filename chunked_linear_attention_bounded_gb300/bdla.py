"""Thin ctypes binding of libbdla.so (see include/bdla.h).

Argument marshalling only: shape/dtype checks, output and workspace
allocation through PyTorch (device memory and streams are all PyTorch is used
for), and one C-ABI call per op.  Every arithmetic step runs in the library's
CUDA kernels.  There is no fallback: if the library is missing or a call
fails, an exception is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbdla.so")

BOUNDED = 0    # BDLA_DECAY_BOUNDED_SIGMOID: log g = b * sigmoid(a)
SOFTPLUS = 1   # BDLA_DECAY_NEG_SOFTPLUS:    log g = -softplus(a)   (ablation)
CHUNK = 16
OP_FWD, OP_BWD, OP_DECAY = 0, 1, 2

# bdla_status values (include/bdla.h)
OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_ALIGN, ERR_RANGE, ERR_UNSUPPORTED = 0, 1, 2, 3, 4, 5, 6
ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_DEVICE, ERR_TOO_LARGE = 7, 8, 9, 10, 11
STATUS_NAMES = {OK: "BDLA_OK", ERR_NULL: "BDLA_ERR_NULL", ERR_SHAPE: "BDLA_ERR_SHAPE",
                ERR_DTYPE: "BDLA_ERR_DTYPE", ERR_ALIGN: "BDLA_ERR_ALIGN", ERR_RANGE: "BDLA_ERR_RANGE",
                ERR_UNSUPPORTED: "BDLA_ERR_UNSUPPORTED", ERR_WORKSPACE: "BDLA_ERR_WORKSPACE",
                ERR_CUDA: "BDLA_ERR_CUDA", ERR_TIMEOUT: "BDLA_ERR_TIMEOUT", ERR_DEVICE: "BDLA_ERR_DEVICE",
                ERR_TOO_LARGE: "BDLA_ERR_TOO_LARGE"}

# Every symbol include/*.h declares.
EXPORTS = ("bdla_workspace_bytes", "bdla_decay", "bdla_fwd", "bdla_fwd_varlen", "bdla_bwd",
           "bdla_bwd_varlen", "bdla_read_device_status", "bdla_status_string", "bdla_version",
           "bdla_set_kernel_events", "bdla_fwd_noalloc", "bdla_noalloc_read_status",
           "bdla_set_seq_split", "bdla_decode", "bdla_set_wait_limit_ns", "bdla_set_test_stall",
           "bdla_workspace_bytes_vec", "bdla_fwd_vec", "bdla_bwd_vec", "bdla_workspace_bytes_delta",
           "bdla_fwd_delta", "bdla_bwd_delta", "bdla_tile_states_bytes",
           "bdla_qk_norm", "bdla_qk_norm_bwd", "bdla_attn_fwd", "bdla_attn_bwd", "bdla_cache_append",
           "bdla_attn_cached", "bdla_workspace_bytes_attn")
ATTN_FWD, ATTN_BWD, ATTN_NORM_BWD, ATTN_APPEND, ATTN_CACHED = 0, 1, 2, 3, 4
KERNEL_DECAY, KERNEL_FWD, KERNEL_BWD, KERNEL_STATES, KERNEL_SEG = 0, 1, 2, 3, 4
KERNEL_ATTN_FWD, KERNEL_ATTN_BWD, KERNEL_ATTN_CACHED = 5, 6, 7
STALL_NONE, STALL_PRODUCER, STALL_MMA, STALL_EPILOGUE = 0, 1, 2, 3


class BdlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int)]


class AttnDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("Hk", ctypes.c_int),
                ("d", ctypes.c_int)]


class QkNormArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_token", ctypes.c_int64),
                ("q_head", ctypes.c_int64), ("k_token", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("wq", ctypes.c_void_p), ("wk", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("base", ctypes.c_double), ("eps", ctypes.c_float),
                ("rotary", ctypes.c_int), ("interleaved", ctypes.c_int), ("n_docs", ctypes.c_int)]


class CacheArgs(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("n_pages", ctypes.c_int), ("page", ctypes.c_int),
                ("max_pages", ctypes.c_int)]


_lib = None


def lib():
    """Loads libbdla.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libbdla.so is not built ({LIB_PATH}); run "
                               "chunked_linear_attention_bounded_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32, f32, ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_float, ctypes.c_int
        L.bdla_workspace_bytes.argtypes = [ci, Dims, ci, ci, ci]
        L.bdla_workspace_bytes.restype = sz
        L.bdla_decay.argtypes = [vp, f32, ci, vp, ci, vp, Dims, ci, vp, sz, vp]
        L.bdla_fwd.argtypes = [vp, vp, vp, vp, f32, ci, vp, vp, ci, vp, vp, ci, ci, Dims, ci, vp, sz,
                               vp]
        L.bdla_fwd_varlen.argtypes = [vp, vp, vp, vp, f32, ci, vp, ci, vp, vp, ci, vp, vp, ci, ci, Dims,
                                      ci, vp, sz, vp]
        L.bdla_bwd.argtypes = [vp, vp, vp, vp, f32, ci, vp, vp, vp, vp, ci, ci, vp, vp, vp, vp, vp, Dims,
                               ci, vp, sz, vp]
        L.bdla_bwd_varlen.argtypes = [vp, vp, vp, vp, f32, ci, vp, ci, vp, vp, vp, vp, ci, ci, vp, vp, vp,
                                      vp, vp, Dims, ci, vp, sz, vp]
        for name in ("bdla_decay", "bdla_fwd", "bdla_fwd_varlen", "bdla_bwd", "bdla_bwd_varlen",
                     "bdla_read_device_status", "bdla_noalloc_read_status"):
            getattr(L, name).restype = ci
        L.bdla_read_device_status.argtypes = [vp, vp]
        L.bdla_noalloc_read_status.argtypes = [vp]
        L.bdla_status_string.argtypes = [ci]
        L.bdla_status_string.restype = ctypes.c_char_p
        L.bdla_version.restype = ci
        L.bdla_set_kernel_events.argtypes = [ci, vp, vp]
        L.bdla_set_kernel_events.restype = ci
        L.bdla_fwd_noalloc.argtypes = [vp, vp, vp, vp, f32, ci, vp, vp, ci, vp, Dims, ci, vp]
        L.bdla_fwd_noalloc.restype = ci
        L.bdla_set_seq_split.argtypes = [ci]
        L.bdla_set_seq_split.restype = ci
        L.bdla_decode.argtypes = [vp, vp, vp, vp, f32, vp, vp, ci, Dims, ci, vp]
        L.bdla_decode.restype = ci
        L.bdla_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        L.bdla_set_wait_limit_ns.restype = ci
        L.bdla_set_test_stall.argtypes = [ci, ci]
        L.bdla_set_test_stall.restype = ci
        L.bdla_workspace_bytes_vec.argtypes = [ci, Dims, ci]
        L.bdla_workspace_bytes_vec.restype = sz
        L.bdla_fwd_vec.argtypes = [vp, vp, vp, vp, f32, ci, vp, ci, vp, vp, ci, vp, vp, Dims, ci, vp, sz, vp]
        L.bdla_fwd_vec.restype = ci
        L.bdla_bwd_vec.argtypes = [vp, vp, vp, vp, f32, ci, vp, ci, vp, vp, vp, vp, vp, vp, vp, vp, vp, Dims,
                                   ci, vp, sz, vp]
        L.bdla_bwd_vec.restype = ci
        L.bdla_workspace_bytes_delta.argtypes = [ci, Dims, ci]
        L.bdla_workspace_bytes_delta.restype = sz
        L.bdla_fwd_delta.argtypes = [vp, vp, vp, vp, vp, f32, ci, vp, ci, vp, vp, ci, vp, vp, Dims, ci, vp, sz,
                                     vp]
        L.bdla_fwd_delta.restype = ci
        L.bdla_bwd_delta.argtypes = [vp, vp, vp, vp, vp, f32, ci, vp, ci, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                     Dims, ci, vp, sz, vp]
        L.bdla_tile_states_bytes.argtypes = [Dims, ci]
        L.bdla_tile_states_bytes.restype = sz
        L.bdla_bwd_delta.restype = ci
        L.bdla_qk_norm.argtypes = [QkNormArgs, vp, vp, AttnDims, vp]
        L.bdla_qk_norm_bwd.argtypes = [QkNormArgs, vp, vp, ci, vp, vp, vp, vp, AttnDims, vp, sz, vp]
        L.bdla_attn_fwd.argtypes = [vp, vp, vp, vp, ci, f32, vp, vp, AttnDims, vp, sz, vp]
        L.bdla_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, f32, vp, vp, vp, AttnDims, vp, sz, vp]
        L.bdla_cache_append.argtypes = [vp, vp, CacheArgs, vp, vp, AttnDims, vp, sz, vp]
        L.bdla_attn_cached.argtypes = [vp, CacheArgs, vp, f32, vp, vp, AttnDims, vp, sz, vp]
        for name in ("bdla_qk_norm", "bdla_qk_norm_bwd", "bdla_attn_fwd", "bdla_attn_bwd", "bdla_cache_append",
                     "bdla_attn_cached"):
            getattr(L, name).restype = ci
        L.bdla_workspace_bytes_attn.argtypes = [ci, AttnDims, ci, ctypes.c_int64]
        L.bdla_workspace_bytes_attn.restype = sz
        del i32
        _lib = L
    return _lib


def set_kernel_events(kernel: int, start=None, stop=None):
    """Measurement hook: record torch.cuda.Event `start`/`stop` around every
    later launch of `kernel` (KERNEL_*); pass None to clear."""
    h = lambda e: None if e is None else ctypes.c_void_p(e.cuda_event)
    st = lib().bdla_set_kernel_events(int(kernel), h(start), h(stop))
    if st:
        raise BdlaError(st, "bdla_set_kernel_events")


def set_wait_limit_ns(ns: int):
    """Limit of the kernels' pipeline waits for later launches (0 = the
    default 2 s); a test hook (include/bdla_tuning.h)."""
    lib().bdla_set_wait_limit_ns(int(ns))


def set_test_stall(kernel: int, role: int):
    """Test hook: `role` (STALL_*) of `kernel` (KERNEL_*) waits on a barrier
    nothing arrives at, so the bounded wait runs out (STALL_NONE clears)."""
    st = lib().bdla_set_test_stall(int(kernel), int(role))
    if st:
        raise BdlaError(st, "bdla_set_test_stall")


_seq_split = 0


def set_seq_split(blocks: int):
    """Sequence segments of 128-token blocks: 0 automatic, < 0 never, > 0
    always this many blocks per segment (process-wide)."""
    global _seq_split
    lib().bdla_set_seq_split(int(blocks))
    _seq_split = int(blocks)


def segments_engaged(q_shape, dv: int, n_docs: int = 0) -> bool:
    """Whether calls of this shape cut documents into segments under the
    current setting (the segment buffers then appear in the workspace)."""
    cur = _seq_split
    with_cut = workspace_bytes(OP_FWD, q_shape, dv, n_docs)
    set_seq_split(-1)
    try:
        return with_cut > workspace_bytes(OP_FWD, q_shape, dv, n_docs)
    finally:
        set_seq_split(cur)


def status_string(s: int) -> str:
    try:
        return lib().bdla_status_string(int(s)).decode()
    except Exception:  # pragma: no cover
        return "?"


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# the two questions that every call asks, without torch.cuda's checks of its own set-up (a tensor is there already)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _here(t, name: str):
    """The library launches on the current device, whose streams and sizes it takes."""
    if t.get_device() != _current_device():
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{_current_device()}: "
                         f"make the call within torch.cuda.device({t.device.index})")


def _check(t: torch.Tensor, name: str, dtype, ndim: int, here: bool = False):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if here:
        _here(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dims(q: torch.Tensor, v: torch.Tensor) -> Dims:
    B, T, H, dk = q.shape
    return Dims(B, T, H, dk, v.shape[-1])


def n_slots(tokens: int, n_docs: int, stride: int) -> int:
    """Checkpoint slots for `tokens` packed tokens in `n_docs` documents."""
    return (tokens + stride - 1) // stride + n_docs


def _scope(stream):
    """Allocations made in it belong to `stream` (None: the current stream)."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class Workspace:
    """Caller-owned device scratch for the library (status word first).  A call
    that needs more grows it on the call's stream, and what the device has
    recorded stays to be read.  A buffer that a captured graph uses lives as
    long as the workspace, since replays write to it however the workspace has
    grown.  Growing inside a capture puts the new buffer, and the clearing of
    its record, into the graph: size it before."""

    def __init__(self, nbytes: int, device):
        self.nbytes = max(int(nbytes), 256)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device)
        self.device = self.buf.device
        self.in_graph = False   # a graph may hold the present buffer
        self.held = []          # outgrown buffers that one may hold; their records are read where they are

    def ensure(self, nbytes: int, stream=None):
        if nbytes > self.nbytes:
            with _scope(stream):
                old, buf = self.buf, torch.zeros(int(nbytes), dtype=torch.uint8, device=self.device)
                if self.in_graph or _capturing():
                    self.held.append(old)   # (and a captured copy would bring the old record back at every replay)
                else:
                    buf[:256] = old[:256]
                    if old.is_cuda:
                        old.record_stream(torch.cuda.current_stream(self.device))
            self.buf, self.nbytes = buf, int(nbytes)
        return self

    def note_call(self, device, stream=None):
        """To be told of every call that takes the buffer, before it is launched."""
        if self.device != device:
            raise ValueError(f"ws is on {self.device}, expected {device}")
        if not self.in_graph:
            self.in_graph = _capturing()
            if stream is not None and not self.in_graph:
                with torch.cuda.stream(stream):
                    self.in_graph = _capturing()

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())

    def read_device_status(self, stream=None) -> int:
        """An error that the device has recorded since the last read (the first of each buffer is kept), OK if none;
        waits for `stream`."""
        handle = _stream_handle(stream)
        read = [int(lib().bdla_read_device_status(ctypes.c_void_p(b.data_ptr()), handle)) for b in (*self.held, self.buf)]
        return next((st for st in read if st != OK), OK)


def _workspace(need: int, device, ws: Optional[Workspace], stream) -> Workspace:
    """The caller's workspace, grown to `need` bytes, or a new one, made on the call's stream."""
    if ws is not None:
        ws.note_call(device, stream)
        return ws.ensure(need, stream)
    with _scope(stream):
        return Workspace(need, device)


def workspace_bytes(op: int, q_shape, dv: int, n_docs: int = 0, mode: int = BOUNDED,
                    ckpt_stride: int = 0) -> int:
    B, T, H, dk = q_shape
    return int(lib().bdla_workspace_bytes(op, Dims(B, T, H, dk, dv), n_docs, mode, ckpt_stride))


def _ws_for(op, q, v, n_docs, mode, ckpt_stride, ws: Optional[Workspace], stream) -> Workspace:
    need = workspace_bytes(op, tuple(q.shape), v.shape[-1], n_docs, mode, ckpt_stride)
    if need == 0:
        raise BdlaError(ERR_SHAPE, "bdla_workspace_bytes")
    return _workspace(need, q.device, ws, stream)


def decay(a: torch.Tensor, b: float = -5.0, cu_seqlens: Optional[torch.Tensor] = None,
          mode: int = BOUNDED, ws: Optional[Workspace] = None, stream=None) -> torch.Tensor:
    """Tile-local inclusive cumsum Gamma of the log-decay, fp32 [H, B*T]
    (head-major)."""
    _check(a, "a", torch.float32, 3, here=True)
    B, T, H = a.shape
    gamma = torch.empty((H, B * T), dtype=torch.float32, device=a.device)
    n_docs = 0
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, 1)
        n_docs = cu_seqlens.numel() - 1
    ws = _workspace(256, a.device, ws, stream)
    st = lib().bdla_decay(_p(a), b, CHUNK, _p(cu_seqlens), n_docs, _p(gamma),
                          Dims(B, T, H, 64, 64), mode, ws.ptr, ws.nbytes, _stream_handle(stream))
    if st:
        raise BdlaError(st, "bdla_decay")
    return gamma


def decode(q, k, v, a, state, b: float = -5.0, mode: int = BOUNDED, o_dtype=torch.bfloat16,
           out=None, stream=None) -> torch.Tensor:
    """One recurrent step per sequence: q, k [B, H, dk], v [B, H, dv] bf16,
    a [B, H] fp32; `state` fp32 [B, H, dk, dv] is updated in place
    (S <- e^{lambda} S + k v^T).  Returns o = S^T q [B, H, dv]."""
    _check(q, "q", torch.bfloat16, 3, here=True)
    _check(k, "k", torch.bfloat16, 3)
    _check(v, "v", torch.bfloat16, 3)
    _check(a, "a", torch.float32, 2)
    _check(state, "state", torch.float32, 4)
    B, H, dk = q.shape
    dv = v.shape[-1]
    if tuple(state.shape) != (B, H, dk, dv) or tuple(a.shape) != (B, H):
        raise BdlaError(ERR_SHAPE, "decode shapes")
    o = out if out is not None else torch.empty((B, H, dv), dtype=o_dtype, device=q.device)
    st = lib().bdla_decode(_p(q), _p(k), _p(v), _p(a), b, _p(state), _p(o), _dtype_code(o.dtype),
                           Dims(B, 1, H, dk, dv), mode, _stream_handle(stream))
    if st:
        raise BdlaError(st, "bdla_decode")
    return o


def _dtype_code(dt) -> int:
    if dt == torch.bfloat16:
        return 0
    if dt == torch.float32:
        return 1
    raise ValueError(f"unsupported dtype {dt}")


def fwd(q, k, v, a, b: float = -5.0, h0=None, cu_seqlens=None, mode: int = BOUNDED,
        o_dtype=torch.bfloat16, want_hT: bool = True, ckpt_stride: int = 0,
        ckpt_dtype=torch.float32, ws: Optional[Workspace] = None, out=None, hT_out=None,
        ckpt_out=None, stream=None):
    """Forward pass.  Returns (o, hT, ckpt); hT / ckpt are None when not asked
    for.  ckpt_stride > 0 also writes the state every ckpt_stride tokens
    ([H, n_slots, dk, dv], ckpt_dtype), which bwd() can reuse."""
    _check(q, "q", torch.bfloat16, 4, here=True)
    _check(k, "k", torch.bfloat16, 4)
    _check(v, "v", torch.bfloat16, 4)
    _check(a, "a", torch.float32, 3)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or a.shape != q.shape[:3]:
        raise ValueError("q, k, v, a shapes disagree")
    n_docs = 0
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, 1)
        n_docs = cu_seqlens.numel() - 1
    n_seq = n_docs if n_docs else B
    if h0 is not None:
        _check(h0, "h0", torch.float32, 4)
        if tuple(h0.shape) != (n_seq, H, dk, dv):
            raise ValueError("h0 must be [n_docs, H, dk, dv]")
    dev = q.device
    o = out if out is not None else torch.empty((B, T, H, dv), dtype=o_dtype, device=dev)
    hT = hT_out
    if hT is None and want_hT:
        hT = torch.empty((n_seq, H, dk, dv), dtype=torch.float32, device=dev)
    ckpt = ckpt_out
    if ckpt is None and ckpt_stride:
        ckpt = torch.empty((H, n_slots(B * T, n_seq, ckpt_stride), dk, dv), dtype=ckpt_dtype,
                           device=dev)
    ws = _ws_for(OP_FWD, q, v, n_docs, mode, 0, ws, stream)
    odt = 1 if o.dtype == torch.float32 else 0
    ckdt = _dtype_code(ckpt.dtype) if ckpt is not None else 1
    args_tail = (_p(h0), _p(o), odt, _p(hT), _p(ckpt), int(ckpt_stride), ckdt, _dims(q, v), mode,
                 ws.ptr, ws.nbytes, _stream_handle(stream))
    L = lib()
    if n_docs:
        st = L.bdla_fwd_varlen(_p(q), _p(k), _p(v), _p(a), b, CHUNK, _p(cu_seqlens), n_docs,
                               *args_tail)
    else:
        st = L.bdla_fwd(_p(q), _p(k), _p(v), _p(a), b, CHUNK, *args_tail)
    if st:
        raise BdlaError(st, "bdla_fwd")
    return o, hT, ckpt


def bwd(q, k, v, a, dO, b: float = -5.0, h0=None, dhT=None, cu_seqlens=None, ckpt=None,
        ckpt_stride: int = 0, mode: int = BOUNDED, want_dh0: bool = False,
        ws: Optional[Workspace] = None, outs=None, stream=None):
    """Backward pass.  Returns (dq, dk, dv, da, dh0); dh0 is None unless asked for."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dO, "dO")):
        _check(t, n, torch.bfloat16, 4, here=t is q)
    _check(a, "a", torch.float32, 3)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if dO.shape != v.shape:
        raise ValueError("dO must match v")
    n_docs = 0
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, 1)
        n_docs = cu_seqlens.numel() - 1
    n_seq = n_docs if n_docs else B
    for t, n in ((h0, "h0"), (dhT, "dhT")):
        if t is not None:
            _check(t, n, torch.float32, 4)
            if tuple(t.shape) != (n_seq, H, dk, dv):
                raise ValueError(f"{n} must be [n_docs, H, dk, dv]")
    ckdt = 1
    if ckpt is not None:
        _check(ckpt, "ckpt", ckpt.dtype, 4)
        ckdt = _dtype_code(ckpt.dtype)
        if not ckpt_stride:
            raise ValueError("ckpt needs its ckpt_stride")
    dev = q.device
    if outs is None:
        dq = torch.empty((B, T, H, dk), dtype=torch.float32, device=dev)
        dkk = torch.empty((B, T, H, dk), dtype=torch.float32, device=dev)
        dvv = torch.empty((B, T, H, dv), dtype=torch.float32, device=dev)
        da = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    else:
        dq, dkk, dvv, da = outs
    dh0 = torch.empty((n_seq, H, dk, dv), dtype=torch.float32, device=dev) if want_dh0 else None
    stride = int(ckpt_stride) if ckpt is not None else 0
    ws_stride = stride if (ckdt == 1 or dv <= 128) else 0
    ws = _ws_for(OP_BWD, q, v, n_docs, mode, ws_stride, ws, stream)
    args_tail = (_p(h0), _p(dO), _p(dhT), _p(ckpt), stride, ckdt, _p(dq), _p(dkk), _p(dvv), _p(da),
                 _p(dh0), _dims(q, v), mode, ws.ptr, ws.nbytes, _stream_handle(stream))
    L = lib()
    if n_docs:
        st = L.bdla_bwd_varlen(_p(q), _p(k), _p(v), _p(a), b, CHUNK, _p(cu_seqlens), n_docs,
                               *args_tail)
    else:
        st = L.bdla_bwd(_p(q), _p(k), _p(v), _p(a), b, CHUNK, *args_tail)
    if st:
        raise BdlaError(st, "bdla_bwd")
    return dq, dkk, dvv, da, dh0


# ---------------------------------------------------------------- per-channel decay
def _vec_checks(q, k, v, a, cu_seqlens, h0):
    _check(q, "q", torch.bfloat16, 4, here=True)
    _check(k, "k", torch.bfloat16, 4)
    _check(v, "v", torch.bfloat16, 4)
    _check(a, "a", torch.float32, 4)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or a.shape != q.shape:
        raise ValueError("q, k, v, a shapes disagree (a is [B, T, H, dk] for per-channel decay)")
    n_docs = 0
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, 1)
        n_docs = cu_seqlens.numel() - 1
    n_seq = n_docs if n_docs else B
    if h0 is not None:
        _check(h0, "h0", torch.float32, 4)
        if tuple(h0.shape) != (n_seq, H, dk, dv):
            raise ValueError("h0 must be [n_docs, H, dk, dv]")
    return B, T, H, dk, dv, n_docs, n_seq


def _ws_vec(op, q, v, n_docs, ws, stream):
    B, T, H, dk = q.shape
    need = int(lib().bdla_workspace_bytes_vec(op, Dims(B, T, H, dk, v.shape[-1]), n_docs))
    if need == 0:
        raise BdlaError(ERR_UNSUPPORTED, "bdla_workspace_bytes_vec")
    return _workspace(need, q.device, ws, stream)


def tile_states(q, v, cu_seqlens=None):
    """An uninitialised bf16 buffer for the state before every 16-token tile
    ([H, slots, dk, dv]), the `states` hand-off of the per-channel and
    delta-rule paths."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    n_docs = cu_seqlens.numel() - 1 if cu_seqlens is not None else 0
    nbytes = int(lib().bdla_tile_states_bytes(Dims(B, T, H, dk, dv), n_docs))
    if nbytes == 0:
        raise BdlaError(ERR_UNSUPPORTED, "bdla_tile_states_bytes")
    return torch.empty((H, nbytes // (2 * H * dk * dv), dk, dv), dtype=torch.bfloat16, device=q.device)


def fwd_vec(q, k, v, a, b: float = -5.0, h0=None, cu_seqlens=None, mode: int = BOUNDED,
            o_dtype=torch.bfloat16, ws: Optional[Workspace] = None, states_out=None, stream=None):
    """Forward pass with one log-decay per key channel (a [B, T, H, dk]).
    Returns (o, hT); with `states_out` (from tile_states) it also writes the
    state before every tile there, for bwd_vec."""
    B, T, H, dk, dv, n_docs, n_seq = _vec_checks(q, k, v, a, cu_seqlens, h0)
    o = torch.empty((B, T, H, dv), dtype=o_dtype, device=q.device)
    hT = torch.empty((n_seq, H, dk, dv), dtype=torch.float32, device=q.device)
    ws = _ws_vec(OP_FWD, q, v, n_docs, ws, stream)
    st = lib().bdla_fwd_vec(_p(q), _p(k), _p(v), _p(a), b, CHUNK, _p(cu_seqlens), n_docs, _p(h0), _p(o),
                            _dtype_code(o.dtype), _p(hT), _p(states_out), _dims(q, v), mode, ws.ptr, ws.nbytes,
                            _stream_handle(stream))
    if st:
        raise BdlaError(st, "bdla_fwd_vec")
    return o, hT


def bwd_vec(q, k, v, a, dO, b: float = -5.0, h0=None, dhT=None, cu_seqlens=None, mode: int = BOUNDED,
            want_dh0: bool = False, ws: Optional[Workspace] = None, outs=None, states=None, stream=None):
    """Backward pass with one log-decay per key channel.  Returns
    (dq, dk, dv, da, dh0) with da [B, T, H, dk]; dh0 is None unless asked for."""
    B, T, H, dk, dv, n_docs, n_seq = _vec_checks(q, k, v, a, cu_seqlens, h0)
    _check(dO, "dO", torch.bfloat16, 4)
    if dO.shape != v.shape:
        raise ValueError("dO must match v")
    if dhT is not None:
        _check(dhT, "dhT", torch.float32, 4)
    dev = q.device
    if outs is None:
        outs = (torch.empty(q.shape, dtype=torch.float32, device=dev),
                torch.empty(k.shape, dtype=torch.float32, device=dev),
                torch.empty(v.shape, dtype=torch.float32, device=dev),
                torch.empty(a.shape, dtype=torch.float32, device=dev))
    dq, dk_, dv_, da = outs
    dh0 = torch.empty((n_seq, H, dk, dv), dtype=torch.float32, device=dev) if want_dh0 else None
    ws = _ws_vec(OP_BWD, q, v, n_docs, ws, stream)
    st = lib().bdla_bwd_vec(_p(q), _p(k), _p(v), _p(a), b, CHUNK, _p(cu_seqlens), n_docs, _p(h0), _p(dO),
                            _p(dhT), _p(states), _p(dq), _p(dk_), _p(dv_), _p(da), _p(dh0), _dims(q, v), mode,
                            ws.ptr, ws.nbytes, _stream_handle(stream))
    if st:
        raise BdlaError(st, "bdla_bwd_vec")
    return dq, dk_, dv_, da, dh0


# ---------------------------------------------------------------- gated delta rule
def _delta_checks(q, k, v, a, beta, cu_seqlens, h0):
    _check(q, "q", torch.bfloat16, 4, here=True)
    _check(k, "k", torch.bfloat16, 4)
    _check(v, "v", torch.bfloat16, 4)
    _check(a, "a", torch.float32, 3)
    _check(beta, "beta", torch.float32, 3)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or a.shape != q.shape[:3] or beta.shape != a.shape:
        raise ValueError("q, k, v, a, beta shapes disagree")
    n_docs = 0
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, 1)
        n_docs = cu_seqlens.numel() - 1
    n_seq = n_docs if n_docs else B
    if h0 is not None:
        _check(h0, "h0", torch.float32, 4)
        if tuple(h0.shape) != (n_seq, H, dk, dv):
            raise ValueError("h0 must be [n_docs, H, dk, dv]")
    return B, T, H, dk, dv, n_docs, n_seq


def _ws_delta(op, q, v, n_docs, ws, stream):
    B, T, H, dk = q.shape
    need = int(lib().bdla_workspace_bytes_delta(op, Dims(B, T, H, dk, v.shape[-1]), n_docs))
    if need == 0:
        raise BdlaError(ERR_UNSUPPORTED, "bdla_workspace_bytes_delta")
    return _workspace(need, q.device, ws, stream)


def fwd_delta(q, k, v, a, beta, b: float = -5.0, h0=None, cu_seqlens=None, mode: int = BOUNDED,
              o_dtype=torch.bfloat16, ws: Optional[Workspace] = None, out=None, hT_out=None, states_out=None,
              stream=None):
    """Gated delta rule forward (a, beta [B, T, H]).  Returns (o, hT); with
    `states_out` (from tile_states) it also writes the state before every
    tile there, for bwd_delta."""
    B, T, H, dk, dv, n_docs, n_seq = _delta_checks(q, k, v, a, beta, cu_seqlens, h0)
    o = out if out is not None else torch.empty((B, T, H, dv), dtype=o_dtype, device=q.device)
    hT = hT_out if hT_out is not None else torch.empty((n_seq, H, dk, dv), dtype=torch.float32, device=q.device)
    ws = _ws_delta(OP_FWD, q, v, n_docs, ws, stream)
    st = lib().bdla_fwd_delta(_p(q), _p(k), _p(v), _p(a), _p(beta), b, CHUNK, _p(cu_seqlens), n_docs, _p(h0),
                              _p(o), _dtype_code(o.dtype), _p(hT), _p(states_out), _dims(q, v), mode, ws.ptr,
                              ws.nbytes, _stream_handle(stream))
    if st:
        raise BdlaError(st, "bdla_fwd_delta")
    return o, hT


def bwd_delta(q, k, v, a, beta, dO, b: float = -5.0, h0=None, dhT=None, cu_seqlens=None, mode: int = BOUNDED,
              want_dh0: bool = False, ws: Optional[Workspace] = None, outs=None, states=None, stream=None):
    """Gated delta rule backward.  Returns (dq, dk, dv, da, dbeta, dh0);
    dh0 is None unless asked for."""
    B, T, H, dk, dv, n_docs, n_seq = _delta_checks(q, k, v, a, beta, cu_seqlens, h0)
    _check(dO, "dO", torch.bfloat16, 4)
    if dO.shape != v.shape:
        raise ValueError("dO must match v")
    if dhT is not None:
        _check(dhT, "dhT", torch.float32, 4)
    dev = q.device
    if outs is None:
        outs = (torch.empty(q.shape, dtype=torch.float32, device=dev),
                torch.empty(k.shape, dtype=torch.float32, device=dev),
                torch.empty(v.shape, dtype=torch.float32, device=dev),
                torch.empty(a.shape, dtype=torch.float32, device=dev),
                torch.empty(beta.shape, dtype=torch.float32, device=dev))
    dq, dk_, dv_, da, dbeta = outs
    dh0 = torch.empty((n_seq, H, dk, dv), dtype=torch.float32, device=dev) if want_dh0 else None
    ws = _ws_delta(OP_BWD, q, v, n_docs, ws, stream)
    st = lib().bdla_bwd_delta(_p(q), _p(k), _p(v), _p(a), _p(beta), b, CHUNK, _p(cu_seqlens), n_docs, _p(h0),
                              _p(dO), _p(dhT), _p(states), _p(dq), _p(dk_), _p(dv_), _p(da), _p(dbeta), _p(dh0),
                              _dims(q, v), mode, ws.ptr, ws.nbytes, _stream_handle(stream))
    if st:
        raise BdlaError(st, "bdla_bwd_delta")
    return dq, dk_, dv_, da, dbeta, dh0


# ---------------------------------------------------------------- softmax layer
# A decode step makes these calls once a layer, and their kernels run for a few
# microseconds: every check below is one comparison on the good path.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(t: torch.Tensor, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(t.device.index)
    return torch.cuda.current_stream(t.device).cuda_stream


def _on(t, name: str, dtype, shape, device):
    """A contiguous tensor of this type and shape on `device` (a CUDA device)."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device \
            and t.is_contiguous():
        return t.data_ptr()
    _check(t, name, dtype, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, expected {device}")


def _new(device, stream, *outs):
    """Outputs, (shape, dtype) each, that belong to the stream the call runs on."""
    if stream is None:
        return [torch.empty(s, dtype=t, device=device) for s, t in outs]
    with torch.cuda.stream(stream):
        return [torch.empty(s, dtype=t, device=device) for s, t in outs]


def _with_ws(where, op, d: AttnDims, n_docs, max_keys, ws, device, stream, call):
    """Makes the call with the caller's workspace; one that is missing or too
    small is made or grown first, as the library's answer says."""
    st = ERR_WORKSPACE
    if ws is not None:
        ws.note_call(device, stream)
        st = call(ws.buf.data_ptr(), ws.nbytes)
    if st == ERR_WORKSPACE:
        need = int(lib().bdla_workspace_bytes_attn(op, d, n_docs, max_keys))
        if need == 0:   # sizes that the call refuses, before it looks at the workspace or launches: with which status
            raise BdlaError(call(None, 0), where)
        ws = _workspace(need, device, ws, stream)
        st = call(ws.buf.data_ptr(), ws.nbytes)
    if st:
        raise BdlaError(st, where)


def _documents(cu_seqlens, B, device):
    """(pointer, count) of packed documents, (None, 0) for fixed-length rows."""
    if cu_seqlens is None:
        return None, 0
    if not isinstance(cu_seqlens, torch.Tensor):
        raise TypeError("cu_seqlens must be a torch.Tensor")
    p = _on(cu_seqlens, "cu_seqlens", torch.int32, (cu_seqlens.numel(),), device)
    if B != 1:
        raise ValueError("packed documents need B = 1")
    if cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens needs at least two offsets")
    return p, cu_seqlens.numel() - 1


def _strided(t: torch.Tensor, name: str):
    """Element strides (token, head) of a [B, T, H, d] tensor whose features are
    contiguous and whose batch rows follow each other."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16 or t.dim() != 4:
        raise ValueError(f"{name} must be bf16 [B, T, H, d]")
    return _token_strides(t.shape, t.stride(), name)


def _token_strides(shape, strides, name: str):
    """The strides that tell two tokens, or two heads, apart; where there are no two, what torch holds means nothing."""
    B, T, H, d = shape
    sb, st, sh, sd = strides
    if d > 1 and sd != 1:
        raise ValueError(f"{name}: features must be contiguous")
    if B * T <= 1:
        st = H * d
    elif T == 1:
        st = sb   # one token a row: the batch stride steps from token to token
    elif B > 1 and sb != T * st:
        raise ValueError(f"{name}: batch rows must follow each other (batch stride = T * token stride)")
    return st, (sh if H > 1 else d)


def _norm_args(q, k, wq, wk, rotary, base, interleaved, positions, cu_seqlens, eps):
    qt, qh = _strided(q, "q")
    kt, kh = _strided(k, "k")
    B, T, Hq, d = q.shape
    Bk, Tk, Hk, dk = k.shape
    if Bk != B or Tk != T or dk != d:
        raise ValueError("q and k shapes disagree")
    device = q.device
    if k.device != device:
        raise ValueError("q and k are on different devices")
    _here(q, "q")
    cu, n_docs = _documents(cu_seqlens, B, device)
    a = QkNormArgs(q.data_ptr(), k.data_ptr(), qt, qh, kt, kh, _on(wq, "wq", torch.float32, (d,), device),
                   _on(wk, "wk", torch.float32, (d,), device),
                   None if positions is None else _on(positions, "positions", torch.int32, (B, T), device), cu, base,
                   eps, d if rotary is None else rotary, int(interleaved), n_docs)
    return a, AttnDims(B, T, Hq, Hk, d)


def qk_norm(q, k, wq, wk, rotary: Optional[int] = None, base: float = 10000.0, interleaved: bool = False,
            positions=None, cu_seqlens=None, eps: float = 1e-6, stream=None):
    """RMS norm of every head of q [B, T, Hq, d] and k [B, T, Hk, d] (bf16; views
    of one projection are fine) with weights wq, wk (fp32 [d]), then the
    rotation of the first `rotary` features (all by default, 0 for none) by
    the token's position: `positions` (int32 [B, T]), or its index in its
    document.  Returns (qn, kn), contiguous.  Inputs used on another stream
    than their own are the caller's to keep alive, as for every call here."""
    a, d = _norm_args(q, k, wq, wk, rotary, base, interleaved, positions, cu_seqlens, eps)
    qn, kn = _new(q.device, stream, (q.shape, q.dtype), (k.shape, q.dtype))
    st = lib().bdla_qk_norm(a, qn.data_ptr(), kn.data_ptr(), d, _stream_of(q, stream))
    if st:
        raise BdlaError(st, "bdla_qk_norm")
    return qn, kn


def qk_norm_bwd(q, k, wq, wk, dqn, dkn, rotary: Optional[int] = None, base: float = 10000.0,
                interleaved: bool = False, positions=None, cu_seqlens=None, eps: float = 1e-6,
                ws: Optional[Workspace] = None, stream=None):
    """Gradient of qk_norm at the same inputs; dqn, dkn both bf16 or both fp32.
    Returns (dq, dk, dwq, dwk): bf16, bf16 and fp32 [d]."""
    a, d = _norm_args(q, k, wq, wk, rotary, base, interleaved, positions, cu_seqlens, eps)
    code = _dtype_code(dqn.dtype)
    gq = _on(dqn, "dqn", dqn.dtype, q.shape, q.device)
    gk = _on(dkn, "dkn", dqn.dtype, k.shape, q.device)
    bf, f32 = torch.bfloat16, torch.float32
    dq, dk, dwq, dwk = _new(q.device, stream, (q.shape, bf), (k.shape, bf), (wq.shape, f32), (wk.shape, f32))
    s = _stream_of(q, stream)
    _with_ws("bdla_qk_norm_bwd", ATTN_NORM_BWD, d, a.n_docs, 0, ws, q.device, stream,
             lambda p, n: lib().bdla_qk_norm_bwd(a, gq, gk, code, dq.data_ptr(), dk.data_ptr(), dwq.data_ptr(),
                                                 dwk.data_ptr(), d, p, n, s))
    return dq, dk, dwq, dwk


def _attn_args(q, k, v):
    _check(q, "q", torch.bfloat16, 4, here=True)
    B, T, Hq, d = q.shape
    _check(k, "k", torch.bfloat16, 4)
    Hk, device = k.shape[2], q.device
    shape = (B, T, Hk, d)
    return (AttnDims(B, T, Hq, Hk, d), q.data_ptr(), _on(k, "k", torch.bfloat16, shape, device),
            _on(v, "v", torch.bfloat16, shape, device))


def attn_fwd(q, k, v, scale: Optional[float] = None, cu_seqlens=None, ws: Optional[Workspace] = None, stream=None):
    """Causal softmax attention of whole documents: q [B, T, Hq, d], k and v
    [B, T, Hk, d] bf16, Hq a multiple of Hk; packed documents with B = 1 and
    cu_seqlens.  scale is 1/sqrt(d) unless given.  Returns (o, lse): o like q,
    lse fp32 [Hq, B*T]."""
    d, pq, pk, pv = _attn_args(q, k, v)
    cu, n_docs = _documents(cu_seqlens, d.B, q.device)
    o, lse = _new(q.device, stream, (q.shape, q.dtype), ((d.Hq, d.B * d.T), torch.float32))
    scale = d.d ** -0.5 if scale is None else scale
    s = _stream_of(q, stream)
    _with_ws("bdla_attn_fwd", ATTN_FWD, d, n_docs, 0, ws, q.device, stream,
             lambda p, n: lib().bdla_attn_fwd(pq, pk, pv, cu, n_docs, scale, o.data_ptr(), lse.data_ptr(), d, p, n, s))
    return o, lse


def attn_bwd(q, k, v, o, lse, dO, scale: Optional[float] = None, cu_seqlens=None, ws: Optional[Workspace] = None,
             stream=None):
    """Gradient of attn_fwd from its inputs, its (o, lse) and dO like o; o and
    lse may also have been joined with a sink's or other keys' (p = e^{s - lse},
    delta = dO . o).  Returns (dq, dk, dv), bf16.  The same inputs give the same
    bits."""
    d, pq, pk, pv = _attn_args(q, k, v)
    po = _on(o, "o", torch.bfloat16, q.shape, q.device)
    pg = _on(dO, "dO", torch.bfloat16, q.shape, q.device)
    pl = _on(lse, "lse", torch.float32, (d.Hq, d.B * d.T), q.device)
    cu, n_docs = _documents(cu_seqlens, d.B, q.device)
    dq, dk, dv = _new(q.device, stream, (q.shape, q.dtype), (k.shape, q.dtype), (v.shape, q.dtype))
    scale = d.d ** -0.5 if scale is None else scale
    s = _stream_of(q, stream)
    _with_ws("bdla_attn_bwd", ATTN_BWD, d, n_docs, 0, ws, q.device, stream,
             lambda p, n: lib().bdla_attn_bwd(pq, pk, pv, po, pl, pg, cu, n_docs, scale, dq.data_ptr(), dk.data_ptr(),
                                              dv.data_ptr(), d, p, n, s))
    return dq, dk, dv


def _cache_args(kcache, vcache, pages, lens, B, device):
    _check(kcache, "kcache", torch.bfloat16, 4)
    _check(pages, "pages", torch.int32, 2)
    shape, width = kcache.shape, pages.shape[1]
    if kcache.device != device or pages.device != device or pages.shape[0] != B:
        _on(kcache, "kcache", torch.bfloat16, shape, device)
        _on(pages, "pages", torch.int32, (B, width), device)   # one of the two says what is wrong
    return CacheArgs(kcache.data_ptr(), _on(vcache, "vcache", torch.bfloat16, shape, device), pages.data_ptr(),
                     _on(lens, "lens", torch.int32, (B,), device), shape[0], shape[1], width)


def cache_append(k, v, kcache, vcache, pages, lens, rows=None, counts=None, ws: Optional[Workspace] = None,
                 stream=None):
    """Writes k, v [B, T, Hk, d] into the paged cache (kcache, vcache
    [n_pages, page, Hk, d]) behind each sequence's lens[b] tokens: the rows
    0 .. T - 1, or the first counts[b] of rows[b] (int32 [B], [B, T]), which is
    how a verified tree's accepted drafts are made consecutive.  pages is the
    int32 page table [B, max_pages]; lens is left as it is."""
    _check(k, "k", torch.bfloat16, 4, here=True)
    B, T, Hk, d = k.shape
    device = k.device
    pv = _on(v, "v", torch.bfloat16, k.shape, device)
    c = _cache_args(kcache, vcache, pages, lens, B, device)
    if kcache.shape[2:] != (Hk, d):
        raise ValueError("kcache must be [n_pages, page, Hk, d] with the heads of k")
    pr = None if rows is None else _on(rows, "rows", torch.int32, (B, T), device)
    pc = None if counts is None else _on(counts, "counts", torch.int32, (B,), device)
    dims = AttnDims(B, T, Hk, Hk, d)
    pk, s = k.data_ptr(), _stream_of(k, stream)
    _with_ws("bdla_cache_append", ATTN_APPEND, dims, 0, 0, ws, device, stream,
             lambda p, n: lib().bdla_cache_append(pk, pv, c, pr, pc, dims, p, n, s))


def attn_cached(q, kcache, vcache, pages, lens, tree=None, scale: Optional[float] = None,
                ws: Optional[Workspace] = None, stream=None):
    """Attention of each sequence's T newest tokens (q [B, T, Hq, d], T <= 64)
    over the paged cache, their own keys and values already appended at
    positions lens[b] .. lens[b] + T - 1.  tree: int64 [B, T] bit masks of the
    new tokens each one sees (None: those up to and with itself).  Returns
    (o like q, lse fp32 [B, T, Hq]); a token that sees nothing gets 0 and -inf."""
    _check(q, "q", torch.bfloat16, 4, here=True)
    B, T, Hq, d = q.shape
    device = q.device
    c = _cache_args(kcache, vcache, pages, lens, B, device)
    if kcache.shape[3] != d:
        raise ValueError("kcache and q have different widths")
    pt = None if tree is None else _on(tree, "tree", torch.int64, (B, T), device)
    dims = AttnDims(B, T, Hq, kcache.shape[2], d)
    o, lse = _new(device, stream, (q.shape, q.dtype), ((B, T, Hq), torch.float32))
    scale = d ** -0.5 if scale is None else scale
    pq, s = q.data_ptr(), _stream_of(q, stream)
    _with_ws("bdla_attn_cached", ATTN_CACHED, dims, 0, c.max_pages * c.page, ws, device, stream,
             lambda p, n: lib().bdla_attn_cached(pq, c, pt, scale, o.data_ptr(), lse.data_ptr(), dims, p, n, s))
    return o, lse
