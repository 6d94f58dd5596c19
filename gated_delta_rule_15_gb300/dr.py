"""ctypes binding of libdr.so (include/dr.h).

Argument marshalling only: shapes and dtypes are read off torch tensors, pointers and the
current CUDA stream are passed to the C ABI, and every step of the computation runs in the
library's CUDA kernels.  There is no CPU path: importing this module loads libdr.so and
raises ImportError if it has not been built.

Host (CPU) tensors are accepted by the ``*_host`` helpers only, which copy inputs to the
device on the current stream, call the same entry point and copy the results back: that
is the end-to-end path a caller with host buffers takes.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libdr.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libdr.so is not built ({LIB_PATH}); run "
                      "`python -c 'import __graft_entry__ as g; g.build()'`")
_lib = ctypes.CDLL(LIB_PATH)

DR_F32, DR_BF16 = 0, 1
DR_GATE_NONE, DR_GATE_SCALAR, DR_GATE_CHANNEL = 0, 1, 2
DR_OK, DR_ERR_INVALID, DR_ERR_UNSUPPORTED, DR_ERR_CUDA, DR_ERR_TIMEOUT, DR_ERR_WORKSPACE = \
    0, -1, -2, -3, -4, -5
# fused neighbours (flags of dr_chunk_fwd_ex / dr_recurrent_step_ex)
DR_FUSE_QK_L2NORM, DR_FUSE_BETA_SIGMOID, DR_FUSE_OUT_SILU_GATE = 1, 2, 4
DR_FUSE_ALL = 7
L2NORM_EPS = 1e-6   # DR_L2NORM_EPS

# queries and keys (dr_qk_norm_rope): norms, rotation layouts, frequency scalings
DR_NORM_NONE, DR_NORM_L2, DR_NORM_RMS = 0, 1, 2
DR_ROPE_HALF, DR_ROPE_INTERLEAVED = 0, 1
DR_ROPE_PLAIN, DR_ROPE_LINEAR, DR_ROPE_BY_PARTS = 0, 1, 2

# Symbols of include/dr.h (checked by tests/test_abi.py against the header).
EXPORTED = ("dr_version", "dr_chunk_fwd_workspace_bytes", "dr_chunk_fwd_min_workspace_bytes",
            "dr_chunk_fwd_ex_workspace_bytes", "dr_chunk_fwd",
            "dr_recurrent_step", "dr_get_device_status", "dr_strerror",
            "dr_chunk_fwd_noalloc", "dr_chunk_fwd_ex", "dr_recurrent_step_ex",
            "dr_chunk_bwd_workspace_bytes", "dr_chunk_bwd", "dr_selftest_bounded_wait",
            "dr_chunk_fwd_host_dev_bytes", "dr_chunk_fwd_host",
            "dr_linrec_fwd_workspace_bytes", "dr_linrec_fwd", "dr_linrec_bwd_workspace_bytes",
            "dr_linrec_bwd", "dr_linrec_zero_rest", "dr_linrec_step", "dr_rope_table", "dr_qk_norm_rope",
            "dr_qk_norm_rope_bwd_workspace_bytes", "dr_qk_norm_rope_bwd")


class ChunkDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64),
                ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("chunk", ctypes.c_int32)]


class StepDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("H", ctypes.c_int64), ("dk", ctypes.c_int64),
                ("dv", ctypes.c_int64), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class LinrecDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64), ("N", ctypes.c_int64),
                ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class QkNormRopeDesc(ctypes.Structure):
    _fields_ = [("n_tok", ctypes.c_int64), ("seq_len", ctypes.c_int64), ("pos0", ctypes.c_int64),
                ("Hq", ctypes.c_int64), ("Hk", ctypes.c_int64), ("d", ctypes.c_int64),
                ("rot", ctypes.c_int64), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
                ("k_out_stride", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("norm", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("eps", ctypes.c_float),
                ("rot_scale", ctypes.c_float)]


_vp = ctypes.c_void_p
_lib.dr_version.argtypes = []
_lib.dr_version.restype = ctypes.c_int
_lib.dr_chunk_fwd_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDesc),
                                              ctypes.POINTER(ctypes.c_size_t)]
_lib.dr_chunk_fwd_workspace_bytes.restype = ctypes.c_int
_lib.dr_chunk_fwd_min_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDesc),
                                                  ctypes.POINTER(ctypes.c_size_t)]
_lib.dr_chunk_fwd_min_workspace_bytes.restype = ctypes.c_int
_lib.dr_chunk_fwd_ex_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDesc), ctypes.c_uint32,
                                                 ctypes.POINTER(ctypes.c_size_t)]
_lib.dr_chunk_fwd_ex_workspace_bytes.restype = ctypes.c_int
_lib.dr_chunk_fwd.argtypes = [ctypes.POINTER(ChunkDesc), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                              _vp, _vp, ctypes.c_size_t, _vp]
_lib.dr_chunk_fwd.restype = ctypes.c_int
_lib.dr_recurrent_step.argtypes = [ctypes.POINTER(StepDesc), _vp, _vp, _vp, _vp, _vp, _vp,
                                   _vp, _vp]
_lib.dr_recurrent_step.restype = ctypes.c_int
_lib.dr_chunk_fwd_ex.argtypes = [ctypes.POINTER(ChunkDesc), ctypes.c_uint32, _vp, _vp, _vp, _vp,
                                 _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.dr_chunk_fwd_ex.restype = ctypes.c_int
_lib.dr_recurrent_step_ex.argtypes = [ctypes.POINTER(StepDesc), ctypes.c_uint32, _vp, _vp, _vp,
                                      _vp, _vp, _vp, _vp, _vp, _vp]
_lib.dr_recurrent_step_ex.restype = ctypes.c_int
_lib.dr_chunk_bwd_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDesc),
                                              ctypes.POINTER(ctypes.c_size_t)]
_lib.dr_chunk_bwd_workspace_bytes.restype = ctypes.c_int
_lib.dr_chunk_bwd.argtypes = [ctypes.POINTER(ChunkDesc)] + [_vp] * 15 + [ctypes.c_size_t, _vp]
_lib.dr_chunk_bwd.restype = ctypes.c_int
_lib.dr_chunk_fwd_host_dev_bytes.argtypes = [ctypes.POINTER(ChunkDesc), ctypes.c_int,
                                             ctypes.POINTER(ctypes.c_size_t)]
_lib.dr_chunk_fwd_host_dev_bytes.restype = ctypes.c_int
_lib.dr_chunk_fwd_host.argtypes = [ctypes.POINTER(ChunkDesc), ctypes.c_int] + [_vp] * 9 + \
    [ctypes.c_size_t, _vp]
_lib.dr_chunk_fwd_host.restype = ctypes.c_int
_lib.dr_selftest_bounded_wait.argtypes = [ctypes.c_longlong, _vp]
_lib.dr_selftest_bounded_wait.restype = ctypes.c_int
_lib.dr_get_device_status.argtypes = [_vp]
_lib.dr_get_device_status.restype = ctypes.c_int
_lib.dr_strerror.argtypes = [ctypes.c_int]
_lib.dr_strerror.restype = ctypes.c_char_p
_lib.dr_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(ChunkDesc), _vp, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _vp]
_lib.dr_chunk_fwd_noalloc.restype = ctypes.c_int
for _name in ("dr_linrec_fwd_workspace_bytes", "dr_linrec_bwd_workspace_bytes"):
    getattr(_lib, _name).argtypes = [ctypes.POINTER(LinrecDesc), ctypes.POINTER(ctypes.c_size_t)]
_lib.dr_linrec_fwd.argtypes = [ctypes.POINTER(LinrecDesc)] + [_vp] * 9 + [ctypes.c_size_t, _vp]
_lib.dr_linrec_bwd.argtypes = [ctypes.POINTER(LinrecDesc)] + [_vp] * 14 + [ctypes.c_size_t, _vp]
_lib.dr_linrec_zero_rest.argtypes = [ctypes.POINTER(LinrecDesc)] + [_vp] * 6
_lib.dr_linrec_step.argtypes = [ctypes.POINTER(StepDesc)] + [_vp] * 7
_lib.dr_rope_table.argtypes = [ctypes.c_int64, ctypes.c_double, ctypes.c_int32] + \
    [ctypes.c_double] * 4 + [_vp]
_lib.dr_qk_norm_rope.argtypes = [ctypes.POINTER(QkNormRopeDesc)] + [_vp] * 9
_lib.dr_qk_norm_rope_bwd_workspace_bytes.argtypes = [ctypes.POINTER(QkNormRopeDesc),
                                                     ctypes.POINTER(ctypes.c_size_t)]
_lib.dr_qk_norm_rope_bwd.argtypes = [ctypes.POINTER(QkNormRopeDesc)] + [_vp] * 13 + \
    [ctypes.c_size_t, _vp]
for _name in EXPORTED:
    if "linrec" in _name or "rope" in _name:
        getattr(_lib, _name).restype = ctypes.c_int
NOALLOC_SCRATCH_BYTES = 64 << 20   # DR_NOALLOC_SCRATCH_BYTES of include/dr.h

_DT = {torch.float32: DR_F32, torch.bfloat16: DR_BF16}
_TORCH_DT = {DR_F32: torch.float32, DR_BF16: torch.bfloat16}


class DrError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {strerror(status)} (status {status})")
        self.status = status


def lib() -> ctypes.CDLL:
    return _lib


def version() -> int:
    return _lib.dr_version()


def strerror(status: int) -> str:
    return _lib.dr_strerror(status).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _gate_of(log_alpha, bth_shape, dk):
    if log_alpha is None:
        return DR_GATE_NONE
    if tuple(log_alpha.shape) == tuple(bth_shape):
        return DR_GATE_SCALAR
    if tuple(log_alpha.shape) == tuple(bth_shape) + (dk,):
        return DR_GATE_CHANNEL
    raise ValueError(f"log_alpha shape {tuple(log_alpha.shape)} fits neither "
                     f"{tuple(bth_shape)} nor {tuple(bth_shape) + (dk,)}")


def _check_dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def fuse_flags(qk_l2norm: bool = False, beta_sigmoid: bool = False, z=None) -> int:
    """DR_FUSE_* bits for the fused neighbours requested."""
    return ((DR_FUSE_QK_L2NORM if qk_l2norm else 0) | (DR_FUSE_BETA_SIGMOID if beta_sigmoid else 0)
            | (DR_FUSE_OUT_SILU_GATE if z is not None else 0))


def chunk_desc(B, T, H, dk, dv, in_dtype, out_dtype, gate, chunk=64) -> ChunkDesc:
    return ChunkDesc(B, T, H, dk, dv, in_dtype, out_dtype, gate, chunk)


def workspace_bytes(desc: ChunkDesc) -> int:
    n = ctypes.c_size_t(0)
    rc = _lib.dr_chunk_fwd_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != DR_OK:
        raise DrError(rc, "dr_chunk_fwd_workspace_bytes")
    return n.value


def min_workspace_bytes(desc: ChunkDesc) -> int:
    n = ctypes.c_size_t(0)
    rc = _lib.dr_chunk_fwd_min_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != DR_OK:
        raise DrError(rc, "dr_chunk_fwd_min_workspace_bytes")
    return n.value


def ex_workspace_bytes(desc: ChunkDesc, fuse: int) -> int:
    n = ctypes.c_size_t(0)
    rc = _lib.dr_chunk_fwd_ex_workspace_bytes(ctypes.byref(desc), fuse, ctypes.byref(n))
    if rc != DR_OK:
        raise DrError(rc, "dr_chunk_fwd_ex_workspace_bytes")
    return n.value


def chunk_fwd(q, k, v, log_alpha, beta, init_state=None, *, chunk: int = 64,
              out_dtype=None, return_final_state: bool = True, out=None,
              final_state=None, workspace=None, stream=None, qk_l2norm: bool = False,
              beta_sigmoid: bool = False, z=None):
    """Chunkwise forward (dr_chunk_fwd, or dr_chunk_fwd_ex with fused neighbours) on
    device tensors.

    q, k [B,T,H,dk]; v [B,T,H,dv]; beta [B,T,H] (q's dtype); log_alpha None, fp32
    [B,T,H] or [B,T,H,dk]; init_state None or fp32 [B,H,dk,dv].  Returns
    (out [B,T,H,dv], final_state [B,H,dk,dv] fp32 or None).  ``final_state`` may be the
    ``init_state`` tensor for an in-place carry.  Fused neighbours: ``qk_l2norm`` divides
    q and k rows by their norms, ``beta_sigmoid`` reads beta as logits, ``z``
    ([B,T,H,dv], q's dtype) gates the output by silu(z).
    """
    _check_dev(q, k, v, log_alpha, beta, init_state, out, final_state, workspace, z)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DT or k.dtype != q.dtype or v.dtype != q.dtype or beta.dtype != q.dtype:
        raise ValueError("q, k, v, beta must share one dtype (float32 or bfloat16)")
    if tuple(k.shape) != (B, T, H, dk) or tuple(v.shape[:3]) != (B, T, H) \
            or tuple(beta.shape) != (B, T, H):
        raise ValueError("inconsistent shapes")
    if log_alpha is not None and log_alpha.dtype != torch.float32:
        raise ValueError("log_alpha must be float32")
    if init_state is not None and (init_state.dtype != torch.float32
                                   or tuple(init_state.shape) != (B, H, dk, dv)):
        raise ValueError("init_state must be float32 [B,H,dk,dv]")
    if z is not None and (z.dtype != q.dtype or tuple(z.shape) != (B, T, H, dv)):
        raise ValueError("z must have q's dtype and shape [B,T,H,dv]")
    fuse = fuse_flags(qk_l2norm, beta_sigmoid, z)
    gate = _gate_of(log_alpha, (B, T, H), dk)
    odt = _DT[out_dtype or q.dtype]
    desc = chunk_desc(B, T, H, dk, dv, _DT[q.dtype], odt, gate, chunk)
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=_TORCH_DT[odt], device=q.device)
    if final_state is None and return_final_state:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    need = ex_workspace_bytes(desc, fuse) if fuse else workspace_bytes(desc)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if fuse:
        rc = _lib.dr_chunk_fwd_ex(ctypes.byref(desc), fuse, _ptr(q), _ptr(k), _ptr(v),
                                  _ptr(log_alpha), _ptr(beta), _ptr(z), _ptr(init_state),
                                  _ptr(out), _ptr(final_state), _ptr(workspace), wbytes,
                                  _stream_handle(stream))
        if rc != DR_OK:
            raise DrError(rc, "dr_chunk_fwd_ex")
        return out, final_state
    rc = _lib.dr_chunk_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                           _ptr(beta), _ptr(init_state), _ptr(out), _ptr(final_state),
                           _ptr(workspace), wbytes, _stream_handle(stream))
    if rc != DR_OK:
        raise DrError(rc, "dr_chunk_fwd")
    return out, final_state


def bwd_workspace_bytes(desc: ChunkDesc) -> int:
    n = ctypes.c_size_t(0)
    rc = _lib.dr_chunk_bwd_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != DR_OK:
        raise DrError(rc, "dr_chunk_bwd_workspace_bytes")
    return n.value


def chunk_bwd(q, k, v, log_alpha, beta, init_state, d_out, d_final_state=None, *,
              chunk: int = 64, return_d_init: bool = True, workspace=None, stream=None):
    """Backward of chunk_fwd (dr_chunk_bwd): gradients of <d_out, out> +
    <d_final_state, final_state>.  Inputs as for chunk_fwd; d_out [B,T,H,dv] in the
    forward output's dtype; d_final_state None or fp32 [B,H,dk,dv].  Returns (dq, dk, dv,
    d_log_alpha, d_beta, d_init_state): the first three and d_beta in the inputs' dtype,
    d_log_alpha fp32 with log_alpha's shape (None without a gate), d_init_state fp32
    [B,H,dk,dv] (None unless return_d_init)."""
    _check_dev(q, k, v, log_alpha, beta, init_state, d_out, d_final_state, workspace)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DT or k.dtype != q.dtype or v.dtype != q.dtype or beta.dtype != q.dtype:
        raise ValueError("q, k, v, beta must share one dtype (float32 or bfloat16)")
    if d_out.dtype not in _DT or tuple(d_out.shape) != (B, T, H, dv):
        raise ValueError("d_out must be float32 or bfloat16 [B,T,H,dv]")
    for t in (init_state, d_final_state):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (B, H, dk, dv)):
            raise ValueError("states must be float32 [B,H,dk,dv]")
    gate = _gate_of(log_alpha, (B, T, H), dk)
    desc = chunk_desc(B, T, H, dk, dv, _DT[q.dtype], _DT[d_out.dtype], gate, chunk)
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dla = None if log_alpha is None else torch.empty_like(log_alpha)
    dbeta = torch.empty_like(beta)
    dinit = (torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
             if return_d_init else None)
    need = bwd_workspace_bytes(desc)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.dr_chunk_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                           _ptr(beta), _ptr(init_state), _ptr(d_out), _ptr(d_final_state),
                           _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dla), _ptr(dbeta), _ptr(dinit),
                           _ptr(workspace), wbytes, _stream_handle(stream))
    if rc != DR_OK:
        raise DrError(rc, "dr_chunk_bwd")
    return dq, dk_, dv_, dla, dbeta, dinit


def chunk_fwd_noalloc(q, k, v, log_alpha, beta, init_state, out, final_state, *,
                      chunk: int = 64, stream=None):
    """dr_chunk_fwd_noalloc: the chunk forward for callers that cannot allocate device
    memory (a host framework that owns all memory through its own pool, a plugin whose
    execute callback must not allocate, a loop that cannot pay cudaMalloc's implicit
    synchronisation).  The caller passes preallocated ``out`` and ``final_state`` (or
    None); the library's static 64 MiB device scratch replaces the workspace.  Calls that
    overlap on the GPU race on that scratch; the first call on a device must precede any
    stream capture.  Returns the status code (0 on success)."""
    _check_dev(q, k, v, log_alpha, beta, init_state, out, final_state)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    desc = chunk_desc(B, T, H, dk, dv, _DT[q.dtype], _DT[out.dtype],
                      _gate_of(log_alpha, (B, T, H), dk), chunk)
    return _lib.dr_chunk_fwd_noalloc(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v),
                                     _ptr(log_alpha), _ptr(beta), _ptr(init_state),
                                     _ptr(out), _ptr(final_state), _stream_handle(stream))


def recurrent_step(q, k, v, log_alpha, beta, state, *, out=None, out_dtype=None,
                   stream=None, qk_l2norm: bool = False, beta_sigmoid: bool = False, z=None):
    """One decode step (dr_recurrent_step, or dr_recurrent_step_ex with fused neighbours,
    flags as for chunk_fwd; z [B,H,dv]); ``state`` [B,H,dk,dv] fp32 is updated in
    place.  q, k [B,H,dk]; v [B,H,dv]; beta [B,H]; log_alpha None, [B,H] or [B,H,dk].
    Returns out [B,H,dv]."""
    _check_dev(q, k, v, log_alpha, beta, state, out, z)
    B, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DT or k.dtype != q.dtype or v.dtype != q.dtype or beta.dtype != q.dtype:
        raise ValueError("q, k, v, beta must share one dtype (float32 or bfloat16)")
    if state.dtype != torch.float32 or tuple(state.shape) != (B, H, dk, dv):
        raise ValueError("state must be float32 [B,H,dk,dv]")
    if log_alpha is not None and log_alpha.dtype != torch.float32:
        raise ValueError("log_alpha must be float32")
    if z is not None and (z.dtype != q.dtype or tuple(z.shape) != (B, H, dv)):
        raise ValueError("z must have q's dtype and shape [B,H,dv]")
    fuse = fuse_flags(qk_l2norm, beta_sigmoid, z)
    gate = _gate_of(log_alpha, (B, H), dk)
    odt = _DT[out_dtype or q.dtype]
    desc = StepDesc(B, H, dk, dv, _DT[q.dtype], odt, gate, 0)
    if out is None:
        out = torch.empty((B, H, dv), dtype=_TORCH_DT[odt], device=q.device)
    if fuse:
        rc = _lib.dr_recurrent_step_ex(ctypes.byref(desc), fuse, _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(log_alpha), _ptr(beta), _ptr(z), _ptr(state),
                                       _ptr(out), _stream_handle(stream))
        if rc != DR_OK:
            raise DrError(rc, "dr_recurrent_step_ex")
        return out
    rc = _lib.dr_recurrent_step(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v),
                                _ptr(log_alpha), _ptr(beta), _ptr(state), _ptr(out),
                                _stream_handle(stream))
    if rc != DR_OK:
        raise DrError(rc, "dr_recurrent_step")
    return out


def selftest_bounded_wait(cycles: int = 2_000_000, stream=None) -> int:
    """dr_selftest_bounded_wait: a wait that runs out on purpose (no fault); the next
    device_status() returns DR_ERR_TIMEOUT.  Returns the enqueue status."""
    return _lib.dr_selftest_bounded_wait(int(cycles), _stream_handle(stream))


def device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the sticky device status word."""
    return _lib.dr_get_device_status(_stream_handle(stream))


class HostChunkRunner:
    """End-to-end chunk forward for callers holding HOST buffers, through dr_chunk_fwd_host.

    Owns the device staging buffer and pinned host result buffers for one problem shape.
    Each call enqueues, behind the current stream, the host -> device copies of the inputs,
    the forward and the device -> host copies of out and final_state, the sequence split
    into `pieces` time ranges so that copies and kernels overlap; with `sync` it waits for
    the stream.  Returns the pinned host result tensors (reused across calls).  The host
    inputs should be pinned."""

    def __init__(self, like: dict, *, chunk: int = 64, out_dtype=None, pieces: int = 4,
                 device="cuda"):
        q, v = like["q"], like["v"]
        B, T, H, dk = q.shape
        dv = v.shape[-1]
        odt = out_dtype or q.dtype
        self.pieces = pieces
        self.out_h = torch.empty((B, T, H, dv), dtype=odt, pin_memory=True)
        self.fin_h = torch.empty((B, H, dk, dv), dtype=torch.float32, pin_memory=True)
        gate = _gate_of(like["log_alpha"], (B, T, H), dk)
        self.desc = chunk_desc(B, T, H, dk, dv, _DT[q.dtype], _DT[odt], gate, chunk)
        self.with_init = like.get("init_state") is not None
        n = ctypes.c_size_t(0)
        rc = _lib.dr_chunk_fwd_host_dev_bytes(ctypes.byref(self.desc), pieces, ctypes.byref(n))
        if rc != DR_OK:
            raise DrError(rc, "dr_chunk_fwd_host_dev_bytes")
        self.dev = torch.empty(n.value + 256, dtype=torch.uint8, device=device)
        self.dev_off = (-self.dev.data_ptr()) % 256     # 256-byte aligned start
        self.dev_bytes = n.value
        self.h2d_bytes = sum(t.numel() * t.element_size() for t in like.values()
                             if t is not None)
        self.d2h_bytes = (self.out_h.numel() * self.out_h.element_size()
                          + self.fin_h.numel() * self.fin_h.element_size())

    def __call__(self, host: dict, sync: bool = True):
        for t in host.values():
            if t is not None and t.is_cuda:
                raise ValueError("HostChunkRunner takes host tensors")
        rc = _lib.dr_chunk_fwd_host(
            ctypes.byref(self.desc), self.pieces, _ptr(host["q"]), _ptr(host["k"]), _ptr(host["v"]),
            _ptr(host["log_alpha"]), _ptr(host["beta"]), _ptr(host.get("init_state")),
            _ptr(self.out_h), _ptr(self.fin_h),
            ctypes.c_void_p(self.dev.data_ptr() + self.dev_off), self.dev_bytes,
            _stream_handle(None))
        if rc != DR_OK:
            raise DrError(rc, "dr_chunk_fwd_host")
        if sync:
            torch.cuda.current_stream().synchronize()
        return self.out_h, self.fin_h


def chunk_fwd_host(q, k, v, log_alpha, beta, init_state=None, *, chunk: int = 64,
                   out_dtype=None, pieces: int = 4):
    """One-shot end-to-end call for host tensors (see HostChunkRunner)."""
    like = {"q": q, "k": k, "v": v, "log_alpha": log_alpha, "beta": beta,
            "init_state": init_state}
    return HostChunkRunner(like, chunk=chunk, out_dtype=out_dtype, pieces=pieces)(like)


# ------------------------------------------------------------ additive gated recurrence
# These calls also serve single tokens, where the host's time counts: addresses go to ctypes as
# integers, shapes are compared as they are, the device and the stream are asked for without
# torch.cuda's own checks where this torch has the plain getters.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on_one_device(*ts):
    """Contiguous tensors of the current device, or ValueError."""
    dev = _current_device()
    for t in ts:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous and on the current CUDA device")


_NO_SCOPE = contextlib.nullcontext()


def _stream_scope(stream):
    """Buffers allocated for a call belong to the stream that the call runs on."""
    return _NO_SCOPE if stream is None else torch.cuda.stream(stream)


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _current_raw_stream(_current_device())


def _at(t):
    return None if t is None else t.data_ptr()


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _like(t, shape, dtype, what):
    if t is not None and (t.dtype != dtype or t.shape != shape):
        raise ValueError(f"{what} must be {dtype} {list(shape)}")


def _linrec_desc(q, k, v, log_alpha, cu_seqlens, out_dtype):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B,T,H,d]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DT or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share one dtype (float32 or bfloat16)")
    if k.shape != q.shape or v.shape[:3] != q.shape[:3]:
        raise ValueError("inconsistent shapes")
    if out_dtype not in _DT:
        raise ValueError("out_dtype must be float32 or bfloat16")
    _like(log_alpha, (B, T, H), torch.float32, "log_alpha")
    N = 0
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int64 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be int64 [N + 1], N >= 1")
        if B != 1:
            raise ValueError("packed sequences come as one batch row (B = 1)")
        N = cu_seqlens.numel() - 1
    return LinrecDesc(B, T, H, dk, dv, N, _DT[q.dtype], _DT[out_dtype],
                      DR_GATE_NONE if log_alpha is None else DR_GATE_SCALAR, 0)


def _workspace(query, desc, workspace, device, what):
    n = ctypes.c_size_t(0)
    rc = query(ctypes.byref(desc), ctypes.byref(n))
    if rc != DR_OK:
        raise DrError(rc, what)
    if workspace is None and n.value > 0:
        workspace = torch.empty(n.value, dtype=torch.uint8, device=device)
    return workspace


def _zero_rest(desc, cu_seqlens, dq, dk, out, d_log_alpha, stream):
    """New buffers of packed problems: zeros in the rows of no sequence, so that sums over all rows are
    right."""
    if cu_seqlens is None:
        return
    rc = _lib.dr_linrec_zero_rest(ctypes.byref(desc), _at(cu_seqlens), _at(dq), _at(dk), _at(out),
                                  _at(d_log_alpha), _raw_stream(stream))
    if rc != DR_OK:
        raise DrError(rc, "dr_linrec_zero_rest")


def linrec_fwd(q, k, v, log_alpha=None, init_state=None, *, cu_seqlens=None, out_dtype=None,
               return_final_state: bool = True, out=None, final_state=None, workspace=None,
               stream=None):
    """The additive gated linear recurrence S_t = exp(log_alpha_t) S_{t-1} + k_t v_t^T,
    o_t = S_t^T q_t (dr_linrec_fwd).

    q, k [B,T,H,dk]; v [B,T,H,dv]; log_alpha None or fp32 [B,T,H]; init_state None or fp32
    [N,H,dk,dv].  With ``cu_seqlens`` (int64 [N + 1] on the device) the T rows of the one
    batch row hold N sequences behind one another; without, N = B.  Returns (out
    [B,T,H,dv], final_state fp32 [N,H,dk,dv] or None); ``final_state`` may be the
    ``init_state`` tensor.  Rows of no sequence are zero in a new ``out`` and left as they are
    in a given one."""
    _on_one_device(q, k, v, log_alpha, cu_seqlens, init_state, out, final_state, workspace)
    desc = _linrec_desc(q, k, v, log_alpha, cu_seqlens, out_dtype or (q.dtype if out is None else out.dtype))
    states = (desc.N or desc.B, desc.H, desc.dk, desc.dv)
    _like(init_state, states, torch.float32, "init_state")
    _like(final_state, states, torch.float32, "final_state")
    _like(out, v.shape, _TORCH_DT[desc.out_dtype], "out")
    rest = None
    with _stream_scope(stream):
        if out is None:
            out = torch.empty(v.shape, dtype=_TORCH_DT[desc.out_dtype], device=q.device)
            rest = out
        if final_state is None and return_final_state:
            final_state = torch.empty(states, dtype=torch.float32, device=q.device)
        workspace = _workspace(_lib.dr_linrec_fwd_workspace_bytes, desc, workspace, q.device,
                               "dr_linrec_fwd_workspace_bytes")
        rc = _lib.dr_linrec_fwd(ctypes.byref(desc), _at(q), _at(k), _at(v), _at(log_alpha),
                                _at(cu_seqlens), _at(init_state), _at(out), _at(final_state),
                                _at(workspace), _bytes(workspace), _raw_stream(stream))
    if rc != DR_OK:
        raise DrError(rc, "dr_linrec_fwd")
    if rest is not None:
        _zero_rest(desc, cu_seqlens, None, None, rest, None, stream)
    return out, final_state


def linrec_bwd(q, k, v, log_alpha, init_state, d_out, d_final_state=None, *, cu_seqlens=None,
               return_d_init: bool = True, grads=None, workspace=None, stream=None):
    """Gradients of <d_out, out> + <d_final_state, final_state> of linrec_fwd
    (dr_linrec_bwd).  Returns (dq, dk, dv, d_log_alpha, d_init_state): the first three in
    q's dtype, d_log_alpha fp32 (None without a gate), d_init_state fp32 (None unless
    return_d_init).  ``grads``: buffers (dq, dk, dv, d_log_alpha) to write into; their rows
    of no sequence are left as they are (new ones hold zeros there)."""
    _on_one_device(q, k, v, log_alpha, cu_seqlens, init_state, d_out, d_final_state, workspace)
    desc = _linrec_desc(q, k, v, log_alpha, cu_seqlens, d_out.dtype)
    states = (desc.N or desc.B, desc.H, desc.dk, desc.dv)
    _like(init_state, states, torch.float32, "init_state")
    _like(d_final_state, states, torch.float32, "d_final_state")
    _like(d_out, v.shape, d_out.dtype, "d_out")
    new = grads is None
    with _stream_scope(stream):
        if new:
            grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                     None if log_alpha is None else torch.empty_like(log_alpha))
        else:
            if len(grads) != 4 or (grads[3] is None) != (log_alpha is None):
                raise ValueError("grads must be (dq, dk, dv, d_log_alpha or None)")
            _on_one_device(*grads)
            for g, x, n in zip(grads, (q, k, v, log_alpha), ("dq", "dk", "dv", "d_log_alpha")):
                if x is not None and (g is None or g.dtype != x.dtype or g.shape != x.shape):
                    raise ValueError(f"{n} must be {x.dtype} {list(x.shape)}")
        dq, dk, dv, dla = grads
        dinit = torch.empty(states, dtype=torch.float32, device=q.device) if return_d_init else None
        workspace = _workspace(_lib.dr_linrec_bwd_workspace_bytes, desc, workspace, q.device,
                               "dr_linrec_bwd_workspace_bytes")
        rc = _lib.dr_linrec_bwd(ctypes.byref(desc), _at(q), _at(k), _at(v), _at(log_alpha),
                                _at(cu_seqlens), _at(init_state), _at(d_out),
                                _at(d_final_state), _at(dq), _at(dk), _at(dv), _at(dla),
                                _at(dinit), _at(workspace), _bytes(workspace),
                                _raw_stream(stream))
    if rc != DR_OK:
        raise DrError(rc, "dr_linrec_bwd")
    if new:
        _zero_rest(desc, cu_seqlens, dq, dk, dv, dla, stream)
    return dq, dk, dv, dla, dinit


def linrec_step(q, k, v, log_alpha, state, *, out=None, out_dtype=None, stream=None):
    """One token of linrec_fwd for every chain (dr_linrec_step): ``state`` fp32 [B,H,dk,dv] is
    updated in place.  q, k [B,H,dk]; v [B,H,dv]; log_alpha None or fp32 [B,H].  Returns out
    [B,H,dv]."""
    _on_one_device(q, k, v, log_alpha, state, out)
    if q.dim() != 3 or v.dim() != 3 or k.shape != q.shape or v.shape[:2] != q.shape[:2]:
        raise ValueError("inconsistent shapes")
    B, H, dk = q.shape
    dv = v.shape[-1]
    odt = out_dtype or (q.dtype if out is None else out.dtype)
    if q.dtype not in _DT or k.dtype != q.dtype or v.dtype != q.dtype or odt not in _DT:
        raise ValueError("q, k, v must share one dtype (float32 or bfloat16)")
    if state is None:
        raise ValueError("state must be given")
    _like(state, (B, H, dk, dv), torch.float32, "state")
    _like(log_alpha, (B, H), torch.float32, "log_alpha")
    _like(out, (B, H, dv), odt, "out")
    desc = StepDesc(B, H, dk, dv, _DT[q.dtype], _DT[odt],
                    DR_GATE_NONE if log_alpha is None else DR_GATE_SCALAR, 0)
    if out is None:
        with _stream_scope(stream):
            out = torch.empty((B, H, dv), dtype=odt, device=q.device)
    rc = _lib.dr_linrec_step(ctypes.byref(desc), _at(q), _at(k), _at(v), _at(log_alpha),
                             _at(state), _at(out), _raw_stream(stream))
    if rc != DR_OK:
        raise DrError(rc, "dr_linrec_step")
    return out


# ------------------------------------------------------------ queries and keys
_NORMS = {None: DR_NORM_NONE, "none": DR_NORM_NONE, "l2": DR_NORM_L2, "rms": DR_NORM_RMS}
_LAYOUTS = {"half": DR_ROPE_HALF, "interleaved": DR_ROPE_INTERLEAVED}


def rope_table(rot: int, *, base: float = 10000.0, scaling=None, device="cuda"):
    """The rotation's frequencies for qk_norm_rope (dr_rope_table), int64 [rot / 2] on
    ``device``: base^(-2 i / rot), scaled for long contexts by ``scaling``: None,
    {"kind": "linear", "factor"} or {"kind": "by_parts", "factor", "original", "low",
    "high"} (include/dr.h has the formulas)."""
    sc = dict(scaling or {})
    kind = sc.pop("kind", None)
    kinds = {None: (DR_ROPE_PLAIN, ()), "linear": (DR_ROPE_LINEAR, ("factor",)),
             "by_parts": (DR_ROPE_BY_PARTS, ("factor", "original", "low", "high"))}
    if kind not in kinds or set(sc) != set(kinds[kind][1]):
        raise ValueError(f"scaling {scaling!r}: kind linear (factor) or by_parts (factor, original, low, high)")
    t = torch.empty(max(rot, 0) // 2, dtype=torch.int64)
    rc = _lib.dr_rope_table(rot, base, kinds[kind][0], *(float(sc.get(n, 0.0)) for n in
                            ("factor", "original", "low", "high")), t.data_ptr() if t.numel() else 8)
    if rc != DR_OK:
        raise DrError(rc, "dr_rope_table")
    return t.to(device)


def _rows_of(x, what):
    """(rows, heads, d, elements between rows) of [rows, H, d] or [B, T, H, d]."""
    if x.dim() not in (3, 4):
        raise ValueError(f"{what} must be [rows, H, d] or [B, T, H, d]")
    H, d = x.shape[-2:]
    if x.numel() and ((d > 1 and x.stride(-1) != 1) or (H > 1 and x.stride(-2) != d)):
        raise ValueError(f"{what}: a row's heads must lie behind one another")
    n = x.shape[0] if x.dim() == 3 else x.shape[0] * x.shape[1]
    step = x.stride(-3) if x.shape[-3] > 1 else (x.stride(0) if x.dim() == 4 and x.shape[0] > 1 else H * d)
    if x.dim() == 4 and x.shape[0] > 1 and x.shape[1] > 1 and x.stride(0) != x.shape[1] * step:
        raise ValueError(f"{what}: rows must be equally far apart")
    if n > 1 and step < H * d:   # a broadcast row's 0 would mean contiguous rows
        raise ValueError(f"{what}: rows must not share memory")
    return n, H, d, step


def _rows_into(given, x, what):
    """The buffer to write x-shaped rows into and the distance of its rows."""
    if x is None:
        if given is not None:
            raise ValueError(f"{what} without its input")
        return None, 0
    if given is None:
        return torch.empty(x.shape, dtype=x.dtype, device=x.device), 0
    if given.get_device() != x.get_device() or given.dtype != x.dtype \
            or given.shape != x.shape:
        raise ValueError(f"{what} must have its input's shape, dtype and device")
    return given, _rows_of(given, what)[3]


def _qk_desc(q, k, table, positions, offset, norm, wq, wk, eps, layout, rot_scale):
    dev = _current_device()
    for t in (q, k):
        if t is not None and t.get_device() != dev:
            raise ValueError("q and k must be on the current CUDA device")
    _on_one_device(table, positions, wq, wk)
    if q.dtype not in _DT or (k is not None and k.dtype != q.dtype):
        raise ValueError("q and k must share one dtype (float32 or bfloat16)")
    if norm not in _NORMS or layout not in _LAYOUTS:
        raise ValueError("norm must be none, l2 or rms; layout half or interleaved")
    n, Hq, d, qs = _rows_of(q, "q")
    Hk, ks = 0, 0
    if k is not None:
        if k.shape[:-2] != q.shape[:-2] or k.shape[-1] != d:
            raise ValueError("inconsistent shapes")
        _, Hk, _, ks = _rows_of(k, "k")
    if table is not None and (table.dtype != torch.int64 or table.dim() != 1):
        raise ValueError("table must be rope_table's int64 [rot / 2]")
    if positions is not None and (positions.dtype != torch.int64 or positions.shape != q.shape[:-2]):
        raise ValueError("positions must be int64, one per row")
    _like(wq, (d,), torch.float32, "wq")
    _like(wk, (d,), torch.float32, "wk")
    return QkNormRopeDesc(n, q.shape[1] if q.dim() == 4 else 0, int(offset), Hq, Hk, d,
                          0 if table is None else 2 * table.numel(), qs, ks, 0, 0, _DT[q.dtype],
                          _NORMS[norm], _LAYOUTS[layout], 0, eps, rot_scale)


def qk_norm_rope(q, k, table, *, positions=None, offset: int = 0, norm="rms", wq=None, wk=None,
                 eps: float = 1e-6, layout="half", rot_scale: float = 1.0, q_out=None, k_out=None,
                 stream=None):
    """Every head's row of q [..., Hq, d] and k [..., Hk, d] (or None) normalised (``norm``:
    "rms" or "l2" with optional fp32 weights wq, wk [d], or "none") and its first
    2 * len(table) values rotated by the row's position (dr_qk_norm_rope).  Leading shape
    [rows] or [B, T]; rows may be strided, as parts of a fused projection's output.
    ``positions`` int64, one per row, or None: offset + t within each of the B sequences.
    Returns (q_out, k_out): new contiguous tensors, or the given buffers (strided rows, or
    q, k themselves)."""
    desc = _qk_desc(q, k, table, positions, offset, norm, wq, wk, eps, layout, rot_scale)
    with _stream_scope(stream):
        q_out, desc.q_out_stride = _rows_into(q_out, q, "q_out")
        k_out, desc.k_out_stride = _rows_into(k_out, k, "k_out")
    rc = _lib.dr_qk_norm_rope(ctypes.byref(desc), _at(q), _at(k), _at(wq), _at(wk), _at(table),
                              _at(positions), _at(q_out), _at(k_out), _raw_stream(stream))
    if rc != DR_OK:
        raise DrError(rc, "dr_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_bwd(q, k, table, dq_out, dk_out, *, positions=None, offset: int = 0, norm="rms",
                     wq=None, wk=None, eps: float = 1e-6, layout="half", rot_scale: float = 1.0,
                     dq=None, dk=None, workspace=None, stream=None):
    """Gradients of qk_norm_rope from its inputs and the outputs' gradients (contiguous):
    (dq, dk, dwq, dwk), the last two fp32 [d] or None without weights.  ``dq``, ``dk``:
    buffers to write into (strided rows, as parts of a fused gradient, or q, k
    themselves)."""
    desc = _qk_desc(q, k, table, positions, offset, norm, wq, wk, eps, layout, rot_scale)
    _on_one_device(dq_out, dk_out, workspace)
    if dq_out.dtype != q.dtype or dq_out.shape != q.shape or (dk_out is None) != (k is None):
        raise ValueError("dq_out, dk_out must have q's, k's dtype and shape")
    if k is not None and (dk_out.dtype != k.dtype or dk_out.shape != k.shape):
        raise ValueError("dq_out, dk_out must have q's, k's dtype and shape")
    with _stream_scope(stream):
        dq, desc.q_out_stride = _rows_into(dq, q, "dq")
        dk, desc.k_out_stride = _rows_into(dk, k, "dk")
        dwq = None if wq is None else torch.empty_like(wq)
        dwk = None if wk is None else torch.empty_like(wk)
        if dwq is not None or dwk is not None:
            workspace = _workspace(_lib.dr_qk_norm_rope_bwd_workspace_bytes, desc, workspace, q.device,
                                   "dr_qk_norm_rope_bwd_workspace_bytes")
        rc = _lib.dr_qk_norm_rope_bwd(ctypes.byref(desc), _at(q), _at(k), _at(wq), _at(wk),
                                      _at(table), _at(positions), _at(dq_out), _at(dk_out),
                                      _at(dq), _at(dk), _at(dwq), _at(dwk), _at(workspace),
                                      _bytes(workspace), _raw_stream(stream))
    if rc != DR_OK:
        raise DrError(rc, "dr_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk
