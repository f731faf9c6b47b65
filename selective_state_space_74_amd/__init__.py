"""MI355X (gfx950) selective scan: Python binding over libssm.so.

This module only marshals arguments: it checks tensor placement and dtypes,
allocates outputs through torch, fills the C argument blocks declared in
include/ssm.h and calls the library on torch's current HIP stream.  Every step
of the computation runs in the HIP kernels of libssm.so; there is no Python or
CPU fallback, and importing a missing library raises.

    selective_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None,
                       delta_softplus=True, h0=None, return_last_state=False,
                       checkpoints=None)
        -> out, or (out, last_state)
    selective_scan_bwd(dout, u, delta, A, B, C, checkpoints, D=None, z=None,
                       delta_bias=None, delta_softplus=True, h0=None, dlast=None)
        -> dict of gradients (du, ddelta, dB, dC, dA and dz, dD,
           ddelta_bias, dh0 for the inputs that were given)
    selective_state_update(state, x, dt, A, B, C, D=None, z=None,
                           dt_bias=None, dt_softplus=True) -> out  (state updated in place)
    selective_state_update_cached(codes, scales, x, dt, A, B, C, ..., slots=None, seed=None)
        -> out  (the same step on states held in an int8 cache, updated in place)
    state_cache_write(codes, scales, states, slots=None, format="int8")
    state_cache_read(codes, scales, slots=None, format="int8", dtype=float32) -> states
        (a cache of states in int8, e4m3 or e2m1 with a scale per 32 values)
    gated_scan_fwd(x, gate_a, gate_x, lam, c=8.0, h0=None, cu_seqlens=None,
                   return_last_state=False, checkpoints=None) -> out, or (out, last_state)
    gated_scan_bwd(dout, x, gate_a, gate_x, lam, checkpoints, ...) -> dict of gradients
    gated_scan(x, gate_a, gate_x, lam, ...)  (the two as a differentiable torch op)
    gated_state_update(state, x, gate_a, gate_x, lam, c=8.0, slots=None) -> out
        (a gated linear recurrence with one state per channel, token-major,
        batched or packed: prefill, gradients, and its single-token step)

Shapes (N = dstate, 1..64): u, delta, z (batch, dim, L) with time stride 1;
B, C (batch, N, L), or (batch, G, N, L) for G groups of dim // G channels,
with time stride 1; A (dim, N) fp32; D, delta_bias (dim,) fp32; h0 and
last_state (batch, dim, N) fp32.  Decode: state (batch, dim, N) fp32 with
state stride 1; x, dt, z (batch, dim); B, C (batch, N) or (batch, G, N).
IO tensors are float32 or bfloat16 (all of one dtype).
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssm.so")

SSM_ABI_VERSION = 8
CHECKPOINT_TOKENS = 16
GATED_CHECKPOINT_TOKENS = 8
MAX_CONV = 8
SSM_F32, SSM_BF16 = 0, 1
STATUS = {0: "SSM_OK", 1: "SSM_ERR_NULL", 2: "SSM_ERR_SHAPE", 3: "SSM_ERR_STRIDE",
          4: "SSM_ERR_DTYPE", 5: "SSM_ERR_ALIGN", 6: "SSM_ERR_ALIAS", 7: "SSM_ERR_UNSUPPORTED",
          8: "SSM_ERR_HIP", 9: "SSM_ERR_SCRATCH"}
NOALLOC_SCRATCH_BYTES = 32 << 20

CACHE_BLOCK = 32
CACHE_FORMATS = {"int8": 0, "fp8": 1, "fp4": 2}

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32


class ScanArgs(ctypes.Structure):
    """Mirror of ssm_scan_args."""
    _fields_ = [("batch", _I64), ("dim", _I64), ("seqlen", _I64), ("dstate", _I64),
                ("io_dtype", _I32), ("delta_softplus", _I32),
                ("u", _P), ("u_batch_stride", _I64), ("u_dim_stride", _I64),
                ("delta", _P), ("delta_batch_stride", _I64), ("delta_dim_stride", _I64),
                ("z", _P), ("z_batch_stride", _I64), ("z_dim_stride", _I64),
                ("B", _P), ("B_batch_stride", _I64), ("B_state_stride", _I64),
                ("C", _P), ("C_batch_stride", _I64), ("C_state_stride", _I64),
                ("A", _P), ("A_dim_stride", _I64), ("A_state_stride", _I64),
                ("D", _P), ("delta_bias", _P), ("h0", _P), ("last_state", _P),
                ("out", _P), ("out_batch_stride", _I64), ("out_dim_stride", _I64),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t),
                ("checkpoints", _P),
                ("conv_weight", _P), ("conv_bias", _P), ("conv_state_in", _P),
                ("conv_state_out", _P),
                ("conv_out", _P), ("conv_out_batch_stride", _I64), ("conv_out_dim_stride", _I64),
                ("d_conv", _I32), ("conv_silu", _I32),
                ("ngroups", _I64), ("B_group_stride", _I64), ("C_group_stride", _I64)]


class ScanBwdArgs(ctypes.Structure):
    """Mirror of ssm_scan_bwd_args."""
    _fields_ = [("batch", _I64), ("dim", _I64), ("seqlen", _I64), ("dstate", _I64),
                ("io_dtype", _I32), ("delta_softplus", _I32),
                ("u", _P), ("u_batch_stride", _I64), ("u_dim_stride", _I64),
                ("delta", _P), ("delta_batch_stride", _I64), ("delta_dim_stride", _I64),
                ("z", _P), ("z_batch_stride", _I64), ("z_dim_stride", _I64),
                ("B", _P), ("B_batch_stride", _I64), ("B_state_stride", _I64),
                ("C", _P), ("C_batch_stride", _I64), ("C_state_stride", _I64),
                ("A", _P), ("A_dim_stride", _I64), ("A_state_stride", _I64),
                ("D", _P), ("delta_bias", _P), ("h0", _P), ("checkpoints", _P),
                ("dout", _P), ("dout_batch_stride", _I64), ("dout_dim_stride", _I64),
                ("dlast", _P),
                ("du", _P), ("du_batch_stride", _I64), ("du_dim_stride", _I64),
                ("ddelta", _P), ("ddelta_batch_stride", _I64), ("ddelta_dim_stride", _I64),
                ("dz", _P), ("dz_batch_stride", _I64), ("dz_dim_stride", _I64),
                ("dB", _P), ("dC", _P), ("dA", _P), ("dD", _P), ("ddelta_bias", _P),
                ("dh0", _P),
                ("ngroups", _I64), ("B_group_stride", _I64), ("C_group_stride", _I64),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class UpdateArgs(ctypes.Structure):
    """Mirror of ssm_update_args."""
    _fields_ = [("batch", _I64), ("dim", _I64), ("dstate", _I64),
                ("io_dtype", _I32), ("dt_softplus", _I32),
                ("state", _P), ("state_batch_stride", _I64), ("state_dim_stride", _I64),
                ("x", _P), ("x_batch_stride", _I64),
                ("dt", _P), ("dt_batch_stride", _I64),
                ("z", _P), ("z_batch_stride", _I64),
                ("B", _P), ("B_batch_stride", _I64),
                ("C", _P), ("C_batch_stride", _I64),
                ("A", _P), ("A_dim_stride", _I64),
                ("D", _P), ("dt_bias", _P),
                ("out", _P), ("out_batch_stride", _I64),
                ("conv_state", _P), ("conv_weight", _P), ("conv_bias", _P),
                ("d_conv", _I32), ("conv_silu", _I32),
                ("ngroups", _I64), ("B_group_stride", _I64), ("C_group_stride", _I64)]


class SsdArgs(ctypes.Structure):
    """Mirror of ssm_ssd_args."""
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("nheads", _I64), ("headdim", _I64),
                ("ngroups", _I64), ("dstate", _I64),
                ("io_dtype", _I32), ("dt_softplus", _I32),
                ("x", _P), ("x_batch_stride", _I64), ("x_seq_stride", _I64), ("x_head_stride", _I64),
                ("dt", _P), ("dt_batch_stride", _I64), ("dt_seq_stride", _I64),
                ("z", _P), ("z_batch_stride", _I64), ("z_seq_stride", _I64), ("z_head_stride", _I64),
                ("B", _P), ("B_batch_stride", _I64), ("B_seq_stride", _I64), ("B_group_stride", _I64),
                ("C", _P), ("C_batch_stride", _I64), ("C_seq_stride", _I64), ("C_group_stride", _I64),
                ("A", _P), ("D", _P), ("dt_bias", _P), ("h0", _P), ("last_state", _P),
                ("out", _P), ("out_batch_stride", _I64), ("out_seq_stride", _I64),
                ("out_head_stride", _I64), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class GatedArgs(ctypes.Structure):
    """Mirror of ssm_gated_args."""
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("dim", _I64), ("nseq", _I64),
                ("io_dtype", _I32), ("zero_outside", _I32), ("c", ctypes.c_float),
                ("x", _P), ("x_batch_stride", _I64), ("x_seq_stride", _I64),
                ("gate_a", _P), ("gate_a_batch_stride", _I64), ("gate_a_seq_stride", _I64),
                ("gate_x", _P), ("gate_x_batch_stride", _I64), ("gate_x_seq_stride", _I64),
                ("lam", _P), ("cu_seqlens", _P), ("h0", _P), ("last_state", _P),
                ("out", _P), ("out_batch_stride", _I64), ("out_seq_stride", _I64),
                ("checkpoints", _P), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class GatedBwdArgs(ctypes.Structure):
    """Mirror of ssm_gated_bwd_args."""
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("dim", _I64), ("nseq", _I64),
                ("io_dtype", _I32), ("c", ctypes.c_float),
                ("x", _P), ("x_batch_stride", _I64), ("x_seq_stride", _I64),
                ("gate_a", _P), ("gate_a_batch_stride", _I64), ("gate_a_seq_stride", _I64),
                ("gate_x", _P), ("gate_x_batch_stride", _I64), ("gate_x_seq_stride", _I64),
                ("lam", _P), ("cu_seqlens", _P), ("h0", _P), ("checkpoints", _P),
                ("dout", _P), ("dout_batch_stride", _I64), ("dout_seq_stride", _I64),
                ("dlast", _P),
                ("dx", _P), ("dx_batch_stride", _I64), ("dx_seq_stride", _I64),
                ("dgate_a", _P), ("dgate_a_batch_stride", _I64), ("dgate_a_seq_stride", _I64),
                ("dgate_x", _P), ("dgate_x_batch_stride", _I64), ("dgate_x_seq_stride", _I64),
                ("dlam", _P), ("dh0", _P), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class GatedUpdateArgs(ctypes.Structure):
    """Mirror of ssm_gated_update_args."""
    _fields_ = [("batch", _I64), ("nslots", _I64), ("dim", _I64),
                ("io_dtype", _I32), ("c", ctypes.c_float),
                ("state", _P), ("state_slot_stride", _I64),
                ("x", _P), ("x_batch_stride", _I64),
                ("gate_a", _P), ("gate_a_batch_stride", _I64),
                ("gate_x", _P), ("gate_x_batch_stride", _I64),
                ("lam", _P), ("slots", _P), ("out", _P), ("out_batch_stride", _I64)]


class StateCacheArgs(ctypes.Structure):
    """Mirror of ssm_state_cache_args."""
    _fields_ = [("batch", _I64), ("nslots", _I64), ("outer", _I64), ("inner", _I64),
                ("format", _I32), ("io_dtype", _I32),
                ("codes", _P), ("codes_slot_stride", _I64),
                ("scales", _P), ("scales_slot_stride", _I64),
                ("states", _P), ("states_batch_stride", _I64), ("slots", _P)]


class CachedUpdateArgs(ctypes.Structure):
    """Mirror of ssm_cached_update_args."""
    _fields_ = [("batch", _I64), ("nslots", _I64), ("dim", _I64), ("dstate", _I64),
                ("io_dtype", _I32), ("dt_softplus", _I32),
                ("codes", _P), ("codes_slot_stride", _I64),
                ("scales", _P), ("scales_slot_stride", _I64),
                ("x", _P), ("x_batch_stride", _I64),
                ("dt", _P), ("dt_batch_stride", _I64),
                ("z", _P), ("z_batch_stride", _I64),
                ("B", _P), ("B_batch_stride", _I64), ("B_group_stride", _I64),
                ("C", _P), ("C_batch_stride", _I64), ("C_group_stride", _I64),
                ("A", _P), ("A_dim_stride", _I64), ("D", _P), ("dt_bias", _P),
                ("out", _P), ("out_batch_stride", _I64),
                ("slots", _P), ("seed", _P), ("ngroups", _I64)]


class SSMError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")


_lib = None


def lib():
    """The loaded libssm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libssm.so not found at {LIB_PATH}; build it with "
                              "`python -m selective_state_space_74_amd._build`")
        L = ctypes.CDLL(LIB_PATH)
        L.ssm_abi_version.restype = ctypes.c_int
        L.ssm_scan_args_size.restype = ctypes.c_size_t
        L.ssm_scan_bwd_args_size.restype = ctypes.c_size_t
        L.ssm_update_args_size.restype = ctypes.c_size_t
        L.ssm_ssd_args_size.restype = ctypes.c_size_t
        L.ssm_status_string.restype = ctypes.c_char_p
        L.ssm_status_string.argtypes = [ctypes.c_int]
        for name, T in (("ssm_validate_scan", ScanArgs), ("ssm_validate_update", UpdateArgs),
                        ("ssm_validate_scan_bwd", ScanBwdArgs), ("ssm_validate_ssd", SsdArgs)):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [ctypes.POINTER(T)]
        L.ssm_scan_workspace_size.restype = ctypes.c_size_t
        L.ssm_scan_workspace_size.argtypes = [ctypes.POINTER(ScanArgs)]
        L.ssm_scan_bwd_workspace_size.restype = ctypes.c_size_t
        L.ssm_scan_bwd_workspace_size.argtypes = [ctypes.POINTER(ScanBwdArgs)]
        L.ssm_ssd_workspace_size.restype = ctypes.c_size_t
        L.ssm_ssd_workspace_size.argtypes = [ctypes.POINTER(SsdArgs)]
        L.ssm_selective_scan_fwd.restype = ctypes.c_int
        L.ssm_selective_scan_fwd.argtypes = [ctypes.POINTER(ScanArgs), _P]
        L.ssm_selective_scan_fwd_noalloc.restype = ctypes.c_int
        L.ssm_selective_scan_fwd_noalloc.argtypes = [ctypes.POINTER(ScanArgs), _P]
        L.ssm_selective_scan_bwd.restype = ctypes.c_int
        L.ssm_selective_scan_bwd.argtypes = [ctypes.POINTER(ScanBwdArgs), _P]
        L.ssm_selective_state_update.restype = ctypes.c_int
        L.ssm_selective_state_update.argtypes = [ctypes.POINTER(UpdateArgs), _P]
        L.ssm_ssd_scan_fwd.restype = ctypes.c_int
        L.ssm_ssd_scan_fwd.argtypes = [ctypes.POINTER(SsdArgs), _P]
        for name, T in (("gated_scan_fwd", GatedArgs), ("gated_scan_bwd", GatedBwdArgs),
                        ("gated_state_update", GatedUpdateArgs), ("state_cache_write", StateCacheArgs),
                        ("state_cache_read", StateCacheArgs),
                        ("selective_state_update_cached", CachedUpdateArgs)):
            f = getattr(L, "ssm_" + name)
            f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(T), _P]
        for name, T in (("gated", GatedArgs), ("gated_bwd", GatedBwdArgs),
                        ("gated_update", GatedUpdateArgs), ("state_cache_write", StateCacheArgs),
                        ("state_cache_read", StateCacheArgs), ("cached_update", CachedUpdateArgs)):
            f = getattr(L, "ssm_validate_" + name)
            f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(T)]
        for name, T in (("gated_scan", GatedArgs), ("gated_scan_bwd", GatedBwdArgs)):
            f = getattr(L, "ssm_%s_workspace_size" % name)
            f.restype, f.argtypes = ctypes.c_size_t, [ctypes.POINTER(T)]
        if L.ssm_abi_version() != SSM_ABI_VERSION:
            raise ImportError(f"libssm.so ABI {L.ssm_abi_version()} != {SSM_ABI_VERSION}")
        if (L.ssm_scan_args_size() != ctypes.sizeof(ScanArgs)
                or L.ssm_scan_bwd_args_size() != ctypes.sizeof(ScanBwdArgs)
                or L.ssm_update_args_size() != ctypes.sizeof(UpdateArgs)
                or L.ssm_ssd_args_size() != ctypes.sizeof(SsdArgs)):
            raise ImportError("libssm.so argument struct layout differs from the binding")
        for name, T in (("gated", GatedArgs), ("gated_bwd", GatedBwdArgs), ("gated_update", GatedUpdateArgs),
                        ("state_cache", StateCacheArgs), ("cached_update", CachedUpdateArgs)):
            f = getattr(L, "ssm_%s_args_size" % name)
            f.restype = ctypes.c_size_t
            if f() != ctypes.sizeof(T):
                raise ImportError("libssm.so argument struct layout differs from the binding")
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ssm_status_string(int(status)).decode()


def validate_scan(args: ScanArgs) -> int:
    return lib().ssm_validate_scan(ctypes.byref(args))


def validate_scan_bwd(args: ScanBwdArgs) -> int:
    return lib().ssm_validate_scan_bwd(ctypes.byref(args))


def validate_update(args: UpdateArgs) -> int:
    return lib().ssm_validate_update(ctypes.byref(args))


def scan_workspace_size(args: ScanArgs) -> int:
    return lib().ssm_scan_workspace_size(ctypes.byref(args))


def scan_bwd_workspace_size(args: "ScanBwdArgs") -> int:
    return lib().ssm_scan_bwd_workspace_size(ctypes.byref(args))


def scan_fwd_raw(args: ScanArgs, stream: int = 0) -> int:
    return lib().ssm_selective_scan_fwd(ctypes.byref(args), _P(stream or None))


def scan_fwd_noalloc_raw(args: ScanArgs, stream: int = 0) -> int:
    return lib().ssm_selective_scan_fwd_noalloc(ctypes.byref(args), _P(stream or None))


def validate_ssd(args: SsdArgs) -> int:
    return lib().ssm_validate_ssd(ctypes.byref(args))


def ssd_workspace_size(args: SsdArgs) -> int:
    return lib().ssm_ssd_workspace_size(ctypes.byref(args))


def ssd_fwd_raw(args: SsdArgs, stream: int = 0) -> int:
    return lib().ssm_ssd_scan_fwd(ctypes.byref(args), ctypes.c_void_p(stream))


def scan_bwd_raw(args: ScanBwdArgs, stream: int = 0) -> int:
    return lib().ssm_selective_scan_bwd(ctypes.byref(args), _P(stream or None))


def checkpoint_shape(batch: int, dim: int, seqlen: int, dstate: int = 16):
    """Shape of the fp32 state checkpoints the forward writes for the backward."""
    return (batch, dim, (seqlen + CHECKPOINT_TOKENS - 1) // CHECKPOINT_TOKENS, dstate)


def state_update_raw(args: UpdateArgs, stream: int = 0) -> int:
    return lib().ssm_selective_state_update(ctypes.byref(args), _P(stream or None))


# ---------------------------------------------------------------------------
# torch-level wrappers

def _torch():
    import torch
    return torch


def _io_code(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return SSM_F32
    if t.dtype == torch.bfloat16:
        return SSM_BF16
    raise TypeError(f"IO tensors must be float32 or bfloat16, got {t.dtype}")


def _check_dev(name, t, device, dtype=None):
    if t is None:
        return
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _contig_f32(name, t, shape):
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _bc_groups(B, C, batch, dim, N, tail):
    """B/C groups from the shape of B: (batch, N, *tail) is one group shared
    by every channel, (batch, G, N, *tail) is G groups of dim // G channels."""
    if tuple(B.shape) != tuple(C.shape):
        raise ValueError("B and C must have the same shape")
    if tuple(B.shape) == (batch, N) + tuple(tail):
        return 0
    if B.dim() == 3 + len(tail) and tuple(B.shape[2:]) == (N,) + tuple(tail) \
            and B.shape[0] == batch and B.shape[1] >= 1 and dim % B.shape[1] == 0:
        return int(B.shape[1])
    raise ValueError("B and C must be (batch, dstate%s) or (batch, ngroups, dstate%s) with "
                     "ngroups dividing dim" % ((", L",) * 2 if tail else ("", "")))


def _set_bc(a, B, C, G, time):
    """B/C pointers and strides into an argument block (0 groups: 3-D B/C)."""
    a.B, a.C, a.ngroups = _ptr(B), _ptr(C), G
    if time:
        if G:
            a.B_batch_stride, a.B_group_stride, a.B_state_stride = B.stride()[:3]
            a.C_batch_stride, a.C_group_stride, a.C_state_stride = C.stride()[:3]
        else:
            a.B_batch_stride, a.B_state_stride = B.stride()[:2]
            a.C_batch_stride, a.C_state_stride = C.stride()[:2]
    else:
        a.B_batch_stride, a.C_batch_stride = B.stride(0), C.stride(0)
        if G:
            a.B_group_stride, a.C_group_stride = B.stride(1), C.stride(1)


def _stream(stream):
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def selective_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True,
                       h0=None, return_last_state=False, out=None, last_state=None, stream=None,
                       workspace=None, checkpoints=None, conv_weight=None, conv_bias=None,
                       conv_state_in=None, conv_state_out=None, conv_out=None, conv_silu=True,
                       noalloc=False):
    """Prefill selective scan on the GPU (see the module docstring).

    `workspace` (optional): a device tensor reused across calls; when None,
    one of the size the library asks for is allocated through torch; False
    passes no workspace (the scan then runs each sequence as one segment).
    `checkpoints` (optional): an fp32 tensor of checkpoint_shape(...) that
    receives the state entering every 16-token block, for the backward.
    Fused conv branch: with conv_weight (dim, d_conv) fp32, `u` is the conv
    input x and the SSM input is silu(conv_bias + causal depthwise conv of
    x) (no SiLU with conv_silu=False).  conv_state_in (batch, dim, d_conv)
    fp32 holds the inputs before the sequence; conv_state_out (same shape,
    filled with the last d_conv inputs) and conv_out (like u, the SSM
    input) are optional output tensors.
    `noalloc=True` calls ssm_selective_scan_fwd_noalloc, which keeps the
    segment aggregates in the library's static device scratch (no workspace
    is passed or allocated; pass `out` and `last_state` to allocate
    nothing at all)."""
    torch = _torch()
    if u.dim() != 3:
        raise ValueError("u must be (batch, dim, L)")
    batch, dim, L = u.shape
    N = A.shape[1] if A.dim() == 2 else -1
    dev = u.device
    io = u.dtype
    code = _io_code(u)
    for name, t in (("delta", delta), ("z", z), ("B", B), ("C", C)):
        _check_dev(name, t, dev, io)
    for name, t in (("A", A), ("D", D), ("delta_bias", delta_bias), ("h0", h0),
                    ("last_state", last_state)):
        _check_dev(name, t, dev, torch.float32)
    if tuple(delta.shape) != (batch, dim, L) or (z is not None and tuple(z.shape) != (batch, dim, L)):
        raise ValueError("delta and z must match u's shape")
    G = _bc_groups(B, C, batch, dim, N, (L,))
    if tuple(A.shape) != (dim, N):
        raise ValueError("A must be (dim, dstate)")
    for name, t in (("u", u), ("delta", delta), ("z", z), ("B", B), ("C", C)):
        if t is not None and L > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must have time stride 1")
    _contig_f32("D", D, (dim,))
    _contig_f32("delta_bias", delta_bias, (dim,))
    _contig_f32("h0", h0, (batch, dim, N))
    if out is None:
        out = torch.empty((batch, dim, L), dtype=io, device=dev)
    _check_dev("out", out, dev, io)
    if tuple(out.shape) != (batch, dim, L) or (L > 1 and out.stride(2) != 1):
        raise ValueError("out must be (batch, dim, L) with time stride 1")
    if return_last_state and last_state is None:
        last_state = torch.empty((batch, dim, N), dtype=torch.float32, device=dev)
    if last_state is not None:
        _contig_f32("last_state", last_state, (batch, dim, N))
    a = ScanArgs()
    a.batch, a.dim, a.seqlen, a.dstate = batch, dim, L, N
    a.io_dtype, a.delta_softplus = code, int(bool(delta_softplus))
    a.u, (a.u_batch_stride, a.u_dim_stride) = _ptr(u), u.stride()[:2]
    a.delta, (a.delta_batch_stride, a.delta_dim_stride) = _ptr(delta), delta.stride()[:2]
    if z is not None:
        a.z, (a.z_batch_stride, a.z_dim_stride) = _ptr(z), z.stride()[:2]
    _set_bc(a, B, C, G, time=True)
    a.A, (a.A_dim_stride, a.A_state_stride) = _ptr(A), A.stride()
    a.D, a.delta_bias, a.h0 = _ptr(D), _ptr(delta_bias), _ptr(h0)
    a.last_state = _ptr(last_state)
    a.out, (a.out_batch_stride, a.out_dim_stride) = _ptr(out), out.stride()[:2]
    if checkpoints is not None:
        _contig_f32("checkpoints", checkpoints, checkpoint_shape(batch, dim, L, N))
        _check_dev("checkpoints", checkpoints, dev, torch.float32)
        a.checkpoints = _ptr(checkpoints)
    if conv_weight is not None:
        if conv_weight.dim() != 2 or conv_weight.shape[0] != dim:
            raise ValueError("conv_weight must be (dim, d_conv)")
        K = conv_weight.shape[1]
        _check_dev("conv_weight", conv_weight, dev, torch.float32)
        _contig_f32("conv_weight", conv_weight, (dim, K))
        for name, t, shp in (("conv_bias", conv_bias, (dim,)),
                             ("conv_state_in", conv_state_in, (batch, dim, K)),
                             ("conv_state_out", conv_state_out, (batch, dim, K))):
            _check_dev(name, t, dev, torch.float32)
            _contig_f32(name, t, shp)
        a.conv_weight, a.conv_bias = _ptr(conv_weight), _ptr(conv_bias)
        a.conv_state_in, a.conv_state_out = _ptr(conv_state_in), _ptr(conv_state_out)
        a.d_conv, a.conv_silu = K, int(bool(conv_silu))
        if conv_out is not None:
            _check_dev("conv_out", conv_out, dev, io)
            if tuple(conv_out.shape) != (batch, dim, L) or (L > 1 and conv_out.stride(2) != 1):
                raise ValueError("conv_out must be (batch, dim, L) with time stride 1")
            a.conv_out = _ptr(conv_out)
            a.conv_out_batch_stride, a.conv_out_dim_stride = conv_out.stride()[:2]
    if noalloc:
        st = scan_fwd_noalloc_raw(a, _stream(stream))
        if st != 0:
            raise SSMError(st, "ssm_selective_scan_fwd_noalloc")
        return (out, last_state) if return_last_state else out
    need = scan_workspace_size(a) if workspace is not False else 0
    if need:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        _check_dev("workspace", workspace, dev)
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    st = scan_fwd_raw(a, _stream(stream))
    if st != 0:
        raise SSMError(st, "ssm_selective_scan_fwd")
    return (out, last_state) if return_last_state else out


def selective_state_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True,
                           out=None, stream=None, conv_state=None, conv_weight=None,
                           conv_bias=None, conv_silu=True):
    """Single-token decode update on the GPU; `state` is updated in place.
    With conv_weight (dim, d_conv), x is the conv input and conv_state
    (batch, dim, d_conv) fp32 is shifted in place (the fused conv branch)."""
    torch = _torch()
    if state.dim() != 3:
        raise ValueError("state must be (batch, dim, dstate)")
    batch, dim, N = state.shape
    dev = state.device
    io = x.dtype
    code = _io_code(x)
    _check_dev("state", state, dev, torch.float32)
    for name, t in (("x", x), ("dt", dt), ("z", z), ("B", B), ("C", C)):
        _check_dev(name, t, dev, io)
    for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias)):
        _check_dev(name, t, dev, torch.float32)
    for name, t in (("x", x), ("dt", dt), ("z", z)):
        if t is not None and (tuple(t.shape) != (batch, dim) or (dim > 1 and t.stride(1) != 1)):
            raise ValueError(f"{name} must be (batch, dim) with dim stride 1")
    G = _bc_groups(B, C, batch, dim, N, ())
    for name, t in (("B", B), ("C", C)):
        if N > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must have state stride 1")
    if tuple(A.shape) != (dim, N) or (N > 1 and A.stride(1) != 1):
        raise ValueError("A must be (dim, dstate) with state stride 1")
    if N > 1 and state.stride(2) != 1:
        raise ValueError("state must have state stride 1")
    _contig_f32("D", D, (dim,))
    _contig_f32("dt_bias", dt_bias, (dim,))
    if out is None:
        out = torch.empty((batch, dim), dtype=io, device=dev)
    _check_dev("out", out, dev, io)
    if tuple(out.shape) != (batch, dim) or (dim > 1 and out.stride(1) != 1):
        raise ValueError("out must be (batch, dim) with dim stride 1")
    a = UpdateArgs()
    a.batch, a.dim, a.dstate = batch, dim, N
    a.io_dtype, a.dt_softplus = code, int(bool(dt_softplus))
    a.state, (a.state_batch_stride, a.state_dim_stride) = _ptr(state), state.stride()[:2]
    a.x, a.x_batch_stride = _ptr(x), x.stride(0)
    a.dt, a.dt_batch_stride = _ptr(dt), dt.stride(0)
    if z is not None:
        a.z, a.z_batch_stride = _ptr(z), z.stride(0)
    _set_bc(a, B, C, G, time=False)
    a.A, a.A_dim_stride = _ptr(A), A.stride(0)
    a.D, a.dt_bias = _ptr(D), _ptr(dt_bias)
    a.out, a.out_batch_stride = _ptr(out), out.stride(0)
    if conv_weight is not None:
        if conv_weight.dim() != 2 or conv_weight.shape[0] != dim:
            raise ValueError("conv_weight must be (dim, d_conv)")
        K = conv_weight.shape[1]
        if conv_state is None:
            raise ValueError("conv_state is required with conv_weight")
        for name, t, shp in (("conv_weight", conv_weight, (dim, K)), ("conv_bias", conv_bias, (dim,)),
                             ("conv_state", conv_state, (batch, dim, K))):
            _check_dev(name, t, dev, torch.float32)
            _contig_f32(name, t, shp)
        a.conv_state, a.conv_weight, a.conv_bias = _ptr(conv_state), _ptr(conv_weight), _ptr(conv_bias)
        a.d_conv, a.conv_silu = K, int(bool(conv_silu))
    st = state_update_raw(a, _stream(stream))
    if st != 0:
        raise SSMError(st, "ssm_selective_state_update")
    return out


# the backward's workspace is allocated automatically only up to this size
BWD_WORKSPACE_AUTO_MAX = 2 << 30


def selective_scan_bwd(dout, u, delta, A, B, C, checkpoints, D=None, z=None, delta_bias=None,
                       delta_softplus=True, h0=None, dlast=None, stream=None, workspace=None):
    """Gradients of selective_scan_fwd for the upstream gradient dout on out
    (and dlast on last_state), from the checkpoints that forward wrote.
    Returns a dict: du, ddelta (IO dtype, shaped like u), dB, dC (fp32, like
    B), dA (fp32, like A) and, for the inputs that were given, dz, dD,
    ddelta_bias, dh0 (fp32).  The sums over channels (dB, dC) and batch rows
    (dA, dD, ddelta_bias) are formed from partials in a workspace, in fixed
    order (deterministic), or with device atomics without one (their last
    bits may then vary between runs).
    `workspace`: a device tensor reused across calls; None allocates one of
    the size the library asks for (up to BWD_WORKSPACE_AUTO_MAX bytes);
    False passes none (dB/dC then always by atomics)."""
    torch = _torch()
    if u.dim() != 3:
        raise ValueError("u must be (batch, dim, L)")
    batch, dim, L = u.shape
    N = A.shape[1] if A.dim() == 2 else -1
    dev, io = u.device, u.dtype
    code = _io_code(u)
    for name, t in (("delta", delta), ("z", z), ("B", B), ("C", C), ("dout", dout)):
        _check_dev(name, t, dev, io)
    for name, t in (("A", A), ("D", D), ("delta_bias", delta_bias), ("h0", h0),
                    ("checkpoints", checkpoints), ("dlast", dlast)):
        _check_dev(name, t, dev, torch.float32)
    for name, t in (("delta", delta), ("z", z), ("dout", dout)):
        if t is not None and tuple(t.shape) != (batch, dim, L):
            raise ValueError(f"{name} must match u's shape")
    G = _bc_groups(B, C, batch, dim, N, (L,))
    if tuple(A.shape) != (dim, N):
        raise ValueError("A must be (dim, dstate)")
    for name, t in (("u", u), ("delta", delta), ("z", z), ("B", B), ("C", C), ("dout", dout)):
        if t is not None and L > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must have time stride 1")
    _contig_f32("D", D, (dim,))
    _contig_f32("delta_bias", delta_bias, (dim,))
    _contig_f32("h0", h0, (batch, dim, N))
    _contig_f32("dlast", dlast, (batch, dim, N))
    _contig_f32("checkpoints", checkpoints, checkpoint_shape(batch, dim, L, N))
    g = dict(du=torch.empty((batch, dim, L), dtype=io, device=dev),
             ddelta=torch.empty((batch, dim, L), dtype=io, device=dev),
             dB=torch.empty(tuple(B.shape), dtype=torch.float32, device=dev),
             dC=torch.empty(tuple(C.shape), dtype=torch.float32, device=dev),
             dA=torch.empty((dim, N), dtype=torch.float32, device=dev))
    if z is not None:
        g["dz"] = torch.empty((batch, dim, L), dtype=io, device=dev)
    if D is not None:
        g["dD"] = torch.empty(dim, dtype=torch.float32, device=dev)
    if delta_bias is not None:
        g["ddelta_bias"] = torch.empty(dim, dtype=torch.float32, device=dev)
    if h0 is not None:
        g["dh0"] = torch.empty((batch, dim, N), dtype=torch.float32, device=dev)
    a = ScanBwdArgs()
    a.batch, a.dim, a.seqlen, a.dstate = batch, dim, L, N
    a.io_dtype, a.delta_softplus = code, int(bool(delta_softplus))
    a.u, (a.u_batch_stride, a.u_dim_stride) = _ptr(u), u.stride()[:2]
    a.delta, (a.delta_batch_stride, a.delta_dim_stride) = _ptr(delta), delta.stride()[:2]
    if z is not None:
        a.z, (a.z_batch_stride, a.z_dim_stride) = _ptr(z), z.stride()[:2]
        a.dz, (a.dz_batch_stride, a.dz_dim_stride) = _ptr(g["dz"]), g["dz"].stride()[:2]
    _set_bc(a, B, C, G, time=True)
    a.A, (a.A_dim_stride, a.A_state_stride) = _ptr(A), A.stride()
    a.D, a.delta_bias, a.h0 = _ptr(D), _ptr(delta_bias), _ptr(h0)
    a.checkpoints, a.dlast = _ptr(checkpoints), _ptr(dlast)
    a.dout, (a.dout_batch_stride, a.dout_dim_stride) = _ptr(dout), dout.stride()[:2]
    a.du, (a.du_batch_stride, a.du_dim_stride) = _ptr(g["du"]), g["du"].stride()[:2]
    a.ddelta, (a.ddelta_batch_stride, a.ddelta_dim_stride) = _ptr(g["ddelta"]), g["ddelta"].stride()[:2]
    a.dB, a.dC, a.dA = _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dA"])
    a.dD, a.ddelta_bias, a.dh0 = _ptr(g.get("dD")), _ptr(g.get("ddelta_bias")), _ptr(g.get("dh0"))
    need = scan_bwd_workspace_size(a) if workspace is not False else 0
    if need > 0:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = (torch.empty(need, dtype=torch.uint8, device=dev)
                         if need <= BWD_WORKSPACE_AUTO_MAX else None)
        if workspace is not None:
            _check_dev("workspace", workspace, dev)
            a.workspace = _ptr(workspace)
            a.workspace_bytes = workspace.numel() * workspace.element_size()
    st = scan_bwd_raw(a, _stream(stream))
    if st != 0:
        raise SSMError(st, "ssm_selective_scan_bwd")
    return g


def ssd_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, h0=None,
                 return_last_state=False, out=None, last_state=None, stream=None, workspace=None):
    """Mamba-2 SSM (SSD layer) prefill on the GPU.

    x, z: (batch, L, nheads, headdim) with headdim stride 1; dt: (batch, L,
    nheads) with head stride 1 (IO dtype); B, C: (batch, L, ngroups, dstate)
    with state stride 1; A, D, dt_bias: (nheads,) fp32; h0: (batch, nheads,
    headdim, dstate) fp32.  Returns out (like x) or (out, last_state).
    `workspace`: as for selective_scan_fwd (None allocates what the library
    asks for, False passes none: each sequence then runs as one segment)."""
    torch = _torch()
    if x.dim() != 4:
        raise ValueError("x must be (batch, L, nheads, headdim)")
    batch, L, H, P = x.shape
    dev, io = x.device, x.dtype
    code = _io_code(x)
    for name, t in (("dt", dt), ("z", z), ("B", B), ("C", C)):
        _check_dev(name, t, dev, io)
    for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias), ("h0", h0),
                    ("last_state", last_state)):
        _check_dev(name, t, dev, torch.float32)
    if B.dim() != 4 or tuple(B.shape) != tuple(C.shape) or tuple(B.shape[:2]) != (batch, L):
        raise ValueError("B and C must be (batch, L, ngroups, dstate)")
    G, N = B.shape[2], B.shape[3]
    if tuple(dt.shape) != (batch, L, H) or (z is not None and tuple(z.shape) != tuple(x.shape)):
        raise ValueError("dt must be (batch, L, nheads) and z shaped like x")
    for name, t in (("x", x), ("z", z), ("dt", dt), ("B", B), ("C", C)):
        if t is not None and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must have a unit innermost stride")
    _contig_f32("A", A, (H,))
    _contig_f32("D", D, (H,))
    _contig_f32("dt_bias", dt_bias, (H,))
    _contig_f32("h0", h0, (batch, H, P, N))
    if out is None:
        out = torch.empty_like(x)
    _check_dev("out", out, dev, io)
    if tuple(out.shape) != tuple(x.shape) or (P > 1 and out.stride(-1) != 1):
        raise ValueError("out must be shaped like x with headdim stride 1")
    if return_last_state and last_state is None:
        last_state = torch.empty((batch, H, P, N), dtype=torch.float32, device=dev)
    if last_state is not None:
        _contig_f32("last_state", last_state, (batch, H, P, N))
    a = SsdArgs()
    a.batch, a.seqlen, a.nheads, a.headdim, a.ngroups, a.dstate = batch, L, H, P, G, N
    a.io_dtype, a.dt_softplus = code, int(bool(dt_softplus))
    a.x, (a.x_batch_stride, a.x_seq_stride, a.x_head_stride) = _ptr(x), x.stride()[:3]
    a.dt, (a.dt_batch_stride, a.dt_seq_stride) = _ptr(dt), dt.stride()[:2]
    if z is not None:
        a.z, (a.z_batch_stride, a.z_seq_stride, a.z_head_stride) = _ptr(z), z.stride()[:3]
    a.B, (a.B_batch_stride, a.B_seq_stride, a.B_group_stride) = _ptr(B), B.stride()[:3]
    a.C, (a.C_batch_stride, a.C_seq_stride, a.C_group_stride) = _ptr(C), C.stride()[:3]
    a.A, a.D, a.dt_bias, a.h0 = _ptr(A), _ptr(D), _ptr(dt_bias), _ptr(h0)
    a.last_state = _ptr(last_state)
    a.out, (a.out_batch_stride, a.out_seq_stride, a.out_head_stride) = _ptr(out), out.stride()[:3]
    need = ssd_workspace_size(a) if workspace is not False else 0
    if need:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        _check_dev("workspace", workspace, dev)
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    st = ssd_fwd_raw(a, _stream(stream))
    if st != 0:
        raise SSMError(st, "ssm_ssd_scan_fwd")
    return (out, last_state) if return_last_state else out


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True):
    """selective_scan_fwd as a differentiable torch op: the forward keeps the
    state checkpoints and the backward runs ssm_selective_scan_bwd on them.
    Gradients flow to u, delta, A, B, C and, when given, D, z and delta_bias
    (d_state 1..64; B/C shared or in groups that keep 16-channel blocks whole)."""
    torch = _torch()

    class _Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, u, delta, A, B, C, D, z, delta_bias):
            batch, dim, L = u.shape
            ck = torch.empty(checkpoint_shape(batch, dim, L, A.shape[1]), dtype=torch.float32,
                             device=u.device)
            out = selective_scan_fwd(u, delta, A, B, C, D=D, z=z, delta_bias=delta_bias,
                                     delta_softplus=delta_softplus, checkpoints=ck)
            ctx.save_for_backward(u, delta, A, B, C, D, z, delta_bias, ck)
            return out

        @staticmethod
        def backward(ctx, dout):
            u, delta, A, B, C, D, z, delta_bias, ck = ctx.saved_tensors
            g = selective_scan_bwd(dout.contiguous(), u, delta, A, B, C, ck, D=D, z=z,
                                   delta_bias=delta_bias, delta_softplus=delta_softplus)
            return (g["du"], g["ddelta"], g["dA"], g["dB"].to(B.dtype), g["dC"].to(C.dtype),
                    g.get("dD"), g.get("dz"), g.get("ddelta_bias"))

    return _Scan.apply(u, delta, A, B, C, D, z, delta_bias)


# ---------------------------------------------------------------------------
# the gated linear recurrence and the quantised state cache

def validate_gated(args: GatedArgs) -> int:
    return lib().ssm_validate_gated(ctypes.byref(args))


def validate_gated_bwd(args: GatedBwdArgs) -> int:
    return lib().ssm_validate_gated_bwd(ctypes.byref(args))


def validate_gated_update(args: GatedUpdateArgs) -> int:
    return lib().ssm_validate_gated_update(ctypes.byref(args))


def validate_state_cache_write(args: StateCacheArgs) -> int:
    return lib().ssm_validate_state_cache_write(ctypes.byref(args))


def validate_state_cache_read(args: StateCacheArgs) -> int:
    return lib().ssm_validate_state_cache_read(ctypes.byref(args))


def validate_cached_update(args: CachedUpdateArgs) -> int:
    return lib().ssm_validate_cached_update(ctypes.byref(args))


def gated_scan_workspace_size(args: GatedArgs) -> int:
    return lib().ssm_gated_scan_workspace_size(ctypes.byref(args))


def gated_scan_bwd_workspace_size(args: GatedBwdArgs) -> int:
    return lib().ssm_gated_scan_bwd_workspace_size(ctypes.byref(args))


class _Current:
    """The current stream as a context: nothing to switch."""
    __slots__ = ("raw",)

    def __init__(self, raw):
        self.raw = raw

    def __enter__(self):
        return self.raw

    def __exit__(self, *exc):
        return False


@contextlib.contextmanager
def _switched(device, stream):
    torch = _torch()
    if hasattr(stream, "device") and stream.device.index != device:
        raise ValueError(f"stream is of {stream.device}, the tensors are on device {device}")
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        with torch.cuda.stream(stream):
            yield stream.cuda_stream


def _on(device, stream):
    """The tensors' device (its index) and the call's stream as the current
    ones, and the stream's handle: what is allocated meanwhile belongs to that
    stream."""
    C = _torch()._C
    if stream is None and device == C._cuda_getDevice():
        return _Current(C._cuda_getCurrentRawStream(device))
    return _switched(device, stream)


def _gpu(name, t):
    """The index of the GPU a tensor is on."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    return device


def _placed(name, t, dtype, device):
    if t.get_device() != device or t.dtype != dtype:
        _check_dev(name, t, _torch().device("cuda", device), dtype)


def _empty(like, shape, dtype, device):
    """A new tensor of this shape, by the shorter way where `like` has it."""
    torch = _torch()
    if like.shape == shape and like.dtype == dtype and like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(shape, dtype=dtype, device=device)


def _launch(name, args, stream):
    st = getattr(lib(), name)(ctypes.byref(args), stream or None)
    if st != 0:
        raise SSMError(st, name)


def _tokens(name, t, shape, dtype, device):
    """Pointer and (batch, token) strides of a tensor shaped and typed like x; a
    packed (tokens, dim) tensor is one batch row."""
    _placed(name, t, dtype, device)
    if t.shape != shape:
        raise ValueError(f"{name} must be shaped like x")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must have dim stride 1")
    return (t.data_ptr(), st[0], st[1]) if len(st) == 3 else (t.data_ptr(), 0, st[0])


def _fp32(name, t, shape, device):
    """Pointer of a contiguous fp32 tensor of this shape, None for None."""
    if t is None:
        return None
    _placed(name, t, _torch().float32, device)
    if t.shape != shape or not t.is_contiguous():
        _contig_f32(name, t, shape)
    return t.data_ptr()


def _decay_constant(c):
    c = float(c)
    if not 0.0 < c < float("inf"):
        raise ValueError("c must be positive and finite")
    return c


def _gated_sizes(x, cu_seqlens):
    """(batch, tokens of a row, number of sequences, nseq field, bounds' pointer)."""
    torch = _torch()
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError("x must be (batch, L, dim), or (tokens, dim) with cu_seqlens")
        return x.shape[0], x.shape[1], x.shape[0], 0, None
    if x.dim() != 2:
        raise ValueError("x must be (tokens, dim) with cu_seqlens")
    _placed("cu_seqlens", cu_seqlens, torch.int32, x.get_device())
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous int32 vector of nseq + 1 entries")
    n = cu_seqlens.numel() - 1
    return 1, x.shape[0], n, n, cu_seqlens.data_ptr()


def _set_workspace(a, need, workspace, device):
    if not need:
        return None
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = _torch().empty(need, dtype=_torch().uint8, device=device)
    else:
        _placed("workspace", workspace, workspace.dtype, device)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    return workspace


def gated_checkpoint_shape(shape):
    """Shape of the fp32 checkpoints that gated_scan_fwd writes for the
    backward, for x of the given shape."""
    shape = tuple(shape)
    return shape[:-2] + ((shape[-2] + GATED_CHECKPOINT_TOKENS - 1) // GATED_CHECKPOINT_TOKENS, shape[-1])


def gated_scan_fwd(x, gate_a, gate_x, lam, c=8.0, h0=None, cu_seqlens=None, return_last_state=False,
                   out=None, last_state=None, checkpoints=None, stream=None, workspace=None):
    """Gated linear recurrence over whole sequences on the GPU:
        a_t = exp(-c softplus(lam) sigmoid(gate_a_t))
        h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(gate_x_t) x_t,   out_t = h_t

    x, gate_a, gate_x: (batch, L, dim), or (tokens, dim) with cu_seqlens, the
    int32 device tensor of nseq + 1 sequence bounds; dim stride 1, any token
    stride, float32 or bfloat16.  lam (dim,) fp32; h0 (batch or nseq, dim)
    fp32.  Returns out, or (out, last_state); an empty sequence's last state
    is its h0.  Tokens outside every sequence: zero rows in an `out` made
    here, left as they were in one that is given.
    `checkpoints` (optional): an fp32 tensor of gated_checkpoint_shape(x.shape)
    for gated_scan_bwd.  `last_state` may be h0 itself.  `workspace`: a device
    tensor reused across calls, by one call at a time (calls on two streams or
    two captured graphs take one each); None allocates one."""
    torch = _torch()
    code = _io_code(x)
    shape, dev, io = x.shape, _gpu("x", x), x.dtype
    batch, L, n, nseq, cu = _gated_sizes(x, cu_seqlens)
    dim = shape[-1]
    inputs = _tokens("x", x, shape, io, dev) + _tokens("gate_a", gate_a, shape, io, dev) + \
        _tokens("gate_x", gate_x, shape, io, dev)
    lam_p, h0_p = _fp32("lam", lam, (dim,), dev), _fp32("h0", h0, (n, dim), dev)
    c = _decay_constant(c)
    with _on(dev, stream) as s:
        made = out is None
        if made:
            out = _empty(x, shape, io, dev)
        if return_last_state and last_state is None:
            last_state = _empty(x if h0 is None else h0, (n, dim), torch.float32, dev)
        a = GatedArgs(batch, L, dim, nseq, code, made, c, *inputs, lam_p, cu, h0_p,
                      _fp32("last_state", last_state, (n, dim), dev), *_tokens("out", out, shape, io, dev),
                      checkpoints if checkpoints is None else
                      _fp32("checkpoints", checkpoints, gated_checkpoint_shape(shape), dev))
        workspace = _set_workspace(a, gated_scan_workspace_size(a), workspace, dev)
        _launch("ssm_gated_scan_fwd", a, s)
    return (out, last_state) if return_last_state else out


def gated_scan_bwd(dout, x, gate_a, gate_x, lam, checkpoints, c=8.0, h0=None, cu_seqlens=None,
                   dlast=None, stream=None, workspace=None):
    """Gradients of gated_scan_fwd for the upstream gradient dout on out (and
    dlast on last_state), from the checkpoints that forward wrote.  Returns a
    dict: dx, dgate_a, dgate_x (like x), dlam (fp32) and, with h0, dh0 (fp32).
    The inputs are those that the forward read; h0 too, so not a tensor that it
    has since carried in place.
    Rows of tokens outside every sequence are zero.  Every output is the same
    bits from run to run.  `workspace`: as for gated_scan_fwd."""
    torch = _torch()
    code = _io_code(x)
    shape, dev, io = x.shape, _gpu("x", x), x.dtype
    batch, L, n, nseq, cu = _gated_sizes(x, cu_seqlens)
    dim = shape[-1]
    inputs = _tokens("x", x, shape, io, dev) + _tokens("gate_a", gate_a, shape, io, dev) + \
        _tokens("gate_x", gate_x, shape, io, dev)
    lam_p, h0_p = _fp32("lam", lam, (dim,), dev), _fp32("h0", h0, (n, dim), dev)
    ck_p = _fp32("checkpoints", checkpoints, gated_checkpoint_shape(shape), dev)
    upstream = _tokens("dout", dout, shape, io, dev)
    dlast_p = _fp32("dlast", dlast, (n, dim), dev)
    c = _decay_constant(c)
    with _on(dev, stream) as s:
        dx, dga, dgx = (_empty(dout, shape, io, dev) for _ in range(3))
        g = dict(dx=dx, dgate_a=dga, dgate_x=dgx, dlam=torch.empty_like(lam))
        if h0 is not None:
            g["dh0"] = torch.empty_like(h0)
        # the three gradients have the same strides: a row of tokens after another
        rows = (L * dim, dim)
        a = GatedBwdArgs(batch, L, dim, nseq, code, c, *inputs, lam_p, cu, h0_p, ck_p, *upstream, dlast_p,
                         dx.data_ptr(), *rows, dga.data_ptr(), *rows, dgx.data_ptr(), *rows, g["dlam"].data_ptr(),
                         _ptr(g.get("dh0")))
        workspace = _set_workspace(a, gated_scan_bwd_workspace_size(a), workspace, dev)
        _launch("ssm_gated_scan_bwd", a, s)
    return g


def gated_scan(x, gate_a, gate_x, lam, c=8.0, h0=None, cu_seqlens=None, return_last_state=False):
    """gated_scan_fwd as a differentiable torch op: gradients flow to x,
    gate_a, gate_x, lam and h0, from out and from the last state."""
    torch = _torch()
    recording = torch.is_grad_enabled()   # asked here: within forward it never is

    class _GatedScan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, gate_a, gate_x, lam, h0):
            ctx.set_materialize_grads(False)
            ck = None
            if recording and any(ctx.needs_input_grad):
                ck = torch.empty(gated_checkpoint_shape(x.shape), dtype=torch.float32, device=x.device)
            out, last = gated_scan_fwd(x, gate_a, gate_x, lam, c=c, h0=h0, cu_seqlens=cu_seqlens,
                                       return_last_state=True, checkpoints=ck)
            ctx.save_for_backward(x, gate_a, gate_x, lam, h0, cu_seqlens, ck)
            return out, last

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout, dlast):
            x, gate_a, gate_x, lam, h0, cu, ck = ctx.saved_tensors
            dout = torch.zeros_like(x, memory_format=torch.contiguous_format) if dout is None else dout.contiguous()
            g = gated_scan_bwd(dout, x, gate_a, gate_x, lam, ck, c=c, h0=h0, cu_seqlens=cu,
                               dlast=None if dlast is None else dlast.contiguous())
            return g["dx"], g["dgate_a"], g["dgate_x"], g["dlam"], g.get("dh0")

    out, last = _GatedScan.apply(x, gate_a, gate_x, lam, h0)
    return (out, last) if return_last_state else out


def _check_slots(slots, batch, nslots, device):
    if slots is None:
        if batch > nslots:
            raise ValueError("without slots, the batch must not be larger than the pool")
        return
    _placed("slots", slots, _torch().int32, device)
    if slots.shape != (batch,) or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous int32 vector with one entry per batch row")


def _row_tokens(name, t, shape, dtype, device):
    """Pointer and row stride of a (batch, dim) tensor, (None, 0) for None."""
    if t is None:
        return None, 0
    _placed(name, t, dtype, device)
    st = t.stride()
    if t.shape != shape or (st[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be (batch, dim) with dim stride 1")
    return t.data_ptr(), st[0]


def gated_state_update(state, x, gate_a, gate_x, lam, c=8.0, slots=None, out=None, stream=None):
    """Single-token step of the gated recurrence; `state` (nslots, dim) fp32 is
    updated in place.  x, gate_a, gate_x: (batch, dim).  slots: int32 (batch,),
    the pool row of each batch row (None: row b on state b); a slot outside
    the pool marks a padding row (no state touched, zero out), and rows naming
    the same slot are taken in order."""
    torch = _torch()
    if state.dim() != 2 or x.dim() != 2:
        raise ValueError("state must be (nslots, dim) and x (batch, dim)")
    code = _io_code(x)
    (nslots, dim), dev, io = state.shape, _gpu("state", state), x.dtype
    shape = (x.shape[0], dim)
    _placed("state", state, torch.float32, dev)
    pool = state.stride()
    if dim > 1 and pool[1] != 1:
        raise ValueError("state must have dim stride 1")
    inputs = _row_tokens("x", x, shape, io, dev) + _row_tokens("gate_a", gate_a, shape, io, dev) + \
        _row_tokens("gate_x", gate_x, shape, io, dev)
    lam_p = _fp32("lam", lam, (dim,), dev)
    _check_slots(slots, shape[0], nslots, dev)
    c = _decay_constant(c)
    with _on(dev, stream) as s:
        if out is None:
            out = _empty(x, shape, io, dev)
        a = GatedUpdateArgs(shape[0], nslots, dim, code, c, state.data_ptr(), pool[0], *inputs, lam_p, _ptr(slots),
                            *_row_tokens("out", out, shape, io, dev))
        _launch("ssm_gated_state_update", a, s)
    return out


def state_cache_shape(nslots, shape, format="int8"):
    """Shapes of the two uint8 tensors (codes, scales) of a cache of nslots
    states of the given shape; its last axis is cut into blocks of
    CACHE_BLOCK values with one scale each."""
    shape = tuple(shape)
    if format not in CACHE_FORMATS:
        raise ValueError(f"format must be one of {sorted(CACHE_FORMATS)}")
    if not shape:
        raise ValueError("a state has at least one axis")
    if format == "fp4" and shape[-1] % 2:
        raise ValueError("fp4 needs an even last axis")
    held = shape[-1] // 2 if format == "fp4" else shape[-1]
    return (nslots,) + shape[:-1] + (held,), (nslots,) + shape[:-1] + (-(-shape[-1] // CACHE_BLOCK),)


def _inner_contiguous(t):
    """Whether each t[i] is contiguous."""
    return t.shape[0] == 0 or t[0].is_contiguous()


def _cache_fields(codes, scales, shape, format, device):
    """Pointers and slot strides of a cache's two tensors, for states of a shape."""
    uint8 = _torch().uint8
    want = state_cache_shape(codes.shape[0] if codes.dim() else 0, shape, format)
    for name, t, w in (("codes", codes, want[0]), ("scales", scales, want[1])):
        _placed(name, t, uint8, device)
        if t.shape != w:
            raise ValueError(f"{name} must have shape {w} for this state and format, got {tuple(t.shape)}")
        if not t.is_contiguous() and not _inner_contiguous(t):
            raise ValueError(f"{name} must be contiguous within a slot")
    return codes.data_ptr(), codes.stride(0), scales.data_ptr(), scales.stride(0)


def _cache_args(codes, scales, states, slots, format):
    dev, shape = _gpu("codes", codes), states.shape
    if len(shape) < 2:
        raise ValueError("states must be (batch, ...)")
    fields = _cache_fields(codes, scales, shape[1:], format, dev)
    code = _io_code(states)
    _placed("states", states, states.dtype, dev)
    if not states.is_contiguous() and not _inner_contiguous(states):
        raise ValueError("states must be contiguous within a batch row")
    nslots = codes.shape[0]
    _check_slots(slots, shape[0], nslots, dev)
    return StateCacheArgs(shape[0], nslots, math.prod(shape[1:-1]), shape[-1], CACHE_FORMATS[format], code,
                          *fields, states.data_ptr(), states.stride(0), _ptr(slots))


def state_cache_write(codes, scales, states, slots=None, format="int8", stream=None):
    """Quantise states (batch, *shape), float32 or bfloat16, into slots of a
    cache (codes, scales: uint8, of state_cache_shape(nslots, shape, format)).
    Each block of 32 values along the last axis shares a power-of-two scale;
    int8, e4m3 ("fp8") or e2m1 ("fp4") codes, rounded to nearest even.
    slots: int32 (batch,); None: row b to slot b.  A slot outside the cache is
    not written; of rows naming the same slot the last is.  A block with a NaN
    or an infinity reads back as NaN."""
    a = _cache_args(codes, scales, states, slots, format)
    with _on(codes.get_device(), stream) as s:
        _launch("ssm_state_cache_write", a, s)


def state_cache_read(codes, scales, slots=None, format="int8", dtype=None, out=None, stream=None):
    """The states held in slots of a cache (all of it without slots), as
    float32 or `dtype` bfloat16, or into `out`.  A slot outside the cache reads
    as a zero state."""
    torch = _torch()
    if codes.dim() < 2:
        raise ValueError("codes must be (nslots, ...)")
    if format not in CACHE_FORMATS:
        raise ValueError(f"format must be one of {sorted(CACHE_FORMATS)}")
    dev = _gpu("codes", codes)
    batch = codes.shape[0] if slots is None else slots.shape[0]
    shape = (batch,) + tuple(codes.shape[1:-1]) + (codes.shape[-1] * (2 if format == "fp4" else 1),)
    if out is not None and (tuple(out.shape) != shape or (dtype is not None and out.dtype != dtype)):
        raise ValueError(f"out must have shape {shape} and the dtype asked for")
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty(shape, dtype=dtype or torch.float32, device=dev)
        _launch("ssm_state_cache_read", _cache_args(codes, scales, out, slots, format), s)
    return out


def selective_state_update_cached(codes, scales, x, dt, A, B, C, D=None, z=None, dt_bias=None,
                                  dt_softplus=True, slots=None, seed=None, out=None, stream=None):
    """selective_state_update on states held in an int8 cache, updated in place:
    codes (nslots, dim, dstate) and scales (nslots, dim, ceil(dstate / 32)),
    uint8, as state_cache_write fills them.  slots: int32 (batch,), the slot of
    each batch row (None: row b on slot b); a slot outside the cache marks a
    padding row (no state touched, zero out), and rows naming the same slot are
    taken in order.  seed: an int64 device tensor of one element; the new
    states are then rounded stochastically (unbiased), with random bytes that
    its value determines: give every step another value.  None rounds to
    nearest, in which changes below half a code are lost.  out is computed
    before the rounding."""
    torch = _torch()
    if codes.dim() != 3 or x.dim() != 2:
        raise ValueError("codes must be (nslots, dim, dstate) and x (batch, dim)")
    code = _io_code(x)
    (nslots, dim, N), dev, io = codes.shape, _gpu("codes", codes), x.dtype
    shape = (x.shape[0], dim)
    held = _cache_fields(codes, scales, (dim, N), "int8", dev)
    inputs = _row_tokens("x", x, shape, io, dev) + _row_tokens("dt", dt, shape, io, dev) + \
        _row_tokens("z", z, shape, io, dev)
    for name, t in (("B", B), ("C", C)):
        _placed(name, t, io, dev)
        if N > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must have state stride 1")
    G = _bc_groups(B, C, shape[0], dim, N, ())
    _placed("A", A, torch.float32, dev)
    if A.shape != (dim, N) or (N > 1 and A.stride(1) != 1):
        raise ValueError("A must be (dim, dstate) with state stride 1")
    D_p, bias_p = _fp32("D", D, (dim,), dev), _fp32("dt_bias", dt_bias, (dim,), dev)
    _check_slots(slots, shape[0], nslots, dev)
    if seed is not None:
        _placed("seed", seed, torch.int64, dev)
        if seed.numel() != 1:
            raise ValueError("seed must hold one int64")
    with _on(dev, stream) as s:
        if out is None:
            out = _empty(x, shape, io, dev)
        a = CachedUpdateArgs(shape[0], nslots, dim, N, code, bool(dt_softplus), *held, *inputs,
                             B.data_ptr(), B.stride(0), B.stride(1) if G else 0,
                             C.data_ptr(), C.stride(0), C.stride(1) if G else 0, A.data_ptr(), A.stride(0), D_p, bias_p,
                             *_row_tokens("out", out, shape, io, dev), _ptr(slots), _ptr(seed), G)
        _launch("ssm_selective_state_update_cached", a, s)
    return out
