"""Selective state-space scan for AMD Instinct MI355X (gfx950).

Python binding of the C ABI in include/mamba_scan.h, include/mamba_layers.h
and include/mamba_gated.h. It only marshals
arguments: it checks shapes and dtypes, allocates outputs and scratch with
torch on the tensors' device, and passes raw device pointers and the current
HIP stream to libmamba_scan.so, whose kernels do every step of the scan.
There is no other code path: without the built library every call raises.

    y, hL = scan_fwd(x, delta, A, B, C, D=None, z=None, h0=None,
                     delta_bias=None, delta_softplus=False)
    scan_fwd_noalloc(x, delta, A, B, C, D, z, h0, y=y, hL=hL)  # outputs given, nothing allocated
    y = state_update(h, x, delta, A, B, C, D=None, z=None,
                     delta_bias=None, delta_softplus=False)   # h updated in place
    grads = scan_bwd(x, delta, A, B, C, D=None, z=None, h0=None, dy=dy, dhL=None,
                     delta_bias=None, delta_softplus=False)      # dict of gradients
    y, hL = ssd_fwd(x, dt, A_heads, B, C, D=None, z=None, h0=None)   # Mamba-2 dual form
    y, state = conv1d_fwd(x, weight, bias=None, state_in=None, silu=True)
    y = conv1d_update(state, x, weight, bias=None, silu=True)  # state updated in place
    o, hL = linear_attn_fwd(q, k, v, log_decay, h0=None, lengths=None)
    grads = linear_attn_bwd(q, k, v, log_decay, h0=None, do=do, dhL=None, lengths=None)
    o = linear_attn_update(h, q, k, v, log_decay)              # h updated in place
    y, mean, rstd = layer_norm_fwd(x, weight=None, bias=None, groups=1)
    grads = layer_norm_bwd(x, weight, mean, rstd, dy=dy, groups=1)
    y, hL, block_states = gated_scan_fwd(x, decay_gate, log_decay, input_gate=None, h0=None)
    grads = gated_scan_bwd(x, decay_gate, log_decay, input_gate, block_states=block_states,
                           dy=dy, dhL=None)
    y = gated_scan_update(h, x, decay_gate, log_decay, input_gate=None)   # h updated in place
    y, rstd = gated_norm_fwd(x, z=None, weight=None, groups=1, gate_first=True)
    grads = gated_norm_bwd(x, z, weight, rstd, dy=dy, groups=1, gate_first=True)
    y, total, rstd = residual_norm_fwd(x, residual, scale=None, weight=None)
    grads = residual_norm_bwd(total, weight, rstd, x, scale, dy=dy, dtotal=None)

Shapes (row-major, contiguous): x, delta, z, y (batch, L, dim); B, C
(batch, L, N); A (dim, N) fp32; D and delta_bias (dim,) fp32; h0, hL
(batch, dim, N) fp32. With delta_softplus the kernels use
softplus(delta + delta_bias) in place of delta. The short convolution takes
x, y (batch, L, dim), weight (dim, W) fp32, bias (dim,) fp32 and a state of
the last W inputs (batch, dim, W) in the dtype of x.
x, delta, z, B and C share one dtype, float32 or bfloat16, and y has it too.
Linear attention takes q, o (batch, L, heads, dk or dv), k, v (batch, L,
kv_heads, dk or dv), log_decay (heads,) fp32, states (batch, heads, dk, dv) fp32
and lengths (batch,) int32; layer norm x, y (..., dim), weight and bias (dim,)
fp32, mean and rstd (..., groups) fp32. The gated recurrence takes x, gates and y
(batch, L, dim), log_decay (dim,) fp32 and states (batch, dim) fp32; the gated
norm x, z, y (..., dim), weight (dim,) fp32, rstd (..., groups) fp32; the residual
norm x, y (..., dim), the residual stream (..., dim) in the dtype of x or fp32,
scale and weight (dim,) fp32. x, z and the gates of the gated operators may be
slices of a wider tensor's channels (rows a fixed stride apart) that start on 16
bytes: the second half of a tensor of 2 dim channels does where dim is a multiple of
8 in bfloat16, of 4 in float32; other slices raise MambaScanError and are copied
first (contiguous()).
"""
import collections
import ctypes
import functools
import os

import torch

__all__ = ["scan_fwd", "scan_fwd_noalloc", "NOALLOC_SCRATCH_BYTES", "scan_bwd", "ssd_fwd", "state_update", "conv1d_fwd", "conv1d_update",
           "linear_attn_fwd", "linear_attn_bwd", "linear_attn_update", "layer_norm_fwd",
           "layer_norm_bwd", "gated_scan_fwd", "gated_scan_bwd", "gated_scan_update",
           "GATED_SCAN_BLOCK", "gated_norm_fwd", "gated_norm_bwd", "residual_norm_fwd",
           "residual_norm_bwd", "workspace_size", "resolve_plan", "library_path",
           "load_library", "MambaScanError", "MAX_DSTATE", "ScanPlan", "ScanOptions", "Plan",
           "CARRY_AUTO", "CARRY_RERUN", "CARRY_REPAIR", "HALVES_AUTO", "HALVES_NONE"]

MAX_DSTATE = 16
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024  # MAMBA_NOALLOC_SCRATCH_BYTES
GATED_SCAN_BLOCK = 64   # MAMBA_GATED_SCAN_BLOCK: tokens between block_states
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None
_WS = {}


CARRY_AUTO, CARRY_RERUN, CARRY_REPAIR = 0, 1, 2


HALVES_AUTO, HALVES_NONE = 0, -1


class ScanPlan(ctypes.Structure):
    """mamba_scan_plan: chunk_len (tokens per parallel chunk), state_split
    (waves sharing one channel's states), carry (CARRY_RERUN: summary pass
    and a rerun of every chunk; CARRY_REPAIR: one pass from zero states and a
    rerun of each chunk's head while the entering state still counts) and
    halves (the last channel groups run as two 32-channel halves; -1 none,
    k > 0 the last k groups); 0 means automatic."""
    _fields_ = [("chunk_len", ctypes.c_int64), ("state_split", ctypes.c_int32),
                ("carry", ctypes.c_int32), ("halves", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


Plan = collections.namedtuple("Plan", "chunk_len state_split carry halves workspace_bytes")


class ScanOptions(ctypes.Structure):
    """mamba_scan_options: optional delta bias (device pointer) and softplus."""
    _fields_ = [("delta_bias", ctypes.c_void_p), ("delta_softplus", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class MambaScanError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(msg)
        self.status = status


def library_path():
    return os.environ.get("MAMBA_SCAN_LIB", os.path.join(_HERE, "libmamba_scan.so"))


def load_library():
    """Load libmamba_scan.so (built in-tree by __graft_entry__.build())."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise MambaScanError(-5, f"HIP library not built: {path} is missing "
                                 "(run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    pp = ctypes.POINTER(ScanPlan)
    po = ctypes.POINTER(ScanOptions)
    lib.ssm_scan_fwd_workspace_size.argtypes = [i64, i64, i64, i32, i32, pp, pp,
                                                ctypes.POINTER(ctypes.c_size_t)]
    lib.ssm_scan_fwd_workspace_size.restype = i32
    lib.ssm_scan_fwd.argtypes = ([i64, i64, i64, i32, i32] + [vp] * 10 +
                                 [po, pp, vp, ctypes.c_size_t, vp])
    lib.ssm_scan_fwd.restype = i32
    lib.ssm_scan_fwd_noalloc.argtypes = [i64, i64, i64, i32, i32] + [vp] * 10 + [po, pp, vp]
    lib.ssm_scan_fwd_noalloc.restype = i32
    lib.ssm_state_update.argtypes = [i64, i64, i32, i32] + [vp] * 9 + [po, vp]
    lib.ssm_state_update.restype = i32
    lib.ssm_scan_bwd_workspace_size.argtypes = [i64, i64, i64, i32, i32, pp, pp,
                                                ctypes.POINTER(ctypes.c_size_t)]
    lib.ssm_scan_bwd_workspace_size.restype = i32
    lib.ssm_scan_bwd.argtypes = ([i64, i64, i64, i32, i32] + [vp] * 8 + [po, pp] + [vp] * 11 +
                                 [vp, ctypes.c_size_t, vp])
    lib.ssm_scan_bwd.restype = i32
    lib.ssd_fwd.argtypes = [i64, i64, i64, i64, i32, i32] + [vp] * 10 + [po, vp]
    lib.ssd_fwd.restype = i32
    lib.causal_conv1d_fwd.argtypes = [i64, i64, i64, i32, i32] + [vp] * 6 + [i32, vp]
    lib.causal_conv1d_fwd.restype = i32
    lib.causal_conv1d_update.argtypes = [i64, i64, i32, i32] + [vp] * 5 + [i32, vp]
    lib.causal_conv1d_update.restype = i32
    sz = ctypes.c_size_t
    for fn in (lib.linear_attn_fwd_workspace_size, lib.linear_attn_bwd_workspace_size):
        fn.argtypes = [i64] * 6 + [i32, i64, ctypes.POINTER(sz)]
        fn.restype = i32
    f32 = ctypes.c_float
    lib.linear_attn_fwd.argtypes = [i64] * 6 + [i32] + [vp] * 6 + [f32] + [vp] * 2 + [i64, vp, sz, vp]
    lib.linear_attn_fwd.restype = i32
    lib.linear_attn_bwd.argtypes = [i64] * 6 + [i32] + [vp] * 6 + [f32] + [vp] * 7 + [i64, vp, sz, vp]
    lib.linear_attn_bwd.restype = i32
    lib.linear_attn_update.argtypes = [i64] * 5 + [i32] + [vp] * 5 + [f32, vp, vp]
    lib.linear_attn_update.restype = i32
    lib.layer_norm_fwd.argtypes = [i64] * 3 + [i32] + [vp] * 3 + [f32] + [vp] * 4
    lib.layer_norm_fwd.restype = i32
    lib.layer_norm_bwd_workspace_size.argtypes = [i64] * 3 + [i32, ctypes.POINTER(sz)]
    lib.layer_norm_bwd_workspace_size.restype = i32
    lib.layer_norm_bwd.argtypes = [i64] * 3 + [i32] + [vp] * 9 + [sz, vp]
    lib.layer_norm_bwd.restype = i32
    psz = ctypes.POINTER(sz)
    for fn in (lib.gated_scan_fwd_workspace_size, lib.gated_scan_bwd_workspace_size):
        fn.argtypes = [i64] * 3 + [i32, psz]
        fn.restype = i32
    gates = [vp, i64, vp, i64, vp, vp, i64]   # x, decay_gate, log_decay, input_gate, strides
    lib.gated_scan_fwd.argtypes = [i64] * 3 + [i32] + gates + [vp] * 5 + [vp, sz, vp]
    lib.gated_scan_fwd.restype = i32
    lib.gated_scan_bwd.argtypes = [i64] * 3 + [i32] + gates + [vp] * 9 + [vp, sz, vp]
    lib.gated_scan_bwd.restype = i32
    lib.gated_scan_update.argtypes = [i64] * 2 + [i32, vp] + gates + [vp, vp]
    lib.gated_scan_update.restype = i32
    lib.gated_norm_fwd.argtypes = [i64] * 3 + [i32] * 2 + [vp, i64, vp, i64, vp, f32] + [vp] * 3
    lib.gated_norm_fwd.restype = i32
    lib.gated_norm_bwd_workspace_size.argtypes = [i64] * 3 + [i32, psz]
    lib.gated_norm_bwd_workspace_size.restype = i32
    lib.gated_norm_bwd.argtypes = ([i64] * 3 + [i32] * 2 + [vp, i64, vp, i64] + [vp] * 6 +
                                   [vp, sz, vp])
    lib.gated_norm_bwd.restype = i32
    lib.residual_norm_fwd.argtypes = [i64] * 2 + [i32] * 2 + [vp] * 4 + [f32] + [vp] * 4
    lib.residual_norm_fwd.restype = i32
    lib.residual_norm_bwd_workspace_size.argtypes = [i64] * 2 + [i32] * 2 + [psz]
    lib.residual_norm_bwd_workspace_size.restype = i32
    lib.residual_norm_bwd.argtypes = [i64] * 2 + [i32] * 2 + [vp] * 11 + [vp, sz, vp]
    lib.residual_norm_bwd.restype = i32
    lib.mamba_status_string.argtypes = [i32]
    lib.mamba_status_string.restype = ctypes.c_char_p
    _LIB = lib
    return lib


def _check(status, what):
    if status != 0:
        msg = load_library().mamba_status_string(status).decode()
        raise MambaScanError(status, f"{what}: {msg}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, shape, dtype, device):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _options(delta_bias, delta_softplus):
    if delta_bias is None and not delta_softplus:
        return None
    return ctypes.byref(ScanOptions(None if delta_bias is None else delta_bias.data_ptr(),
                                    1 if delta_softplus else 0, 0))


def resolve_plan(batch, seqlen, dim, dstate, dtype=torch.bfloat16, chunk_len=0, state_split=0,
                 carry=CARRY_AUTO, halves=HALVES_AUTO):
    """The plan ssm_scan_fwd uses for this shape, and its scratch bytes, as a
    Plan (chunk_len, state_split, carry, halves, workspace_bytes); halves is
    the number of channel groups split. Automatic fields query the current
    device."""
    req = ScanPlan(chunk_len, state_split, carry, halves, 0)
    out = ScanPlan(0, 0, 0, 0, 0)
    nbytes = ctypes.c_size_t(0)
    _check(load_library().ssm_scan_fwd_workspace_size(batch, seqlen, dim, dstate, _DTYPES[dtype],
                                                      ctypes.byref(req), ctypes.byref(out),
                                                      ctypes.byref(nbytes)),
           "ssm_scan_fwd_workspace_size")
    return Plan(out.chunk_len, out.state_split, out.carry, out.halves, nbytes.value)


def resolve_bwd_plan(batch, seqlen, dim, dstate, dtype=torch.bfloat16, chunk_len=0,
                     halves=HALVES_AUTO):
    """The plan ssm_scan_bwd uses for this shape, and its scratch bytes, as a
    Plan (chunk_len: the chunk length, the whole sequence when uncut; halves:
    the channel groups split; state_split and carry 0)."""
    req = ScanPlan(chunk_len, 0, 0, halves, 0)
    out = ScanPlan(0, 0, 0, 0, 0)
    nbytes = ctypes.c_size_t(0)
    _check(load_library().ssm_scan_bwd_workspace_size(batch, seqlen, dim, dstate, _DTYPES[dtype],
                                                      ctypes.byref(req), ctypes.byref(out),
                                                      ctypes.byref(nbytes)),
           "ssm_scan_bwd_workspace_size")
    return Plan(out.chunk_len, 0, 0, out.halves, nbytes.value)


def workspace_size(batch, seqlen, dim, dstate, dtype=torch.bfloat16, chunk_len=0, state_split=0,
                   carry=CARRY_AUTO, halves=HALVES_AUTO):
    """Scratch bytes ssm_scan_fwd needs for this shape and plan."""
    return resolve_plan(batch, seqlen, dim, dstate, dtype, chunk_len, state_split, carry,
                        halves).workspace_bytes


def _workspace(device, nbytes, kind="fwd"):
    if nbytes == 0:
        return None
    key = (device, torch.cuda.current_stream(device).cuda_stream, kind)
    buf = _WS.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _WS[key] = buf
    return buf


def scan_fwd(x, delta, A, B, C, D=None, z=None, h0=None, *, delta_bias=None,
             delta_softplus=False, chunk_len=0, state_split=0, carry=CARRY_AUTO,
             halves=HALVES_AUTO, return_state=True, out=None, state_out=None):
    """Selective scan over whole sequences; returns (y, hL) (hL is None when
    return_state is False). `delta_bias` (dim,) fp32 is added to delta and
    `delta_softplus` applies softplus after it, inside the kernels.
    `chunk_len` > 0 forces the parallel chunk length, `state_split` > 0 the
    number of waves sharing a channel's states, `carry` how chunks join
    (CARRY_RERUN or CARRY_REPAIR) and `halves` how many of the last channel
    groups run as two 32-channel halves (HALVES_NONE: none)."""
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be (batch, L, dim)")
    batch, seqlen, dim = x.shape
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError("A must be (dim, N)")
    dstate = A.shape[1]
    dev, dt = x.device, x.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported I/O dtype {dt}")
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _need(x, "x", (batch, seqlen, dim), dt, dev)
    _need(delta, "delta", (batch, seqlen, dim), dt, dev)
    _need(A, "A", (dim, dstate), torch.float32, dev)
    _need(B, "B", (batch, seqlen, dstate), dt, dev)
    _need(C, "C", (batch, seqlen, dstate), dt, dev)
    _need(D, "D", (dim,), torch.float32, dev)
    _need(z, "z", (batch, seqlen, dim), dt, dev)
    _need(h0, "h0", (batch, dim, dstate), torch.float32, dev)
    _need(delta_bias, "delta_bias", (dim,), torch.float32, dev)
    y = out if out is not None else torch.empty_like(x)
    _need(y, "out", (batch, seqlen, dim), dt, dev)
    hL = None
    if return_state:
        hL = state_out if state_out is not None else torch.empty(batch, dim, dstate,
                                                                 dtype=torch.float32, device=dev)
        _need(hL, "state_out", (batch, dim, dstate), torch.float32, dev)
    plan = ScanPlan(chunk_len, state_split, carry, halves, 0)
    with torch.cuda.device(dev):
        nbytes = workspace_size(batch, seqlen, dim, dstate, dt, chunk_len, state_split, carry,
                                halves)
        ws = _workspace(dev, nbytes)
        st = lib.ssm_scan_fwd(batch, seqlen, dim, dstate, _DTYPES[dt], _ptr(x), _ptr(delta),
                              _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(y),
                              _ptr(hL), _options(delta_bias, delta_softplus), ctypes.byref(plan),
                              _ptr(ws), nbytes, _stream(dev))
    _check(st, "ssm_scan_fwd")
    return y, hL


def scan_fwd_noalloc(x, delta, A, B, C, D=None, z=None, h0=None, *, y, hL=None,
                     delta_bias=None, delta_softplus=False, chunk_len=0, state_split=0,
                     carry=CARRY_AUTO, halves=HALVES_AUTO):
    """scan_fwd through ssm_scan_fwd_noalloc: the caller passes the outputs
    y (like x) and hL ((batch, dim, N) fp32 or None) and nothing is
    allocated, on the device or by torch; a chunked plan uses the library's
    fixed per-GPU scratch (NOALLOC_SCRATCH_BYTES), which calls that overlap
    on one GPU share. Returns (y, hL)."""
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be (batch, L, dim)")
    batch, seqlen, dim = x.shape
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError("A must be (dim, N)")
    dstate = A.shape[1]
    dev, dt = x.device, x.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported I/O dtype {dt}")
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _need(x, "x", (batch, seqlen, dim), dt, dev)
    _need(delta, "delta", (batch, seqlen, dim), dt, dev)
    _need(A, "A", (dim, dstate), torch.float32, dev)
    _need(B, "B", (batch, seqlen, dstate), dt, dev)
    _need(C, "C", (batch, seqlen, dstate), dt, dev)
    _need(D, "D", (dim,), torch.float32, dev)
    _need(z, "z", (batch, seqlen, dim), dt, dev)
    _need(h0, "h0", (batch, dim, dstate), torch.float32, dev)
    _need(delta_bias, "delta_bias", (dim,), torch.float32, dev)
    if y is None:
        raise ValueError("y (the output) is required")
    _need(y, "y", (batch, seqlen, dim), dt, dev)
    _need(hL, "hL", (batch, dim, dstate), torch.float32, dev)
    plan = ScanPlan(chunk_len, state_split, carry, halves, 0)
    with torch.cuda.device(dev):
        st = lib.ssm_scan_fwd_noalloc(batch, seqlen, dim, dstate, _DTYPES[dt], _ptr(x),
                                      _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                      _ptr(h0), _ptr(y), _ptr(hL),
                                      _options(delta_bias, delta_softplus), ctypes.byref(plan),
                                      _stream(dev))
    _check(st, "ssm_scan_fwd_noalloc")
    return y, hL


def scan_bwd(x, delta, A, B, C, D=None, z=None, h0=None, *, dy, dhL=None, delta_bias=None,
             delta_softplus=False, want_dh0=True, halves=HALVES_AUTO, chunk_len=0):
    """Gradients of sum(dy * y) + sum(dhL * hL) for the scan_fwd call with the
    same inputs. Returns a dict: dx, ddelta, dz (like x, I/O dtype); dB, dC
    (batch, L, N) fp32; dA (dim, N) fp32; dD, ddelta_bias (dim,) fp32; dh0
    (batch, dim, N) fp32. Entries of absent optional inputs are None.
    `halves` is the number of the last channel groups run as two 32-channel
    halves (HALVES_AUTO: the library's choice, HALVES_NONE: none; N 13..16);
    `chunk_len` > 0 (a multiple of 8) cuts the sequence into chunks that run
    in parallel (0: the library's choice)."""
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be (batch, L, dim)")
    batch, seqlen, dim = x.shape
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError("A must be (dim, N)")
    dstate = A.shape[1]
    dev, dt = x.device, x.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported I/O dtype {dt}")
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _need(x, "x", (batch, seqlen, dim), dt, dev)
    _need(delta, "delta", (batch, seqlen, dim), dt, dev)
    _need(A, "A", (dim, dstate), torch.float32, dev)
    _need(B, "B", (batch, seqlen, dstate), dt, dev)
    _need(C, "C", (batch, seqlen, dstate), dt, dev)
    _need(D, "D", (dim,), torch.float32, dev)
    _need(z, "z", (batch, seqlen, dim), dt, dev)
    _need(h0, "h0", (batch, dim, dstate), torch.float32, dev)
    _need(delta_bias, "delta_bias", (dim,), torch.float32, dev)
    _need(dy, "dy", (batch, seqlen, dim), dt, dev)
    _need(dhL, "dhL", (batch, dim, dstate), torch.float32, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    g = dict(dx=torch.empty_like(x), ddelta=torch.empty_like(x),
             dA=torch.empty(dim, dstate, **f32), dB=torch.empty(batch, seqlen, dstate, **f32),
             dC=torch.empty(batch, seqlen, dstate, **f32),
             dD=None if D is None else torch.empty(dim, **f32),
             dz=None if z is None else torch.empty_like(x),
             dh0=torch.empty(batch, dim, dstate, **f32) if want_dh0 else None,
             ddelta_bias=None if delta_bias is None else torch.empty(dim, **f32))
    with torch.cuda.device(dev):
        plan = ScanPlan(chunk_len, 0, 0, halves, 0)
        nbytes = ctypes.c_size_t(0)
        _check(lib.ssm_scan_bwd_workspace_size(batch, seqlen, dim, dstate, _DTYPES[dt],
                                               ctypes.byref(plan), None, ctypes.byref(nbytes)),
               "ssm_scan_bwd_workspace_size")
        ws = _workspace(dev, nbytes.value, "bwd")
        st = lib.ssm_scan_bwd(batch, seqlen, dim, dstate, _DTYPES[dt], _ptr(x), _ptr(delta),
                              _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0),
                              _options(delta_bias, delta_softplus),
                              ctypes.byref(plan), _ptr(dy), _ptr(dhL),
                              _ptr(g["dx"]), _ptr(g["ddelta"]), _ptr(g["dA"]), _ptr(g["dB"]),
                              _ptr(g["dC"]), _ptr(g["dD"]), _ptr(g["dz"]), _ptr(g["dh0"]),
                              _ptr(g["ddelta_bias"]), _ptr(ws), nbytes.value, _stream(dev))
    _check(st, "ssm_scan_bwd")
    return g


def state_update(h, x, delta, A, B, C, D=None, z=None, *, delta_bias=None,
                 delta_softplus=False, out=None):
    """One decode step: h (batch, dim, N) fp32 is updated in place; returns y
    (batch, dim). delta_bias and delta_softplus act as in scan_fwd."""
    lib = load_library()
    if h.dim() != 3:
        raise ValueError("h must be (batch, dim, N)")
    batch, dim, dstate = h.shape
    dev, dt = x.device, x.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported I/O dtype {dt}")
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _need(h, "h", (batch, dim, dstate), torch.float32, dev)
    _need(x, "x", (batch, dim), dt, dev)
    _need(delta, "delta", (batch, dim), dt, dev)
    _need(A, "A", (dim, dstate), torch.float32, dev)
    _need(B, "B", (batch, dstate), dt, dev)
    _need(C, "C", (batch, dstate), dt, dev)
    _need(D, "D", (dim,), torch.float32, dev)
    _need(z, "z", (batch, dim), dt, dev)
    _need(delta_bias, "delta_bias", (dim,), torch.float32, dev)
    y = out if out is not None else torch.empty_like(x)
    _need(y, "out", (batch, dim), dt, dev)
    with torch.cuda.device(dev):
        st = lib.ssm_state_update(batch, dim, dstate, _DTYPES[dt], _ptr(h), _ptr(x), _ptr(delta),
                                  _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(y),
                                  _options(delta_bias, delta_softplus), _stream(dev))
    _check(st, "ssm_state_update")
    return y


def conv1d_fwd(x, weight, bias=None, state_in=None, *, silu=True, return_state=True, out=None,
               state_out=None):
    """Short causal depthwise convolution over whole sequences; returns
    (y, state_out) where state_out (batch, dim, W) holds the last W inputs
    (None when return_state is False). state_in (batch, dim, W), in the dtype
    of x, holds the W inputs before the sequence (None: zeros); state_out may
    be the same tensor."""
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be (batch, L, dim)")
    batch, seqlen, dim = x.shape
    if weight.dim() != 2 or weight.shape[0] != dim:
        raise ValueError("weight must be (dim, W)")
    width = weight.shape[1]
    dev, dt = x.device, x.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported I/O dtype {dt}")
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _need(x, "x", (batch, seqlen, dim), dt, dev)
    _need(weight, "weight", (dim, width), torch.float32, dev)
    _need(bias, "bias", (dim,), torch.float32, dev)
    _need(state_in, "state_in", (batch, dim, width), dt, dev)
    y = out if out is not None else torch.empty_like(x)
    _need(y, "out", (batch, seqlen, dim), dt, dev)
    st = None
    if return_state:
        st = state_out if state_out is not None else torch.empty(batch, dim, width, dtype=dt,
                                                                 device=dev)
        _need(st, "state_out", (batch, dim, width), dt, dev)
    with torch.cuda.device(dev):
        rc = lib.causal_conv1d_fwd(batch, seqlen, dim, width, _DTYPES[dt], _ptr(x), _ptr(weight),
                                   _ptr(bias), _ptr(state_in), _ptr(y), _ptr(st),
                                   1 if silu else 0, _stream(dev))
    _check(rc, "causal_conv1d_fwd")
    return y, st


def conv1d_update(state, x, weight, bias=None, *, silu=True, out=None):
    """One decode step of the convolution: state (batch, dim, W), in the
    dtype of x, is updated in place; returns y (batch, dim)."""
    lib = load_library()
    if state.dim() != 3:
        raise ValueError("state must be (batch, dim, W)")
    batch, dim, width = state.shape
    dev, dt = x.device, x.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported I/O dtype {dt}")
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _need(state, "state", (batch, dim, width), dt, dev)
    _need(x, "x", (batch, dim), dt, dev)
    _need(weight, "weight", (dim, width), torch.float32, dev)
    _need(bias, "bias", (dim,), torch.float32, dev)
    y = out if out is not None else torch.empty_like(x)
    _need(y, "out", (batch, dim), dt, dev)
    with torch.cuda.device(dev):
        rc = lib.causal_conv1d_update(batch, dim, width, _DTYPES[dt], _ptr(state), _ptr(x),
                                      _ptr(weight), _ptr(bias), _ptr(y), 1 if silu else 0,
                                      _stream(dev))
    _check(rc, "causal_conv1d_update")
    return y


SSD_HEADDIM = 64


def ssd_fwd(x, dt, A, B, C, D=None, z=None, h0=None, *, dt_bias=None, dt_softplus=False,
            return_state=True, out=None, state_out=None):
    """Mamba-2 dual form: heads of 64 channels share the step dt (batch, L,
    nheads) and the decay a_h (A: (nheads,) fp32). x, z (batch, L, nheads*64)
    and B, C (batch, L, N) are bf16; N is 64 or 128. Returns (y, hL) with
    hL (batch, nheads, 64, N) fp32 (None when return_state is False)."""
    lib = load_library()
    if x.dim() != 3 or dt.dim() != 3:
        raise ValueError("x must be (batch, L, nheads*64) and dt (batch, L, nheads)")
    batch, seqlen, dim = x.shape
    nheads = dt.shape[2]
    if dim != nheads * SSD_HEADDIM:
        raise ValueError(f"x has {dim} channels, expected nheads*{SSD_HEADDIM}")
    dstate = B.shape[2]
    dev, dtp = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _need(x, "x", (batch, seqlen, dim), dtp, dev)
    _need(dt, "dt", (batch, seqlen, nheads), dtp, dev)
    _need(A, "A", (nheads,), torch.float32, dev)
    _need(B, "B", (batch, seqlen, dstate), dtp, dev)
    _need(C, "C", (batch, seqlen, dstate), dtp, dev)
    _need(D, "D", (dim,), torch.float32, dev)
    _need(z, "z", (batch, seqlen, dim), dtp, dev)
    _need(h0, "h0", (batch, nheads, SSD_HEADDIM, dstate), torch.float32, dev)
    _need(dt_bias, "dt_bias", (nheads,), torch.float32, dev)
    y = out if out is not None else torch.empty_like(x)
    _need(y, "out", (batch, seqlen, dim), dtp, dev)
    hL = None
    if return_state:
        hL = state_out if state_out is not None else torch.empty(
            batch, nheads, SSD_HEADDIM, dstate, dtype=torch.float32, device=dev)
        _need(hL, "state_out", (batch, nheads, SSD_HEADDIM, dstate), torch.float32, dev)
    with torch.cuda.device(dev):
        st = lib.ssd_fwd(batch, seqlen, nheads, SSD_HEADDIM, dstate, _DTYPES.get(dtp, -1),
                         _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                         _ptr(h0), _ptr(y), _ptr(hL), _options(dt_bias, dt_softplus),
                         _stream(dev))
    _check(st, "ssd_fwd")
    return y, hL


def _require(t, name, shape, dtype, dev):
    """The address of a tensor that _need accepts; None for None. The cheap
    test comes first, _need says what is wrong."""
    if t is None:
        return None
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev.index
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, shape, dtype, dev)
    return t.data_ptr()


def _must(t, name, shape, dtype, dev):
    if t is None:
        raise ValueError(f"{name} is required")
    return _require(t, name, shape, dtype, dev)


def _output(t, name, shape, dtype, dev):
    """The caller's tensor for an output, or a new one, and its address."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=dev)
        return t, t.data_ptr()
    return t, _require(t, name, shape, dtype, dev)


def _output_like(t, name, x, dtype, dev):
    """_output for one of an input's shape and dtype: dense, and quicker made from an
    input that is."""
    if t is None and x.is_contiguous():
        t = torch.empty_like(x)
        return t, t.data_ptr()
    return _output(t, name, x.shape, dtype, dev)


class _Stay:
    """The device that is current already."""

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_STAY = _Stay()
_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(dev):
    """The tensors' device made current for a call, if it is not already."""
    return _STAY if _device_now() == dev.index else torch.cuda.device(dev)


# the current stream's handle, without the object around it where torch has a
# function for that
_raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(dev):
    if _raw_stream_of is not None:
        return _raw_stream_of(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _scratch(dev, nbytes):
    """Scratch of one call, from torch's allocator on the current stream: a
    captured graph keeps its own, and calls on different streams share none."""
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


def _attn_shapes(q, k, v, ndim):
    """(batch, L, heads, kv_heads, dk, dv) of q, k and v and their addresses,
    checked against each other; L is 1 for single tokens (ndim 3). The cheap
    test comes first, _attn_checked says what is wrong."""
    try:
        if ndim == 4:
            batch, seqlen, heads, dk = q.shape
            kb, kl, kv_heads, kd = k.shape
            vb, vl, vh, dv = v.shape
        else:
            (batch, heads, dk), (kb, kv_heads, kd), (vb, vh, dv) = q.shape, k.shape, v.shape
            seqlen = kl = vl = 1
        dt, index = q.dtype, q.get_device()
        if (kb == batch == vb and kl == seqlen == vl and kd == dk and kv_heads == vh > 0
                and heads % vh == 0 and dt in _DTYPES and k.dtype is dt and v.dtype is dt
                and index >= 0 and k.get_device() == index and v.get_device() == index
                and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
            return ((batch, seqlen, heads, kv_heads, dk, dv),
                    (q.data_ptr(), k.data_ptr(), v.data_ptr()))
    except (AttributeError, ValueError, TypeError):
        pass
    return _attn_checked(q, k, v, ndim)


def _attn_checked(q, k, v, ndim):
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != ndim:
            raise ValueError(f"{name} must be (batch, {'L, ' if ndim == 4 else ''}heads, size)")
    dev, dt = q.device, q.dtype
    if ndim == 4:
        batch, seqlen, heads, dk = q.shape
        kv_heads, dv = v.shape[2], v.shape[3]
        kv = (batch, seqlen, kv_heads)
    else:
        batch, heads, dk = q.shape
        seqlen = 1
        kv_heads, dv = v.shape[1], v.shape[2]
        kv = (batch, kv_heads)
    if heads % kv_heads if kv_heads else heads:
        raise ValueError(f"q has {heads} heads, not a multiple of the {kv_heads} of k and v")
    if dt not in _DTYPES:
        raise ValueError(f"unsupported I/O dtype {dt}")
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    addresses = (_require(q, "q", q.shape, dt, dev), _require(k, "k", (*kv, dk), dt, dev),
                 _require(v, "v", (*kv, dv), dt, dev))
    return (batch, seqlen, heads, kv_heads, dk, dv), addresses


@functools.lru_cache(maxsize=1024)
def _scratch_bytes(call, index, *sizes):
    """Scratch bytes of a call: a function of its sizes and the GPU's kind."""
    nbytes = ctypes.c_size_t(0)
    _check(getattr(load_library(), call)(*sizes, ctypes.byref(nbytes)), call)
    return nbytes.value


def linear_attn_fwd(q, k, v, log_decay, h0=None, *, lengths=None, scale=None, return_state=True,
                    out=None, state_out=None, segment_len=0):
    """Linear attention with a decay exp(log_decay[h]) for each head over whole
    sequences: S_t = decay S_(t-1) + k_t^T v_t, o_t = scale q_t S_t. q (batch, L,
    heads, dk); k, v (batch, L, kv_heads, dk or dv), each shared by heads /
    kv_heads heads; `lengths` (batch,) int32 the tokens of each row (None: L),
    behind which o is zero; h0 (batch, heads, dk, dv) fp32; `scale` dk ** -0.5
    by default. Returns (o, hL), hL (None when return_state is False) the state
    after each row's last token; state_out may be h0. `segment_len` > 0 (a
    multiple of 64) forces the parallel segments' length."""
    lib = load_library()
    sizes, (pq, pk, pv) = _attn_shapes(q, k, v, 4)
    batch, seqlen, heads, _, dk, dv = sizes
    dev, dt = q.device, q.dtype
    state = (batch, heads, dk, dv)
    pg = _must(log_decay, "log_decay", (heads,), torch.float32, dev)
    p0 = _require(h0, "h0", state, torch.float32, dev)
    pl = _require(lengths, "lengths", (batch,), torch.int32, dev)
    o, po = _output(out, "out", (batch, seqlen, heads, dv), dt, dev)
    hL = ph = None
    if return_state:
        hL, ph = _output(state_out, "state_out", state, torch.float32, dev)
    code = _DTYPES[dt]
    with _on(dev):
        nbytes = _scratch_bytes("linear_attn_fwd_workspace_size", dev.index, *sizes, code,
                                segment_len)
        ws = _scratch(dev, nbytes)
        st = lib.linear_attn_fwd(*sizes, code, pq, pk, pv, pg, pl, p0,
                                 dk ** -0.5 if scale is None else scale, po, ph, segment_len,
                                 None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev))
    if st:
        _check(st, "linear_attn_fwd")
    return o, hL


def linear_attn_bwd(q, k, v, log_decay, h0=None, *, do, dhL=None, lengths=None, scale=None,
                    want_dlog_decay=True, want_dh0=True, segment_len=0):
    """Gradients of sum(do * o) + sum(dhL * hL) for the linear_attn_fwd call
    with the same inputs. Returns a dict: dq, dk, dv (like q, k, v; zero behind
    a row's length); dlog_decay (heads,) fp32 and dh0 (batch, heads, dk, dv)
    fp32, None when not wanted."""
    lib = load_library()
    sizes, (pq, pk, pv) = _attn_shapes(q, k, v, 4)
    batch, seqlen, heads, _, dk, dv = sizes
    dev, dt = q.device, q.dtype
    state = (batch, heads, dk, dv)
    pg = _must(log_decay, "log_decay", (heads,), torch.float32, dev)
    p0 = _require(h0, "h0", state, torch.float32, dev)
    pl = _require(lengths, "lengths", (batch,), torch.int32, dev)
    pdo = _must(do, "do", (batch, seqlen, heads, dv), dt, dev)
    pdh = _require(dhL, "dhL", state, torch.float32, dev)
    g = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
             dlog_decay=(torch.empty(heads, dtype=torch.float32, device=dev) if want_dlog_decay
                         else None),
             dh0=torch.empty(state, dtype=torch.float32, device=dev) if want_dh0 else None)
    code = _DTYPES[dt]
    with _on(dev):
        nbytes = _scratch_bytes("linear_attn_bwd_workspace_size", dev.index, *sizes, code,
                                segment_len)
        ws = _scratch(dev, nbytes)
        st = lib.linear_attn_bwd(*sizes, code, pq, pk, pv, pg, pl, p0,
                                 dk ** -0.5 if scale is None else scale, pdo, pdh,
                                 *(None if t is None else t.data_ptr() for t in g.values()),
                                 segment_len, None if ws is None else ws.data_ptr(), nbytes,
                                 _raw_stream(dev))
    if st:
        _check(st, "linear_attn_bwd")
    return g


def linear_attn_update(h, q, k, v, log_decay, *, scale=None, out=None):
    """One token of linear attention: h (batch, heads, dk, dv) fp32 is updated
    in place; q (batch, heads, dk), k, v (batch, kv_heads, dk or dv); returns o
    (batch, heads, dv)."""
    lib = load_library()
    (batch, _, heads, kv_heads, dk, dv), (pq, pk, pv) = _attn_shapes(q, k, v, 3)
    dev, dt = q.device, q.dtype
    ph = _must(h, "h", (batch, heads, dk, dv), torch.float32, dev)
    pg = _must(log_decay, "log_decay", (heads,), torch.float32, dev)
    o, po = _output(out, "out", (batch, heads, dv), dt, dev)
    with _on(dev):
        st = lib.linear_attn_update(batch, heads, kv_heads, dk, dv, _DTYPES[dt], ph, pq, pk, pv, pg,
                                    dk ** -0.5 if scale is None else scale, po, _raw_stream(dev))
    if st:
        _check(st, "linear_attn_update")
    return o


def _norm_shapes(x, groups):
    """(rows, dim) of x, and its address. The cheap test comes first,
    _norm_checked says what is wrong."""
    try:
        dim = x.shape[-1]
        if (groups > 0 and dim > 0 and dim % groups == 0 and x.dtype in _DTYPES
                and x.get_device() >= 0 and x.is_contiguous()):
            return x.numel() // dim, dim, x.data_ptr()
    except (AttributeError, IndexError, TypeError):
        pass
    return _norm_checked(x, groups)


def _norm_checked(x, groups):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() < 1:
        raise ValueError("x must be (..., dim)")
    dim = x.shape[-1]
    if groups < 1 or dim % groups or dim == 0:
        raise ValueError(f"{dim} channels do not split into {groups} groups")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported I/O dtype {x.dtype}")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    return x.numel() // dim, dim, _require(x, "x", x.shape, x.dtype, dev)


def layer_norm_fwd(x, weight=None, bias=None, *, groups=1, eps=1e-5, out=None):
    """Layer norm over each of the `groups` equal parts of the last dimension:
    y = (x - mean) * rstd * weight + bias with rstd = (var + eps) ** -0.5.
    weight and bias (dim,) fp32. Returns (y, mean, rstd), mean and rstd
    (..., groups) fp32, which layer_norm_bwd takes; out may be x."""
    lib = load_library()
    rows, dim, px = _norm_shapes(x, groups)
    dev, dt = x.device, x.dtype
    pw = _require(weight, "weight", (dim,), torch.float32, dev)
    pb = _require(bias, "bias", (dim,), torch.float32, dev)
    y, py = _output(out, "out", x.shape, dt, dev)
    mean = torch.empty((*x.shape[:-1], groups), dtype=torch.float32, device=dev)
    rstd = torch.empty_like(mean)
    with _on(dev):
        st = lib.layer_norm_fwd(rows, dim, groups, _DTYPES[dt], px, pw, pb, eps, py, mean.data_ptr(),
                                rstd.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "layer_norm_fwd")
    return y, mean, rstd


def layer_norm_bwd(x, weight, mean, rstd, *, dy, groups=1, want_dbias=True, out=None):
    """Gradients of sum(dy * y) for the layer_norm_fwd call with the same x and
    weight, mean and rstd from it. Returns a dict: dx (like x; out may be dy),
    dweight (dim,) fp32 (None without a weight) and dbias (dim,) fp32 (None
    when not wanted)."""
    lib = load_library()
    rows, dim, px = _norm_shapes(x, groups)
    dev, dt = x.device, x.dtype
    stats = (*x.shape[:-1], groups)
    pw = _require(weight, "weight", (dim,), torch.float32, dev)
    pm = _must(mean, "mean", stats, torch.float32, dev)
    pr = _must(rstd, "rstd", stats, torch.float32, dev)
    pdy = _must(dy, "dy", x.shape, dt, dev)
    dx, pdx = _output(out, "out", x.shape, dt, dev)
    dw = None if weight is None else torch.empty(dim, dtype=torch.float32, device=dev)
    db = torch.empty(dim, dtype=torch.float32, device=dev) if want_dbias else None
    code = _DTYPES[dt]
    with _on(dev):
        nbytes = _scratch_bytes("layer_norm_bwd_workspace_size", dev.index, rows, dim, groups, code)
        ws = _scratch(dev, nbytes)
        st = lib.layer_norm_bwd(rows, dim, groups, code, px, pw, pm, pr, pdy, pdx,
                                None if dw is None else dw.data_ptr(),
                                None if db is None else db.data_ptr(),
                                None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev))
    if st:
        _check(st, "layer_norm_bwd")
    return dict(dx=dx, dweight=dw, dbias=db)


def _rows(t, name, shape, dtype, dev):
    """The address of an input and the elements between its rows of channels: a
    dense tensor, or a slice of a wider one's channels. The cheap test comes
    first, _rows_checked says what is wrong."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev.index
                and t.is_contiguous()):
            return t.data_ptr(), shape[-1]
    except AttributeError:
        pass
    return _rows_checked(t, name, shape, dtype, dev)


def _rows_checked(t, name, shape, dtype, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape or t.dtype is not dtype or t.device != dev:
        _need(t, name, shape, dtype, dev)
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.numel() == 0:
        return t.data_ptr(), shape[-1]
    at, step, size = t.stride(), None, 1
    for n, stride in zip(reversed(shape[:-1]), reversed(at[:-1])):
        if n != 1:
            if step is None:
                step = stride // size if stride % size == 0 else -1
            if stride != step * size:
                step = -1
            if step < shape[-1]:
                break
        size *= n
    step = shape[-1] if step is None else step
    if (at[-1] != 1 and shape[-1] != 1) or step < shape[-1]:
        raise ValueError(f"{name}: rows of neighbouring channels a fixed stride apart are needed, "
                         f"strides are {at}")
    return t.data_ptr(), step


def _gated_shape(x, ndim):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() != ndim:
        raise ValueError(f"x must be (batch, {'L, ' if ndim == 3 else ''}dim)")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported I/O dtype {x.dtype}")
    if x.device.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    return x.shape


def _gates(x, decay_gate, log_decay, input_gate, shape, dt, dev):
    """The arguments of a recurrence that its three calls share."""
    i = (None, 0) if input_gate is None else _rows(input_gate, "input_gate", shape, dt, dev)
    return (*_rows(x, "x", shape, dt, dev), *_rows(decay_gate, "decay_gate", shape, dt, dev),
            _must(log_decay, "log_decay", shape[-1:], torch.float32, dev), *i)


def gated_scan_fwd(x, decay_gate, log_decay, input_gate=None, h0=None, *, lengths=None,
                   return_state=True, return_block_states=False, out=None, state_out=None):
    """Gated linear recurrence over whole sequences: h_t = a_t h_(t-1) + sqrt(1 -
    a_t^2) sigmoid(input_gate_t) x_t with a_t = exp(log_decay sigmoid(decay_gate_t)).
    x and the gates (batch, L, dim), input_gate None: 1; log_decay (dim,) fp32,
    <= 0; h0 (batch, dim) fp32; `lengths` (batch,) int32 the tokens of each row
    (None: L), behind which y is zero. Returns (y, hL, block_states): y the states
    in the dtype of x, hL (batch, dim) fp32 the one after each row's last token (None
    when return_state is False; state_out may be h0), block_states (batch, ceil(L /
    64), dim) fp32 those entering every 64 tokens, which gated_scan_bwd takes (None
    unless wanted)."""
    lib = load_library()
    shape = _gated_shape(x, 3)
    batch, seqlen, dim = shape
    dev, dt = x.device, x.dtype
    gates = _gates(x, decay_gate, log_decay, input_gate, shape, dt, dev)
    pl = _require(lengths, "lengths", (batch,), torch.int32, dev)
    p0 = _require(h0, "h0", (batch, dim), torch.float32, dev)
    y, py = _output_like(out, "out", x, dt, dev)
    hL = ph = states = ps = None
    if return_state:
        hL, ph = _output(state_out, "state_out", (batch, dim), torch.float32, dev)
    if return_block_states:
        states, ps = _output(None, "block_states", (batch, -(-seqlen // GATED_SCAN_BLOCK), dim),
                             torch.float32, dev)
    code = _DTYPES[dt]
    with _on(dev):
        nbytes = _scratch_bytes("gated_scan_fwd_workspace_size", dev.index, batch, seqlen, dim, code)
        ws = _scratch(dev, nbytes)
        st = lib.gated_scan_fwd(batch, seqlen, dim, code, *gates, pl, p0, py, ph, ps,
                                None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev))
    if st:
        _check(st, "gated_scan_fwd")
    return y, hL, states


def gated_scan_bwd(x, decay_gate, log_decay, input_gate=None, *, block_states, dy, dhL=None,
                   lengths=None, want_dlog_decay=True, want_dh0=True):
    """Gradients of sum(dy * y) + sum(dhL * hL) for the gated_scan_fwd call with the
    same inputs, block_states from it. Returns a dict: dx, ddecay_gate, dinput_gate
    (like x; zero behind a row's length; dinput_gate None without an input gate),
    dlog_decay (dim,) fp32 and dh0 (batch, dim) fp32, None when not wanted."""
    lib = load_library()
    shape = _gated_shape(x, 3)
    batch, seqlen, dim = shape
    dev, dt = x.device, x.dtype
    gates = _gates(x, decay_gate, log_decay, input_gate, shape, dt, dev)
    pl = _require(lengths, "lengths", (batch,), torch.int32, dev)
    ps = _must(block_states, "block_states", (batch, -(-seqlen // GATED_SCAN_BLOCK), dim),
               torch.float32, dev)
    pdy = _must(dy, "dy", shape, dt, dev)
    pdh = _require(dhL, "dhL", (batch, dim), torch.float32, dev)

    like = torch.empty_like   # dense, as dy and log_decay are
    g = dict(dx=like(dy), ddecay_gate=like(dy), dinput_gate=None if input_gate is None else like(dy),
             dlog_decay=like(log_decay) if want_dlog_decay else None,
             dh0=torch.empty((batch, dim), dtype=torch.float32, device=dev) if want_dh0 else None)
    code = _DTYPES[dt]
    with _on(dev):
        nbytes = _scratch_bytes("gated_scan_bwd_workspace_size", dev.index, batch, seqlen, dim, code)
        ws = _scratch(dev, nbytes)
        st = lib.gated_scan_bwd(batch, seqlen, dim, code, *gates, pl, ps, pdy, pdh,
                                *(None if t is None else t.data_ptr() for t in g.values()),
                                None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev))
    if st:
        _check(st, "gated_scan_bwd")
    return g


def gated_scan_update(h, x, decay_gate, log_decay, input_gate=None, *, out=None):
    """One token of the gated recurrence: h (batch, dim) fp32 is updated in place;
    x and the gates (batch, dim); returns y (batch, dim), the new state in the dtype
    of x."""
    lib = load_library()
    shape = _gated_shape(x, 2)
    dev, dt = x.device, x.dtype
    gates = _gates(x, decay_gate, log_decay, input_gate, shape, dt, dev)
    ph = _must(h, "h", shape, torch.float32, dev)
    y, py = _output_like(out, "out", x, dt, dev)
    with _on(dev):
        st = lib.gated_scan_update(*shape, _DTYPES[dt], ph, *gates, py, _raw_stream(dev))
    if st:
        _check(st, "gated_scan_update")
    return y


def _norm_rows(x, groups):
    """(rows, dim) of a norm's input, whose rows may be a stride apart."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() < 1:
        raise ValueError("x must be (..., dim)")
    dim = x.shape[-1]
    if groups < 1 or dim == 0 or dim % groups:
        raise ValueError(f"{dim} channels do not split into {groups} groups")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported I/O dtype {x.dtype}")
    if x.device.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    return x.numel() // dim, dim


def _gate_code(z, gate_first):
    return 0 if z is None else 1 if gate_first else 2   # mamba_norm_gate


def gated_norm_fwd(x, z=None, weight=None, *, groups=1, eps=1e-5, gate_first=True, out=None):
    """The norm behind a block with its gate, over each of the `groups` equal parts
    of the last dimension: y = v * rstd * weight with v = x * silu(z) and rstd =
    (mean(v^2) + eps) ** -0.5; with gate_first False v = x and y = v * rstd * weight *
    silu(z); without z no gate. weight (dim,) fp32. Returns (y, rstd), rstd (...,
    groups) fp32, which gated_norm_bwd takes; out may be x or z where that is
    dense."""
    lib = load_library()
    rows, dim = _norm_rows(x, groups)
    dev, dt, shape = x.device, x.dtype, x.shape
    px = _rows(x, "x", shape, dt, dev)
    pz = (None, 0) if z is None else _rows(z, "z", shape, dt, dev)
    pw = _require(weight, "weight", (dim,), torch.float32, dev)
    y, py = _output_like(out, "out", x, dt, dev)
    rstd = torch.empty((*shape[:-1], groups), dtype=torch.float32, device=dev)
    with _on(dev):
        st = lib.gated_norm_fwd(rows, dim, groups, _DTYPES[dt], _gate_code(z, gate_first), *px, *pz,
                                pw, eps, py, rstd.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "gated_norm_fwd")
    return y, rstd


def gated_norm_bwd(x, z, weight, rstd, *, dy, groups=1, gate_first=True, out=None):
    """Gradients of sum(dy * y) for the gated_norm_fwd call with the same x, z and
    weight, rstd from it. Returns a dict: dx (like x; out may be dy), dz (None without
    z) and dweight (dim,) fp32 (None without a weight)."""
    lib = load_library()
    rows, dim = _norm_rows(x, groups)
    dev, dt, shape = x.device, x.dtype, x.shape
    px = _rows(x, "x", shape, dt, dev)
    pz = (None, 0) if z is None else _rows(z, "z", shape, dt, dev)
    pw = _require(weight, "weight", (dim,), torch.float32, dev)
    pr = _must(rstd, "rstd", (*shape[:-1], groups), torch.float32, dev)
    pdy = _must(dy, "dy", shape, dt, dev)
    dx, pdx = _output_like(out, "out", x, dt, dev)
    dz = None if z is None else torch.empty_like(dy)   # dense, as dy is
    dw = None if weight is None else torch.empty_like(weight)
    code = _DTYPES[dt]
    with _on(dev):
        nbytes = 0
        if dw is not None:
            nbytes = _scratch_bytes("gated_norm_bwd_workspace_size", dev.index, rows, dim, groups, code)
        ws = _scratch(dev, nbytes)
        st = lib.gated_norm_bwd(rows, dim, groups, code, _gate_code(z, gate_first), *px, *pz, pw, pr,
                                pdy, pdx, None if dz is None else dz.data_ptr(),
                                None if dw is None else dw.data_ptr(),
                                None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev))
    if st:
        _check(st, "gated_norm_bwd")
    return dict(dx=dx, dz=dz, dweight=dw)


def _stream_dtype(t, name, dt):
    """The dtype code of the residual stream: the I/O dtype or fp32."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dt and t.dtype is not torch.float32:
        raise ValueError(f"{name} must be {dt} or torch.float32, is {t.dtype}")
    return t.dtype


def residual_norm_fwd(x, residual, scale=None, weight=None, *, eps=1e-5, out=None, total_out=None):
    """The norm before a block with the residual sum: total = residual + scale * x,
    y = total * rstd * weight with rstd = (mean(total^2) + eps) ** -0.5 over the last
    dimension. residual (..., dim) in the dtype of x or fp32; scale and weight (dim,)
    fp32, None: ones. Returns (y, total, rstd): y in the dtype of x, total in that of
    residual, rstd (..., 1) fp32; residual_norm_bwd takes the last two. out may be x,
    total_out residual."""
    lib = load_library()
    rows, dim = _norm_rows(x, 1)
    dev, dt, shape = x.device, x.dtype, x.shape
    px = _must(x, "x", shape, dt, dev)
    rt = _stream_dtype(residual, "residual", dt)
    pres = _must(residual, "residual", shape, rt, dev)
    psc = _require(scale, "scale", (dim,), torch.float32, dev)
    pw = _require(weight, "weight", (dim,), torch.float32, dev)
    y, py = _output_like(out, "out", x, dt, dev)
    total, pt = _output_like(total_out, "total_out", residual, rt, dev)
    rstd = torch.empty((*shape[:-1], 1), dtype=torch.float32, device=dev)
    with _on(dev):
        st = lib.residual_norm_fwd(rows, dim, _DTYPES[dt], _DTYPES[rt], px, pres, psc, pw, eps, py, pt,
                                   rstd.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "residual_norm_fwd")
    return y, total, rstd


def residual_norm_bwd(total, weight, rstd, x=None, scale=None, *, dy, dtotal=None):
    """Gradients of sum(dy * y) + sum(dtotal * total) for the residual_norm_fwd call
    that gave total and rstd; x and scale as given to it (x is looked at with a scale
    only). Returns a dict: dx (like dy), dresidual (like total), dscale (dim,) fp32
    (None without a scale) and dweight (dim,) fp32 (None without a weight). Without a
    scale and with a total in the dtype of dy, dx is dresidual, the same tensor."""
    lib = load_library()
    rows, dim = _norm_rows(dy, 1)
    dev, dt, shape = dy.device, dy.dtype, dy.shape
    pdy = _must(dy, "dy", shape, dt, dev)
    rt = _stream_dtype(total, "total", dt)
    pt = _must(total, "total", shape, rt, dev)
    pw = _require(weight, "weight", (dim,), torch.float32, dev)
    pr = _must(rstd, "rstd", (*shape[:-1], 1), torch.float32, dev)
    psc = _require(scale, "scale", (dim,), torch.float32, dev)
    px = None if scale is None else _must(x, "x", shape, dt, dev)
    pdt = _require(dtotal, "dtotal", shape, rt, dev)
    dres = torch.empty_like(total)   # dense, as total is
    dx = dres if scale is None and rt is dt else torch.empty_like(dy)
    dsc = None if scale is None else torch.empty_like(scale)
    dw = None if weight is None else torch.empty_like(weight)
    codes = _DTYPES[dt], _DTYPES[rt]
    with _on(dev):
        nbytes = 0
        if dsc is not None or dw is not None:
            nbytes = _scratch_bytes("residual_norm_bwd_workspace_size", dev.index, rows, dim, *codes)
        ws = _scratch(dev, nbytes)
        st = lib.residual_norm_bwd(rows, dim, *codes, pt, pw, pr, px, psc, pdy, pdt,
                                   None if dx is dres else dx.data_ptr(), dres.data_ptr(),
                                   None if dsc is None else dsc.data_ptr(),
                                   None if dw is None else dw.data_ptr(),
                                   None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev))
    if st:
        _check(st, "residual_norm_bwd")
    return dict(dx=dx, dresidual=dres, dscale=dsc, dweight=dw)
