"""The gated block's C ABI on the host, without a GPU: exports of
include/mamba_gated.h, and every refusal with its documented status before any HIP
call. Also the binding's own argument checks."""
import ctypes
import os
import re

import pytest
import torch

import selective_state_space_40_amd as ms

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "mamba_gated.h")

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, -1, -2, -3, -4

# fake device addresses: never dereferenced, every call below is refused or a
# no-op before any HIP call
P = ctypes.c_void_p(0x10000)
PM = ctypes.c_void_p(0x10008)   # not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    return ms.load_library()


def test_library_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^int\s+(\w+)\s*\(", text, flags=re.M)))
    assert names == ["gated_norm_bwd", "gated_norm_bwd_workspace_size", "gated_norm_fwd", "gated_scan_bwd",
                     "gated_scan_bwd_workspace_size", "gated_scan_fwd", "gated_scan_fwd_workspace_size",
                     "gated_scan_update", "residual_norm_bwd", "residual_norm_bwd_workspace_size",
                     "residual_norm_fwd"]
    for n in names:
        assert hasattr(lib, n), n


def _inputs(p, dim, strides):
    s = dict(x=dim, decay_gate=dim, input_gate=dim)
    s.update(strides or {})
    return [p["x"], s["x"], p["decay_gate"], s["decay_gate"], p["log_decay"], p["input_gate"], s["input_gate"]]


def _fwd(lib, batch=2, seqlen=64, dim=64, dtype=1, ptrs=None, strides=None, ws=P, wsb=1 << 40):
    p = dict(x=P, decay_gate=P, log_decay=P, input_gate=P, lengths=None, h0=None, y=P, hL=P, states=None)
    p.update(ptrs or {})
    return lib.gated_scan_fwd(batch, seqlen, dim, dtype, *_inputs(p, dim, strides), p["lengths"], p["h0"], p["y"],
                              p["hL"], p["states"], ws, wsb, None)


def _bwd(lib, batch=2, seqlen=64, dim=64, dtype=1, ptrs=None, strides=None, ws=P, wsb=1 << 40):
    p = dict(x=P, decay_gate=P, log_decay=P, input_gate=P, lengths=None, states=P, dy=P, dhL=None, dx=P, ddecay=P,
             dinput=P, dlog_decay=P, dh0=P)
    p.update(ptrs or {})
    return lib.gated_scan_bwd(batch, seqlen, dim, dtype, *_inputs(p, dim, strides), p["lengths"], p["states"],
                              p["dy"], p["dhL"], p["dx"], p["ddecay"], p["dinput"], p["dlog_decay"], p["dh0"], ws,
                              wsb, None)


def _update(lib, batch=2, dim=64, dtype=1, ptrs=None, strides=None, **_):
    p = dict(h=P, x=P, decay_gate=P, log_decay=P, input_gate=P, y=P)
    p.update(ptrs or {})
    return lib.gated_scan_update(batch, dim, dtype, p["h"], *_inputs(p, dim, strides), p["y"], None)


def test_scan_refuses_bad_shapes(lib):
    for call in (_fwd, _bwd, _update):
        assert call(lib, batch=-1) == INVALID
        assert call(lib, dim=-1) == INVALID
        assert call(lib, dtype=2) == INVALID
        assert call(lib, dtype=-1) == INVALID
        assert call(lib, dim=(1 << 20) + 1) == UNSUPPORTED
        assert call(lib, batch=1 << 40) == UNSUPPORTED
        assert call(lib, batch=1 << 14, dim=1 << 20) == UNSUPPORTED    # more threads than a launch counts
        for name in ("x", "decay_gate", "input_gate"):
            assert call(lib, strides={name: 63}) == INVALID, name
            assert call(lib, strides={name: (1 << 20) + 1}) == UNSUPPORTED, name
        assert call(lib, ptrs=dict(x=None), strides=dict(x=1)) == INVALID
    for call in (_fwd, _bwd):
        assert call(lib, seqlen=-1) == INVALID
        assert call(lib, seqlen=1 << 40) == UNSUPPORTED
        assert call(lib, batch=1 << 16, seqlen=1 << 20, dim=1) == UNSUPPORTED
    need = ctypes.c_size_t(0)
    for size in (lib.gated_scan_fwd_workspace_size, lib.gated_scan_bwd_workspace_size):
        assert size(2, 64, 64, 1, None) == INVALID
        assert size(-1, 64, 64, 1, ctypes.byref(need)) == INVALID
        assert size(2, 64, 1 << 21, 1, ctypes.byref(need)) == UNSUPPORTED


def test_scan_refuses_null_and_misaligned(lib):
    for name in ("x", "decay_gate", "log_decay", "y"):
        assert _fwd(lib, ptrs={name: None}) == INVALID, name
    for name in ("x", "decay_gate", "log_decay", "input_gate", "lengths", "h0", "y", "hL", "states"):
        assert _fwd(lib, ptrs={name: PM}) == MISALIGNED, name
    for name in ("x", "decay_gate", "log_decay", "states", "dy", "dx", "ddecay", "dinput"):
        assert _bwd(lib, ptrs={name: None}) == INVALID, name
    for name in ("x", "decay_gate", "log_decay", "input_gate", "lengths", "states", "dy", "dhL", "dx", "ddecay",
                 "dinput", "dlog_decay", "dh0"):
        assert _bwd(lib, ptrs={name: PM}) == MISALIGNED, name
    for name in ("h", "x", "decay_gate", "log_decay", "y"):
        assert _update(lib, ptrs={name: None}) == INVALID, name
    for name in ("h", "x", "decay_gate", "log_decay", "input_gate", "y"):
        assert _update(lib, ptrs={name: PM}) == MISALIGNED, name
    assert _fwd(lib, ws=PM) == MISALIGNED and _bwd(lib, ws=PM) == MISALIGNED


def test_scan_no_ops(lib):
    none = dict(x=None, decay_gate=None, log_decay=None, input_gate=None)
    assert _fwd(lib, batch=0, ptrs=none) == OK
    assert _fwd(lib, dim=0, ptrs=none) == OK
    assert _fwd(lib, seqlen=0, ptrs=dict(none, y=None, hL=None)) == OK
    assert _bwd(lib, dim=0, ptrs=none) == OK
    assert _bwd(lib, batch=0, ptrs=dict(none, dlog_decay=None, dh0=None)) == OK
    assert _update(lib, batch=0, ptrs=none) == OK


def _norm(lib, rows=4, dim=64, groups=1, dtype=1, gate=1, eps=1e-5, ptrs=None, xs=None, zs=None):
    p = dict(x=P, z=P, weight=None, y=P, rstd=P)
    p.update(ptrs or {})
    return lib.gated_norm_fwd(rows, dim, groups, dtype, gate, p["x"], dim if xs is None else xs, p["z"],
                              dim if zs is None else zs, p["weight"], eps, p["y"], p["rstd"], None)


def _norm_bwd(lib, rows=4, dim=64, groups=1, dtype=1, gate=1, ptrs=None, xs=None, zs=None, **_):
    p = dict(x=P, z=P, weight=None, rstd=P, dy=P, dx=P, dz=P, dweight=None)
    p.update(ptrs or {})
    return lib.gated_norm_bwd(rows, dim, groups, dtype, gate, p["x"], dim if xs is None else xs, p["z"],
                              dim if zs is None else zs, p["weight"], p["rstd"], p["dy"], p["dx"], p["dz"],
                              p["dweight"], None, 0, None)


def test_gated_norm_refuses_bad_arguments(lib):
    for call in (_norm, _norm_bwd):
        assert call(lib, rows=-1) == INVALID
        assert call(lib, dim=-4) == INVALID
        assert call(lib, groups=0) == INVALID
        assert call(lib, groups=3) == INVALID
        assert call(lib, dtype=9) == INVALID
        assert call(lib, gate=3) == INVALID
        assert call(lib, gate=-1) == INVALID
        assert call(lib, dim=16385) == UNSUPPORTED
        assert call(lib, rows=1 << 40) == UNSUPPORTED
        assert call(lib, dim=1 << 28, groups=1 << 16) == UNSUPPORTED
        assert call(lib, rows=1 << 30, dim=64, groups=64) == UNSUPPORTED
        assert call(lib, xs=63) == INVALID and call(lib, zs=63) == INVALID
        assert call(lib, xs=(1 << 27) + 1) == UNSUPPORTED and call(lib, zs=(1 << 27) + 1) == UNSUPPORTED
        for name in ("x", "z"):
            assert call(lib, ptrs={name: None}) == INVALID, name
    for eps in (-1.0, float("nan"), float("inf")):
        assert _norm(lib, eps=eps) == INVALID
    assert _norm(lib, ptrs=dict(y=None)) == INVALID
    for name in ("x", "z", "weight", "y", "rstd"):
        assert _norm(lib, ptrs={name: PM}) == MISALIGNED, name
    for name in ("rstd", "dy", "dx", "dz"):
        assert _norm_bwd(lib, ptrs={name: None}) == INVALID, name
    for name in ("x", "z", "weight", "rstd", "dy", "dx", "dz", "dweight"):
        assert _norm_bwd(lib, ptrs={name: PM}) == MISALIGNED, name
    assert lib.gated_norm_bwd_workspace_size(4, 64, 1, 1, None) == INVALID
    none = dict(x=None, z=None, y=None, rstd=None, dy=None, dx=None, dz=None)
    for call in (_norm, _norm_bwd):
        assert call(lib, rows=0, ptrs=none) == OK
        assert call(lib, dim=0, ptrs=none) == OK


def _res(lib, rows=4, dim=64, dtype=1, total=0, eps=1e-5, ptrs=None):
    p = dict(x=P, residual=P, scale=None, weight=None, y=P, total=P, rstd=P)
    p.update(ptrs or {})
    return lib.residual_norm_fwd(rows, dim, dtype, total, p["x"], p["residual"], p["scale"], p["weight"], eps,
                                 p["y"], p["total"], p["rstd"], None)


def _res_bwd(lib, rows=4, dim=64, dtype=1, total=0, ptrs=None, **_):
    p = dict(total=P, weight=None, rstd=P, x=P, scale=None, dy=P, dtotal=None, dx=P, dresidual=P, dscale=None,
             dweight=None)
    p.update(ptrs or {})
    return lib.residual_norm_bwd(rows, dim, dtype, total, p["total"], p["weight"], p["rstd"], p["x"], p["scale"],
                                 p["dy"], p["dtotal"], p["dx"], p["dresidual"], p["dscale"], p["dweight"], None, 0,
                                 None)


def test_residual_norm_refuses_bad_arguments(lib):
    for call in (_res, _res_bwd):
        assert call(lib, rows=-1) == INVALID
        assert call(lib, dim=-4) == INVALID
        assert call(lib, dtype=9) == INVALID
        assert call(lib, total=9) == INVALID
        assert call(lib, dtype=0, total=1) == UNSUPPORTED      # a stream of fewer bits than the I/O
        assert call(lib, dim=16385) == UNSUPPORTED
        assert call(lib, rows=1 << 40) == UNSUPPORTED
    for eps in (-1.0, float("nan"), float("inf")):
        assert _res(lib, eps=eps) == INVALID
    for name in ("x", "residual", "y", "total"):
        assert _res(lib, ptrs={name: None}) == INVALID, name
    for name in ("x", "residual", "scale", "weight", "y", "total", "rstd"):
        assert _res(lib, ptrs={name: PM}) == MISALIGNED, name
    for name in ("total", "rstd", "dy", "dresidual"):
        assert _res_bwd(lib, ptrs={name: None}) == INVALID, name
    assert _res_bwd(lib, ptrs=dict(dscale=P)) == INVALID                      # no scale to have one
    assert _res_bwd(lib, ptrs=dict(dscale=P, scale=P, x=None)) == INVALID
    for name in ("total", "weight", "rstd", "x", "scale", "dy", "dtotal", "dx", "dresidual", "dweight"):
        assert _res_bwd(lib, ptrs={name: PM}) == MISALIGNED, name
    assert lib.residual_norm_bwd_workspace_size(4, 64, 1, 1, None) == INVALID
    none = dict(x=None, residual=None, y=None, total=None, rstd=None, dy=None, dresidual=None)
    for call in (_res, _res_bwd):
        assert call(lib, rows=0, ptrs=none) == OK
        assert call(lib, dim=0, ptrs=none) == OK


def test_binding_checks_its_arguments():
    t = lambda *s: torch.zeros(*s)   # noqa: E731
    x, lam = t(2, 8, 16), t(16)
    with pytest.raises(ValueError, match="GPU"):
        ms.gated_scan_fwd(x, x, lam)
    with pytest.raises(ValueError, match="batch"):
        ms.gated_scan_fwd(t(2, 16), x, lam)
    with pytest.raises(ValueError, match="batch"):
        ms.gated_scan_update(t(2, 16), x, x, lam)
    with pytest.raises(TypeError):
        ms.gated_scan_fwd(None, x, lam)
    with pytest.raises(ValueError, match="dtype"):
        ms.gated_scan_fwd(x.half(), x.half(), lam)
    with pytest.raises(ValueError, match="dtype"):
        ms.gated_scan_bwd(x.double(), x, lam, block_states=t(2, 1, 16), dy=x)
    for call in (ms.gated_norm_fwd, lambda v, **kw: ms.residual_norm_fwd(v, v)):
        with pytest.raises(ValueError, match="GPU"):
            call(t(4, 10))
        with pytest.raises(ValueError, match="dtype"):
            call(t(4, 10).double())
        with pytest.raises(TypeError):
            call(None)
        for shape in ((4, 0), (0,), (2, 3, 0)):
            with pytest.raises(ValueError, match="channels"):
                call(t(*shape))
    with pytest.raises(ValueError, match="groups"):
        ms.gated_norm_fwd(t(4, 10), groups=3)


def test_binding_takes_rows_a_fixed_stride_apart():
    from selective_state_space_40_amd import _rows
    dev, f = torch.device("cpu"), torch.float32
    wide = torch.zeros(3, 5, 24)
    at = lambda t: _rows(t, "x", t.shape, f, t.device)   # noqa: E731
    # a CPU tensor has no device number to match, so the checks behind the cheap test run
    assert at(wide) == (wide.data_ptr(), 24)
    part = wide[..., 8:16]
    assert at(part) == (part.data_ptr(), 24)
    assert at(part[1])[1] == 24 and at(part[:1, :1])[1] == 8 and at(part[:, :1])[1] == 120
    assert at(wide[..., :1])[1] == 24
    for bad in (wide.transpose(0, 1), wide[..., ::2], wide[:, ::2], wide[:1].expand(3, 5, 24),
                torch.zeros(24).expand(5, 24), wide.transpose(1, 2)):
        with pytest.raises(ValueError, match="stride"):
            at(bad)
    with pytest.raises(ValueError, match="shape"):
        _rows(wide, "x", (3, 5, 8), f, dev)
    with pytest.raises(ValueError, match="dtype"):
        _rows(wide, "x", wide.shape, torch.bfloat16, dev)
    with pytest.raises(TypeError):
        _rows(None, "x", wide.shape, f, dev)
