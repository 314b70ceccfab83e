"""The norms around a block on the GPU against 64 bits (gated_ref.py, where the
bounds are derived): the norm behind a block with its gate, and the norm before one
with the residual sum, forward and gradients."""
import sys

import pytest
import torch

import gated_ref as ref
import selective_state_space_40_amd as ms

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch.cuda.synchronize()


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _gated(rows, dim, dtype, seed, weight=True, fused=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    both = r(rows, 2 * dim).to(dtype).to(DEV)
    x, z = both[:, :dim], both[:, dim:]
    if not fused:
        x, z = x.clone(), z.clone()   # on addresses of their own
    return x, z, (1 + 0.2 * r(dim)).to(DEV) if weight else None, r(rows, dim).to(dtype).to(DEV)


def _each_gate(x, z, w, dy, groups, what):
    _say(f"case {what}")
    ref.check_gated(ms, x, z, w, dy, groups, True, f"{what} first")
    ref.check_gated(ms, x, z, w, dy, groups, False, f"{what} behind")
    ref.check_gated(ms, x, None, w, dy, groups, True, f"{what} none")


# at the edges of a team's lanes, of waves and of runs, odd ones, one value
WIDTHS = [1, 2, 7, 8, 9, 64, 120, 127, 128, 129, 136, 255, 256, 504, 511, 512, 513, 520, 1000, 1024, 1531, 2048,
          4095, 4104, 5120, 8185, 8191, 8192, 8193, 8200, 10001, 12288, 14223, 16376, 16383, 16384]


@TYPES
@pytest.mark.parametrize("dim", WIDTHS)
def test_gated_widths(dim, dtype):
    for rows in (1, 5, 67):
        _each_gate(*_gated(rows, dim, dtype, dim + rows, weight=rows != 5), 1, f"{rows} x {dim} {dtype}")


@TYPES
@pytest.mark.parametrize("case", [(33, 1024, 16), (7, 24, 8), (130, 37 * 3, 3), (300, 4096, 2), (9, 12, 12),
                                  (2000, 640, 5), (5, 16384 * 3, 3), (40, 5120, 8)], ids=lambda c: "x".join(map(str, c)))
def test_gated_groups(case, dtype):
    rows, dim, groups = case
    _each_gate(*_gated(rows, dim, dtype, sum(case), fused=dim % 8 == 0), groups, f"groups {case} {dtype}")


@TYPES
def test_gated_many_rows(dtype):
    for rows, dim in ((20011, 64), (5003, 520), (2051, 1531), (9001, 136)):
        x, z, w, dy = _gated(rows, dim, dtype, rows)
        _say(f"case rows {rows} x {dim} {dtype}")
        ref.check_gated(ms, x, z, w, dy, 1, True, f"rows {rows} x {dim}")


def _residual(rows, dim, dtype, seed, wide=False, scale=True, weight=True, dtotal=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    rt = F32 if wide else dtype
    to = lambda t, dt: t.to(dt).to(DEV)   # noqa: E731
    return (to(r(rows, dim), dtype), to(2 * r(rows, dim) + r(dim), rt), to(0.5 * r(dim), F32) if scale else None,
            to(1 + 0.2 * r(dim), F32) if weight else None, to(r(rows, dim), dtype),
            to(r(rows, dim), rt) if dtotal else None)


STREAMS = pytest.mark.parametrize("kind", ["bf16", "bf16-f32", "f32"])


def _types(kind):
    return (F32 if kind == "f32" else BF), kind == "bf16-f32"


@STREAMS
@pytest.mark.parametrize("dim", WIDTHS)
def test_residual_widths(dim, kind):
    dtype, wide = _types(kind)
    for rows in (1, 5, 67):
        _say(f"case {rows} x {dim} {kind}")
        args = _residual(rows, dim, dtype, dim + rows, wide, scale=rows != 5, weight=rows != 1)
        ref.check_residual(ms, *args, f"{rows} x {dim} {kind}")


@STREAMS
def test_residual_many_rows_and_parts(kind):
    dtype, wide = _types(kind)
    for rows, dim in ((20011, 64), (5003, 520), (2051, 1531)):
        _say(f"case rows {rows} x {dim} {kind}")
        ref.check_residual(ms, *_residual(rows, dim, dtype, rows, wide, dtotal=dim != 520), f"rows {rows} x {dim}")


def test_residual_gradient_shared_or_apart():
    x, res, _, w, dy, dt = _residual(30, 200, BF, 1, scale=False)
    y, total, rstd = ms.residual_norm_fwd(x, res, None, w)
    g = ms.residual_norm_bwd(total, w, rstd, dy=dy, dtotal=dt)
    assert g["dx"] is g["dresidual"] and g["dscale"] is None
    y, total, rstd = ms.residual_norm_fwd(x, res.float(), None, w)
    g = ms.residual_norm_bwd(total, w, rstd, dy=dy, dtotal=dt.float())
    assert g["dx"].dtype == BF and g["dresidual"].dtype == F32
    assert torch.equal(g["dx"], g["dresidual"].to(BF))


def test_in_place_and_shapes():
    x, z, w, dy = _gated(24, 200, BF, 3)
    y, rstd = ms.gated_norm_fwd(x, z, w, groups=2)
    g = ms.gated_norm_bwd(x, z, w, rstd, dy=dy, groups=2)
    y3, r3 = ms.gated_norm_fwd(x.view(2, 12, 200), z.view(2, 12, 200), w, groups=2)
    assert torch.equal(y3.view_as(y), y) and r3.shape == (2, 12, 2)
    for which in (x, z):
        a = {id(t): t.clone() for t in (x, z)}
        o = a[id(which)]
        assert ms.gated_norm_fwd(a[id(x)], a[id(z)], w, groups=2, out=o)[0] is o and torch.equal(o, y)
    d = dy.clone()
    g2 = ms.gated_norm_bwd(x, z, w, rstd, dy=d, groups=2, out=d)
    assert torch.equal(d, g["dx"]) and torch.equal(g2["dz"], g["dz"]) and torch.equal(g2["dweight"], g["dweight"])
    x, res, sc, w, dy, dt = _residual(24, 200, BF, 4)
    y, total, rstd = ms.residual_norm_fwd(x, res, sc, w)
    xc, rc = x.clone(), res.clone()
    yo, to, _ = ms.residual_norm_fwd(xc, rc, sc, w, out=xc, total_out=rc)
    assert yo is xc and to is rc and torch.equal(yo, y) and torch.equal(to, total)
    assert rstd.shape == (24, 1)


def test_no_rows():
    x, z, w, dy = _gated(0, 96, BF, 5)
    y, rstd = ms.gated_norm_fwd(x, z, w)
    g = ms.gated_norm_bwd(x, z, w, rstd, dy=dy)
    assert y.shape == (0, 96) and (g["dweight"] == 0).all()
    x, res, sc, w, dy, dt = _residual(0, 96, BF, 5)
    y, total, rstd = ms.residual_norm_fwd(x, res, sc, w)
    g = ms.residual_norm_bwd(total, w, rstd, x, sc, dy=dy, dtotal=dt)
    assert (g["dweight"] == 0).all() and (g["dscale"] == 0).all()


def test_special_values_stay_in_their_row():
    x, z, w, dy = _gated(5, 300, F32, 6)
    clean, _ = ms.gated_norm_fwd(x, z, w)
    x[1, 7] = float("nan")
    z[2, 299] = float("nan")
    x[3, 5] = float("inf")
    x[4] = 0.0
    y, rstd = ms.gated_norm_fwd(x, z, w)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all() and torch.isnan(y[3, 5])
    assert torch.equal(y[0], clean[0]) and not y[4].any() and abs(rstd[4].item() - 1e-5 ** -0.5) < 1e-3
    g = ms.gated_norm_bwd(x, z, w, rstd, dy=dy)
    assert torch.isfinite(g["dx"][[0, 4]]).all() and torch.isnan(g["dx"][1]).all()
    # gates far out: silu is 0 or the value itself. A sigmoid below 2^-126 may count as
    # zero, its silu is then off by up to 200 * 2^-126 = 2.4e-36; times |x|, |dy| < 5, rstd
    # and weights < 4 and 4 rows that is below 1e-33
    far = torch.tensor([-200.0, -90.0, -30.0, 30.0, 90.0, 200.0], device=DEV).repeat(4, 50)
    ref.check_gated(ms, x[[0, 0, 0, 0]], far, w, dy[:4], 1, False, "far gates", floor=1e-33)


def test_a_long_stride_and_one_row():
    # rows a long way apart, one row of any stride, channels not a multiple of a run
    for dtype in (BF, F32):
        base = torch.randn(7, 4096, device=DEV).to(dtype)
        z, w, dy = (torch.randn(7, 333, device=DEV).to(dtype), torch.rand(333, device=DEV),
                    torch.randn(7, 333, device=DEV).to(dtype))
        x = base[:, 16:349]
        got = ms.gated_norm_fwd(x, z, w)
        want = ms.gated_norm_fwd(x.contiguous(), z, w)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        a = ms.gated_norm_bwd(x, z, w, got[1], dy=dy)
        b = ms.gated_norm_bwd(x.contiguous(), z, w, got[1], dy=dy)
        assert all(torch.equal(a[k], b[k]) for k in a)
        one = base[:1, 16:349]
        assert torch.equal(ms.gated_norm_fwd(one)[0], ms.gated_norm_fwd(one.contiguous())[0])


def test_gradients_against_differences():
    # central differences of the 64-bit definition, error O(step^2)
    gen = torch.Generator().manual_seed(7)
    x, z, w, dy = _gated(5, 40, F32, 8)
    for first in (True, False):
        y, rstd = ms.gated_norm_fwd(x, z, w, groups=2, gate_first=first)
        g = ms.gated_norm_bwd(x, z, w, rstd, dy=dy, groups=2, gate_first=first)
        args = dict(x=ref.d64(x), z=ref.d64(z), weight=ref.d64(w))
        for name in args:
            d = torch.randn(args[name].shape, generator=gen, dtype=torch.float64)
            loss = [(ref.gated(**{**args, name: args[name] + s * 1e-4 * d}, groups=2, gate_first=first)[0]
                     * ref.d64(dy)).sum().item() for s in (1, -1)]
            want = (ref.d64(g["d" + name]) * d).sum().item()
            size = (ref.d64(g["d" + name]).norm() * d.norm()).item()
            assert abs((loss[0] - loss[1]) / 2e-4 - want) <= 1e-5 * size, name
    x, res, sc, w, dy, dt = _residual(5, 40, F32, 9)
    _, total, rstd = ms.residual_norm_fwd(x, res, sc, w)
    g = ms.residual_norm_bwd(total, w, rstd, x, sc, dy=dy, dtotal=dt)
    args = dict(x=ref.d64(x), residual=ref.d64(res), scale=ref.d64(sc), weight=ref.d64(w))

    def loss_of(x, residual, scale, weight):
        t = residual + scale * x
        y = t * (t.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * weight
        return ((y * ref.d64(dy)).sum() + (t * ref.d64(dt)).sum()).item()

    for name in args:
        d = torch.randn(args[name].shape, generator=gen, dtype=torch.float64)
        ends = [loss_of(**{**args, name: args[name] + s * 1e-4 * d}) for s in (1, -1)]
        want = (ref.d64(g["d" + name]) * d).sum().item()
        size = (ref.d64(g["d" + name]).norm() * d.norm()).item()
        assert abs((ends[0] - ends[1]) / 2e-4 - want) <= 1e-5 * size, name


def test_captured_calls_replay():
    x, z, w, dy = _gated(700, 1000, BF, 10)
    a, res, sc, w2, dy2, dt = _residual(700, 1000, BF, 11, wide=True)

    def calls():
        y, rstd = ms.gated_norm_fwd(x, z, w, groups=4)
        g = ms.gated_norm_bwd(x, z, w, rstd, dy=dy, groups=4)
        y2, total, r2 = ms.residual_norm_fwd(a, res, sc, w2)
        g2 = ms.residual_norm_bwd(total, w2, r2, a, sc, dy=dy2, dtotal=dt)
        return [y, rstd, *g.values(), y2, total, r2, *g2.values()]

    want = calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for r in range(4):
        for t in got:
            t.fill_(float("nan"))
        torch.randn(1 << 16, device=DEV).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for p, e in zip(got, want):
            assert torch.equal(p, e), f"replay {r}"
