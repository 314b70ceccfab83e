"""The gated operators' scratch and pointers through the C ABI: what a call needs,
what it takes as it finds it, and what may share memory."""
import ctypes

import pytest
import torch

import selective_state_space_40_amd as ms

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
OK, WORKSPACE = 0, -4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch.cuda.synchronize()


def _p(t):
    return None if t is None else t.data_ptr()


def _code(dtype):
    return 1 if dtype == BF else 0


def _stream():
    return torch.cuda.current_stream(DEV).cuda_stream


def _size(call, *sizes):
    n = ctypes.c_size_t()
    assert getattr(ms.load_library(), call)(*sizes, ctypes.byref(n)) == OK
    return n.value


def _sequences(b, n, d, dtype, seed, lengths=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=dtype: torch.randn(*s, generator=g).to(dt).to(DEV)   # noqa: E731
    return dict(x=r(b, n, d), decay_gate=r(b, n, d), log_decay=-torch.logspace(-3, 1, d).to(DEV),
                input_gate=r(b, n, d), h0=r(b, d, dt=F32), dy=r(b, n, d), dhL=r(b, d, dt=F32),
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV))


def _forward(c, ws):
    """(status, y, hL, block states) with the scratch ws."""
    b, n, d = c["x"].shape
    y, hL = torch.empty_like(c["x"]), torch.empty(b, d, device=DEV)
    states = torch.zeros(b, -(-n // ms.GATED_SCAN_BLOCK), d, device=DEV)
    st = ms.load_library().gated_scan_fwd(
        b, n, d, _code(c["x"].dtype), _p(c["x"]), d, _p(c["decay_gate"]), d, _p(c["log_decay"]), _p(c["input_gate"]), d,
        _p(c["lengths"]), _p(c["h0"]), _p(y), _p(hL), _p(states), _p(ws), 0 if ws is None else ws.numel(), _stream())
    return st, y, hL, states


def _backward(c, states, ws, dlog=True):
    """(status, gradients) with the scratch ws; without dlog_decay where dlog is False."""
    b, n, d = c["x"].shape
    g = dict(dx=torch.empty_like(c["x"]), ddecay_gate=torch.empty_like(c["x"]), dinput_gate=torch.empty_like(c["x"]),
             dlog_decay=torch.empty(d, device=DEV) if dlog else None, dh0=torch.empty(b, d, device=DEV))
    st = ms.load_library().gated_scan_bwd(
        b, n, d, _code(c["x"].dtype), _p(c["x"]), d, _p(c["decay_gate"]), d, _p(c["log_decay"]), _p(c["input_gate"]), d,
        _p(c["lengths"]), _p(states), _p(c["dy"]), _p(c["dhL"]), *(_p(t) for t in g.values()), _p(ws),
        0 if ws is None else ws.numel(), _stream())
    return st, g


@pytest.mark.parametrize("b,d", [(1, 1), (3, 70), (700, 5121)])
def test_no_tokens_read_nothing(b, d):
    # x, gates and log_decay are NULL: hL = h0, dh0 = dhL, in place as well
    lib, state = ms.load_library(), torch.randn(b, d, generator=torch.Generator().manual_seed(d)).to(DEV)
    none = [None, 0, None, 0, None, None, 0]
    for h0 in (state, None):
        hL = torch.full_like(state, 7.0)
        assert lib.gated_scan_fwd(b, 0, d, 1, *none, None, _p(h0), None, _p(hL), None, None, 0, _stream()) == OK
        dh0, dlog = torch.full_like(state, 7.0), torch.full((d,), 7.0, device=DEV)
        assert lib.gated_scan_bwd(b, 0, d, 1, *none, None, None, None, _p(h0), None, None, None, _p(dlog), _p(dh0),
                                  None, 0, _stream()) == OK
        torch.cuda.synchronize()
        for t in (hL, dh0):
            assert torch.equal(t, state if h0 is not None else torch.zeros_like(state))
        assert not bool(dlog.any())
    same = state.clone()
    assert lib.gated_scan_fwd(b, 0, d, 0, *none, None, _p(same), None, _p(same), None, None, 0, _stream()) == OK
    torch.cuda.synchronize()
    assert torch.equal(same, state)


@pytest.mark.parametrize("kind", ["bf16", "bf16-f32", "f32"])
@pytest.mark.parametrize("rows,dim", [(5, 7), (900, 333), (3001, 645), (2003, 1531), (1501, 2560), (701, 5001),
                                      (401, 9001), (301, 16383), (301, 12288)])
def test_residual_gradients_in_place(rows, dim, kind):
    # dresidual over dtotal and dx over dy. At odd widths the last 8 values overlap the
    # run before, in a lane of another wave where a part takes more than one: both read
    # before the barrier of the row's sum and write behind it
    g = torch.Generator().manual_seed(dim)
    dtype = F32 if kind == "f32" else BF
    wide = F32 if kind == "bf16-f32" else dtype
    r = lambda *s, dt=dtype: torch.randn(*s, generator=g).to(dt).to(DEV)   # noqa: E731
    total, dtotal = r(rows, dim, dt=wide), r(rows, dim, dt=wide)
    x, dy, scale, weight = r(rows, dim), r(rows, dim), r(dim, dt=F32), r(dim, dt=F32)
    rstd = (total.float().square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    print(f"case {rows} x {dim} {kind}", flush=True)
    want = ms.residual_norm_bwd(total, weight, rstd, x, scale, dy=dy, dtotal=dtotal)
    need = _size("residual_norm_bwd_workspace_size", rows, dim, _code(dtype), _code(wide))
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    dscale, dweight = torch.empty(dim, device=DEV), torch.empty(dim, device=DEV)
    for _ in range(3):
        d, dx = dtotal.clone(), dy.clone()
        assert ms.load_library().residual_norm_bwd(
            rows, dim, _code(dtype), _code(wide), _p(total), _p(weight), _p(rstd), _p(x), _p(scale), _p(dx), _p(d),
            _p(dx), _p(d), _p(dscale), _p(dweight), _p(ws), need, _stream()) == OK
        torch.cuda.synchronize()
        for name, t in dict(dresidual=d, dx=dx, dscale=dscale, dweight=dweight).items():
            assert torch.equal(t, want[name]), name


@TYPES
def test_no_scratch_where_none_is_used(dtype):
    # a row walked keeps its share of the decay's gradient in scratch, and nothing else
    c = _sequences(3, 200, 70, dtype, 1, [200, 0, 77])
    st, _, _, states = _forward(c, None)
    assert st == OK and _size("gated_scan_fwd_workspace_size", 3, 200, 70, _code(dtype)) == 0
    need = _size("gated_scan_bwd_workspace_size", 3, 200, 70, _code(dtype))
    assert need > 0
    st, want = _backward(c, states, torch.empty(need, dtype=torch.uint8, device=DEV))
    assert st == OK
    assert _backward(c, states, None)[0] == WORKSPACE
    assert _backward(c, states, torch.empty(need - 4, dtype=torch.uint8, device=DEV))[0] == WORKSPACE
    st, got = _backward(c, states, None, dlog=False)
    assert st == OK
    torch.cuda.synchronize()
    for k, t in got.items():
        assert t is None or torch.equal(t, want[k]), k
    # a chain's tiles learn from each other through it in any case
    c = _sequences(1, 4000, 70, dtype, 2)
    need = _size("gated_scan_bwd_workspace_size", 1, 4000, 70, _code(dtype))
    states = _forward(c, torch.empty(need, dtype=torch.uint8, device=DEV))[3]
    assert _backward(c, states, None, dlog=False)[0] == WORKSPACE


@TYPES
@pytest.mark.parametrize("b,n,d,lens", [(2, 9000, 130, [9000, 7001]), (1, 4100, 65, None), (513, 1500, 8, "many")], ids=str)
def test_results_whatever_the_scratch_holds(b, n, d, lens, dtype):
    # each call's scratch filled by the test: zeros (states and sums of nothing), all
    # ones (a word that is not there yet), 0x7f, what the call before left, and what one
    # of other sizes left
    if lens == "many":
        lens = torch.randint(0, n + 1, (b,), generator=torch.Generator().manual_seed(b)).tolist()
    c, other = _sequences(b, n, d, dtype, 6, lens), _sequences(1, 7777, 192, dtype, 7)
    sizes = [_size(f"gated_scan_{w}_workspace_size", *s, _code(dtype)) for w in ("fwd", "bwd")
             for s in ((b, n, d), (1, 7777, 192))]
    assert min(sizes) > 0
    ws = torch.empty(max(sizes), dtype=torch.uint8, device=DEV)
    print(f"case {b} x {n} x {d} {dtype}", flush=True)
    want = None
    for fill in (0, 0xff, 0x7f, "left", "other"):
        for call in ("forward", "backward"):
            if fill == "other":
                st, _, _, s = _forward(other, ws)
                assert st == OK and _backward(other, s, ws)[0] == OK
            elif fill != "left":
                ws.fill_(fill)
            if call == "forward":
                st, *got = _forward(c, ws)
            else:
                st, g = _backward(c, got[2], ws)
                got += g.values()
            assert st == OK
        torch.cuda.synchronize()
        want = want or [t.clone() for t in got]
        for i, (t, e) in enumerate(zip(got, want)):
            assert torch.equal(t, e), (fill, i)
    f = ms.gated_scan_fwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"], c["h0"], lengths=c["lengths"])
    assert torch.equal(f[0], want[0]) and torch.equal(f[1], want[1])


@TYPES
@pytest.mark.parametrize("rows,dim", [(900, 333), (3001, 645), (2003, 1531), (701, 5001), (401, 9001), (301, 16383)])
def test_norms_in_place_at_odd_widths(rows, dim, dtype):
    # outputs over inputs, where runs of neighbouring lanes and waves overlap
    g = torch.Generator().manual_seed(dim)
    r = lambda *s, dt=dtype: torch.randn(*s, generator=g).to(dt).to(DEV)   # noqa: E731
    x, z, dy, w, sc = r(rows, dim), r(rows, dim), r(rows, dim), r(dim, dt=F32), r(dim, dt=F32)
    print(f"case {rows} x {dim} {dtype}", flush=True)
    for first in (True, False):
        y, rstd = ms.gated_norm_fwd(x, z, w, gate_first=first)
        grads = ms.gated_norm_bwd(x, z, w, rstd, dy=dy, gate_first=first)
        for which in (0, 1):
            a = [x.clone(), z.clone()]
            assert torch.equal(ms.gated_norm_fwd(*a, w, gate_first=first, out=a[which])[0], y)
        d = dy.clone()
        more = ms.gated_norm_bwd(x, z, w, rstd, dy=d, gate_first=first, out=d)
        for k, t in grads.items():
            assert torch.equal(more[k], t), k
    for res in (r(rows, dim), r(rows, dim, dt=F32)):
        want = ms.residual_norm_fwd(x, res, sc, w)
        a, b = x.clone(), res.clone()
        for t, e in zip(ms.residual_norm_fwd(a, b, sc, w, out=a, total_out=b), want):
            assert torch.equal(t, e)
