"""A gated recurrent block as a model runs it: residual norm, projections, gated
recurrence, gated norm, projection; its training step and its serving, token by
token, against 64 bits. And what is between the norms' calls: neighbouring groups,
streams, graphs."""
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


WIDTH, INNER, GROUPS, LAYERS = 48, 96, 4, 2


def _weights(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    return [dict(scale=1 + 0.1 * r(WIDTH), norm=1 + 0.1 * r(WIDTH), into=r(WIDTH, 4 * INNER) / WIDTH ** 0.5,
                 log_decay=-torch.pow(10.0, -2.0 * torch.rand(INNER, generator=g)), gnorm=1 + 0.1 * r(INNER),
                 out=r(INNER, WIDTH) / INNER ** 0.5) for _ in range(LAYERS)]


def _plain(x, stream, weights, lengths):
    """The block's layers in 64 bits, differentiable: (last branch, last stream)."""
    n = x.shape[1]
    live = (torch.arange(n) < lengths[:, None])[..., None]
    for w in weights:
        stream = stream + w["scale"] * x
        u = stream * (stream.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w["norm"]
        v, dg, ig, z = (u @ w["into"]).split(INNER, -1)
        g = w["log_decay"] * torch.sigmoid(dg)
        add = (-torch.expm1(2 * g)).sqrt() * torch.sigmoid(ig) * v
        h, hs = torch.zeros_like(v[:, 0]), []
        for t in range(n):
            h = torch.where(live[:, t], g[:, t].exp() * h + add[:, t], h)
            hs.append(h)
        y = torch.where(live, torch.stack(hs, 1), 0.0)
        y, _ = ref.gated(y, z, w["gnorm"], GROUPS, True)
        x = y @ w["out"]
    return x, stream


def _forward(x, stream, weights, lengths, saved=None):
    for w in weights:
        u, total, rstd = ms.residual_norm_fwd(x, stream, w["scale"], w["norm"])
        mixed = u @ w["into"]
        v, dg, ig, z = mixed.split(INNER, -1)
        y, _, states = ms.gated_scan_fwd(v, dg, w["log_decay"], ig, lengths=lengths, return_block_states=True)
        n, nrstd = ms.gated_norm_fwd(y, z, w["gnorm"], groups=GROUPS)
        if saved is not None:
            saved.append((x, total, rstd, u, mixed, y, states, n, nrstd))
        x, stream = n @ w["out"], total
    return x, stream


def _backward(dx, dstream, weights, lengths, saved):
    grads = []
    flat = lambda t: t.reshape(-1, t.shape[-1])   # noqa: E731
    for w, (x, total, rstd, u, mixed, y, states, n, nrstd) in zip(weights[::-1], saved[::-1]):
        g = dict(out=flat(n).T @ flat(dx))
        v, dg, ig, z = mixed.split(INNER, -1)
        gn = ms.gated_norm_bwd(y, z, w["gnorm"], nrstd, dy=dx @ w["out"].T, groups=GROUPS)
        gs = ms.gated_scan_bwd(v, dg, w["log_decay"], ig, block_states=states, dy=gn["dx"], lengths=lengths)
        dmixed = torch.cat([gs["dx"], gs["ddecay_gate"], gs["dinput_gate"], gn["dz"]], -1)
        g.update(gnorm=gn["dweight"], log_decay=gs["dlog_decay"], into=flat(u).T @ flat(dmixed))
        gr = ms.residual_norm_bwd(total, w["norm"], rstd, x, w["scale"], dy=dmixed @ w["into"].T, dtotal=dstream)
        dx, dstream = gr["dx"], gr["dresidual"]
        g.update(norm=gr["dweight"], scale=gr["dscale"])
        grads.append(g)
    return dx, dstream, grads[::-1]


def _close(got, want, what):
    # 10 operators a layer, forward and backward, each within 4e-6 of what its values
    # add up to; sums of some terms of either sign: up to 3 times the values' norm
    rel = ((got.double().cpu() - want).norm() / want.norm()).item()
    _say(f"case {what}: {rel:.1e}")
    assert rel <= 10 * LAYERS * 3 * 4e-6, what


def test_training_step():
    b, n = 3, 200
    host = _weights(1)
    g = torch.Generator().manual_seed(2)
    x, stream, rx, rs = (torch.randn(b, n, WIDTH, generator=g) for _ in range(4))
    lengths = torch.tensor([n, 77, 130], dtype=torch.int32)
    # behind a row's end the recurrence gives zeros; the weights of the loss are its
    rx, rs = (torch.where((torch.arange(n) < lengths[:, None])[..., None], t, 0.0) for t in (rx, rs))
    leaves = [{k: t.double().requires_grad_() for k, t in w.items()} for w in host]
    xd, sd = x.double().requires_grad_(), stream.double().requires_grad_()
    xo, so = _plain(xd, sd, leaves, lengths)
    want = torch.autograd.grad((xo * rx).sum() + (so * rs).sum(), [xd, sd] + [t for w in leaves for t in w.values()])
    dev = [{k: t.to(DEV) for k, t in w.items()} for w in host]
    saved, lens = [], lengths.to(DEV)
    gx, gs = _forward(x.to(DEV), stream.to(DEV), dev, lens, saved)
    _close(gx, xo.detach(), "output")
    _close(gs, so.detach(), "stream")
    dx, ds, grads = _backward(rx.to(DEV), rs.to(DEV), dev, lens, saved)
    _close(dx, want[0], "dx")
    _close(ds, want[1], "dstream")
    names = [(i, k) for i, w in enumerate(leaves) for k in w]
    for (i, k), t in zip(names, want[2:]):
        _close(grads[i][k], t, f"layer {i} {k}")


def test_serving_continues_a_prompt():
    b, n, more = 2, 150, 12
    host = _weights(3)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(b, n + more, WIDTH, generator=g)
    dev = [{k: t.to(DEV) for k, t in w.items()} for w in host]
    want, _ = _plain(x.double(), torch.zeros_like(x).double(),
                     [{k: t.double() for k, t in w.items()} for w in host], torch.tensor([n + more] * b))
    branch, stream, states = x[:, :n].to(DEV), torch.zeros(b, n, WIDTH, device=DEV), []
    for w in dev:
        u, stream, _ = ms.residual_norm_fwd(branch, stream, w["scale"], w["norm"])
        v, dg, ig, z = (u @ w["into"]).split(INNER, -1)
        y, h, _ = ms.gated_scan_fwd(v, dg, w["log_decay"], ig)
        states.append(h)
        branch = ms.gated_norm_fwd(y, z, w["gnorm"], groups=GROUPS)[0] @ w["out"]
    _close(branch, want[:, :n], "prompt")
    for t in range(n, n + more):
        branch, stream = x[:, t].to(DEV), torch.zeros(b, WIDTH, device=DEV)
        for w, h in zip(dev, states):
            u, stream, _ = ms.residual_norm_fwd(branch, stream, w["scale"], w["norm"])
            v, dg, ig, z = (u @ w["into"]).split(INNER, -1)
            y = ms.gated_scan_update(h, v, dg, w["log_decay"], ig)
            branch = ms.gated_norm_fwd(y, z, w["gnorm"], groups=GROUPS)[0] @ w["out"]
        _close(branch, want[:, t], f"token {t}")


def test_captured_training_step_replays():
    b, n = 2, 600   # the recurrence's tiles learn from each other
    dev = [{k: t.to(DEV) for k, t in w.items()} for w in _weights(5)]
    g = torch.Generator(DEV).manual_seed(6)
    x, stream, rx, rs = (torch.randn(b, n, WIDTH, generator=g, device=DEV) for _ in range(4))
    lens = torch.tensor([n, 555], dtype=torch.int32, device=DEV)

    def step():
        saved = []
        out = _forward(x, stream, dev, lens, saved)
        dx, ds, grads = _backward(rx, rs, dev, lens, saved)
        return [*out, dx, ds, *(t for w in grads for t in w.values())]

    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for r in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        for a, e, w in zip(got, eager, want):
            # the projections are the library's, which may add up in another order
            assert (a - w).norm() <= 1e-5 * w.norm() and (e - w).norm() <= 1e-5 * w.norm(), f"replay {r}"


@TYPES
@pytest.mark.parametrize("case", [(700, 3, 64), (900, 16, 64), (513, 80, 64), (40, 7, 60), (301, 6, 128), (65, 5, 130),
                                  (257, 12, 256), (33, 10, 250), (129, 6, 300), (77, 3, 520), (50, 6, 640), (21, 4, 1000),
                                  (19, 8, 768), (35, 2, 1531), (4000, 32, 8), (77, 9, 5), (3, 64, 1)],
                         ids=lambda c: "x".join(map(str, c)))
def test_neighbouring_groups(case, dtype):
    rows, groups, part = case
    g = torch.Generator().manual_seed(sum(case))
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    x, z, dy = (r(rows, groups * part).to(dtype).to(DEV) for _ in range(3))
    w = (1 + 0.2 * r(groups * part)).to(DEV)
    _say(f"case {case} {dtype}")
    ref.check_gated(ms, x, z, w, dy, groups, True, "first")
    ref.check_gated(ms, x, z, w, dy, groups, False, "behind")


def test_norms_of_two_streams_at_once():
    g = torch.Generator(DEV).manual_seed(7)
    r = lambda *s, dt=BF: torch.randn(*s, generator=g, device=DEV).to(dt)   # noqa: E731
    cases = [(r(6000, 5120), r(6000, 5120), r(6000, 5120), 8), (r(700, 16384), r(700, 16384), r(700, 16384), 1)]

    def gated(x, z, dy, groups):
        w = torch.ones(x.shape[-1], device=DEV)
        y, rstd = ms.gated_norm_fwd(x, z, w, groups=groups)
        grads = ms.gated_norm_bwd(x, z, w, rstd, dy=dy, groups=groups)
        a, total, rs = ms.residual_norm_fwd(y, z, w, w)
        more = ms.residual_norm_bwd(total, w, rs, y, w, dy=dy, dtotal=x)
        return [y, rstd, *grads.values(), a, total, *more.values()]

    want = [gated(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in cases]
    for _ in range(3):
        got = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream(DEV))
            with torch.cuda.stream(s):
                got.append(gated(*c))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for t, e in zip(a, b):
                assert torch.equal(t, e)


@TYPES
def test_gradients_in_place(dtype):
    # dx may be dy and dresidual dtotal, where a part's last values are held twice too
    for rows, dim in ((9, 1531), (300, 12345), (50, 5121), (700, 61), (5, 9)):
        g = torch.Generator(DEV).manual_seed(dim)
        r = lambda *s, dt=dtype: torch.randn(*s, generator=g, device=DEV).to(dt)   # noqa: E731
        x, z, dy, dt = r(rows, dim), r(rows, dim), r(rows, dim), r(rows, dim)
        w, sc = r(dim, dt=F32), r(dim, dt=F32)
        y, rstd = ms.gated_norm_fwd(x, z, w)
        want = ms.gated_norm_bwd(x, z, w, rstd, dy=dy)
        lib, code = ms.load_library(), 1 if dtype == BF else 0
        ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        p = lambda t: None if t is None else t.data_ptr()   # noqa: E731
        mine, dz, dw = dy.clone(), torch.empty_like(z), torch.empty_like(w)
        stream = torch.cuda.current_stream(DEV).cuda_stream
        assert lib.gated_norm_bwd(rows, dim, 1, code, 1, p(x), dim, p(z), dim, p(w), p(rstd), p(mine), p(mine), p(dz),
                                  p(dw), p(ws), ws.numel(), stream) == 0
        assert torch.equal(mine, want["dx"]) and torch.equal(dz, want["dz"]) and torch.equal(dw, want["dweight"])
        a, total, rs = ms.residual_norm_fwd(x, z, sc, w)
        want = ms.residual_norm_bwd(total, w, rs, x, sc, dy=dy, dtotal=dt)
        into, inta = dt.clone(), dy.clone()
        ds = torch.empty_like(w)
        assert lib.residual_norm_bwd(rows, dim, code, code, p(total), p(w), p(rs), p(x), p(sc), p(inta), p(into), p(inta),
                                     p(into), p(ds), p(dw), p(ws), ws.numel(), stream) == 0
        assert torch.equal(inta, want["dx"]) and torch.equal(into, want["dresidual"])
        assert torch.equal(ds, want["dscale"]) and torch.equal(dw, want["dweight"])
