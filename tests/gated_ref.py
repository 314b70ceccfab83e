"""The gated recurrence and the norms around a block in 64 bits on the CPU, from
their definitions, for the tests of the GPU kernels: states token by token,
gradients by differentiating the definitions.

Also the tests' bounds, each in proportion to what a value is made of.

Recurrence, fp32 arithmetic. sigmoid(r) takes the rounding of r log2(e) (half a
step of up to 40: |r| 2^-25, below 4 * 2^-24 for |r| <= 8), one step of exp2, an
addition and one step of the reciprocal: 9 * 2^-24. log a adds 2 roundings. w =
sqrt(s) q takes half of the error of s (log a's and 2e-7), the root's and the other
sigmoid's: 20 * 2^-24, and w x one more. A state adds the terms w x behind it,
decayed: each is off by that, by its decay's error, |G| e^-|G| 11 * 2^-24 with G the
decay's logarithm, below 4 * 2^-24, and by the roundings of at most 16 tokens, 16
segments and 2 a tile: in all below 64 * 2^-24 = 4e-6 (STATE) of the sum of the
terms' absolute values, which is the recurrence run over |w x| from |h0|. Adjoints
alike, over |dy| from |dhL|. A product of two such sums is off by STATE of each. With
bf16 a result is rounded once more, by 2^-8 of itself.

Norms. A mean of squares adds at most 16 values in a lane, 6 times across a wave and
16 waves: 40 * 2^-24, half of which reaches rstd, with 4 more roundings; silu is off
by 12 * 2^-24. y is a product, off by their sum, twice silu's where it is part of the
squares: 56 * 2^-24 < 4e-6 (NORM) of itself. dx and dz are differences of a term and a
mean of terms, off by twice that of their sizes.
"""
import torch

STATE = 4e-6
NORM = 4e-6


def d64(t):
    return None if t is None else t.detach().double().cpu()


def within(got, want, bound, what):
    """Every value of `got` within `bound` of 64 bits, and a bf16 one's rounding."""
    g, w = got.detach().double().cpu(), want.double()
    assert g.shape == w.shape, f"{what}: shape {tuple(g.shape)}, expected {tuple(w.shape)}"
    if w.numel() == 0:
        return
    assert torch.isfinite(g).all(), f"{what}: non-finite values"
    bound = bound.expand_as(w)
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (w.abs() + bound)
    worst = ((g - w).abs() - bound).max().item()
    at = ((g - w).abs() / (bound + 1e-300)).max().item()
    assert worst <= 0, f"{what}: {at:.3g} times the bound"


def _step(x, decay_gate, log_decay, input_gate):
    """(log a, w x) of every token."""
    g = log_decay * torch.sigmoid(decay_gate)
    w = (-torch.expm1(2.0 * g)).sqrt()
    if input_gate is not None:
        w = w * torch.sigmoid(input_gate)
    return g, w * x


def scan(x, decay_gate, log_decay, input_gate=None, h0=None, lengths=None, dy=None, dhL=None):
    """(y, hL, block states) and their magnitudes, in a dict; with `dy` gradients
    and the magnitudes that bound them as well (keys ending in _size)."""
    x, decay_gate, log_decay, input_gate, h0, dy, dhL = map(
        d64, (x, decay_gate, log_decay, input_gate, h0, dy, dhL))
    b, n, d = x.shape
    lens = [n] * b if lengths is None else [max(0, min(n, int(v))) for v in lengths.cpu()]
    live = (torch.arange(n) < torch.tensor(lens)[:, None])[..., None]
    clean = lambda t: None if t is None else torch.where(live, t, 0.0)   # noqa: E731
    x, decay_gate, input_gate, dy = map(clean, (x, decay_gate, input_gate, dy))
    g, u = _step(x, decay_gate, log_decay, input_gate)
    a, u = torch.where(live, g.exp(), 1.0), clean(u)
    h = torch.zeros(b, d, dtype=torch.float64) if h0 is None else h0.clone()
    size = h.abs()
    before, hs, bs, ss = [], [], [], []
    for t in range(n):
        before.append(h)
        bs.append(size)
        h = a[:, t] * h + u[:, t]
        size = a[:, t] * size + u[:, t].abs()
        hs.append(h)
        ss.append(size)
    pile = lambda v: torch.stack(v, 1) if v else torch.zeros(b, 0, d, dtype=torch.float64)   # noqa: E731
    before, before_size = pile(before), pile(bs)
    out = dict(y=clean(pile(hs)), y_size=pile(ss), hL=h, hL_size=size,
               block_states=before[:, ::64], block_states_size=before_size[:, ::64])
    if dy is None:
        return out
    adj = torch.zeros_like(h) if dhL is None else dhL.clone()
    size = adj.abs()
    As, sizes = [], []
    for t in reversed(range(n)):
        adj, size = dy[:, t] + adj, dy[:, t].abs() + size
        As.append(adj)
        sizes.append(size)
        adj, size = a[:, t] * adj, a[:, t] * size
    A, As_size = clean(pile(As[::-1])), clean(pile(sizes[::-1]))
    leaves = [t.clone().requires_grad_() for t in (x, decay_gate, log_decay)]
    if input_gate is not None:
        leaves.append(input_gate.clone().requires_grad_())
    gg, uu = _step(*leaves, *([] if input_gate is not None else [None]))
    grads = torch.autograd.grad((A * (gg.exp() * before + uu)).sum(), leaves)
    out.update(dx=grads[0], ddecay_gate=grads[1], dlog_decay=grads[2], dh0=adj, dh0_size=size)
    p = torch.sigmoid(decay_gate)
    s = -torch.expm1(2.0 * g)
    q = 1.0 if input_gate is None else torch.sigmoid(input_gate)
    w = s.sqrt() * q
    per_g = As_size * a * (before_size + q * x.abs() * a / s.sqrt())
    out.update(dx_size=As_size * w, ddecay_gate_size=per_g * g.abs() * torch.sigmoid(-decay_gate),
               dlog_decay_size=(per_g * p).sum((0, 1)))
    if input_gate is not None:
        out.update(dinput_gate=grads[3], dinput_gate_size=As_size * u.abs() * torch.sigmoid(-input_gate))
    return out


# what each result adds up to, in units of STATE: one sum, or a product of two
SCAN_UNITS = dict(y=1, hL=1, block_states=1, dh0=1, dx=1.5, dinput_gate=1.5, ddecay_gate=3, dlog_decay=3)


def check_scan(got, want, what):
    """Each of the dict's results against scan()'s."""
    for name, t in got.items():
        if t is not None:
            within(t, want[name], SCAN_UNITS[name] * STATE * want[name + "_size"], f"{what} {name}")


def _split(t, groups):
    return t.reshape(*t.shape[:-1], groups, -1)


def gated(x, z=None, weight=None, groups=1, gate_first=True, eps=1e-5):
    """(y, rstd), differentiable in 64-bit inputs."""
    silu = None if z is None else z * torch.sigmoid(z)
    v = x if z is None or not gate_first else x * silu
    rstd = (_split(v, groups).square().mean(-1) + eps).rsqrt()
    y = (_split(v, groups) * rstd[..., None]).reshape(v.shape)
    if weight is not None:
        y = y * weight
    if z is not None and not gate_first:
        y = y * silu
    return y, rstd


def check_gated(ms, x, z, weight, dy, groups, gate_first, what, eps=1e-5, floor=0.0):
    """Forward and gradients of the GPU's calls against 64 bits; returns them. `floor`
    is added to every bound."""
    y, rstd = ms.gated_norm_fwd(x, z, weight, groups=groups, gate_first=gate_first, eps=eps)
    grads = ms.gated_norm_bwd(x, z, weight, rstd, dy=dy, groups=groups, gate_first=gate_first)
    leaves = {k: None if t is None else d64(t).requires_grad_() for k, t in (("x", x), ("z", z), ("weight", weight))}
    yr, rr = gated(*leaves.values(), groups, gate_first, eps)
    within(y, yr.detach(), NORM * yr.detach().abs() + floor, f"{what} y")
    within(rstd, rr.detach(), NORM * rr.detach(), f"{what} rstd")
    used = {k: t for k, t in leaves.items() if t is not None}
    want = dict(zip(used, torch.autograd.grad((yr * d64(dy)).sum(), list(used.values()))))
    assert (grads["dz"] is None) == (z is None) and (grads["dweight"] is None) == (weight is None)
    xd, dyd, r = d64(x), d64(dy).abs(), _split(torch.ones_like(d64(x)), groups) * rr.detach()[..., None]
    r = r.reshape(xd.shape)
    w = 1.0 if weight is None else d64(weight).abs()
    silu, dsilu = 1.0, 0.0
    if z is not None:
        zd = d64(z)
        silu = zd * torch.sigmoid(zd)
        dsilu = torch.sigmoid(zd) * (1 + zd.abs() * torch.sigmoid(-zd))
    first = z is not None and gate_first
    v = (xd * silu if first else xd).abs()
    n = v * r
    up = dyd * (1.0 if z is None or gate_first else silu.abs())
    mean = _split(up * w * n, groups).mean(-1, keepdim=True).expand(*_split(n, groups).shape).reshape(n.shape)
    dv = r * (up * w + n * mean)
    within(grads["dx"], want["x"], 2 * NORM * dv * (silu.abs() if first else 1.0) + floor, f"{what} dx")
    if z is not None:
        size = dv * xd.abs() * dsilu if first else dyd * n * w * dsilu
        within(grads["dz"], want["z"], 2 * NORM * size + floor, f"{what} dz")
    if weight is not None:
        size = (up * n).reshape(-1, x.shape[-1]).sum(0)
        within(grads["dweight"], want["weight"], 2 * NORM * size + floor, f"{what} dweight")
    return y, rstd, grads


def check_residual(ms, x, residual, scale, weight, dy, dtotal, what, eps=1e-5):
    """Forward and gradients of the GPU's calls against 64 bits; returns them."""
    y, total, rstd = ms.residual_norm_fwd(x, residual, scale, weight, eps=eps)
    g = ms.residual_norm_bwd(total, weight, rstd, x, scale, dy=dy, dtotal=dtotal)
    xd, res = d64(x), d64(residual)
    sc = torch.ones(x.shape[-1], dtype=torch.float64) if scale is None else d64(scale)
    w = torch.ones(x.shape[-1], dtype=torch.float64) if weight is None else d64(weight)
    t = res + sc * xd
    size = res.abs() + (sc * xd).abs()
    r = (t.square().mean(-1, keepdim=True) + eps).rsqrt()
    # a sum's rounding is in proportion to its terms, in the norm of the row as well
    rel = NORM * r * (size.square().mean(-1, keepdim=True) + eps).sqrt()
    within(total, t, 2.0 ** -23 * size, f"{what} total")
    within(rstd, r, rel * r, f"{what} rstd")
    within(y, t * r * w, (2.0 ** -23 * size * r + rel * (t * r).abs()) * w.abs(), f"{what} y")
    # the gradients are those at the total and the statistics that the call was given
    t, r = d64(total), d64(rstd)
    n, dyd = t * r, d64(dy)
    wdy = dyd * w
    dt = 0.0 if dtotal is None else d64(dtotal)
    d = dt + r * (wdy - n * (wdy * n).mean(-1, keepdim=True))
    dsize = (torch.as_tensor(dt).abs() + r * (wdy.abs() + n.abs() * (wdy * n).abs().mean(-1, keepdim=True)))
    within(g["dresidual"], d, NORM * dsize, f"{what} dresidual")
    within(g["dx"], d * sc, NORM * dsize * sc.abs(), f"{what} dx")
    assert (g["dscale"] is None) == (scale is None) and (g["dweight"] is None) == (weight is None)
    rows = lambda v: v.reshape(-1, x.shape[-1]).sum(0)   # noqa: E731
    if scale is not None:
        within(g["dscale"], rows(d * xd), NORM * rows(dsize * xd.abs()), f"{what} dscale")
    if weight is not None:
        within(g["dweight"], rows(dyd * n), NORM * rows((dyd * n).abs()), f"{what} dweight")
    return y, total, rstd, g
