"""Linear attention and layer norm in 64 bits on the CPU, token by token from
their definitions, for the tests of the GPU kernels. Holds no chunk algebra.

Also the tests' tolerances. A value rounded to bf16 is off by at most 2^-8 of
itself and, as a rounding error is spread evenly over its half step and
mantissas over an octave, by about 2^-8 / sqrt(3) * 0.72 < 1.7e-3 in the
root mean square; an fp32 rounding by 2^-24 likewise.

bf16 outputs: the output's rounding, that of P (its terms are independent, so
the sum's relative error is P's) and that of the state as an operand, each
1.7e-3 of the part it acts on; P and the state act on different parts of the
sum, so two of the three together: sqrt(2) * 1.7e-3 = 2.4e-3, taken as 4e-3.
Elementwise: 2^-8 of the value for the output and 2^-8 of terms that add up
incoherently to the largest outputs; 2.5 * 2^-8 < 1e-2 of the largest value.

fp32 results, from fp32 or bf16 inputs (products of bf16 values are exact and
what the kernel splits into three bf16 terms keeps 2^-25): sums of n = dk + 64 + chunks terms in fp32 round n times, errors
independent, each 2^-24 / sqrt(3) of a partial sum: sqrt(400) * 3.5e-8 = 7e-7
for the longest here; the powers of the decay add 2^-23; taken as 3e-6, and
1.5e-5 of the largest elementwise.

The decay's gradient adds terms of the same fp32 accuracy, 7e-7 of their size,
with errors that add up no faster than the terms. It is bounded by the sum over
tokens of |dS_t . lam S_(t-1)|, in which the pairs of tokens that a token lies
between add up with any sign, to about the root of their number (under 200
here): sqrt(200) * 7e-7 = 1e-5 of that sum. Where the decay's own power is below
2^-126, the smallest normal fp32 number, fp32 holds none of it: the gradient may
be off by 2^-126 times the sum of |S| |dS|, under 1e8 here.
"""
import torch

TWO_NORM = {"bf16": 4e-3, "f32": 3e-6}
LARGEST = {"bf16": 1e-2, "f32": 1.5e-5}
DECAY_GRAD = 1e-5


def check(got, want, kind, what):
    g, w = got.detach().double().cpu(), want.double().cpu()
    assert g.shape == w.shape, f"{what}: shape {tuple(g.shape)}, expected {tuple(w.shape)}"
    assert torch.isfinite(g).all(), f"{what}: non-finite values"
    if w.numel() == 0:
        return
    err, norm = (g - w).norm().item(), w.norm().item()
    assert err <= TWO_NORM[kind] * norm, f"{what}: error {err / max(norm, 1e-300):.3e} (2-norm)"
    worst, top = (g - w).abs().max().item(), w.abs().max().item()
    assert worst <= LARGEST[kind] * top, f"{what}: error {worst / max(top, 1e-300):.3e} (largest)"


def _heads(x, heads):
    return x.double().cpu().repeat_interleave(heads // x.shape[-2], -2)


def attn(q, k, v, log_decay, h0=None, lengths=None, scale=None, do=None, dhL=None):
    """(o, hL), and with `do` the gradients' dict as well, with `decay_scale`:
    per head the sum over tokens of |dS_t . lam S_(t-1)|."""
    b, n, h, dk = q.shape
    dv = v.shape[-1]
    scale = dk ** -0.5 if scale is None else scale
    qd, kd, vd = q.double().cpu(), _heads(k, h), _heads(v, h)
    lam = log_decay.double().cpu().exp()[:, None, None]
    start = torch.zeros(b, h, dk, dv, dtype=torch.float64) if h0 is None else h0.double().cpu()
    lens = [n] * b if lengths is None else [max(0, min(n, int(x))) for x in lengths.cpu()]
    o = torch.zeros(b, n, h, dv, dtype=torch.float64)
    end = start.clone()
    states = []
    for r in range(b):
        s, kept = start[r], []
        for t in range(lens[r]):
            kept.append(s)
            s = lam * s + kd[r, t][:, :, None] * vd[r, t][:, None, :]
            o[r, t] = scale * (qd[r, t][:, None, :] @ s)[:, 0]
        end[r] = s
        states.append(kept)
    if do is None:
        return o, end
    dod = do.double().cpu()
    dq, dkk = torch.zeros_like(qd), torch.zeros_like(kd)
    dvv = torch.zeros_like(vd)
    dh0 = torch.zeros_like(start) if dhL is None else dhL.double().cpu().clone()
    dg, mag = torch.zeros(h, dtype=torch.float64), torch.zeros(h, dtype=torch.float64)
    for r in range(b):
        adj = dh0[r].clone()
        for t in reversed(range(lens[r])):
            before = states[r][t]
            s = lam * before + kd[r, t][:, :, None] * vd[r, t][:, None, :]
            adj = adj + scale * qd[r, t][:, :, None] * dod[r, t][:, None, :]
            dq[r, t] = scale * (s @ dod[r, t][:, :, None])[:, :, 0]
            dkk[r, t] = (adj @ vd[r, t][:, :, None])[:, :, 0]
            dvv[r, t] = (kd[r, t][:, None, :] @ adj)[:, 0]
            term = (adj * lam * before).sum((1, 2))
            dg, mag = dg + term, mag + term.abs()
            adj = lam * adj
        dh0[r] = adj
    rep = h // k.shape[-2]
    share = lambda x: x.view(b, n, h // rep, rep, -1).sum(3)   # noqa: E731
    return o, end, dict(dq=dq, dk=share(dkk), dv=share(dvv), dlog_decay=dg, dh0=dh0,
                        decay_scale=mag)


def attn_token(h, q, k, v, log_decay, scale=None):
    """(o, new state) of one token."""
    heads = q.shape[1]
    o, s = attn(q[:, None], k[:, None], v[:, None], log_decay, h, scale=scale)
    assert s.shape[1] == heads
    return o[:, 0], s


def check_grads(got, want, dtype, what):
    kind = "bf16" if dtype == torch.bfloat16 else "f32"
    for name in ("dq", "dk", "dv"):
        check(got[name], want[name], kind, f"{what} {name}")
    if got["dh0"] is not None:
        check(got["dh0"], want["dh0"], "f32", f"{what} dh0")
    if got["dlog_decay"] is not None:
        err = (got["dlog_decay"].double().cpu() - want["dlog_decay"]).abs()
        bound = DECAY_GRAD * want["decay_scale"] + 2.0 ** -126 * 1e8
        assert (err <= bound).all(), (f"{what} dlog_decay: {err.tolist()} beyond {bound.tolist()}, "
                                      f"values {want['dlog_decay'].tolist()}")


def norm(x, weight=None, bias=None, groups=1, eps=1e-5):
    """(y, mean, rstd)."""
    xd = x.double().cpu()
    parts = xd.reshape(*x.shape[:-1], groups, x.shape[-1] // groups)
    mean = parts.mean(-1)
    rstd = ((parts - mean[..., None]).square().mean(-1) + eps).rsqrt()
    y = ((parts - mean[..., None]) * rstd[..., None]).reshape(xd.shape)
    if weight is not None:
        y = y * weight.double().cpu()
    if bias is not None:
        y = y + bias.double().cpu()
    return y, mean, rstd


def norm_grads(x, weight, dy, groups=1, eps=1e-5):
    """(dx, dweight, dbias) of sum(dy * y) by differentiating norm() itself."""
    xd = x.double().cpu().requires_grad_()
    w = (torch.ones(x.shape[-1], dtype=torch.float64) if weight is None
         else weight.double().cpu()).requires_grad_()
    b = torch.zeros(x.shape[-1], dtype=torch.float64, requires_grad=True)
    y, _, _ = norm(xd, w, b, groups, eps)
    return torch.autograd.grad((y * dy.double().cpu()).sum(), (xd, w, b))
