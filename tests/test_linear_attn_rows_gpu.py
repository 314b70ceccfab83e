"""Linear attention on the GPU, every row and head by itself: a norm over a whole
tensor is set by its largest part, so the shortest rows and the fastest heads are
held to their own sizes here (test_linear_attn_fading_gpu.py derives the bounds).
Also the plans that the gradients of unlike widths take, and bf16 gradients
against differences of the definition."""
import pytest
import torch

import layers_ref as ref
import selective_state_space_40_amd as ms
from test_linear_attn_fading_gpu import BF, DEV, F32, STATE, TOKEN, _reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch.cuda.synchronize()


def _make(lengths, length, heads, kv_heads, dk, dv, dtype, seed, decays):
    g = torch.Generator().manual_seed(seed)
    b = len(lengths)

    def n(*shape, dt=F32):
        return torch.randn(*shape, generator=g).to(dt).to(DEV)

    return dict(q=n(b, length, heads, dk, dt=dtype), k=n(b, length, kv_heads, dk, dt=dtype),
                v=n(b, length, kv_heads, dv, dt=dtype), do=n(b, length, heads, dv, dt=dtype),
                log_decay=torch.tensor(decays).to(DEV), h0=n(b, heads, dk, dv), dhL=n(b, heads, dk, dv),
                lengths=torch.tensor(lengths, dtype=torch.int32, device=DEV))


def _rows(i):
    """The definition's results per row: what _reference gives for the row's own
    tokens with its heads' keys and values, gradients of shared ones summed."""
    heads, kv = i["q"].shape[2], i["k"].shape[2]
    out = []
    for r, n in enumerate(i["lengths"].tolist()):
        if n == 0:
            out.append(None)
            continue
        one = {x: i[x][r:r + 1, :n].cpu() for x in ("q", "k", "v", "do")}
        for x in ("k", "v"):
            one[x] = one[x].repeat_interleave(heads // kv, 2)
        tokens, states, dg = _reference(dict(one, log_decay=i["log_decay"], h0=i["h0"][r:r + 1],
                                             dhL=i["dhL"][r:r + 1]))
        for x in ("dk", "dv"):
            g, size = tokens[x]
            share = lambda t: t.unflatten(2, (kv, heads // kv))   # noqa: E731
            tokens[x] = share(g).sum(3), share(size).square().sum(3).sqrt()
        out.append((tokens, states, dg))
    return out


LENGTHS = [0, 1, 31, 32, 33, 63, 64, 65, 130]
DECAYS = [0.0, -0.003, -0.05, -0.2, -0.6, -3.0]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 72), (200, 136), (16, 256)])
def test_every_row_and_head(dk, dv, dtype):
    i = _make(LENGTHS, 130, 6, 3, dk, dv, dtype, dk + 2 * dv, DECAYS)
    rows = _rows(i)
    for seg in (0, 64, 192):
        print(f"case rows {dk}x{dv} {dtype} segment_len={seg}", flush=True)
        o, hL = ms.linear_attn_fwd(i["q"], i["k"], i["v"], i["log_decay"], i["h0"], lengths=i["lengths"],
                                   segment_len=seg)
        got = ms.linear_attn_bwd(i["q"], i["k"], i["v"], i["log_decay"], i["h0"], do=i["do"], dhL=i["dhL"],
                                 lengths=i["lengths"], segment_len=seg)
        torch.cuda.synchronize()
        got.update(o=o, hL=hL)
        got = {k: v.double().cpu() for k, v in got.items()}
        dg, dg_size = torch.zeros(6, dtype=torch.float64), torch.zeros(6, dtype=torch.float64)
        for r, n in enumerate(LENGTHS):
            for x in ("o", "dq", "dk", "dv"):
                assert (got[x][r, n:] == 0).all()
            if n == 0:
                assert torch.equal(got["hL"][r], i["h0"][r].double().cpu())
                assert torch.equal(got["dh0"][r], i["dhL"][r].double().cpu())
                continue
            tokens, states, (g, size) = rows[r]
            dg, dg_size = dg + g, dg_size + size
            for x, (want, size) in tokens.items():
                err = (got[x][r, :n] - want[0]).norm(dim=-1) / (TOKEN[dtype] * size[0])
                assert (err <= 1).all(), f"row {r} {x}: {err.max().item():.3g} times its bound"
            for x, want in states.items():
                err = (got[x][r] - want[0]).flatten(1).norm(dim=-1) / (STATE * want[0].flatten(1).norm(dim=-1))
                assert (err <= 1).all(), f"row {r} {x}: {err.tolist()} times its bound"
        err = (got["dlog_decay"] - dg).abs() / (3e-6 * dg_size)
        assert (err <= 1).all(), f"dlog_decay: {err.tolist()} times its bound"


def _kernels(call):
    from torch.profiler import ProfilerActivity, profile
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    return [e.name for e in p.events() if "linear_attn_kernel<" in e.name]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dk,dv,launches", [(200, 16, 2), (136, 64, 2), (16, 200, 2), (64, 64, 1), (72, 128, 1)])
def test_gradients_launched_at_each_width(dk, dv, launches, dtype):
    # work enough that dq and dk, which contract over dv, and dv, which contracts
    # over dk, are launched apart where the widths' kernels differ
    i = _make([256] * 7 + [201], 256, 16, 16, dk, dv, dtype, dk, [-0.01 * 2 ** (h / 3) for h in range(16)])
    call = lambda: ms.linear_attn_bwd(i["q"], i["k"], i["v"], i["log_decay"], i["h0"], do=i["do"],   # noqa: E731
                                      dhL=i["dhL"], lengths=i["lengths"])
    call()
    names = _kernels(call)
    assert len(names) == launches, names
    _, _, grads = ref.attn(**i)
    ref.check_grads(call(), grads, dtype, f"{dk}x{dv} {dtype}")


def test_bf16_gradients_against_differences():
    # central differences of the 64-bit definition at the inputs as bf16 holds them:
    # the loss is linear in q, k, v and h0, so their quotients are exact; the
    # decay's is off by the step's square. The gradients' own errors, 2.4e-3 in the
    # root mean square and independent, add up along a random direction to 2.4e-3
    # of the two norms' product over the root of their number (4480 at least):
    # 3.6e-5, eight times that allowed. dh0 and the decay's gradient are fp32.
    i = _make([70], 70, 2, 1, 64, 64, BF, 7, [-0.3, -0.02])
    grads = ms.linear_attn_bwd(i["q"], i["k"], i["v"], i["log_decay"], i["h0"], do=i["do"], dhL=i["dhL"])
    _, _, want = ref.attn(**i)

    def loss(**change):
        j = {**i, **change}
        o, h = ref.attn(j["q"], j["k"], j["v"], j["log_decay"], j["h0"])
        return ((o * i["do"].double().cpu()).sum() + (h * i["dhL"].double().cpu()).sum()).item()

    gen = torch.Generator().manual_seed(8)
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("log_decay", "dlog_decay"), ("h0", "dh0")):
        x = i[name].double().cpu()
        d = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        step = 1e-5 if name == "log_decay" else 0.5
        slope = (loss(**{name: x + step * d}) - loss(**{name: x - step * d})) / (2 * step)
        got = (grads[key].double().cpu() * d).sum().item()
        if name == "log_decay":
            bound = 2e-5 * (want["decay_scale"] * d.abs()).sum().item()
        else:
            bound = (3e-6 if name == "h0" else 3e-4) * (want[key].norm() * d.norm()).item()
        assert abs(got - slope) <= bound, f"{name}: {got} against {slope}, bound {bound:.2e}"
