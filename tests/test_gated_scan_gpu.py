"""The gated recurrence on the GPU against 64 bits (gated_ref.py, where the bounds
are derived): sequences, gradients, single tokens."""
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


def _make(b, n, d, dtype, seed, gated=True, state=True, ragged=False, fused=False, decay="mixed"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    both = r(b, n, 2 * d).to(dtype).to(DEV)
    dg, ig = both[..., :d], both[..., d:]
    if not fused:
        dg, ig = dg.clone(), ig.clone()   # on addresses of their own
    u = torch.rand(d, generator=g)
    lam = {"mixed": -torch.pow(10.0, 1.0 - 5.0 * u), "slow": -1e-3 * (0.1 + u), "fast": -1.0 - 7.0 * u}[decay]
    c = dict(x=r(b, n, d).to(dtype).to(DEV), decay_gate=dg, log_decay=lam.to(DEV), input_gate=ig if gated else None,
             h0=r(b, d).to(DEV) if state else None, lengths=None, dy=r(b, n, d).to(dtype).to(DEV),
             dhL=r(b, d).to(DEV) if state else None)
    if ragged:
        lens = torch.randint(0, n + 1, (b,), generator=g, dtype=torch.int32)
        lens[0], lens[-1] = n, 0
        c["lengths"] = lens.to(DEV)
    return c


def _forward(c):
    y, hL, states = ms.gated_scan_fwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"], c["h0"],
                                      lengths=c["lengths"], return_block_states=True)
    return dict(y=y, hL=hL, block_states=states)


def _backward(c, states):
    return ms.gated_scan_bwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"], block_states=states,
                             dy=c["dy"], dhL=c["dhL"], lengths=c["lengths"])


def _drop_behind(c, states):
    """States of blocks that start behind a row's length are not written: zeros."""
    if c["lengths"] is None:
        return states
    first = 64 * torch.arange(states.shape[1], device=DEV)
    return torch.where((first < c["lengths"][:, None])[..., None], states, 0.0)


def _check(c, what):
    _say(f"case {what}")
    got = _forward(c)
    grads = _backward(c, got["block_states"])
    torch.cuda.synchronize()
    want = ref.scan(**c)
    for k in ("block_states", "block_states_size"):
        want[k] = _drop_behind(c, want[k].to(DEV)).cpu()
    got["block_states"] = _drop_behind(c, got["block_states"])
    ref.check_scan(got, want, what)
    ref.check_scan(grads, want, what)
    return got, grads


@TYPES
@pytest.mark.parametrize("n", [1, 2, 7, 16, 63, 64, 65, 127, 128, 129, 192, 257, 300])
def test_lengths(n, dtype):
    _check(_make(2, n, 72, dtype, n), f"2 x {n} x 72 {dtype}")


@TYPES
@pytest.mark.parametrize("d", [1, 2, 3, 8, 63, 64, 65, 66, 128, 130, 191, 200, 513])
def test_widths(d, dtype):
    _check(_make(3, 150, d, dtype, d, fused=d % 8 == 0), f"3 x 150 x {d} {dtype}")


@TYPES
@pytest.mark.parametrize("kw", [dict(gated=False), dict(state=False), dict(ragged=True), dict(ragged=True, state=False),
                                dict(gated=False, ragged=True, fused=True), dict(decay="fast"), dict(decay="slow"),
                                dict(fused=True, decay="slow", ragged=True)],
                         ids=lambda k: "-".join(f"{a}_{b}" for a, b in k.items()))
def test_parts(kw, dtype):
    for d in (96, 77):
        if d % 8 and kw.get("fused"):
            continue
        _check(_make(5, 210, d, dtype, 3, **kw), f"{kw} {d} {dtype}")


@TYPES
def test_many_rows(dtype):
    _check(_make(40, 33, 70, dtype, 9, ragged=True), f"rows {dtype}")


def test_slow_constant_gates_over_long_sequences():
    # the same decay next to 1 at every token: its rounding must not add up. 20,000
    # tokens of memory; every rounding is that of a sum, independent of the others,
    # so that of the 20,000 / 64 tiles adds sqrt(313) * 2 * 2^-24 / sqrt(3) < 2e-6 to
    # the 20 tokens' and segments' 1e-6 and the gates' 1e-6
    n, d = 20000, 64
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1, n, d, generator=g).to(DEV)
    gate = torch.full((1, n, d), 0.3, device=DEV)
    lam = -torch.logspace(-5, -2, d).to(DEV)
    h0 = torch.randn(1, d, generator=g).to(DEV)
    c = dict(x=x, decay_gate=gate, log_decay=lam, input_gate=gate, h0=h0, lengths=None,
             dy=torch.randn(1, n, d, generator=g).to(DEV), dhL=torch.randn(1, d, generator=g).to(DEV))
    got = _forward(c)
    got.update(_backward(c, got["block_states"]))
    want = ref.scan(**c)
    for name, t in got.items():
        err = (t.double().cpu() - want[name]).abs()
        size = want[name + "_size"]
        # a sum of terms of either sign is of the root of their number's size
        units = ref.SCAN_UNITS[name] * ref.STATE
        assert (err <= units * size).all(), f"{name}: {(err / size).max():.2e}"
        rel = (err.norm() / want[name].norm()).item()
        _say(f"case constant gates {name}: {rel:.2e}")
        assert rel <= 4e-6 * (3 if name in ("ddecay_gate", "dlog_decay") else 1), name


def test_remainder_of_a_large_state():
    # what is left of a state far above all that enters behind it
    c = _make(2, 200, 64, F32, 4, decay="fast")
    c["h0"] = 1e20 * torch.ones(2, 64, device=DEV)
    c["x"].zero_()
    c["log_decay"].fill_(-0.1)
    got = _forward(c)
    want = ref.scan(**{k: v for k, v in c.items() if k not in ("dy", "dhL")})
    # log a is off by 11 * 2^-24 of itself, and 200 * 0.1 * sigmoid of it are added
    total = 0.1 * torch.sigmoid(c["decay_gate"].double().cpu()).sum(1)
    bound = (64 + 12 * total) * 2.0 ** -24
    assert ((got["hL"].double().cpu() / want["hL"] - 1).abs() <= bound).all()


@TYPES
def test_tokens_continue_a_sequence(dtype):
    c = _make(3, 70, 88, dtype, 5, fused=True)
    whole = _forward(c)
    cut = {k: (v[:, :60] if k in ("x", "decay_gate", "input_gate") else v) for k, v in c.items()}
    cut["x"] = cut["x"].contiguous()
    cut["decay_gate"], cut["input_gate"] = cut["decay_gate"].contiguous(), cut["input_gate"].contiguous()
    h = _forward(cut)["hL"]
    want = ref.scan(**{k: v for k, v in c.items() if k not in ("dy", "dhL")})
    for t in range(60, 70):
        y = ms.gated_scan_update(h, c["x"][:, t], c["decay_gate"][:, t], c["log_decay"], c["input_gate"][:, t])
        ref.within(y, want["y"][:, t], ref.STATE * want["y_size"][:, t], f"token {t}")
    ref.within(h, want["hL"], ref.STATE * want["hL_size"], "state")
    ref.within(whole["hL"], want["hL"], ref.STATE * want["hL_size"], "whole")


@TYPES
@pytest.mark.parametrize("shape", [(1, 1), (1, 64), (7, 33), (300, 1540), (64, 5120)], ids=str)
def test_single_tokens(shape, dtype):
    b, d = shape
    for gated in (True, False):
        c = _make(b, 1, d, dtype, b + d, gated=gated)
        h = c["h0"].clone()
        _say(f"case token {shape} {dtype} {gated}")
        args = [None if c[k] is None else c[k][:, 0] for k in ("x", "decay_gate", "input_gate")]
        y = ms.gated_scan_update(h, args[0], args[1], c["log_decay"], args[2])
        want = ref.scan(**{k: v for k, v in c.items() if k not in ("dy", "dhL")})
        ref.within(y, want["y"][:, 0], ref.STATE * want["y_size"][:, 0], "y")
        ref.within(h, want["hL"], ref.STATE * want["hL_size"], "state")


def test_large_and_closed_gates():
    # gates far out: sigmoid near 0 and 1, decays from 1 to 0
    n, d = 90, 40
    edge = torch.tensor([-120.0, -60.0, -20.0, -8.0, 8.0, 20.0, 60.0, 120.0])
    g = torch.Generator().manual_seed(8)
    pick = lambda: edge[torch.randint(0, 8, (2, n, d), generator=g)].to(DEV)   # noqa: E731
    c = _make(2, n, d, F32, 8)
    c["decay_gate"], c["input_gate"] = pick(), pick()
    c["log_decay"] = -torch.logspace(-3, 2, d).to(DEV)
    got = _forward(c)
    got.update(_backward(c, got["block_states"]))
    want = ref.scan(**c)
    # |r| 2^-25 more for each sigmoid, |r| up to 120. A sigmoid below 2^-126 may count
    # as zero or as that: 1 - a^2 = 2 |log_decay| p is then off by up to 200 * 2^-126, its
    # root, the weight of one token, by 1.6e-18. 90 tokens of |x| < 5, or adjoints below
    # 90 * 5 times that weight, add up to 7e-16 at most.
    for name, t in got.items():
        w = want[name]
        assert torch.isfinite(t).all(), name
        err = (t.double().cpu() - w).abs()
        bound = ref.SCAN_UNITS[name] * (ref.STATE + 2 * 120 * 2.0 ** -25) * want[name + "_size"] + 7e-16
        assert (err <= bound).all(), f"{name}: {(err / bound).max():.3g}"


def test_nan_and_infinity_stay_in_their_channel():
    for dtype in (BF, F32):
        c = _make(2, 200, 70, dtype, 6, decay="fast")
        clean = _forward(c)
        grads = _backward(c, clean["block_states"])
        c["x"][0, 90, 5] = float("nan")
        c["x"][1, 130, 69] = float("inf")
        got = _forward(c)
        assert torch.equal(got["y"][0, :90], clean["y"][0, :90]) and torch.isnan(got["y"][0, 90:, 5]).all()
        others = [i for i in range(70) if i not in (5, 69)]
        assert torch.equal(got["y"][..., others], clean["y"][..., others])
        assert torch.equal(got["y"][1, :130], clean["y"][1, :130])
        g = _backward(c, got["block_states"])
        for name in ("dx", "ddecay_gate", "dinput_gate"):
            assert torch.equal(g[name][..., others], grads[name][..., others]), name
        assert torch.isnan(g["dlog_decay"][5]) and torch.isfinite(g["dlog_decay"][others]).all()
        c["dy"][0, 40, 8] = float("nan")
        g = _backward(c, got["block_states"])
        assert torch.isnan(g["dx"][0, :41, 8]).all() and torch.isfinite(g["dx"][0, 41:, 8]).all()


def test_what_stands_behind_a_row_is_not_read_and_rows_may_be_empty():
    for dtype in (BF, F32):
        c = _make(4, 140, 66, dtype, 7)
        c["lengths"] = torch.tensor([70, 0, 140, 129], dtype=torch.int32, device=DEV)
        got = _forward(c)
        grads = _backward(c, got["block_states"])
        for k in ("x", "decay_gate", "input_gate", "dy"):
            c[k] = c[k].clone()
            c[k][0, 70:] = float("nan")
            c[k][1] = float("nan")
            c[k][3, 129:] = float("inf")
        again = _forward(c)
        assert torch.equal(again["y"], got["y"]) and torch.equal(again["hL"], got["hL"])
        more = _backward(c, again["block_states"])
        for k in grads:
            assert torch.equal(more[k], grads[k]), k
        assert not got["y"][0, 70:].any() and not got["y"][1].any()
        assert torch.equal(got["hL"][1], c["h0"][1]) and torch.equal(grads["dh0"][1], c["dhL"][1])
        # lengths out of range count as none and all
        c2 = _make(2, 30, 66, dtype, 7)
        full = _forward(c2)
        c2["lengths"] = torch.tensor([31, -1], dtype=torch.int32, device=DEV)
        odd = _forward(c2)
        assert torch.equal(odd["y"][0], full["y"][0]) and not odd["y"][1].any()
        assert torch.equal(odd["hL"][1], c2["h0"][1])


def test_no_tokens_no_rows():
    c = _make(3, 0, 40, F32, 1)
    got = _forward(c)
    assert got["y"].shape == (3, 0, 40) and torch.equal(got["hL"], c["h0"])
    g = _backward(c, got["block_states"])
    assert torch.equal(g["dh0"], c["dhL"]) and not g["dlog_decay"].any()
    c = _make(3, 0, 40, F32, 1, state=False)
    got = _forward(c)
    assert not got["hL"].any()
    c = _make(0, 5, 40, BF, 1)
    g = _backward(c, _forward(c)["block_states"])
    assert g["dx"].shape == (0, 5, 40) and not g["dlog_decay"].any()


def test_outputs_given_and_wanted():
    c = _make(2, 100, 64, BF, 2)
    want = _forward(c)
    out, state = torch.empty_like(c["x"]), c["h0"].clone()
    y, hL, none = ms.gated_scan_fwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"], state, out=out,
                                    state_out=state)
    assert y is out and hL is state and none is None
    assert torch.equal(y, want["y"]) and torch.equal(hL, want["hL"])
    y, hL, _ = ms.gated_scan_fwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"], c["h0"], return_state=False)
    assert hL is None and torch.equal(y, want["y"])
    full = _backward(c, want["block_states"])
    part = ms.gated_scan_bwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"],
                             block_states=want["block_states"], dy=c["dy"], dhL=c["dhL"], want_dlog_decay=False,
                             want_dh0=False)
    assert part["dlog_decay"] is None and part["dh0"] is None
    for k in ("dx", "ddecay_gate", "dinput_gate"):
        assert torch.equal(part[k], full[k])


def test_slices_of_wider_tensors():
    # every input a slice of channels, at odd strides too where they start on 16 bytes
    for dtype, wide in ((BF, 200), (BF, 201), (F32, 200), (F32, 203)):
        g = torch.Generator().manual_seed(wide)
        b, n, d = 1, 90, 64
        c = _make(b, n, d, dtype, wide)
        base = torch.randn(3, b, n, wide, generator=g).to(dtype).to(DEV)
        for i, k in enumerate(("x", "decay_gate", "input_gate")):
            at = base[i].data_ptr() % 16 // base.element_size()
            base[i, ..., at:at + d] = c[k]
            if at == 0:
                c[k + "_s"] = base[i, ..., :d]
        c["x_s"] = c.get("x_s", c["x"])
        want = ref.scan(**{k: c[k] for k in ("x", "decay_gate", "log_decay", "input_gate", "h0")})
        y, hL, _ = ms.gated_scan_fwd(c["x_s"], c.get("decay_gate_s", c["decay_gate"]), c["log_decay"],
                                     c.get("input_gate_s", c["input_gate"]), c["h0"])
        ref.check_scan(dict(y=y, hL=hL), want, f"{dtype} {wide}")


def test_gradients_against_differences():
    # central differences of the 64-bit definition, error O(step^2)
    c = _make(2, 90, 20, F32, 11)
    got = _backward(c, _forward(c)["block_states"])
    names = dict(x="dx", decay_gate="ddecay_gate", input_gate="dinput_gate", log_decay="dlog_decay", h0="dh0")
    base = {k: ref.d64(v) for k, v in c.items()}

    def loss(**change):
        o = ref.scan(**{**{k: v for k, v in base.items() if k not in ("dy", "dhL")}, **change})
        return ((o["y"] * base["dy"]).sum() + (o["hL"] * base["dhL"]).sum()).item()

    g = torch.Generator().manual_seed(12)
    for k, name in names.items():
        d = torch.randn(base[k].shape, generator=g, dtype=torch.float64)
        if k == "log_decay":
            d = d * base[k].abs()
        up, down = loss(**{k: base[k] + 1e-5 * d}), loss(**{k: base[k] - 1e-5 * d})
        want = (got[name].double().cpu() * d).sum().item()
        size = (got[name].double().cpu().norm() * d.norm()).item()
        assert abs((up - down) / 2e-5 - want) <= 2e-5 * size, name


def test_reproducible_and_on_another_stream():
    c = _make(3, 400, 130, BF, 13, ragged=True)
    got = _forward(c)
    grads = _backward(c, got["block_states"])
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    for _ in range(3):
        with torch.cuda.stream(side):
            more = _forward(c)
            mg = _backward(c, _drop_behind(c, more["block_states"]))
        side.synchronize()
        for k in ("y", "hL"):
            assert torch.equal(more[k], got[k]), k
        for k in grads:
            assert torch.equal(mg[k], grads[k]), k


def test_captured_calls_replay():
    c = _make(4, 700, 96, BF, 14, ragged=True)
    h = torch.randn(4, 96, device=DEV)
    first = h.clone()

    def calls():
        f = _forward(c)
        g = _backward(c, f["block_states"])
        y = ms.gated_scan_update(h, c["x"][:, 0], c["decay_gate"][:, 0], c["log_decay"], c["input_gate"][:, 0])
        return [f["y"], f["hL"], *g.values(), y, h]

    want = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for r in range(4):
        for t in got:
            t.fill_(float("nan"))
        h.copy_(first)
        torch.randn(1 << 16, device=DEV).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip(got, want):
            assert torch.equal(a, e), f"replay {r}"
