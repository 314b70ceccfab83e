"""Gates that are closed for good: of the type's lowest value or near it, as masks
write them. What such a gate lets through is zero, forward and in the gradients,
however large the value behind it is."""
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


@TYPES
@pytest.mark.parametrize("first", [True, False], ids=["first", "behind"])
@pytest.mark.parametrize("dim,groups", [(40, 1), (333, 1), (640, 5), (1531, 1), (5120, 1), (9000, 1)])
def test_norm_gate_of_the_lowest_value(dim, groups, first, dtype):
    # silu(z) = z / (1 + exp(-z)) is 0 in fp32 from z = -200 down, where it is below 1e-84:
    # times |x|, |dy| < 6, weights < 2 and rstd <= 1e-5^-0.5 < 317 below 1e-79. A row
    # whose gates are all closed has v = 0: y = 0, and nothing reaches x or z.
    g = torch.Generator().manual_seed(dim)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    rows = 9
    far = torch.tensor([-200.0, -1e5, -1e20, -1e37, torch.finfo(dtype).min])
    shut = torch.rand(rows, dim, generator=g) < 0.3
    shut[4] = True
    z = torch.where(shut, far[torch.randint(0, len(far), (rows, dim), generator=g)], r(rows, dim))
    x, z, dy = (t.to(dtype).to(DEV) for t in (r(rows, dim), z, r(rows, dim)))
    w = (1 + 0.2 * r(dim)).to(DEV)
    _say(f"case {dim} in {groups} {dtype} {first}")
    y, rstd, grads = ref.check_gated(ms, x, z, w, dy, groups, first, f"{dim} in {groups}", floor=1e-79)
    shut = shut.to(DEV)
    assert not bool(y[shut].any()) and not bool(grads["dz"][shut].any())
    assert not first or not bool(grads["dx"][shut].any())


def _sequences(b, n, d, dtype, seed, gated=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=dtype: torch.randn(*s, generator=g).to(dt).to(DEV)   # noqa: E731
    return dict(x=r(b, n, d), decay_gate=r(b, n, d), log_decay=-torch.logspace(-3, 1, d).to(DEV),
                input_gate=r(b, n, d) if gated else None, h0=r(b, d, dt=F32), dy=r(b, n, d),
                dhL=r(b, d, dt=F32)), (torch.rand(b, n, d, generator=g) < 0.3).to(DEV)


def _results(c):
    y, hL, states = ms.gated_scan_fwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"], c["h0"],
                                      return_block_states=True)
    g = ms.gated_scan_bwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"], block_states=states,
                          dy=c["dy"], dhL=c["dhL"])
    return dict(y=y, hL=hL, block_states=states, **g)


@TYPES
@pytest.mark.parametrize("n", [100, 1300])   # walked, and in bf16 and fp32 a chain
@pytest.mark.parametrize("which,gate", [("input_gate", -2000.0), ("input_gate", "lowest"), ("input_gate", "infinite"),
                                        ("decay_gate", -2000.0), ("decay_gate", "lowest"), ("decay_gate", "infinite")])
def test_nothing_enters_through_a_closed_gate(which, gate, n, dtype):
    # exp(-2000) is 0 in 64 bits: the token's weight w is 0 by either gate, so x counts
    # as 0 there, the type's lowest value as well, and it has no gradient
    c, shut = _sequences(2, n, 66, dtype, n, gated=True)
    low = torch.finfo(dtype).min
    value = dict(lowest=low, infinite=float("-inf")).get(gate, gate)
    c[which] = torch.where(shut, torch.tensor(value, dtype=dtype, device=DEV), c[which])
    _say(f"case {which} {gate} {n} {dtype}")
    c["x"] = torch.where(shut, torch.tensor(0, dtype=dtype, device=DEV), c["x"])
    want = _results(c)
    if which == "input_gate" and gate == -2000.0:
        exact = ref.scan(**c)
        # 2000 2^-25 log2(e) more of a sigmoid that is 0 all the same
        ref.check_scan({k: t for k, t in want.items() if k != "block_states"}, exact, "closed")
    c["x"] = torch.where(shut, torch.tensor(low, dtype=dtype, device=DEV), c["x"])
    got = _results(c)
    for k, t in got.items():
        assert bool(torch.isfinite(t).all()), k
        assert bool((t == want[k]).all()), k
    assert not bool(got["dx"][shut].any())


@TYPES
@pytest.mark.parametrize("n", [100, 1300])
def test_decays_of_the_lowest_value(n, dtype):
    # log_decay may be any finite number: next to -1e30, where a is 0 behind any gate
    # that is not closed (exp(-1e30 sigmoid(-40)) is), the lowest one gives the same; behind
    # a closed one a is 1 and nothing enters
    c, shut = _sequences(2, n, 66, dtype, n)
    c["decay_gate"] = torch.where(shut, torch.tensor(float("-inf"), dtype=dtype, device=DEV),
                                  c["decay_gate"].clamp(min=-40))
    low = torch.finfo(F32).min
    _say(f"case {n} {dtype}")
    c["log_decay"][1::2] = -1e30
    want = _results(c)
    h = c["h0"].clone()
    token = ms.gated_scan_update(h, c["x"][:, 0], c["decay_gate"][:, 0], c["log_decay"], c["input_gate"][:, 0])
    for k, t in want.items():
        assert bool(torch.isfinite(t).all()), k
    for value in (low, 0.75 * low):
        c["log_decay"][1::2] = value
        got = _results(c)
        for k, t in got.items():
            assert bool((t == want[k]).all()), (k, value)
        h2 = c["h0"].clone()
        again = ms.gated_scan_update(h2, c["x"][:, 0], c["decay_gate"][:, 0], c["log_decay"], c["input_gate"][:, 0])
        assert bool((again == token).all()) and bool((h2 == h).all())
