"""Which form a call of the gated recurrence runs in, by the kernels that it
launches, and the forms at what other tests leave out: tiles in the rows' own order,
and inputs of unlike odd strides."""
import sys

import pytest
import torch
from torch.profiler import ProfilerActivity, profile

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


def _make(b, n, d, dtype, seed, lengths=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=dtype: torch.randn(*s, generator=g).to(dt).to(DEV)   # noqa: E731
    lam = -torch.pow(10.0, 1.0 - 5.0 * torch.rand(d, generator=g)).to(DEV)
    return dict(x=r(b, n, d), decay_gate=r(b, n, d), log_decay=lam, input_gate=r(b, n, d), h0=r(b, d, dt=F32),
                dy=r(b, n, d), dhL=r(b, d, dt=F32),
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV))


def _forward(c):
    y, hL, states = ms.gated_scan_fwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"], c["h0"],
                                      lengths=c["lengths"], return_block_states=True)
    return dict(y=y, hL=hL, block_states=states)


def _backward(c, states):
    return ms.gated_scan_bwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"], block_states=states,
                             dy=c["dy"], dhL=c["dhL"], lengths=c["lengths"])


def _chained(call):
    """Whether the call's tiles go to workgroups one by one; its result."""
    call()
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        out = call()
        torch.cuda.synchronize()
    names = [e.name for e in p.events() if "gated_scan_" in e.name]
    chains = sum("_chain_kernel" in n for n in names)
    walks = sum("gated_scan_fwd_kernel" in n or "gated_scan_bwd_kernel" in n for n in names)
    assert chains + walks == 1, names
    return chains == 1, out


def _live(c, states):
    """The states of blocks with tokens; zeros for others, which are not written."""
    if c["lengths"] is None:
        return states
    first = 64 * torch.arange(states.shape[1], device=states.device)
    return torch.where((first < c["lengths"].to(states.device)[:, None])[..., None], states, 0.0)


@TYPES
def test_more_rows_than_are_put_in_order(dtype):
    # Above 512 rows a chain's tiles come in the rows' own order, those without tokens
    # between the others. The gradients in bf16 are walked at any such number.
    n, b, d = 1500, 513, 8
    g = torch.Generator().manual_seed(b)
    lens = torch.randint(0, n + 1, (b,), generator=g)
    lens[::7], lens[3::11] = 0, n
    c = _make(b, n, d, dtype, 13, lengths=lens.to(torch.int32).tolist())
    chain, got = _chained(lambda: _forward(c))
    assert chain
    chain, grads = _chained(lambda: _backward(c, got["block_states"]))
    assert chain == (dtype == F32)
    want = ref.scan(**c)
    for k in ("block_states", "block_states_size"):
        want[k] = _live(c, want[k])
    got["block_states"] = _live(c, got["block_states"])
    _say(f"case {b} x {n} x {d} {dtype}")
    ref.check_scan(got, want, "rows in their own order")
    ref.check_scan(grads, want, "rows in their own order")


@pytest.mark.parametrize("b,n,d,ragged,want", [
    (1, 511, 70, False, "walk"), (1, 512, 70, False, "chain"), (1, 600, 63, False, "chain"),
    (200, 600, 64, False, "walk forward"), (9, 2500, 66, True, "chain"), (23, 4000, 70, True, "chain"),
    (2, 9000, 130, True, "chain"), (3, 5000, 130, True, "chain"), (2, 1300, 66, False, "chain"),
    (1, 3000, 192, True, "chain"), (1, 30000, 512, False, "chain"), (2, 17000, 320, False, "chain")], ids=str)
@TYPES
def test_forms_that_other_tests_mean(b, n, d, ragged, want, dtype):
    # the sizes at which tests compare one form with 64 bits, itself or the other form
    c = _make(b, n, d, dtype, n, lengths=[n - 77 * i for i in range(b)] if ragged else None)
    _say(f"case {b} x {n} x {d} {ragged} {dtype}")
    chain, got = _chained(lambda: _forward(c))
    assert chain == (want == "chain")
    if want != "walk forward":
        assert _chained(lambda: _backward(c, got["block_states"]))[0] == chain


def _slice(t, wide):
    """The same values in a wider tensor of its own, whose rows are `wide` apart."""
    base = torch.full((*t.shape[:-1], wide), float("nan"), dtype=t.dtype, device=DEV)
    base[..., :t.shape[-1]] = t
    assert base.data_ptr() % 16 == 0
    return base[..., :t.shape[-1]]


# two channels to a lane forward; the odd stride at each input by turns; all unlike;
# the single token's four channels a lane, and not
STRIDES = [(200, 208, 216), (201, 200, 200), (200, 203, 200), (200, 200, 207), (201, 203, 207), (202, 206, 210)]


@TYPES
@pytest.mark.parametrize("strides", STRIDES, ids=str)
@pytest.mark.parametrize("n,lens", [(90, None), (1300, None), (1300, [1300, 801])], ids=["walk", "chain", "ragged"])
def test_inputs_of_unlike_strides(strides, n, lens, dtype):
    for d in (64, 66):
        c = _make(2, n, d, dtype, d, lengths=lens)
        want = ref.scan(**c)
        for k in ("block_states", "block_states_size"):
            want[k] = _live(c, want[k])
        for k, wide in zip(("x", "decay_gate", "input_gate"), strides):
            c[k] = _slice(c[k], wide)
        _say(f"case {strides} {n} x {d} {dtype}")
        chain, got = _chained(lambda: _forward(c))
        assert chain == (n > 1000)
        grads = _backward(c, got["block_states"])
        got["block_states"] = _live(c, got["block_states"])
        ref.check_scan(got, want, f"{strides}")
        ref.check_scan(grads, want, f"{strides}")


@TYPES
@pytest.mark.parametrize("strides", STRIDES, ids=str)
def test_single_tokens_of_unlike_strides(strides, dtype):
    for d in (64, 66, 63):
        c = _make(5, 1, d, dtype, d)
        want = ref.scan(**{k: v for k, v in c.items() if k not in ("dy", "dhL")})
        h = c["h0"].clone()
        x, dg, ig = (_slice(c[k][:, 0], wide) for k, wide in zip(("x", "decay_gate", "input_gate"), strides))
        _say(f"case token {strides} {d} {dtype}")
        y = ms.gated_scan_update(h, x, dg, c["log_decay"], ig)
        ref.within(y, want["y"][:, 0], ref.STATE * want["y_size"][:, 0], "y")
        ref.within(h, want["hL"], ref.STATE * want["hL_size"], "state")


@TYPES
def test_slices_that_start_off_16_bytes_are_refused(dtype):
    # halves of one projection start on 16 bytes where a half is a multiple of that
    size = 16 // (2 if dtype == BF else 4)
    for d, fits in ((8 * size, True), (8 * size + 1, False), (8 * size + size // 2, False)):
        both = torch.randn(3, 5, 2 * d, device=DEV).to(dtype)
        x, z = both.split(d, -1)
        lam = -torch.rand(d, device=DEV)
        h = torch.zeros(3, d, device=DEV)
        dy = torch.randn(3, 5, d, device=DEV).to(dtype)
        rstd = torch.ones(3, 5, 1, device=DEV)
        states = torch.zeros(3, 1, d, device=DEV)
        calls = [lambda x, z: ms.gated_scan_fwd(x, z, lam)[0],
                 lambda x, z: ms.gated_scan_bwd(x, z, lam, block_states=states, dy=dy)["dx"],
                 lambda x, z: ms.gated_scan_update(h.clone(), x[:, 0], z[:, 0], lam),
                 lambda x, z: ms.gated_norm_fwd(x, z)[0],
                 lambda x, z: ms.gated_norm_bwd(x, z, None, rstd, dy=dy)["dx"]]
        for i, call in enumerate(calls):
            if fits:
                assert torch.equal(call(x, z), call(x.contiguous(), z.contiguous())), i
            else:
                with pytest.raises(ms.MambaScanError) as e:
                    call(x, z)
                assert e.value.status == -3, i
                call(x, z.contiguous())
