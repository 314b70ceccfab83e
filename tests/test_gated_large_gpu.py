"""The gated operators on tensors whose last rows or tokens start past 2^32 elements:
offsets of 32 bits would reach earlier ones. What stands before is empty, zero or far
away, so that the 64-bit reference needs the last only. Takes up to 90 GB of the GPU's
memory."""
import pytest
import torch

import gated_ref as ref
import selective_state_space_40_amd as ms

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
PAST = 1 << 32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info(DEV)[0] < 120 << 30:
        pytest.skip("less than 120 GB of GPU memory free")
    ms.load_library()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _grads(c, states):
    return ms.gated_scan_bwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"], block_states=states,
                             dy=c["dy"], lengths=c["lengths"])


def test_rows_of_a_batch():
    # 17 rows of 65536 tokens by 4096 channels: the last row starts at element 2^32 of
    # each tensor; its 150 tokens are the only ones
    batch, length, dim, n = 17, 65536, 4096, 150
    assert (batch - 1) * length * dim == PAST
    g = torch.Generator(DEV).manual_seed(1)

    def rows():
        t = torch.empty(batch, length, dim, dtype=BF, device=DEV)
        t[0, :n] = float("nan")   # where offsets cut to 32 bits would read
        t[-1, :n] = torch.randn(n, dim, generator=g, device=DEV).to(BF)
        return t

    c = {k: rows() for k in ("x", "decay_gate", "input_gate", "dy")}
    c["log_decay"] = -torch.logspace(0, -3, dim, device=DEV)
    c["lengths"] = torch.zeros(batch, dtype=torch.int32, device=DEV)
    c["lengths"][-1] = n
    last = {k: t[-1:, :n] if t.dim() == 3 else t for k, t in c.items() if k != "lengths"}
    want = ref.scan(**last)
    print("case rows past 2^32 elements", flush=True)
    y, hL, states = ms.gated_scan_fwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"], lengths=c["lengths"],
                                      return_block_states=True)
    torch.cuda.synchronize()
    assert not y[:-1].any() and not y[-1, n:].any() and not hL[:-1].any()
    ref.check_scan(dict(y=y[-1:, :n], hL=hL[-1:], block_states=states[-1:, :3]), want, "rows")
    del y
    got = _grads(c, states)
    torch.cuda.synchronize()
    for k in ("dx", "ddecay_gate", "dinput_gate"):
        assert not got[k][:-1].any() and not got[k][-1, n:].any(), k
        got[k] = got[k][-1:, :n]
    assert not got["dh0"][:-1].any()
    got["dh0"] = got["dh0"][-1:]
    ref.check_scan(got, want, "rows")


def test_tokens_of_a_row():
    # one row of 2^21 + 300 tokens by 2048 channels: the last 300 start at element 2^32.
    # Those before have no inputs and no gradients but what comes from behind, which a
    # decay of e^-0.5 a token leaves nothing of within 300
    length, dim, n = (1 << 21) + 300, 2048, 300
    g = torch.Generator(DEV).manual_seed(2)
    c = {k: torch.zeros(1, length, dim, dtype=BF, device=DEV) for k in ("x", "decay_gate", "input_gate", "dy")}
    for t in c.values():
        t[:, -n:] = torch.randn(n, dim, generator=g, device=DEV).to(BF)
    c["log_decay"] = torch.full((dim,), -1.0, device=DEV)
    c["lengths"] = None
    print("case tokens past 2^32 elements", flush=True)
    y, hL, states = ms.gated_scan_fwd(c["x"], c["decay_gate"], c["log_decay"], c["input_gate"],
                                      return_block_states=True)
    torch.cuda.synchronize()
    want = ref.scan(**{k: t[:, -n:] if t.dim() == 3 else t for k, t in c.items() if k != "lengths"})
    ref.check_scan(dict(y=y[:, -n:], hL=hL), want, "tokens")
    assert not y[:, :-n].any() and not states[:, :(1 << 21) // 64].any()
    ref.within(states[:, -5:], want["block_states"], ref.STATE * want["block_states_size"], "states")
    del y
    got = _grads(c, states)
    torch.cuda.synchronize()
    assert not got["dh0"].any()
    for k in ("dx", "ddecay_gate", "dinput_gate"):
        assert not got[k][:, :1 << 20].any(), k
        got[k] = got[k][:, -n:]
    del got["dh0"], got["dlog_decay"]   # the sum over all tokens has those before as well
    ref.check_scan(got, want, "tokens")


@pytest.mark.parametrize("groups", [1, 64])
def test_norms(groups):
    # 2^20 + 3 rows of 4096: the last three start past 2^32 elements
    rows, dim, last = (1 << 20) + 3, 4096, 3
    assert (rows - last) * dim == PAST
    g = torch.Generator(DEV).manual_seed(3)

    def some():
        t = torch.zeros(rows, dim, dtype=BF, device=DEV)
        t[-last:] = torch.randn(last, dim, generator=g, device=DEV).to(BF)
        return t

    x, z, dy = some(), some(), some()
    w = 1 + 0.2 * torch.randn(dim, generator=g, device=DEV)
    print(f"case norms past 2^32 elements, {groups} groups", flush=True)
    y, rstd = ms.gated_norm_fwd(x, z, w, groups=groups)
    got = ms.gated_norm_bwd(x, z, w, rstd, dy=dy, groups=groups)
    torch.cuda.synchronize()
    wy, wr = ref.gated(ref.d64(x[-last:]), ref.d64(z[-last:]), ref.d64(w), groups)
    ref.within(y[-last:], wy, ref.NORM * wy.abs(), "y")
    ref.within(rstd[-last:], wr, ref.NORM * wr, "rstd")
    assert not y[:-last].any() and not got["dx"][:-last].any() and not got["dz"][:-last].any()
    # the last rows by themselves, which other tests hold to 64 bits
    alone = ms.gated_norm_bwd(x[-last:].clone(), z[-last:].clone(), w, rstd[-last:].clone(), dy=dy[-last:].clone(),
                              groups=groups)
    for k in ("dx", "dz"):
        assert torch.equal(got[k][-last:], alone[k]), k
    ref.within(got["dweight"], ref.d64(alone["dweight"]), 1e-6 * ref.d64(alone["dweight"]).abs() + 1e-6, "dweight")
    if groups > 1:
        return
    del got, y
    y, total, rstd = ms.residual_norm_fwd(x, z, w, w)
    got = ms.residual_norm_bwd(total, w, rstd, x, w, dy=dy, dtotal=z)
    torch.cuda.synchronize()
    assert not y[:-last].any() and not total[:-last].any() and not got["dx"][:-last].any()
    tail = lambda t: t[-last:].clone()   # noqa: E731
    ya, ta, ra = ms.residual_norm_fwd(tail(x), tail(z), w, w)
    assert torch.equal(y[-last:], ya) and torch.equal(total[-last:], ta) and torch.equal(rstd[-last:], ra)
    alone = ms.residual_norm_bwd(ta, w, ra, tail(x), w, dy=tail(dy), dtotal=tail(z))
    for k in ("dx", "dresidual"):
        assert torch.equal(got[k][-last:], alone[k]), k
