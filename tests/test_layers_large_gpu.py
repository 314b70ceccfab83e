"""The layer operators on tensors whose last rows start past 2^32 elements (states
past 2^32 elements): offsets of 32 bits would reach an earlier row. What stands
before the last rows is empty, so that the 64-bit reference needs the last only.
Takes up to 150 GB of the GPU's memory."""
import pytest
import torch

import layers_ref as ref
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
    if torch.cuda.mem_get_info(DEV)[0] < 160 << 30:
        pytest.skip("less than 160 GB of GPU memory free")
    ms.load_library()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_sequences():
    # 17 rows of 16384 tokens, 64 heads of 256: the last row starts at element 2^32
    # of q, o, do and dq and of the fp32 gradients that heads share; its 70 tokens
    # are the only ones
    batch, length, heads, kv, dim, n = 17, 16384, 64, 32, 256, 70
    assert (batch - 1) * length * heads * dim == PAST
    g = torch.Generator(DEV).manual_seed(1)

    def rows(h):
        t = torch.empty(batch, length, h, dim, dtype=BF, device=DEV)
        t[0, :n] = float("nan")         # where offsets cut to 32 bits would read
        t[-1, :n] = torch.randn(n, h, dim, generator=g, device=DEV).to(BF)
        return t

    q, k, v, do = rows(heads), rows(kv), rows(kv), rows(heads)
    decay = -torch.logspace(0, -3, heads, device=DEV)
    lengths = torch.zeros(batch, dtype=torch.int32, device=DEV)
    lengths[-1] = n
    last = dict(q=q[-1:, :n], k=k[-1:, :n], v=v[-1:, :n], do=do[-1:, :n], log_decay=decay)
    want_o, want_h, want = ref.attn(**{x: t.cpu() for x, t in last.items()})
    print("case sequences past 2^32 elements", flush=True)
    o, h = ms.linear_attn_fwd(q, k, v, decay, lengths=lengths, segment_len=length)
    torch.cuda.synchronize()
    ref.check(o[-1:, :n], want_o, "bf16", "o")
    ref.check(h[-1:], want_h, "f32", "hL")
    assert not o[:-1].any() and not o[-1, n:].any() and not h[:-1].any()
    del o, h
    torch.cuda.empty_cache()
    got = ms.linear_attn_bwd(q, k, v, decay, do=do, lengths=lengths, segment_len=length)
    torch.cuda.synchronize()
    for x in ("dq", "dk", "dv"):
        assert not got[x][:-1].any() and not got[x][-1, n:].any(), x
        got[x] = got[x][-1:, :n]
    assert not got["dh0"][:-1].any()
    got["dh0"] = got["dh0"][-1:]
    ref.check_grads(got, want, BF, "sequences")


def test_states_and_cut_sequences():
    # states of 1025 rows of 64 heads of 256 x 256: the last row's start at 2^32
    batch, heads, dim = 1025, 64, 256
    assert (batch - 1) * heads * dim * dim == PAST
    g = torch.Generator(DEV).manual_seed(2)

    def some(*shape, dt=F32):
        return torch.randn(*shape, generator=g, device=DEV).to(dt)

    h = torch.zeros(batch, heads, dim, dim, device=DEV)
    h[-1] = some(heads, dim, dim)
    q, k, v = (some(batch, heads, dim, dt=BF) for _ in range(3))
    k[:-1] = 0.0
    decay = -torch.logspace(0, -3, heads, device=DEV)
    want_o, want_h = ref.attn_token(h[-1:], q[-1:], k[-1:], v[-1:], decay)
    print("case states past 2^32 elements", flush=True)
    o = ms.linear_attn_update(h, q, k, v, decay)
    torch.cuda.synchronize()
    ref.check(o[-1:], want_o, "bf16", "o")
    ref.check(h[-1:], want_h, "f32", "h")
    assert not h[:-1].any() and not o[:-1].any()
    # the same states entering sequences cut into three segments, whose own states
    # pass 2^32 elements as well
    batch = 343
    assert (batch - 1) * heads * 3 * dim * dim > PAST
    h = h[-batch:].contiguous()
    start = h[-1:].clone()
    q, k, v = (torch.zeros(batch, 130, heads if x == "q" else 1, dim, dtype=BF, device=DEV) for x in "qkv")
    for t in (q, k, v):
        t[-1] = some(*t.shape[1:], dt=BF)
    want_o, want_h = ref.attn(q[-1:], k[-1:], v[-1:], decay, start)
    o, end = ms.linear_attn_fwd(q, k, v, decay, h, segment_len=64)
    torch.cuda.synchronize()
    ref.check(o[-1:], want_o, "bf16", "cut o")
    ref.check(end[-1:], want_h, "f32", "cut hL")
    assert not end[:-1].any() and not o[:-1].any()


@pytest.mark.parametrize("groups", [1, 32])
def test_norms(groups):
    # 2^20 + 3 rows of 4096: the last three start past 2^32 elements
    rows, dim, last = (1 << 20) + 3, 4096, 3
    assert (rows - last) * dim == PAST
    g = torch.Generator(DEV).manual_seed(3)
    x, dy = (torch.zeros(rows, dim, dtype=BF, device=DEV) for _ in range(2))
    for t in (x, dy):
        t[-last:] = torch.randn(last, dim, generator=g, device=DEV).to(BF)
    w, b = 1 + 0.2 * torch.randn(dim, generator=g, device=DEV), torch.randn(dim, generator=g, device=DEV)
    print(f"case norms past 2^32 elements, {groups} groups", flush=True)
    y, mean, rstd = ms.layer_norm_fwd(x, w, b, groups=groups)
    got = ms.layer_norm_bwd(x, w, mean, rstd, dy=dy, groups=groups)
    torch.cuda.synchronize()
    yr, mr, rr = ref.norm(x[-last:], w, b, groups)
    dx, dw, db = ref.norm_grads(x[-last:], w, dy[-last:], groups)
    ref.check(y[-last:], yr, "bf16", "y")
    ref.check(mean[-last:], mr, "f32", "mean")
    ref.check(rstd[-last:], rr, "f32", "rstd")
    ref.check(got["dx"][-last:], dx, "bf16", "dx")
    ref.check(got["dweight"], dw, "f32", "dweight")     # rows before add nothing
    ref.check(got["dbias"], db, "f32", "dbias")
    assert torch.equal(y[:4], b.to(BF).expand(4, dim)) and not got["dx"][:-last].any()
