"""Linear attention on the GPU (whole sequences, gradients, single tokens)
against its definition in 64 bits, at the sizes, layouts and values where the
chunked kernels can go wrong."""
import math
import sys

import pytest
import torch

import layers_ref as ref
import selective_state_space_40_amd as ms

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


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


def _make(batch, length, heads, kv_heads, dk, dv, dtype, seed=0, state=True, lengths=None, decay=None):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, dt=F32):
        return torch.randn(*shape, generator=g).to(dt).to(DEV)

    if decay is None:   # from a memory of a third of a token to one of thousands
        decay = -torch.logspace(0.5, -4, heads) if heads > 1 else torch.tensor([-0.05])
    return dict(q=n(batch, length, heads, dk, dt=dtype), k=n(batch, length, kv_heads, dk, dt=dtype),
                v=n(batch, length, kv_heads, dv, dt=dtype), log_decay=torch.as_tensor(decay).float().to(DEV),
                h0=n(batch, heads, dk, dv) if state else None,
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV),
                do=n(batch, length, heads, dv, dt=dtype), dhL=n(batch, heads, dk, dv) if state else None)


def _fwd(i, **kw):
    return ms.linear_attn_fwd(i["q"], i["k"], i["v"], i["log_decay"], i["h0"], lengths=i["lengths"], **kw)


def _bwd(i, **kw):
    return ms.linear_attn_bwd(i["q"], i["k"], i["v"], i["log_decay"], i["h0"], do=i["do"], dhL=i["dhL"],
                              lengths=i["lengths"], **kw)


def _check_all(i, what, segments=(0,), **kw):
    o, hL, grads = ref.attn(**i, **kw)
    dt = i["q"].dtype
    kind = "bf16" if dt == BF else "f32"
    for seg in segments:
        _say(f"case {what} segment_len={seg}")
        got_o, got_h = _fwd(i, segment_len=seg, **kw)
        torch.cuda.synchronize()
        ref.check(got_o, o, kind, f"{what} o")
        ref.check(got_h, hL, "f32", f"{what} hL")
        got = _bwd(i, segment_len=seg, **kw)
        torch.cuda.synchronize()
        ref.check_grads(got, grads, dt, what)


SHAPES = [
    # (batch, length, heads, kv_heads, dk, dv)
    (1, 1, 1, 1, 8, 8), (2, 2, 3, 3, 16, 8), (1, 31, 2, 1, 64, 64), (1, 32, 2, 2, 64, 72),
    (2, 33, 4, 2, 72, 64), (1, 63, 2, 2, 128, 128), (1, 64, 1, 1, 128, 64), (1, 65, 3, 1, 64, 128),
    (2, 97, 2, 2, 136, 40), (1, 130, 2, 1, 40, 136), (1, 200, 2, 2, 256, 256), (1, 320, 4, 4, 96, 80),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape, dtype):
    i = _make(*shape, dtype, seed=sum(shape))
    _check_all(i, f"{shape} {dtype}", segments=(0, 64))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_without_states(dtype):
    i = _make(2, 150, 2, 2, 64, 64, dtype, seed=1, state=False)
    _check_all(i, f"no states {dtype}", segments=(0, 128))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_rows_of_different_lengths(dtype):
    # empty, one token, ends before, at and past a chunk and a segment, beyond
    # the buffer and negative (taken as all and none)
    lengths = [0, 1, 63, 64, 65, 128, 130, 200, 1000, -3]
    i = _make(len(lengths), 200, 2, 1, 64, 72, dtype, seed=2, lengths=lengths)
    _check_all(i, f"lengths {dtype}", segments=(0, 64, 128))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(200, 168), (144, 256), (256, 8), (8, 200)])
def test_wide_heads_of_different_lengths(dk, dv, dtype):
    # two waves share a wide head's columns; rows that are empty, end in the
    # first chunk, at a chunk's end and inside the last, heads of every memory
    lengths = [0, 1, 64, 150]
    i = _make(len(lengths), 150, 4, 2, dk, dv, dtype, seed=dk + dv, lengths=lengths,
              decay=[0.0, -0.01, -0.5, float("-inf")])
    _check_all(i, f"wide {dk}x{dv} {dtype}", segments=(0, 64))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(200, 16), (16, 200), (136, 64), (64, 96)])
def test_gradients_of_heads_of_unlike_widths(dk, dv, dtype):
    # rows and heads enough that the passes over dk and over dv are launched
    # apart, each at its own width
    lengths = [70, 0, 33, 64, 70, 1]
    i = _make(6, 70, 24, 8, dk, dv, dtype, seed=dk, lengths=lengths)
    _check_all(i, f"unlike {dk}x{dv} {dtype}", segments=(0, 64))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("decay", [-0.8, -3.0, -9.0])
def test_large_states_that_fade_fast(decay, dtype):
    # a carried state (and its gradient) far above what a short sequence adds:
    # what remains of it is small, and must not be rounded at its old size
    for length in (1, 3, 43, 64, 70):
        i = _make(2, length, 2, 1, 136 if length == 43 else 64, 64, dtype, seed=length, decay=[decay, 1.5 * decay])
        i["h0"] *= 100.0
        i["dhL"] *= 100.0
        _check_all(i, f"fading {decay} {length} {dtype}", segments=(0, 64))
        h = i["h0"].clone()
        one = [i[n][:, 0].contiguous() for n in ("q", "k", "v")]
        want_o, want_h = ref.attn_token(i["h0"], *one, i["log_decay"])
        o = ms.linear_attn_update(h, *one, i["log_decay"])
        ref.check(o, want_o, "bf16" if dtype == BF else "f32", "token o")
        ref.check(h, want_h, "f32", "token h")


def test_outputs_without_the_final_state():
    # the state then enters with fewer terms, which bf16 outputs do not show
    for dk, dv in ((64, 64), (128, 72), (192, 136)):
        i = _make(2, 300, 2, 1, dk, dv, BF, seed=dk)
        o, _, _ = ref.attn(**i)
        for seg in (0, 128):
            got, none = _fwd(i, return_state=False, segment_len=seg)
            assert none is None
            ref.check(got, o, "bf16", f"{dk}x{dv} o")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_padding_is_neither_read_nor_left(dtype):
    # NaN and infinity behind the rows' ends change nothing, outputs and
    # gradients there are zeros
    lengths = [0, 5, 70, 129]
    i = _make(len(lengths), 130, 2, 2, 64, 64, dtype, seed=3, lengths=lengths)
    want_o, want_h = _fwd(i)
    want = _bwd(i)
    bad = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in i.items()}
    for r, n in enumerate(lengths):
        for name in ("q", "k", "v", "do"):
            bad[name][r, n:] = float("nan")
            bad[name][r, n:][..., ::2] = float("inf")
    for seg in (0, 64):
        _say(f"case padding {dtype} segment_len={seg}")
        out = torch.full_like(want_o, float("nan"))
        got_o, got_h = _fwd(bad, out=out, segment_len=seg)
        got = _bwd(bad, segment_len=seg)
        torch.cuda.synchronize()
        for r, n in enumerate(lengths):
            assert (got_o[r, n:] == 0).all()
            for name in ("dq", "dk", "dv"):
                assert (got[name][r, n:] == 0).all()
        if seg == 0:
            assert torch.equal(got_o, want_o) and torch.equal(got_h, want_h)
            for name in want:
                assert torch.equal(got[name], want[name]), name
        assert all(torch.isfinite(got[name]).all() for name in got)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_decays(dtype):
    # none, one that underflows within a chunk, one that forgets at once
    i = _make(1, 190, 5, 5, 64, 64, dtype, seed=4, decay=[0.0, -1e-6, -2.0, -100.0, -math.inf])
    o, hL, grads = ref.attn(**{**i, "log_decay": i["log_decay"].clamp(min=-1e4)})
    kind = "bf16" if dtype == BF else "f32"
    for seg in (0, 64):
        _say(f"case decays {dtype} segment_len={seg}")
        got_o, got_h = _fwd(i, segment_len=seg)
        ref.check(got_o, o, kind, "o")
        ref.check(got_h, hL, "f32", "hL")
        ref.check_grads(_bwd(i, segment_len=seg), grads, dtype, "decays")


def test_long_memory_does_not_drift():
    # a decay next to 1 over many chunks: its power is that of the definition
    i = _make(1, 6400, 1, 1, 16, 16, F32, seed=5, decay=[-1e-5])
    o, hL, grads = ref.attn(**i)
    for seg in (6400, 640):
        _say(f"case long memory segment_len={seg}")
        got_o, got_h = _fwd(i, segment_len=seg)
        ref.check(got_o, o, "f32", "o")
        ref.check(got_h, hL, "f32", "hL")
        ref.check_grads(_bwd(i, segment_len=seg), grads, F32, "long memory")


def test_scale_and_wanted_outputs():
    i = _make(2, 70, 2, 2, 64, 64, F32, seed=6)
    _check_all(i, "scale", scale=0.3)
    assert _fwd(i, return_state=False)[1] is None
    full = _bwd(i)
    part = _bwd(i, want_dlog_decay=False, want_dh0=False)
    assert part["dlog_decay"] is None and part["dh0"] is None
    for name in ("dq", "dk", "dv"):
        assert torch.equal(part[name], full[name]), name


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_gradients_against_differences(dtype):
    # central differences of the GPU forward pass itself, in fp32 outputs of
    # smooth inputs: the two-sided quotient's own error is O(step^2), and the
    # outputs' rounding over the step
    i = _make(1, 70, 2, 1, 64, 64, F32, seed=7, decay=[-0.3, -0.02])
    grads = _bwd(i)

    def loss(j):
        o, h = _fwd(j)
        return ((o.double() * i["do"].double()).sum() + (h.double() * i["dhL"].double()).sum()).item()

    gen = torch.Generator().manual_seed(8)
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("log_decay", "dlog_decay"), ("h0", "dh0")):
        d = torch.randn(i[name].shape, generator=gen).to(DEV)
        step = 1e-2 if name != "log_decay" else 1e-3
        up = loss({**i, name: i[name] + step * d})
        down = loss({**i, name: i[name] - step * d})
        want = (grads[key].double() * d.double()).sum().item()
        size = (grads[key].double().norm() * d.double().norm()).item()
        _say(f"case differences {name}")
        # q, k, v and h0 enter linearly: the quotient is exact up to rounding,
        # 2^-24 sqrt(outputs) |values| / step < 1e-3 of the gradient's size
        assert abs((up - down) / (2 * step) - want) <= 1e-3 * size, name


def test_split_sequence_carries_state_in_place():
    i = _make(2, 150, 2, 2, 64, 72, BF, seed=9)
    o, hL, _ = ref.attn(**i)
    state = i["h0"].clone()
    m = 77
    outs = []
    for lo, hi in ((0, m), (m, m), (m, 150)):
        j = {k: (i[k][:, lo:hi].contiguous() if k in ("q", "k", "v") else i[k]) for k in i}
        outs.append(ms.linear_attn_fwd(j["q"], j["k"], j["v"], i["log_decay"], state, state_out=state)[0])
    torch.cuda.synchronize()
    ref.check(torch.cat(outs, 1), o, "bf16", "o")
    # two calls' two-term roundings and one more chunk edge: still the state's bound
    ref.check(state, hL, "f32", "state")


def test_empty_calls():
    i = _make(2, 0, 2, 2, 64, 64, F32, seed=10)
    o, hL = _fwd(i)
    assert o.shape == (2, 0, 2, 64) and torch.equal(hL, i["h0"])
    g = _bwd(i)
    assert torch.equal(g["dh0"], i["dhL"]) and (g["dlog_decay"] == 0).all()
    i = _make(0, 5, 2, 2, 64, 64, F32, seed=10)
    assert _fwd(i)[0].shape == (0, 5, 2, 64)
    assert (_bwd(i)["dlog_decay"] == 0).all()


def test_results_are_reproducible():
    i = _make(2, 500, 3, 3, 128, 128, BF, seed=11)
    for seg in (0, 128):
        a, b = _bwd(i, segment_len=seg), _bwd(i, segment_len=seg)
        for name in a:
            assert torch.equal(a[name], b[name]), name


UPDATE = [(1, 1, 1, 8, 8), (3, 4, 2, 64, 64), (2, 2, 2, 128, 128), (2, 3, 1, 72, 200), (1, 2, 2, 256, 256)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", UPDATE, ids=lambda s: "x".join(map(str, s)))
def test_single_tokens(shape, dtype):
    batch, heads, kv_heads, dk, dv = shape
    decay = [0.0, -0.5, -math.inf, -2.0][:heads]
    i = _make(batch, 4, heads, kv_heads, dk, dv, dtype, seed=sum(shape), decay=decay)
    h = i["h0"].clone()
    want = i["h0"].double().cpu()
    finite = i["log_decay"].clamp(min=-1e4)
    _say(f"case update {shape} {dtype}")
    for t in range(4):
        tok = [i[n][:, t].contiguous() for n in ("q", "k", "v")]
        o, want = ref.attn_token(want, *tok, finite)
        got = ms.linear_attn_update(h, *tok, i["log_decay"])
        torch.cuda.synchronize()
        ref.check(got, o, "bf16" if dtype == BF else "f32", f"o {t}")
        ref.check(h, want, "f32", f"h {t}")     # no bf16 operand: fp32 whatever the inputs


def test_tokens_continue_a_prompt():
    # the prompt pass and the single tokens after it are one sequence
    i = _make(2, 75, 4, 2, 64, 64, BF, seed=12)
    o, hL, _ = ref.attn(**i)
    cut = {k: (i[k][:, :70].contiguous() if k in ("q", "k", "v") else i[k]) for k in i}
    first, h = _fwd(cut)
    outs = [first]
    for t in range(70, 75):
        outs.append(ms.linear_attn_update(h, *[i[n][:, t].contiguous() for n in ("q", "k", "v")],
                                          i["log_decay"])[:, None])
    torch.cuda.synchronize()
    ref.check(torch.cat(outs, 1), o, "bf16", "o")
    ref.check(h, hL, "f32", "h")


def test_offsets_past_32_bits():
    # the last row of a batch whose q, k, v and o pass 2^32 bytes, and whose
    # states pass 2^32 elements' worth of bytes
    batch, length, heads, dk = 17, 16384, 16, 256
    g = torch.Generator(DEV).manual_seed(13)
    q, k, v = (torch.randn(batch, length, heads, dk, generator=g, device=DEV).to(BF) for _ in range(3))
    decay = -torch.logspace(0, -3, heads, device=DEV)
    assert q.numel() * 2 > 1 << 31
    _say("case offsets past 32 bits")
    o, h = ms.linear_attn_fwd(q, k, v, decay)
    one = [t[-1:].clone() for t in (q, k, v)]
    o1, h1 = ms.linear_attn_fwd(*one, decay, segment_len=16384)
    torch.cuda.synchronize()
    ref.check(o[-1:], o1, "bf16", "o")
    ref.check(h[-1:], h1, "f32", "h")


@pytest.mark.parametrize("seg", [0, 64])
def test_captured_calls_replay(seg):
    i = _make(2, 200, 2, 2, 64, 64, BF, seed=14)
    h = i["h0"].clone()
    tok = [i[n][:, 0].contiguous() for n in ("q", "k", "v")]
    want = (_fwd(i, segment_len=seg), _bwd(i, segment_len=seg))
    side = torch.cuda.Stream(DEV)
    with torch.cuda.stream(side):
        _fwd(i, segment_len=seg), _bwd(i, segment_len=seg), ms.linear_attn_update(h.clone(), *tok, i["log_decay"])
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):   # two graphs of the same calls share no scratch
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = (_fwd(i, segment_len=seg), _bwd(i, segment_len=seg))
            o = ms.linear_attn_update(h, *tok, i["log_decay"])
        graphs.append((graph, got, o))
    eager = i["h0"].clone()
    for r in range(4):
        torch.randn(1 << 16, device=DEV).sum().item()
        for graph, got, o in graphs:
            for t in (*got[0], *got[1].values()):
                t.fill_(float("nan"))
            graph.replay()
            want_o = ms.linear_attn_update(eager, *tok, i["log_decay"])
            torch.cuda.synchronize()
            for a, b in zip((*got[0], *got[1].values()), (*want[0], *want[1].values())):
                assert torch.equal(a, b), f"replay {r}"
            assert torch.equal(o, want_o) and torch.equal(h, eager), f"replay {r}"


def test_streams_do_not_share_scratch():
    jobs = [_make(2, 300, 2, 2, 64, 64, BF, seed=20 + s) for s in range(3)]
    want = [(_fwd(i, segment_len=64), _bwd(i, segment_len=64)) for i in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in jobs]
    got = [None] * len(jobs)
    for _ in range(3):
        for n, (s, i) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(s):
                got[n] = (_fwd(i, segment_len=64), _bwd(i, segment_len=64))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip((*a[0], *a[1].values()), (*b[0], *b[1].values())):
            assert torch.equal(x, y)


def test_nan_stays_in_its_head_and_after_its_chunk():
    i = _make(2, 200, 2, 2, 64, 64, BF, seed=15, state=False)
    clean, _ = _fwd(i)
    i["v"][0, 100, 1, 3] = float("nan")
    o, h = _fwd(i)
    torch.cuda.synchronize()
    bad = torch.isnan(o)
    assert bad[0, 100:, 1, 3].all() and torch.isnan(h[0, 1, :, 3]).all()
    assert not bad[0, :64].any() and not bad[1].any() and not bad[0, :, 0].any()
    assert torch.equal(o[0, :64], clean[0, :64]) and torch.equal(o[1], clean[1])
