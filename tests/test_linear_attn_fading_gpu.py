"""Linear attention where tokens of unlike size meet a decay that takes much of
a state within a chunk: what remains of a large state, or of its adjoint, is
small and has to keep its own accuracy, whole or cut into segments, in the final
states, in every token's outputs and gradients, and in the decay's gradient.

Everything is compared per (row, head), outputs and gradients per token, since
one norm over a tensor shows its largest part only. A token's output is
sum_j scale lam^(t-j) (q_t . k_j) v_j = scale sum_n q_tn S_n. Its `size` is the
root of the sum of three squares: of the terms scale q_tn lam^(t-j) k_jn v_jp,
added up as independent ones; of scale lam^(t-j) (q_t . k_j) v_j likewise; and of
the output itself. With bf16 I/O S, the weights of v_j and the output are each
rounded to bf16 once, off by at most 2^-8 of the term they act on, with
independent signs: 2^-8 of the size, taken as 4e-3. In fp32 every term is off by
about 7e-7 (layers_ref.py derives it), taken as 3e-6 as there. States and their
gradients are fp32 whatever the inputs: 3e-6 of a (row, head)'s state in the
2-norm. Of the decay's gradient, sum_t <dS_t, lam S_(t-1)>, every token's term is
off by 7e-7 of its own size (its products added up as independent ones) and the
errors of neighbouring tokens may agree: 3e-6 of the sum of the sizes.
"""
import sys

import pytest
import torch

import selective_state_space_40_amd as ms

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
TOKEN = {BF: 4e-3, F32: 3e-6}
STATE = 3e-6
DECAYS = [-0.05, -0.1, -0.15, -0.2, -0.25, -0.3, -0.45]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch.cuda.synchronize()


def _walk(q, k, v, lam, start, scale):
    """The recurrence S = lam S + k^T v, out = scale q S over (batch, L, heads,
    size) inputs in 64 bits: outputs, their sizes, the last state, and for every
    token S and the sum of its terms' squares."""
    b, n, h, _ = q.shape
    lam = lam.view(1, h, 1, 1)
    s = torch.zeros(b, h, k.shape[-1], v.shape[-1], dtype=torch.float64) if start is None else start
    m = s.square()
    outs, sizes, states, squares = [], [], [], []
    for t in range(n):
        s = lam * s + k[:, t, :, :, None] * v[:, t, :, None, :]
        m = lam.square() * m + (k[:, t, :, :, None] * v[:, t, :, None, :]).square()
        o = scale * (q[:, t, :, None, :] @ s)[:, :, 0]
        size = scale ** 2 * (q[:, t, :, None, :].square() @ m)[:, :, 0].sum(-1) + o.square().sum(-1)
        j = torch.arange(t + 1)
        near = (scale * lam.view(1, h, 1) ** (t - j) *
                torch.einsum("bhd,bjhd->bhj", q[:, t], k[:, :t + 1]))
        size = size + (near.square() * v[:, :t + 1].square().sum(-1).transpose(1, 2)).sum(-1)
        outs.append(o)
        sizes.append(size.sqrt())
        states.append(s)
        squares.append(m)
    return torch.stack(outs, 1), torch.stack(sizes, 1), s, states, squares


def _reference(i):
    q, k, v, do = (i[x].double().cpu() for x in ("q", "k", "v", "do"))
    g = i["log_decay"].double().cpu()
    lam, h = g.exp(), q.shape[2]
    h0 = None if i["h0"] is None else i["h0"].double().cpu()
    scale = q.shape[-1] ** -0.5
    o, o_size, hL, states, squares = _walk(q, k, v, lam, h0, scale)
    dq, dq_size, *_ = _walk(do, v, k, lam, None if h0 is None else h0.transpose(-1, -2), scale)
    back = lambda x: x.flip(1)   # noqa: E731
    # _walk scales the output only: the adjoint is scale times its state, and
    # enters the last token without that token's decay
    end = None if i.get("dhL") is None else i["dhL"].double().cpu() / (scale * lam.view(1, h, 1, 1))
    dv, dv_size, first, adj, adj_squares = _walk(back(k), back(q), back(do), lam, end, scale)
    dk, dk_size, *_ = _walk(back(v), back(do), back(q), lam, None if end is None else end.transpose(-1, -2), scale)
    dh0 = scale * lam.view(1, h, 1, 1) * first
    adj, adj_squares = adj[::-1], adj_squares[::-1]
    dg = torch.zeros(h, dtype=torch.float64)
    dg_size = torch.zeros(h, dtype=torch.float64)
    start = torch.zeros_like(states[0]) if h0 is None else h0
    for t in range(len(states)):
        before, sq = (start, start.square()) if t == 0 else (states[t - 1], squares[t - 1])
        dg += (scale * adj[t] * lam.view(1, h, 1, 1) * before).sum((0, 2, 3))
        size = (scale ** 2 * adj_squares[t] * lam.square().view(1, h, 1, 1) * sq).sum((2, 3)).sqrt()
        dg_size += size.sum(0)
    tokens = dict(o=(o, o_size), dq=(dq, dq_size), dk=(back(dk), back(dk_size)), dv=(back(dv), back(dv_size)))
    return tokens, dict(hL=hL, dh0=dh0), (dg, dg_size)


def _check(i, what, segments):
    tokens, states, (dg, dg_size) = _reference(i)
    dt = i["q"].dtype
    wrong = []

    def bound(err, limit, name):
        over = (err / limit.clamp(min=1e-300)).max().item()
        if not over <= 1.0:      # a NaN as well
            wrong.append(f"{name}: {over:.3g} times its bound")

    for seg in segments:
        print(f"case {what} segment_len={seg}", flush=True)
        sys.stdout.flush()
        o, hL = ms.linear_attn_fwd(i["q"], i["k"], i["v"], i["log_decay"], i["h0"], segment_len=seg)
        bare, _ = ms.linear_attn_fwd(i["q"], i["k"], i["v"], i["log_decay"], i["h0"], segment_len=seg,
                                     return_state=False)
        got = ms.linear_attn_bwd(i["q"], i["k"], i["v"], i["log_decay"], i["h0"], do=i["do"],
                                 segment_len=seg)
        plain = ms.linear_attn_bwd(i["q"], i["k"], i["v"], i["log_decay"], i["h0"], do=i["do"],
                                   segment_len=seg, want_dlog_decay=False)
        torch.cuda.synchronize()
        got.update(o=o, hL=hL)
        for source, names in ((got, ("o", "dq", "dk", "dv")), (plain, ("dq", "dk", "dv")),
                              (dict(o=bare), ("o",))):
            for name in names:
                want, size = tokens[name]
                err = (source[name].double().cpu() - want).norm(dim=-1)
                bound(err, TOKEN[dt] * size, f"segment_len {seg} {name}")
        for source, name in ((got, "hL"), (got, "dh0"), (plain, "dh0")):
            err = (source[name].double().cpu() - states[name]).flatten(2).norm(dim=-1)
            bound(err, STATE * states[name].flatten(2).norm(dim=-1), f"segment_len {seg} {name}")
        bound((got["dlog_decay"].double().cpu() - dg).abs(), 3e-6 * dg_size, f"segment_len {seg} dlog_decay")
    assert not wrong, f"{what}: " + "; ".join(wrong)


def _make(length, dk, dv, dtype, seed, decays=DECAYS, state=False):
    g = torch.Generator().manual_seed(seed)
    h = len(decays)
    n = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    return dict(q=n(1, length, h, dk), k=n(1, length, h, dk), v=n(1, length, h, dv), do=n(1, length, h, dv),
                log_decay=torch.tensor(decays), h0=n(1, h, dk, dv) if state else None, dtype=dtype)


def _place(i):
    dt = i.pop("dtype")
    for name in ("q", "k", "v", "do"):
        i[name] = i[name].to(dt).to(DEV)
    for name in ("log_decay", "h0"):
        i[name] = None if i[name] is None else i[name].to(DEV)
    return i


SIZES = [(64, 64), (128, 72), (200, 136)]
types = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])


@types
@pytest.mark.parametrize("dk,dv", SIZES)
def test_tokens_without_keys_behind_others(dk, dv, dtype):
    # keys that are zero behind the first 64 tokens, a loss on the last 64 only:
    # the states and adjoints between are remainders and nothing else
    i = _make(192, dk, dv, dtype, dk + dv)
    i["k"][:, 64:] = 0.0
    i["do"][:, :128] = 0.0
    _check(_place(i), f"remainders {dk}x{dv} {dtype}", (0, 64, 128, 192))


@types
@pytest.mark.parametrize("dk,dv", SIZES)
def test_large_tokens_before_ordinary_ones(dk, dv, dtype):
    # the first 64 tokens carry a hundred times larger keys and values, the last
    # 64 a hundred times larger queries and gradients
    i = _make(200, dk, dv, dtype, dk - dv, state=True)
    for name in ("k", "v"):
        i[name][:, :64] *= 100.0
    for name in ("q", "do"):
        i[name][:, 128:] *= 100.0
    _check(_place(i), f"large {dk}x{dv} {dtype}", (0, 64, 256))


@types
@pytest.mark.parametrize("factor", [1e3, 1e4, 1e6])
def test_one_large_token_at_a_chunks_edge(factor, dtype):
    # just before an edge of 32 or 64 tokens for the state, just behind it for
    # the adjoint
    i = _make(128, 64, 72, dtype, 5, decays=[-0.1, -0.3, -0.45])
    edge = 64 if dtype == BF else 32
    i["v"][:, edge - 1] *= factor
    i["do"][:, 128 - edge] *= factor
    _check(_place(i), f"one token {factor} {dtype}", (0, 64, 128))


def test_remainders_across_a_whole_segment():
    # decays whose product with the segment's 192 tokens rounds by up to 3.8e-6 in
    # fp32: as an exponent that would be as much of the state itself, past the bound
    decays = [-0.4321, -0.4299, -0.436]
    i = _make(385, 64, 64, F32, 11, decays=decays)
    i["k"][:, :188] = 0.0
    i["k"][:, 192:] = 0.0
    i = _place(i)
    lam = i["log_decay"].double().cpu().exp()
    k, v = i["k"].double().cpu(), i["v"].double().cpu()
    want = sum(lam.view(1, 3, 1, 1) ** (384 - t) * k[:, t, :, :, None] * v[:, t, :, None, :]
               for t in range(188, 192))
    for seg in (192, 448):
        print(f"case whole segment segment_len={seg}", flush=True)
        _, hL = ms.linear_attn_fwd(i["q"], i["k"], i["v"], i["log_decay"], segment_len=seg)
        err = (hL.double().cpu() - want).flatten(2).norm(dim=-1) / want.flatten(2).norm(dim=-1)
        assert (err <= STATE).all(), f"segment_len {seg}: {err.tolist()}"


@pytest.mark.parametrize("decay", [0.0, -1e-3, -0.3, -2.0])
def test_infinite_states_of_rows_that_end_and_of_single_tokens(decay):
    # a decay above zero times an infinity is that infinity: a row without tokens
    # keeps its state as it is, whole or cut, and a token adds to it
    inf = float("inf")
    i = _place(_make(130, 16, 24, F32, 12, decays=[decay, 0.5 * decay], state=True))
    h0 = i["h0"].clone()
    h0[0, 0, 3, 5], h0[0, 1, 7, 0] = inf, -inf
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    for seg in (0, 64, 192):
        _, hL = ms.linear_attn_fwd(i["q"], i["k"], i["v"], i["log_decay"], h0, lengths=none, segment_len=seg)
        assert torch.equal(hL, h0), f"segment_len {seg}"
    got = ms.linear_attn_bwd(i["q"], i["k"], i["v"], i["log_decay"], i["h0"], do=i["do"], dhL=h0, lengths=none,
                             segment_len=64)
    assert torch.equal(got["dh0"], h0)
    h, clean = h0.clone(), i["h0"].clone()
    tok = [i[n][:, 0].contiguous() for n in ("q", "k", "v")]
    ms.linear_attn_update(clean, *tok, i["log_decay"])
    ms.linear_attn_update(h, *tok, i["log_decay"])
    torch.cuda.synchronize()
    assert h[0, 0, 3, 5] == inf and h[0, 1, 7, 0] == -inf
    same = torch.isfinite(h0)
    assert torch.equal(h[same], clean[same])
