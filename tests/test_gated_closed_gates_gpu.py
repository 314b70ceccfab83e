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
