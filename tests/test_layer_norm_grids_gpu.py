"""Layer norm on the GPU at the row counts where the launches change shape: the
lanes that share a part, the workgroups' size and how many of them leave partial
sums. References and tolerances as in test_layer_norm_gpu.py."""
import pytest
import torch

import selective_state_space_40_amd as ms
from test_layer_norm_gpu import BF, F32, _check, _make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch.cuda.synchronize()


CASES = [
    # few parts take four waves, more take one; 16-byte loads, value by value
    (255, 1280, 1), (256, 1280, 1), (255, 1026, 1), (256, 1026, 1), (1023, 1101, 1), (1024, 1101, 1),
    (64, 4096, 4), (85, 4 * 1302, 4), (256, 4 * 1302, 4),
    # one workgroup with all rows, small workgroups, large ones
    (16, 384, 1), (17, 384, 1), (32, 384, 1), (33, 384, 1), (2047, 384, 1), (2048, 384, 1), (32, 640, 5), (33, 640, 5), (410, 5 * 120, 5),
    (409, 5 * 120, 5),
    # teams of a wave, of four and of eight: one workgroup for all rows or more
    (8, 1000, 1), (9, 1000, 1), (2, 2048, 1), (3, 2048, 1), (1, 8192, 1), (2, 8192, 1), (500, 2048, 1),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_launch_shapes(case, dtype):
    rows, dim, groups = case
    print(f"case {case} {dtype}", flush=True)
    _check(*_make(rows, dim, dtype, sum(case)), groups, f"{case} {dtype}")
