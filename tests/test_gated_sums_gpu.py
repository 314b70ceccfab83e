"""Sums over very many rows: the gradients of a norm's weight, whose partial sums
are of a bounded number of rows however many groups there are."""
import pytest
import torch

import selective_state_space_40_amd as ms

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.mark.parametrize("rows,dim,groups", [(1 << 18, 521 * 8, 521), (1 << 15, 1031 * 64, 1031), (1 << 21, 136, 1),
                                             (70001, 2085, 3), (257, 1 << 24, 1 << 19)])
def test_weight_gradient_over_many_rows(rows, dim, groups):
    # All rows alike, so that every addition of a long fp32 sum rounds the same way.
    # dweight = rows dy n with n = x rstd: the product rounds once, a sum in registers
    # at most 1024 times, those of at most 32 teams of a workgroup 32 times, the rest is
    # in 64 bits, and the result rounds once more: 1058 * 2^-24 of the value.
    g = torch.Generator().manual_seed(dim)
    x = (0.3 + torch.rand(dim, generator=g)).to(BF).to(DEV)
    dy = (0.3 + torch.rand(dim, generator=g)).to(BF).to(DEV)
    print(f"case {rows} x {dim} in {groups}", flush=True)
    wide, wdy = x.expand(rows, dim).contiguous(), dy.expand(rows, dim).contiguous()
    weight = torch.ones(dim, device=DEV)
    y, rstd = ms.gated_norm_fwd(wide, None, weight, groups=groups)
    del y
    got = ms.gated_norm_bwd(wide, None, weight, rstd, dy=wdy, groups=groups)["dweight"]
    r = rstd[0].double().repeat_interleave(dim // groups)
    want = rows * dy.double() * x.double() * r
    err = (got.double() / want - 1).abs().max().item()
    assert err <= 1058 * 2.0 ** -24, f"{err:.3g}"
