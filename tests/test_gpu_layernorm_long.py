"""layernorm's gradients of rows past 4 GiB: strided dy, x, dres and dx, on every path."""
import pytest
import torch

import convolution_implicit_gemm_amd as c3d
from test_gpu_layernorm import EPS, forward_slack, grad64, ln64
from token_helpers import assert_within, gen, normal, scratch

pytestmark = pytest.mark.gpu

STRIDE = 1 << 20


def far_rows(seed, rows, c, dt):
    v = torch.empty((rows, STRIDE), dtype=dt, device="cuda:0")[:, :c]
    v.copy_(normal(gen(seed), (rows, c), dt))
    return v


# 2100 rows 2 MiB apart: the row blocks with the partials of the weights' sums, and dx alone
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("rows,c", [(2100, 264), (2100, 2056)])
def test_gradients_past_four_gib(rows, c, weights):
    dt = torch.bfloat16
    x, dy, dres, dx = (far_rows(s, rows, c, dt) for s in range(4))
    gamma = normal(gen(6), (c,), dt, 0.3, 1.0)
    y = far_rows(5, rows, c, dt)
    stats = torch.empty((rows, 2), dtype=torch.float32, device="cuda:0")
    c3d.layernorm_bf16(x, gamma, None, y, stats, rows, c, EPS, STRIDE, STRIDE)
    ref, mean, rstd, _ = ln64(x, gamma, None)
    assert_within(y, ref, forward_slack(x, gamma, None, mean, rstd), "y")
    dg, db = (torch.empty_like(gamma), torch.empty_like(gamma)) if weights else (None, None)
    c3d.layernorm_backward_bf16(dy, x, gamma, stats, dres, dx, dg, db, rows, c,
                                scratch(c3d.layernorm_backward_workspace(rows, c)), STRIDE, STRIDE)
    torch.cuda.synchronize()
    refs, slacks = grad64(dy, x, gamma, stats, dres)
    for got, r, s, what in zip((dx, dg, db), refs, slacks, ("dx", "dgamma", "dbeta")):
        if got is not None:
            assert_within(got, r, s, what)


@pytest.mark.parametrize("rows", [2047, 2048])
def test_column_blocks_up_to_four_gib(rows):
    # the most rows that the column blocks walk: their last row begins just below 4 GiB
    c, dt = 264, torch.float16
    x, dy, dx = (far_rows(s, rows, c, dt) for s in range(3))
    gamma = normal(gen(6), (c,), dt, 0.3, 1.0)
    _, mean, rstd, _ = ln64(x, gamma, None)
    stats = torch.cat([mean, rstd], 1).float().contiguous()
    dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
    c3d.layernorm_backward(dy, x, gamma, stats, None, dx, dg, db, rows, c,
                           scratch(c3d.layernorm_backward_workspace(rows, c)), STRIDE, STRIDE)
    torch.cuda.synchronize()
    refs, slacks = grad64(dy, x, gamma, stats, None)
    for got, r, s, what in zip((dx, dg, db), refs, slacks, ("dx", "dgamma", "dbeta")):
        assert_within(got, r, s, what)
