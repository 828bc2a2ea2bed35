"""Large products: workgroups of the 256 x 256 kernel that run several work units in turn,
launches that mix whole and split tiles, and gradients of rows past 4 GiB."""
import pytest
import torch

import convolution_implicit_gemm_amd as c3d
from helpers import env_var
from test_gpu_linear import backward_slacks, check_backward, run_forward
from token_helpers import ACTS, DTYPES, assert_within, gen, linear64, linear_slack, normal, scratch

pytestmark = pytest.mark.gpu

CUS = 256  # the 256 x 256 kernel runs one workgroup on each


def check_plan(plan, tile, wanted):
    info = plan.info()
    assert info.kernel_name.decode() == tile and wanted(info), "not the plan that this test is for"


def several(info):
    return info.grid > CUS


def mixed(info):
    return info.split_tiles > 0 and info.grid > info.split_tiles * info.split_pieces


def check_forward(m, n, k, act, dtype, residual, keep, gap, tile, wanted):
    plan, x, w, b, r, y, z = run_forward(m, n, k, act, dtype, True, residual, keep, gap, m + k, tile)
    check_plan(plan, tile, wanted)
    yr, zr, mag = linear64(x, w, b, r, act)
    zs, ys = linear_slack(k, mag, zr, yr, act)
    assert_within(y, yr, ys, "y")
    if keep:
        assert_within(z, zr, zs, "preact")


# 17 x 17 tiles and more, remainders in rows and columns: two units for some workgroups,
# then two for all and three for some; contractions of one stage (padded to two), two,
# an odd number of them, and many
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(4100, 4104, 40), (4352, 4352, 128), (4097, 4360, 264), (6200, 5400, 200),
                                   (8200, 4104, 72), (4150, 4232, 1032)])
def test_workgroups_run_several_units(m, n, k, dtype):
    check_forward(m, n, k, "gelu_tanh", dtype, True, True, 16, "m256n256k64", several)


@pytest.mark.parametrize("act,residual,keep", [("none", False, False), ("none", True, False), ("silu", False, True),
                                               ("gelu", True, False)])
def test_epilogues_between_units(act, residual, keep):
    check_forward(4200, 4232, 136, act, "bf16", residual, keep, 8, "m256n256k64", several)


@pytest.mark.parametrize("tile,m,n,k", [("m256n256k64", 4100, 4336, 2056), ("m256n256k64", 4612, 3568, 1032),
                                        ("m128n128k64", 2820, 2928, 2056), ("m128n128k64g2", 2308, 1776, 2056),
                                        ("m64n64k64", 1412, 1456, 2056), ("m64n64k64g4", 1156, 880, 4104)])
def test_whole_and_split_tiles_in_one_product(tile, m, n, k):
    check_forward(m, n, k, "silu", "fp16", True, True, 8, tile, mixed)


def test_several_units_are_exact_on_small_integers():
    # a stage read twice, left out or taken from another unit changes an integer
    m, n, k = 4360, 4360, 320
    g = gen(6)
    x = torch.randint(-2, 3, (m, k), generator=g, device="cuda:0").half()
    w = torch.randint(-2, 3, (n, k), generator=g, device="cuda:0").half()
    plan, _, _, _, _, y, _ = run_forward(m, n, k, "none", "fp16", False, False, False, 0, 6, "m256n256k64", x, w)
    check_plan(plan, "m256n256k64", several)
    ref = x.double() @ w.double().t().contiguous()
    assert float(ref.abs().max()) < 2048
    assert torch.equal(y.double(), ref)


# dx has 17 x 17 tiles and more, dw has, both have with split ones among them
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(4100, 136, 4232), (136, 4104, 4232), (4100, 2056, 4336), (2050, 4104, 4104)])
def test_gradients_of_several_units(m, n, k, dtype):
    check_backward(m, n, k, act="silu", dtype=dtype, gap=8, seed=4, tile="m256n256k64")


def test_several_units_repeat_bit_for_bit():
    outs = []
    for _ in range(3):
        _, _, _, _, _, y, z = run_forward(4150, 4232, 1032, "gelu", "bf16", True, True, True, 8, 5, "m256n256k64")
        outs.append((y.clone(), z.clone()))
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)


def far_rows(g, m, cols, dt):
    """[m, cols] values in rows 2^20 elements apart."""
    v = torch.empty((m, 1 << 20), dtype=dt, device="cuda:0")[:, :cols]
    v.copy_(normal(g, (m, cols), dt))
    return v


# 2100 rows 2^20 elements of 2 bytes apart pass 4 GiB of x, y, dy, the residual and dx
@pytest.mark.parametrize("tile", [None, "m64n64k64+pair", "m128n128k64", "m256n256k64"])
def test_operands_and_gradients_past_four_gib(tile):
    m, n, k, stride, dt = 2100, 72, 64, 1 << 20, torch.float16
    g = gen(8)
    x, dy, r = far_rows(g, m, k, dt), far_rows(g, m, n, dt), far_rows(g, m, n, dt)
    w, z = normal(g, (n, k), dt, 0.125), normal(g, (m, n), dt)
    with env_var("CONV3D_LINEAR_TILE", tile):
        plan = c3d.linear_plan(c3d.make_linear_desc(m, n, k, ACTS["silu"], c3d.CONV3D_F_RESIDUAL, stride, stride,
                                                    stride))
    out = far_rows(g, m, n, dt)
    c3d.linear_forward(plan, x, w, None, r, out, None, scratch(plan.workspace_bytes))
    yr, zr, mag = linear64(x, w, None, r, "silu")
    assert_within(out, yr, linear_slack(k, mag, zr, yr, "silu")[1], "y")
    dx, dw, db = far_rows(g, m, k, dt), torch.empty_like(w), torch.empty((n,), dtype=dt, device="cuda:0")
    c3d.linear_backward(plan, dy, x, w, z, dx, dw, db, scratch(c3d.linear_backward_workspace(plan)))
    refs, slacks = backward_slacks(dy, x, w, z, "silu")
    for got, ref, s, what in zip((dx, dw, db), refs, slacks, ("dx", "dw", "dbias")):
        assert_within(got, ref, s, what)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_bias_gradient_of_rows_past_four_gib(dtype):
    # without an activation dbias reads dy itself, by whole columns or by strips
    dt = DTYPES[dtype]
    for m, n in ((2100, 72), (6200, 8)):
        dy = far_rows(gen(m), m, n, dt)
        plan = c3d.linear_plan(c3d.make_linear_desc(m, n, 8, 0, c3d.CONV3D_F_BF16 if dtype == "bf16" else 0, 0, 1 << 20))
        db = torch.empty((n,), dtype=dt, device="cuda:0")
        c3d.linear_backward(plan, dy, None, None, None, None, None, db, scratch(c3d.linear_backward_workspace(plan)))
        _, slacks = backward_slacks(dy, torch.zeros((m, 8), dtype=dt, device="cuda:0"),
                                    torch.zeros((n, 8), dtype=dt, device="cuda:0"), dy, "none")
        assert_within(db, dy.double().sum(0), slacks[2], "dbias")


@pytest.mark.parametrize("m,n", [(6144, 8192), (6144, 8200), (6145, 64), (767, 65536), (769, 65536)])
def test_bias_gradient_by_whole_columns_and_by_strips(m, n):
    # either side of the sizes that are summed by whole columns, alone and beside dx and dw
    check_backward(m, n, 8, act="none", dtype="bf16", gap=8, seed=m)
