"""linear's activations and their slopes at infinite, huge and far negative preactivations.

A product with one column of ones in x makes z exactly w's first column; a
gradient with dy = 1 over one row makes dbias exactly the slope.
"""
import math

import pytest
import torch

import convolution_implicit_gemm_amd as c3d
from helpers import env_var
from test_gpu_linear import backward_slacks
from token_helpers import ACTS, DTYPES, U24, act64, assert_within, gen, normal, scratch, slope64

pytestmark = pytest.mark.gpu

CURVED = ["silu", "gelu", "gelu_tanh"]
INF = float("inf")
# one row each through the kernel of few rows, the join of split tiles and the tiles' two epilogues
KERNELS = [(1, 8, None), (256, 16384, "m128n128k64"), (40, 8, "m64n64k64"), (40, 8, "m256n256k64")]


def make_plan(m, n, k, act, dt, flags=0, tile=None):
    if dt == torch.bfloat16:
        flags |= c3d.CONV3D_F_BF16
    with env_var("CONV3D_LINEAR_TILE", tile):
        return c3d.linear_plan(c3d.make_linear_desc(m, n, k, ACTS[act], flags))


def forward(z, act, m=1, k=8, tile=None, keep=False):
    """y (and the kept preactivations) of m rows whose preactivations are z, all columns alike."""
    n, dt = z.numel(), z.dtype
    x = torch.zeros((m, k), dtype=dt, device="cuda:0")
    x[:, 0] = 1.0
    w = torch.zeros((n, k), dtype=dt, device="cuda:0")
    w[:, 0] = z
    plan = make_plan(m, n, k, act, dt, c3d.CONV3D_F_PREACT if keep else 0, tile)
    y = torch.full((m, n), 12.5, dtype=dt, device="cuda:0")
    kept = torch.full((m, n), 12.5, dtype=dt, device="cuda:0") if keep else None
    c3d.linear_forward(plan, x, w, None, None, y, kept, scratch(plan.workspace_bytes))
    torch.cuda.synchronize()
    return (y, kept) if keep else y


def slopes(z, act):
    """The activation's derivative at z, rounded once."""
    n, dt = z.numel(), z.dtype
    plan = make_plan(1, n, 8, act, dt)
    db = torch.full((n,), 12.5, dtype=dt, device="cuda:0")
    c3d.linear_backward(plan, torch.ones((1, n), dtype=dt, device="cuda:0"), None, None, z[None], None, None, db,
                        scratch(c3d.linear_backward_workspace(plan)))
    torch.cuda.synchronize()
    return db


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("act", CURVED)
@pytest.mark.parametrize("m,k,tile", KERNELS)
def test_infinite_preactivations(m, k, tile, act, dtype):
    # the limits: act(+inf) = +inf, act(-inf) = 0
    z = torch.tensor([INF, -INF, 1.0, -1.0] * 66, device="cuda:0").to(DTYPES[dtype])
    y, kept = forward(z, act, m, k, tile, keep=True)
    assert torch.equal(kept, z.expand(m, -1))
    assert bool((y[:, 0::4] == INF).all()) and bool((y[:, 1::4] == 0).all())
    for col, v in ((2, 1.0), (3, -1.0)):
        ref = act64(torch.full_like(y[:, col::4], v, dtype=torch.float64), act)
        assert_within(y[:, col::4], ref, 2.0 ** -18 * ref.abs(), act)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("act", CURVED)
def test_slopes_at_infinity(act, dtype):
    # 1 at +inf and 0 at -inf, for dbias and through both products
    dt, g = DTYPES[dtype], gen(31)
    z = torch.tensor([INF, -INF] * 4, device="cuda:0").to(dt)
    assert slopes(z, act).tolist() == [1.0, 0.0] * 4
    m, n, k = 70, 136, 72
    dy, x, w, z = normal(g, (m, n), dt), normal(g, (m, k), dt), normal(g, (n, k), dt, k ** -0.5), normal(g, (m, n), dt)
    z[3, 5], z[3, 6], z[69, 135], z[0, 0] = INF, -INF, -INF, INF
    z[17] = -INF
    plan = make_plan(m, n, k, act, dt)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty((n,), dtype=dt, device="cuda:0")
    c3d.linear_backward(plan, dy, x, w, z, dx, dw, db, scratch(c3d.linear_backward_workspace(plan)))
    torch.cuda.synchronize()
    finite = z.clamp(-1e3, 1e3)  # slopes 0 and 1 to the last bit
    refs, slacks = backward_slacks(dy, x, w, finite, act)
    for got, ref, s, what in zip((dx, dw, db), refs, slacks, ("dx", "dw", "dbias")):
        assert_within(got, ref, s, what)
    assert not bool(dx[17].any())


@pytest.mark.parametrize("act", CURVED)
def test_preactivations_below_the_range_of_fp16(act):
    # finite operands, z = -80000 and +80000: y is 0 and +inf, and what is kept for
    # the backward pass is -inf and +inf, whose slopes are 0 and 1
    m, n, k = 33, 72, 40
    g = gen(32)
    x, w = normal(g, (m, k), torch.float16), normal(g, (n, k), torch.float16, k ** -0.5)
    x[4], w[6], w[7] = 0.0, 0.0, 0.0
    x[4, 0], w[6, 0], w[7, 0] = 200.0, -400.0, 400.0
    plan = make_plan(m, n, k, act, torch.float16, c3d.CONV3D_F_PREACT)
    y, z = (torch.empty((m, n), dtype=torch.float16, device="cuda:0") for _ in range(2))
    c3d.linear_forward(plan, x, w, None, None, y, z, scratch(plan.workspace_bytes))
    torch.cuda.synchronize()
    assert (float(z[4, 6]), float(z[4, 7])) == (-INF, INF)
    assert (float(y[4, 6]), float(y[4, 7])) == (0.0, INF)
    dy = normal(g, (m, n), torch.float16)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty((n,), dtype=torch.float16, device="cuda:0")
    c3d.linear_backward(plan, dy, x, w, z, dx, dw, db, scratch(c3d.linear_backward_workspace(plan)))
    torch.cuda.synchronize()
    refs, slacks = backward_slacks(dy, x, w, z.clamp(-6e4, 6e4), act)
    for got, ref, s, what in zip((dx, dw, db), refs, slacks, ("dx", "dw", "dbias")):
        assert_within(got, ref, s, what)


@pytest.mark.parametrize("dtype,big", [("fp16", 1.0), ("bf16", 1.0), ("bf16", 1e30), ("bf16", 5e33)])
@pytest.mark.parametrize("act", CURVED)
def test_large_preactivations_saturate_exactly(act, dtype, big):
    # e^-200 times any value of either type is below its smallest: y is z or 0, the slope 1 or 0
    z = torch.tensor([200.0, -200.0, 3e4, -3e4, 65504.0, -65504.0, 1e3, -1e3], device="cuda:0")
    z = (z * big).to(DTYPES[dtype])
    assert bool(torch.isfinite(z).all())
    for m, k, tile in KERNELS:
        y = forward(z, act, m, k, tile)
        assert torch.equal(y, z.clamp(min=0).expand(m, -1))
    assert torch.equal(slopes(z, act), (z > 0).to(z.dtype))


def exponent(z, act):
    """|the argument of the activation's exponential|."""
    if act == "silu":
        return z.abs()
    return z * z / 2 if act == "gelu" else (2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)).abs()


def relative(z, act):
    # the exponential's argument is rounded three times and its constants once, 2^-24 of
    # it each, which is as much of the exponential; the other steps (two transcendental
    # instructions, the polynomial, a dozen products) stay below 2^-18 together
    return 2.0 ** -18 + 4 * U24 * exponent(z, act)


TAIL = 2.0 ** -122  # below it the instructions may flush to 0, times |z|: bf16 only


def sweep(dtype):
    # fp16: down to where z Phi(z) is below its smallest value
    return torch.linspace(-12.5, 12.5, 8192, device="cuda:0", dtype=torch.float64).to(DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("act", CURVED)
def test_far_negative_preactivations_keep_their_digits(act, dtype):
    z = sweep(dtype)
    zd = z.double()
    ref = act64(zd, act)
    slack = ref.abs() * relative(zd, act) + TAIL * (1 + zd.abs())
    for m, k, tile in KERNELS:
        assert_within(forward(z, act, m, k, tile), ref.expand(m, -1), slack, "%s, %s" % (act, tile))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("act", CURVED)
def test_slopes_of_far_negative_preactivations_keep_their_digits(act, dtype):
    z = sweep(dtype)
    zd = z.double()
    # the two terms of the slope, whose rounding errors stay when they cancel
    if act == "gelu":
        first, second = 0.5 * torch.special.erfc(zd.abs() / math.sqrt(2.0)), \
            zd.abs() * torch.exp(-zd * zd / 2) / math.sqrt(2.0 * math.pi)
    else:
        grow = 1.0 if act == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * zd * zd)
        arg = zd if act == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (zd + 0.044715 * zd ** 3)
        first = torch.sigmoid(arg)
        second = first * zd.abs() * grow * torch.sigmoid(-arg)
    # for positive z, 1 - sigmoid is a difference from 1: 2^-24 times what it multiplies
    far = torch.where(zd > 0, (1.0 + zd.abs() * (1.0 if act == "gelu" else grow)) * 2 * U24, torch.zeros_like(zd))
    slack = (first + second) * relative(zd, act) + far + TAIL * (1 + zd.abs()) ** 3
    assert_within(slopes(z, act), slope64(zd, act), slack, act)
