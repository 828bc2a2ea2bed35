"""layernorm and its gradients against the 64-bit form (bounds: token_helpers.py)."""
import pytest
import torch

import convolution_implicit_gemm_amd as c3d
from token_helpers import DTYPES, U24, assert_unmarked_only, assert_within, gapped, gen, marked, normal, scratch

pytestmark = pytest.mark.gpu

EPS = 1e-6
SIZES = [(1, 8), (1, 1024), (3, 64), (5, 512), (4, 520), (7, 1024), (6, 1032), (9, 2048), (2, 2056), (13, 4096),
         (5, 4104), (3, 8192), (2, 8200), (3, 16384), (257, 264), (1543, 72), (2100, 1160)]


def ln64(x, gamma, beta, eps=EPS):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = (x - mean).pow(2).mean(1, keepdim=True).add(eps).rsqrt()
    xh = (x - mean) * rstd
    y = xh if gamma is None else xh * gamma.double()
    return (y if beta is None else y + beta.double()), mean, rstd, xh


# sums of at most 16384 values are added at most 64 deep, the rest is a dozen fp32 steps: 2^-18
def forward_slack(x, gamma, beta, mean, rstd):
    x = x.double()
    size = (x.abs() + mean.abs()) * rstd
    size = size if gamma is None else size * gamma.double().abs()
    return 2.0 ** -18 * (size if beta is None else size + beta.double().abs())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, dtype):
    rows, c = size
    dt, g = DTYPES[dtype], gen(rows + c)
    x = gapped(g, rows, c, 8, dt, 2.0)
    x += normal(g, (c,), dt, 1.0)
    gamma, beta = normal(g, (c,), dt, 0.3, 1.0), normal(g, (c,), dt, 0.5)
    ybuf, y = marked(rows, c, 24, dt)
    stats = torch.empty((rows, 2), dtype=torch.float32, device="cuda:0")
    c3d.layernorm(x, gamma, beta, y, stats, rows, c, EPS, c + 8, c + 24, bf16=dtype == "bf16")
    torch.cuda.synchronize()
    assert_unmarked_only(ybuf, rows, c, 24)
    ref, mean, rstd, _ = ln64(x, gamma, beta)
    assert_within(y, ref, forward_slack(x, gamma, beta, mean, rstd), "y")
    assert_within(stats[:, :1], mean, 2.0 ** -18 * x.double().abs().mean(1, keepdim=True), "mean")
    assert_within(stats[:, 1:], rstd, 2.0 ** -18 * rstd, "rstd")


@pytest.mark.parametrize("gamma,beta", [(False, False), (True, False), (False, True)])
def test_forward_without_weights_in_place(gamma, beta):
    rows, c = 37, 1032
    g = gen(3)
    x = normal(g, (rows, c), torch.float16, 1.0, 5.0)
    ga = normal(g, (c,), torch.float16) if gamma else None
    be = normal(g, (c,), torch.float16) if beta else None
    ref, mean, rstd, _ = ln64(x, ga, be)
    slack = forward_slack(x, ga, be, mean, rstd)
    c3d.layernorm(x, ga, be, x, None, rows, c, EPS)
    torch.cuda.synchronize()
    assert_within(x, ref, slack, "y")


@pytest.mark.parametrize("c", [8, 1024, 4096, 16384])
def test_rows_without_variance_and_non_finite_rows(c):
    x = torch.zeros((6, c), dtype=torch.float16, device="cuda:0")
    x[1] = 1000.0
    x[2] = -65504.0
    x[3, 0] = float("nan")
    x[4, c - 1] = float("inf")
    x[5] = normal(gen(1), (c,), torch.float16)
    beta = normal(gen(2), (c,), torch.float16)
    y = torch.empty_like(x)
    c3d.layernorm(x, None, beta, y, None, 6, c, EPS)
    torch.cuda.synchronize()
    ref, mean, rstd, _ = ln64(x, None, beta)
    ok = torch.tensor([0, 1, 2, 5], device="cuda:0")
    assert_within(y[ok], ref[ok], forward_slack(x, None, beta, mean, rstd)[ok], "y")
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[4]).all())


def test_a_large_mean_does_not_cancel():
    rows, c = 9, 2048
    x = normal(gen(4), (rows, c), torch.bfloat16, 1.0, 0.0) + 300.0
    y = torch.empty_like(x)
    stats = torch.empty((rows, 2), dtype=torch.float32, device="cuda:0")
    c3d.layernorm_bf16(x, None, None, y, stats, rows, c, EPS)
    ref, mean, rstd, _ = ln64(x, None, None)
    assert_within(y, ref, forward_slack(x, None, None, mean, rstd), "y")
    assert_within(stats[:, 1:], rstd, 2.0 ** -18 * rstd, "rstd")


def make_grad(rows, c, dtype, gap, seed, affine=True, dres=True):
    dt, g = DTYPES[dtype], gen(seed)
    x = gapped(g, rows, c, gap, dt, 2.0)
    x += normal(g, (c,), dt, 1.0)
    dy = gapped(g, rows, c, 2 * gap, dt)
    gamma = normal(g, (c,), dt, 0.3, 1.0) if affine else None
    r = gapped(g, rows, c, gap, dt) if dres else None
    _, mean, rstd, _ = ln64(x, gamma, None)
    return dy, x, gamma, r, torch.cat([mean, rstd], 1).float().contiguous()


def grad64(dy, x, gamma, stats, dres):
    """((dx, dgamma, dbeta), slacks) from the given statistics."""
    rows, c = x.shape
    dy, x, st = dy.double(), x.double(), stats.double()
    r = st[:, 1:]
    xh = (x - st[:, :1]) * r
    g = dy if gamma is None else dy * gamma.double()
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    size = (x.abs() + st[:, :1].abs()) * r  # what xh is the difference of
    sx = 2.0 ** -17 * r * (g.abs() + g.abs().mean(1, keepdim=True) + size * (g.abs() * size).mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
        sx = sx + 2.0 ** -22 * dres.double().abs()
    deep = (128 + rows / 256) * U24
    return (dx, (dy * xh).sum(0), dy.sum(0)), (sx, deep * (dy.abs() * size).sum(0), deep * dy.abs().sum(0))


def run_grad(dy, x, gamma, stats, dres, gap, want=(True, True)):
    rows, c = x.shape
    dxb, dx = marked(rows, c, gap, x.dtype)
    dgb, dg = marked(1, c, 0, x.dtype)
    dbb, db = marked(1, c, 0, x.dtype)
    c3d.layernorm_backward(dy, x, gamma, stats, dres, dx, dg if want[0] else None, db if want[1] else None, rows, c,
                           scratch(c3d.layernorm_backward_workspace(rows, c)), c + gap, c + 2 * gap,
                           bf16=x.dtype == torch.bfloat16)
    torch.cuda.synchronize()
    assert_unmarked_only(dxb, rows, c, gap)
    assert_unmarked_only(dgb, 1, c, 0)
    assert_unmarked_only(dbb, 1, c, 0)
    return dx, dg[0], db[0]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(size, dtype):
    rows, c = size
    dy, x, gamma, dres, stats = make_grad(rows, c, dtype, 8, rows + c, dres=rows % 2 == 1)
    got = run_grad(dy, x, gamma, stats, dres, 8)
    refs, slacks = grad64(dy, x, gamma, stats, dres)
    for a, ref, s, what in zip(got, refs, slacks, ("dx", "dgamma", "dbeta")):
        assert_within(a, ref, s, what)


@pytest.mark.parametrize("rows", [2047, 2048, 2049])
@pytest.mark.parametrize("c", [8, 520, 1032, 2048])
def test_column_sums_either_side_of_2048_rows(rows, c):
    dy, x, gamma, dres, stats = make_grad(rows, c, "bf16", 8, rows + c)
    got = run_grad(dy, x, gamma, stats, dres, 8)
    refs, slacks = grad64(dy, x, gamma, stats, dres)
    for a, ref, s, what in zip(got, refs, slacks, ("dx", "dgamma", "dbeta")):
        assert_within(a, ref, s, what)
    for again, a in zip(run_grad(dy, x, gamma, stats, dres, 8), got):
        assert torch.equal(again, a)


@pytest.mark.parametrize("want", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("affine", [True, False])
def test_backward_computes_only_what_is_asked_for(want, affine):
    dy, x, gamma, dres, stats = make_grad(70, 1032, "fp16", 0, 6, affine, False)
    got = run_grad(dy, x, gamma, stats, dres, 0, want)
    refs, slacks = grad64(dy, x, gamma, stats, dres)
    for asked, a, ref, s in zip((True,) + want, got, refs, slacks):
        if asked:
            assert_within(a, ref, s, "gradient")
        else:
            assert bool((a == 12.5).all())


@pytest.mark.parametrize("which", ["dy", "x", "dres"])
@pytest.mark.parametrize("c", [1032, 4104])
def test_backward_in_place(which, c):
    dy, x, gamma, dres, stats = make_grad(33, c, "fp16", 0, 12)
    refs, slacks = grad64(dy, x, gamma, stats, dres)
    dx = {"dy": dy, "x": x, "dres": dres}[which]
    dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
    c3d.layernorm_backward(dy, x, gamma, stats, dres, dx, dg, db, 33, c,
                           scratch(c3d.layernorm_backward_workspace(33, c)))
    torch.cuda.synchronize()
    for a, ref, s in zip((dx, dg, db), refs, slacks):
        assert_within(a, ref, s, which)


def test_backward_matches_differences():
    rows, c = 5, 72
    g = gen(17)
    dt = torch.float16
    x, gamma, beta = normal(g, (rows, c), dt), normal(g, (c,), dt, 0.3, 1.0), normal(g, (c,), dt)
    dy, y = normal(g, (rows, c), dt), torch.empty((rows, c), dtype=dt, device="cuda:0")
    stats = torch.empty((rows, 2), dtype=torch.float32, device="cuda:0")
    c3d.layernorm(x, gamma, beta, y, stats, rows, c, EPS)
    dx, dg, db = run_grad(dy, x, gamma, stats, None, 0)

    def loss(a):
        return (dy.double() * ln64(*a)[0]).sum()

    args = [x.double(), gamma.double(), beta.double()]
    refs, slacks = grad64(dy, x, gamma, stats, None)
    h = 1e-5
    for i, grad in enumerate((dx, dg, db)):
        v = torch.randn(refs[i].shape, generator=g, device="cuda:0", dtype=torch.float64)
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + h * v, args[i] - h * v
        diff = float((loss(hi) - loss(lo)) / (2 * h))
        # the kept statistics are fp32: 2^-18 of each term once more
        tol = 2 * slacks[i] + 2.0 ** -17 * refs[i].abs() + 2.0 ** -11 * refs[i].abs() + 2.0 ** -25
        assert abs(float((grad.double() * v).sum()) - diff) <= float((tol * v.abs()).sum()) + 1e-6 * abs(diff) + 1e-5


def test_zero_rows():
    x = torch.empty((0, 64), dtype=torch.float16, device="cuda:0")
    w = torch.ones((64,), dtype=torch.float16, device="cuda:0")
    st = torch.empty((0, 2), dtype=torch.float32, device="cuda:0")
    c3d.layernorm(x, w, w, x, st, 0, 64, EPS)
    dg, db = torch.full_like(w, 3.0), torch.full_like(w, 3.0)
    c3d.layernorm_backward(x, x, w, st, None, x, dg, db, 0, 64, None)
    torch.cuda.synchronize()
    assert not bool(dg.any()) and not bool(db.any())


def test_rows_past_four_gib_and_repeatability():
    rows, c, stride = 2100, 264, 1 << 20
    xb = torch.empty((rows, stride), dtype=torch.bfloat16, device="cuda:0")
    x = xb[:, :c]
    x.copy_(normal(gen(5), (rows, c), torch.bfloat16))
    gamma = normal(gen(6), (c,), torch.bfloat16)
    ref, mean, rstd, _ = ln64(x, gamma, None)
    stats = torch.empty((rows, 2), dtype=torch.float32, device="cuda:0")
    y = torch.empty((rows, c), dtype=torch.bfloat16, device="cuda:0")
    c3d.layernorm_bf16(x, gamma, None, y, stats, rows, c, EPS, stride)
    assert_within(y, ref, forward_slack(x, gamma, None, mean, rstd), "y")
    refs, slacks = grad64(y, x, gamma, stats, None)
    outs = []
    for _ in range(2):
        dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
        dx = xb[:, 512:512 + c]
        c3d.layernorm_backward_bf16(y, x.contiguous(), gamma, stats, None, torch.empty_like(y), dg, db, rows, c,
                                    scratch(c3d.layernorm_backward_workspace(rows, c)))
        outs.append((dg, db))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    for a, r, s in zip(outs[0], refs[1:], slacks[1:]):
        assert_within(a, r, s, "weight gradient")


def test_other_stream_and_graph_replay():
    rows, c = 300, 1032
    x, gamma = normal(gen(1), (rows, c), torch.float16), normal(gen(2), (c,), torch.float16)
    dy, y, dx = normal(gen(3), (rows, c), torch.float16), torch.empty_like(x), torch.empty_like(x)
    stats = torch.empty((rows, 2), dtype=torch.float32, device="cuda:0")
    dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
    ws = scratch(c3d.layernorm_backward_workspace(rows, c))

    def step():
        c3d.layernorm(x, gamma, None, y, stats, rows, c, EPS)
        c3d.layernorm_backward(dy, x, gamma, stats, None, dx, dg, db, rows, c, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(normal(gen(100 + i), (rows, c), torch.float16))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, stats, dx, dg, db)]
        for t in (y, stats, dx, dg, db):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(want, (y, stats, dx, dg, db)):
            assert torch.equal(p, q)
