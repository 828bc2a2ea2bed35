"""linear and its gradients against the 64-bit form (bounds: token_helpers.py)."""

import pytest
import torch

import convolution_implicit_gemm_amd as c3d
from helpers import env_var
from token_helpers import (ACTS, DTYPES, U24, act64, assert_unmarked_only, assert_within, gapped, gen, linear64,
                           linear_slack, marked, normal, scratch, slope64)

pytestmark = pytest.mark.gpu

TILES = [None, "m128n128k64", "m256n256k64", "m64n64k64", "m64n64k64g4", "m128n128k64g2"]


def run_forward(m, n, k, act, dtype, bias, residual, keep, gap, seed, tile=None, x=None, w=None):
    dt, g = DTYPES[dtype], gen(seed)
    x = gapped(g, m, k, gap, dt) if x is None else x
    w = normal(g, (n, k), dt, k ** -0.5) if w is None else w
    b = normal(g, (n,), dt, 0.5) if bias else None
    r = gapped(g, m, n, gap, dt) if residual else None
    flags = (c3d.CONV3D_F_BF16 if dtype == "bf16" else 0) | (c3d.CONV3D_F_BIAS if bias else 0) | \
        (c3d.CONV3D_F_RESIDUAL if residual else 0) | (c3d.CONV3D_F_PREACT if keep else 0)
    with env_var("CONV3D_LINEAR_TILE", tile):
        plan = c3d.linear_plan(c3d.make_linear_desc(m, n, k, ACTS[act], flags, k + gap, n + gap, n + gap))
    ybuf, y = marked(m, n, gap, dt)
    zbuf, z = marked(m, n, 0, dt) if keep else (None, None)
    c3d.linear_forward(plan, x, w, b, r, y, z, scratch(plan.workspace_bytes))
    torch.cuda.synchronize()
    assert_unmarked_only(ybuf, m, n, gap)
    if keep:
        assert_unmarked_only(zbuf, m, n, 0)
    return plan, x, w, b, r, y, z


def check_forward(m, n, k, act, dtype, bias=True, residual=False, keep=False, gap=0, seed=1, tile=None):
    _, x, w, b, r, y, z = run_forward(m, n, k, act, dtype, bias, residual, keep, gap, seed, tile)
    yr, zr, mag = linear64(x, w, b, r, act)
    zs, ys = linear_slack(k, mag, zr, yr, act)
    assert_within(y, yr, ys, "y")
    if keep:
        assert_within(z, zr, zs, "preact")


SIZES = [(1, 8, 8), (1, 1024, 1024), (2, 72, 40), (5, 264, 4104), (16, 512, 2048), (17, 1032, 520), (33, 136, 1000),
         (63, 2048, 256), (65, 128, 64), (127, 264, 136), (129, 120, 96), (256, 256, 512), (257, 264, 1032),
         (513, 1544, 72), (1000, 392, 2056)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward_sizes(size, dtype):
    check_forward(*size, act="gelu_tanh", dtype=dtype, residual=True, keep=True, gap=16, seed=sum(size))


@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("bias,residual,keep", [(False, False, False), (True, False, True), (True, True, False)])
@pytest.mark.parametrize("m", [3, 200])
def test_forward_epilogues(m, act, bias, residual, keep):
    check_forward(m, 264, 136, act, "fp16", bias, residual, keep, gap=8, seed=m)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tile", TILES[1:])
@pytest.mark.parametrize("size", [(1, 8, 8), (70, 200, 40), (300, 520, 264), (520, 776, 2000)], ids=str)
def test_forward_every_kernel(size, tile, dtype):
    check_forward(*size, act="silu", dtype=dtype, residual=True, keep=True, gap=8, seed=7, tile=tile)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("size", [(4, 64, 512), (300, 520, 264), (520, 264, 1024)], ids=str)
def test_forward_is_exact_on_small_integers(size, tile):
    # |sum| <= 4 * 1024 values of at most 4: exact in fp32; kept below 2048 by sparsity
    m, n, k = size
    g = gen(5)
    x = torch.randint(-2, 3, (m, k), generator=g, device="cuda:0").half()
    w = (torch.randint(-2, 3, (n, k), generator=g, device="cuda:0") *
         (torch.rand((n, k), generator=g, device="cuda:0") < 0.3)).half()
    _, x, w, _, _, y, _ = run_forward(m, n, k, "none", "fp16", False, False, False, 0, 5, tile, x, w)
    ref = x.double() @ w.double().t().contiguous()
    assert float(ref.abs().max()) < 2048
    assert torch.equal(y.double(), ref)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("m,tile", [(3, None), (300, "m128n128k64"), (300, "m256n256k64"), (300, "m64n64k64g4")])
def test_bias_alone_comes_through_exactly(m, tile, dtype):
    # x = 0: y is the bias bit for bit, subnormal and infinite values too
    dt = DTYPES[dtype]
    n, k = 264, 72
    b = normal(gen(2), (n,), dt)
    b[:8] = torch.tensor([6e-8, -6e-8, 3e-5, -5.9e-5, float("inf"), -float("inf"), 65504.0, 0.0]).to(dt)
    x, w = torch.zeros((m, k), dtype=dt, device="cuda:0"), normal(gen(3), (n, k), dt)
    with env_var("CONV3D_LINEAR_TILE", tile):
        plan = c3d.linear_plan(c3d.make_linear_desc(m, n, k, 0, c3d.CONV3D_F_BIAS |
                                                    (c3d.CONV3D_F_BF16 if dtype == "bf16" else 0)))
    y = torch.empty((m, n), dtype=dt, device="cuda:0")
    c3d.linear_forward(plan, x, w, b, None, y, None, scratch(plan.workspace_bytes))
    torch.cuda.synchronize()
    assert torch.equal(y, b.expand(m, n))


def test_split_contraction_joins_all_pieces():
    # few tiles and a long contraction: the plan splits it, and each piece counts
    plan, x, w, b, r, y, z = run_forward(256, 256, 16384, "gelu", "bf16", True, True, True, 8, 3, "m128n128k64")
    assert plan.info().split_pieces > 1
    yr, zr, mag = linear64(x, w, b, r, "gelu")
    zs, ys = linear_slack(16384, mag, zr, yr, "gelu")
    assert_within(y, yr, ys, "y")
    assert_within(z, zr, zs, "preact")


@pytest.mark.parametrize("m", [2, 40, 300])
def test_infinite_and_nan_rows_stay_in_their_rows(m):
    g = gen(11)
    x, w = normal(g, (m, 136), torch.float16), normal(g, (264, 136), torch.float16, 0.1)
    x[1, 5] = float("inf")
    x[0, 135] = float("nan")
    _, _, _, _, _, y, _ = run_forward(m, 264, 136, "none", "fp16", False, False, False, 0, 1, None, x, w)
    assert bool(torch.isnan(y[0]).all())
    assert not bool(torch.isfinite(y[1]).any())
    assert bool(torch.isfinite(y[2:]).all())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_nan_preactivations_stay_nan(act):
    m, n, k = 40, 72, 64
    g = gen(4)
    dt = torch.float16
    z, dy, x, w = normal(g, (m, n), dt), normal(g, (m, n), dt), normal(g, (m, k), dt), normal(g, (n, k), dt)
    z[3, 5] = float("nan")
    plan = c3d.linear_plan(c3d.make_linear_desc(m, n, k, ACTS[act]))
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty((n,), dtype=dt, device="cuda:0")
    c3d.linear_backward(plan, dy, x, w, z, dx, dw, db, scratch(c3d.linear_backward_workspace(plan)))
    torch.cuda.synchronize()
    assert torch.isnan(dx).nonzero()[:, 0].unique().tolist() == [3] and bool(torch.isnan(dx[3]).all())
    assert torch.isnan(dw).nonzero()[:, 0].unique().tolist() == [5] and bool(torch.isnan(dw[5]).all())
    assert torch.isnan(db).nonzero().flatten().tolist() == [5]
    x[2, 0] = float("nan")
    y = torch.empty((m, n), dtype=dt, device="cuda:0")
    c3d.linear_forward(plan, x, w, None, None, y, None, scratch(plan.workspace_bytes))
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[2]).all()) and not bool(torch.isnan(y[:2]).any()) and not bool(torch.isnan(y[3:]).any())


def test_large_preactivations_saturate():
    # silu and the gelus tend to z and to 0; their derivatives to 1 and 0
    vals = torch.tensor([3e4, -3e4, 65504.0, -65504.0, 200.0, -200.0, 12.0, -12.0], device="cuda:0")
    for act in ("silu", "gelu", "gelu_tanh"):
        for dtype, big in (("fp16", 1.0), ("bf16", 1e30)):
            dt = DTYPES[dtype]
            z = (vals * big).to(dt)
            x = torch.zeros((1, 8), dtype=dt, device="cuda:0")
            x[0, 0] = 1.0
            w = torch.zeros((8, 8), dtype=dt, device="cuda:0")
            w[:, 0] = z
            flags = c3d.CONV3D_F_BF16 if dtype == "bf16" else 0
            plan = c3d.linear_plan(c3d.make_linear_desc(1, 8, 8, ACTS[act], flags))
            y = torch.empty((1, 8), dtype=dt, device="cuda:0")
            c3d.linear_forward(plan, x, w, None, None, y, None, scratch(plan.workspace_bytes))
            zd = z.double()
            assert_within(y[0], act64(zd, act), 4e-6 * (1 + zd.abs()), act)
            dx = torch.empty_like(x)
            dw, db = torch.empty_like(w), torch.empty_like(z)
            c3d.linear_backward(plan, torch.ones_like(y), x, w, z[None], dx, dw, db,
                                scratch(c3d.linear_backward_workspace(plan)))
            assert_within(db, slope64(zd, act), 1e-5 + torch.zeros_like(zd), act + " slope")


def run_backward(m, n, k, act, dtype, gap, seed, tile=None, want=(True, True, True)):
    dt, g = DTYPES[dtype], gen(seed)
    dy, x = gapped(g, m, n, gap, dt), gapped(g, m, k, gap, dt)
    w, z = normal(g, (n, k), dt, k ** -0.5), normal(g, (m, n), dt, 1.5)
    with env_var("CONV3D_LINEAR_TILE", tile):
        plan = c3d.linear_plan(c3d.make_linear_desc(m, n, k, ACTS[act], c3d.CONV3D_F_BF16 if dtype == "bf16" else 0,
                                                    k + gap, n + gap))
    dxb, dx = marked(m, k, gap, dt)
    dwb, dw = marked(n, k, 0, dt)
    dbb, db = marked(1, n, 0, dt)
    ws = scratch(c3d.linear_backward_workspace(plan))
    c3d.linear_backward(plan, dy, x, w, None if act == "none" else z, dx if want[0] else None,
                        dw if want[1] else None, db if want[2] else None, ws)
    torch.cuda.synchronize()
    assert_unmarked_only(dxb, m, k, gap)
    assert_unmarked_only(dwb, n, k, 0)
    assert_unmarked_only(dbb, 1, n, 0)
    return dy, x, w, z, dx, dw, db[0]


def backward_slacks(dy, x, w, z, act):
    """(dx, dw, db) in 64 bits and their slacks.  dz is rounded to the element
    type as an operand of dx and dw (2^-11 / 2^-8 of it, 2^-25 below fp16's normal
    range) and its activation slope errs by less than 1e-5."""
    m, n = dy.shape
    dy64, x64, w64 = dy.double(), x.double(), w.double()
    dz = dy64 * slope64(z.double(), act)
    if act == "none":
        off = torch.zeros_like(dz)
    else:
        off = dz.abs() * (2.0 ** -11 if dy.dtype == torch.float16 else 2.0 ** -8) + 2.0 ** -25 + 1e-5 * dy64.abs()
    dx, dw, db = dz @ w64, dz.t().contiguous() @ x64, dz.sum(0)
    a = dz.abs() + off
    sx = off @ w64.abs() + n * U24 * (a @ w64.abs())
    sw = off.t().contiguous() @ x64.abs() + m * U24 * (a.t().contiguous() @ x64.abs())
    sb = (256 + m / 32) * U24 * dz.abs().sum(0) + (0 if act == "none" else 1e-5) * dy64.abs().sum(0)
    return (dx, dw, db), (sx, sw, sb)


def check_backward(m, n, k, act, dtype, gap=0, seed=1, tile=None):
    dy, x, w, z, dx, dw, db = run_backward(m, n, k, act, dtype, gap, seed, tile)
    refs, slacks = backward_slacks(dy, x, w, z, act)
    for got, ref, s, what in zip((dx, dw, db), refs, slacks, ("dx", "dw", "dbias")):
        assert_within(got, ref, s, what)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tile", ["m128n128k64+pair", "m64n64k64+pair", "m64n64k64g4+pair"])
@pytest.mark.parametrize("size", [(1, 8, 8), (70, 200, 40), (300, 520, 264), (2000, 776, 520), (5000, 72, 72)], ids=str)
def test_backward_in_one_launch(size, tile, dtype):
    check_backward(*size, act="silu", dtype=dtype, gap=8, seed=4, tile=tile)


BACK_SIZES = [(1, 8, 8), (1, 264, 1032), (7, 72, 40), (31, 520, 136), (33, 136, 264), (64, 2056, 72), (129, 264, 392),
              (257, 72, 520), (1001, 264, 136), (2049, 392, 264)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("size", BACK_SIZES, ids=str)
def test_backward_sizes(size, dtype):
    check_backward(*size, act="gelu_tanh", dtype=dtype, gap=16, seed=sum(size))


@pytest.mark.parametrize("tile", [None, "m64n64k64", "m64n64k64g4+pair"])
@pytest.mark.parametrize("m", [1, 63, 65, 1000, 6144, 6145])
def test_backward_bias_without_activation(m, tile):
    check_backward(m, 136, 72, act="none", dtype="bf16", gap=8, seed=m, tile=tile)


@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_backward_activations(act, dtype):
    check_backward(200, 264, 136, act, dtype, gap=8, seed=2)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tile", TILES[1:])
@pytest.mark.parametrize("size", [(1, 8, 8), (70, 200, 40), (300, 520, 264), (2000, 776, 520)], ids=str)
def test_backward_every_kernel(size, tile, dtype):
    check_backward(*size, act="silu", dtype=dtype, gap=8, seed=4, tile=tile)


@pytest.mark.parametrize("want", [(True, False, False), (False, True, False), (False, False, True)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_backward_computes_only_what_is_asked_for(act, want):
    dy, x, w, z, dx, dw, db = run_backward(130, 136, 72, act, "fp16", 8, 9, None, want)
    refs, slacks = backward_slacks(dy, x, w, z, act)
    for asked, got, ref, s in zip(want, (dx, dw, db), refs, slacks):
        if asked:
            assert_within(got, ref, s, "gradient")
        else:
            assert bool((got == 12.5).all())


@pytest.mark.parametrize("act", sorted(ACTS))
def test_backward_matches_differences(act):
    # the directional derivative of L = <dy, y(x, w, b)> in 64 bits against the kernel's gradients
    m, n, k = 37, 72, 40
    g = gen(21)
    dt = torch.float16
    x, w, b = normal(g, (m, k), dt), normal(g, (n, k), dt, k ** -0.5), normal(g, (n,), dt, 0.5)
    dy = normal(g, (m, n), dt)
    plan = c3d.linear_plan(c3d.make_linear_desc(m, n, k, ACTS[act], c3d.CONV3D_F_BIAS | c3d.CONV3D_F_PREACT))
    y, z = torch.empty((m, n), dtype=dt, device="cuda:0"), torch.empty((m, n), dtype=dt, device="cuda:0")
    c3d.linear_forward(plan, x, w, b, None, y, z, scratch(plan.workspace_bytes))
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    c3d.linear_backward(plan, dy, x, w, z, dx, dw, db, scratch(c3d.linear_backward_workspace(plan)))

    def loss(xx, ww, bb):
        return (dy.double() * linear64(xx, ww, bb, None, act)[0]).sum()

    h = 1e-5
    refs, slacks = backward_slacks(dy, x, w, z, act)
    # z was rounded when it was kept: the slope (|act''| <= 1.2) moves by half an ulp of z
    moved = (dy.double().abs() * 1.2 * z.double().abs() * 2.0 ** -11)
    extra = (moved @ w.double().abs(), moved.t().contiguous() @ x.double().abs(), moved.sum(0))
    for i, (grad, ref) in enumerate(zip((dx, dw, db), refs)):
        v = torch.randn(ref.shape, generator=g, device="cuda:0", dtype=torch.float64)
        args = [x.double(), w.double(), b.double()]
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + h * v, args[i] - h * v
        diff = float((loss(*hi) - loss(*lo)) / (2 * h))
        tol = slacks[i] + extra[i] + 2.0 ** -11 * ref.abs() + 2.0 ** -25
        bound = float((tol * v.abs()).sum()) + 1e-6 * abs(diff) + 1e-5
        assert abs(float((grad.double() * v).sum()) - diff) <= bound


def test_zero_rows():
    w = torch.ones((16, 8), dtype=torch.float16, device="cuda:0")
    plan = c3d.linear_plan(c3d.make_linear_desc(0, 16, 8))
    empty = torch.empty((0, 8), dtype=torch.float16, device="cuda:0")
    c3d.linear_forward(plan, empty, w, None, None, torch.empty((0, 16), dtype=torch.float16, device="cuda:0"))
    dw = torch.full_like(w, 3.0)
    db = torch.full((16,), 3.0, dtype=torch.float16, device="cuda:0")
    c3d.linear_backward(plan, torch.empty((0, 16), dtype=torch.float16, device="cuda:0"), empty, w, None, empty, dw,
                        db, scratch(16))
    torch.cuda.synchronize()
    assert not bool(dw.any()) and not bool(db.any())


@pytest.mark.parametrize("tile", TILES)
def test_results_do_not_vary_from_call_to_call(tile):
    outs = []
    for _ in range(3):
        a = run_forward(300, 264, 4096, "gelu", "bf16", True, True, True, 8, 5, tile)
        b = run_backward(3000, 264, 136, "gelu", "bf16", 8, 5, tile)
        outs.append([t.clone() for t in (a[5], a[6]) + tuple(b[4:])])
    for other in outs[1:]:
        for p, q in zip(outs[0], other):
            assert torch.equal(p.view(torch.int16) if p.is_contiguous() else p, q.view(torch.int16)
                               if q.is_contiguous() else q)


def test_rows_past_four_gib():
    # 17 rows 2^20 elements apart take 36 MiB; 2100 rows pass 4 GiB of x and of y
    m, n, k, stride = 2100, 72, 64, 1 << 20
    g = gen(8)
    xb = torch.empty((m, stride), dtype=torch.float16, device="cuda:0")
    yb = torch.empty((m, stride), dtype=torch.float16, device="cuda:0")
    x, y = xb[:, :k], yb[:, :n]
    x.copy_(normal(g, (m, k), torch.float16))
    w = normal(g, (n, k), torch.float16, 0.125)
    plan = c3d.linear_plan(c3d.make_linear_desc(m, n, k, 0, 0, stride, stride))
    c3d.linear_forward(plan, x, w, None, None, y, None, scratch(plan.workspace_bytes))
    yr, zr, mag = linear64(x, w, None, None, "none")
    assert_within(y, yr, linear_slack(k, mag, zr, yr, "none")[1], "y")
    dx, dw = xb[:, 128:128 + k], torch.empty_like(w)
    db = torch.empty((n,), dtype=torch.float16, device="cuda:0")
    plan = c3d.linear_plan(c3d.make_linear_desc(m, n, k, 0, 0, 0, stride))
    dx = torch.empty((m, k), dtype=torch.float16, device="cuda:0")
    c3d.linear_backward(plan, y, x.contiguous(), w, None, dx, dw, db, scratch(c3d.linear_backward_workspace(plan)))
    refs, slacks = backward_slacks(y, x, w, y, "none")
    for got, ref, s in zip((dx, dw, db), refs, slacks):
        assert_within(got, ref, s, "gradient")


def test_other_stream_and_graph_replay():
    m, n, k = 300, 264, 2048
    g = gen(13)
    dt = torch.float16
    x, w, b = normal(g, (m, k), dt), normal(g, (n, k), dt, k ** -0.5), normal(g, (n,), dt)
    dy = normal(g, (m, n), dt)
    plan = c3d.linear_plan(c3d.make_linear_desc(m, n, k, ACTS["gelu"], c3d.CONV3D_F_BIAS | c3d.CONV3D_F_PREACT))
    wsf, wsb = scratch(plan.workspace_bytes), scratch(c3d.linear_backward_workspace(plan))
    y, z = (torch.empty((m, n), dtype=dt, device="cuda:0") for _ in range(2))
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)

    def step():
        c3d.linear_forward(plan, x, w, b, None, y, z, wsf)
        c3d.linear_backward(plan, dy, x, w, z, dx, dw, db, wsb)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    want = [t.clone() for t in (y, z, dx, dw, db)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(normal(gen(100 + i), (m, k), dt))
        step()
        torch.cuda.synchronize()
        eager = [t.clone() for t in (y, z, dx, dw, db)]
        assert i > 0 or not torch.equal(eager[0], want[0])
        for t in (y, z, dx, dw, db):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(eager, (y, z, dx, dw, db)):
            assert torch.equal(p, q)
