"""The token operators' C ABI on the host: planning, validation, error statuses.

Every argument check runs before the device is touched, so fake addresses that
are never dereferenced are enough to reach each status.
"""
import ctypes
import math

import pytest
import torch

import convolution_implicit_gemm_amd as c3d

BAD, UNSUP, WS = c3d.CONV3D_ERR_INVALID_ARG, c3d.CONV3D_ERR_UNSUPPORTED, c3d.CONV3D_ERR_WORKSPACE
A, B, C, D, E, F, G = ((i + 1) << 40 for i in range(7))  # far apart, aligned


def status(call, *args, **kw):
    with pytest.raises(c3d.Conv3dError) as e:
        call(*args, **kw)
    assert c3d.conv3d_last_error()
    return e.value.status


def ldesc(**kw):
    base = dict(m=100, n=64, k=32, act=0, flags=0, x_stride=0, y_stride=0, residual_stride=0)
    base.update(kw)
    return c3d.make_linear_desc(**base)


@pytest.mark.parametrize("bad,want", [
    (dict(m=-1), BAD), (dict(n=0), BAD), (dict(k=0), BAD), (dict(k=-8), BAD), (dict(act=4), BAD), (dict(act=-1), BAD),
    (dict(flags=c3d.CONV3D_F_CHUNK), BAD), (dict(flags=c3d.CONV3D_F_POSITIONS), BAD), (dict(flags=1 << 20), BAD),
    (dict(x_stride=24), BAD), (dict(x_stride=36), BAD), (dict(x_stride=-32), BAD), (dict(y_stride=56), BAD),
    (dict(residual_stride=68), BAD), (dict(n=60), UNSUP), (dict(k=33), UNSUP), (dict(n=65544), UNSUP),
    (dict(k=65544), UNSUP), (dict(m=1 << 30), UNSUP), (dict(x_stride=(1 << 20) + 8), UNSUP)])
def test_linear_plan_refuses(bad, want):
    assert status(c3d.linear_plan, ldesc(**bad)) == want


def test_linear_plan_null_pointers():
    lib = c3d.load_library()
    h, ws, d = ctypes.c_void_p(), ctypes.c_size_t(), ldesc()
    assert lib.linear_plan(None, ctypes.byref(h), ctypes.byref(ws)) == BAD
    assert lib.linear_plan(ctypes.byref(d), None, ctypes.byref(ws)) == BAD
    assert lib.linear_plan(ctypes.byref(d), ctypes.byref(h), None) == BAD
    assert lib.linear_plan_query(None, None) == BAD
    assert lib.linear_forward(None, *([A] * 7), 0, None) == BAD
    assert lib.linear_backward(None, *([A] * 8), 0, None) == BAD
    assert lib.linear_backward_workspace(None) == 0
    lib.linear_plan_destroy(None)


ALL = c3d.CONV3D_F_BIAS | c3d.CONV3D_F_RESIDUAL | c3d.CONV3D_F_PREACT


@pytest.mark.parametrize("args,want", [
    ((0, B, C, D, E, F, None), BAD), ((A, 0, C, D, E, F, None), BAD), ((A, B, 0, D, E, F, None), BAD),
    ((A, B, C, 0, E, F, None), BAD), ((A, B, C, D, 0, F, None), BAD), ((A, B, C, D, E, 0, None), BAD),
    ((A + 8, B, C, D, E, F, None), BAD), ((A, B, C, D, E + 2, F, None), BAD), ((A, B, C, D, A, F, None), BAD),
    ((A, B, C, D, B + 64, F, None), BAD), ((A, B, C, D, D, F, None), BAD), ((A, B, C, D, E, D + 64, None), BAD),
    ((A, B, C, D, E, E + 6400, None), BAD)])
def test_linear_forward_refuses(args, want):
    plan = c3d.linear_plan(ldesc(flags=ALL))
    args = [a or None for a in args]
    assert status(c3d.linear_forward, plan, *args, stream=0) == want


def test_linear_workspace_checks():
    d = ldesc(m=256, n=256, k=32768)
    plan = c3d.linear_plan(d)
    assert plan.workspace_bytes > 0 and plan.info().split_pieces > 1
    assert plan.info().workspace_bytes == plan.workspace_bytes
    assert status(c3d.linear_forward, plan, A, B, None, None, E, None, None, stream=0) == WS
    assert status(c3d.linear_forward, plan, A, B, None, None, E, None, F, plan.workspace_bytes - 1, stream=0) == WS
    assert status(c3d.linear_forward, plan, A, B, None, None, E, None, F + 8, stream=0) == BAD
    assert status(c3d.linear_forward, plan, A, B, None, None, E, None, E, stream=0) == BAD
    assert status(c3d.linear_forward, plan, A, B, None, None, E, None, A, stream=0) == BAD


@pytest.mark.parametrize("args,want", [
    ((0, B, C, D, E, F, G), BAD), ((A, 0, C, D, E, F, G), BAD), ((A, B, 0, D, E, F, G), BAD),
    ((A, B, C, 0, E, F, G), BAD), ((A, B, C, D, 0, 0, 0), BAD), ((A, B, C, D, A, F, G), BAD),
    ((A, B, C, D, E, B, G), BAD), ((A, B, C, D, E, F, C), BAD), ((A, B, C, D, E, E + 64, G), BAD),
    ((A, B, C, D, E + 4, F, G), BAD)])
def test_linear_backward_refuses(args, want):
    plan = c3d.linear_plan(ldesc(act=c3d.CONV3D_ACT_GELU))
    args = [a or None for a in args]
    assert status(c3d.linear_backward, plan, *args, 8 << 40, stream=0) == want


def test_linear_backward_workspace_checks():
    plan = c3d.linear_plan(ldesc(act=c3d.CONV3D_ACT_SILU))
    need = c3d.linear_backward_workspace(plan)
    assert need >= 100 * 64 * 2
    assert status(c3d.linear_backward, plan, A, B, C, D, E, F, G, None, 0, stream=0) == WS
    assert status(c3d.linear_backward, plan, A, B, C, D, E, F, G, 8 << 40, need - 1, stream=0) == WS
    assert status(c3d.linear_backward, plan, A, B, C, D, E, F, G, E, need, stream=0) == BAD


def ln(x=A, gamma=B, beta=C, y=D, stats=E, rows=10, c=64, xs=0, ys=0, eps=1e-6):
    c3d.layernorm(x, gamma, beta, y, stats, rows, c, eps, xs, ys, stream=0)


@pytest.mark.parametrize("bad,want", [
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(rows=-1), BAD), (dict(c=0), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=math.nan), BAD), (dict(xs=60), BAD), (dict(ys=56), BAD), (dict(x=A + 2), BAD), (dict(gamma=B + 2), BAD),
    (dict(stats=E + 4), BAD), (dict(y=A + 16), BAD), (dict(y=A, ys=72), BAD), (dict(y=B), BAD), (dict(stats=A), BAD),
    (dict(stats=D), BAD), (dict(c=60), UNSUP), (dict(c=16392), UNSUP), (dict(rows=1 << 40), UNSUP),
    (dict(xs=(1 << 20) + 8), UNSUP)])
def test_layernorm_refuses(bad, want):
    assert status(lambda: ln(**bad)) == want


def ln_back(dy=A, x=B, gamma=C, stats=D, dres=E, dx=F, dg=G, db=8 << 40, rows=10, c=64, ws=9 << 40, xs=0, ys=0,
            wsb=None):
    c3d.layernorm_backward(dy, x, gamma, stats, dres, dx, dg, db, rows, c, ws, xs, ys, wsb, stream=0)


@pytest.mark.parametrize("bad,want", [
    (dict(dy=None), BAD), (dict(x=None), BAD), (dict(stats=None), BAD), (dict(dx=None), BAD), (dict(rows=-1), BAD),
    (dict(xs=60), BAD), (dict(ys=100), BAD), (dict(dy=A + 2), BAD), (dict(dg=G + 1), BAD), (dict(dx=A, ys=72), BAD),
    (dict(dx=B + 16), BAD), (dict(dx=E + 16), BAD), (dict(dx=C), BAD), (dict(dg=A), BAD), (dict(dg=F), BAD),
    (dict(db=G), BAD), (dict(ws=A), BAD), (dict(ws=F), BAD), (dict(ws=(9 << 40) + 4), BAD), (dict(c=12), UNSUP),
    (dict(c=16392), UNSUP), (dict(ws=None, wsb=0), WS), (dict(wsb=16), WS)])
def test_layernorm_backward_refuses(bad, want):
    assert status(lambda: ln_back(**bad)) == want


def test_layernorm_backward_workspace_of_refused_sizes():
    for rows, c in ((0, 64), (-1, 64), (10, 0), (10, 12), (10, 16392)):
        assert c3d.layernorm_backward_workspace(rows, c) == 0
    assert c3d.layernorm_backward_workspace(10, 64) > 0


def rdesc(**kw):
    base = dict(n=1, t=2, h=3, w=4, heads_q=4, heads_k=2, head_dim=64, dims=(16, 24, 24))
    base.update(kw)
    return c3d.make_rope3d_desc(**base)


@pytest.mark.parametrize("bad,want", [
    (dict(n=-1), BAD), (dict(t=-1), BAD), (dict(h=-2), BAD), (dict(w=-1), BAD), (dict(heads_q=0), BAD),
    (dict(heads_k=-1), BAD), (dict(head_dim=0), BAD), (dict(dims=(15, 24, 24)), BAD), (dict(dims=(-2, 24, 24)), BAD),
    (dict(dims=(0, 0, 0)), BAD), (dict(dims=(32, 24, 24)), BAD), (dict(base=0.0), BAD), (dict(base=-1.0), BAD),
    (dict(base=math.inf), BAD), (dict(base=math.nan), BAD), (dict(pairing=2), BAD), (dict(flags=c3d.CONV3D_F_BIAS), BAD),
    (dict(q_stride=(4, 64, 64)), BAD), (dict(k_out_stride=(-8, 64, 64)), BAD), (dict(head_dim=60, dims=(16, 16, 16)), UNSUP),
    (dict(head_dim=520), UNSUP), (dict(head_dim=512, dims=(128, 128, 64)), UNSUP),
    (dict(pairing=1, dims=(16, 24, 16)), UNSUP), (dict(n=1 << 12, t=1 << 7, h=1 << 6, w=1 << 6), UNSUP),
    (dict(q_stride=(1 << 40, 64, 64)), UNSUP)])
def test_rope3d_plan_refuses(bad, want):
    assert status(c3d.rope3d_plan, rdesc(**bad)) == want


@pytest.mark.parametrize("args", [
    (None, B, C, D, E), (A, None, C, D, E), (A, B, None, D, E), (A, B, C, None, E), (A, B, C, D, None),
    (A + 2, B, C, D, E), (A, B, C, D, E + 2), (A, B, A + 64, D, E), (A, B, C, B + 128, E)])
@pytest.mark.parametrize("call", [c3d.rope3d_forward, c3d.rope3d_backward])
def test_rope3d_calls_refuse(args, call):
    plan = c3d.rope3d_plan(rdesc(flags=c3d.CONV3D_F_POSITIONS))
    assert status(call, plan, *args, 0, 0) == BAD


def test_rope3d_in_place_needs_the_same_strides():
    plan = c3d.rope3d_plan(rdesc(q_out_stride=(24576, 512, 64)))
    assert status(c3d.rope3d_forward, plan, A, B, A, D, None, 0, 0) == BAD
    lib = c3d.load_library()
    assert lib.rope3d_forward(None, A, B, C, D, None, 0, None) == BAD
    assert lib.rope3d_plan(None, None) == BAD
    lib.rope3d_plan_destroy(None)


def test_binding_checks_tensors_before_the_call():
    plan = c3d.linear_plan(ldesc())
    cpu = torch.zeros((100, 32), dtype=torch.float16)
    with pytest.raises(c3d.Conv3dError, match="x is on cpu"):
        c3d.linear_forward(plan, cpu, B, None, None, E, None, None, stream=0)


def test_conv_plans_refuse_the_token_flags():
    d = c3d.make_desc(1, 4, 8, 8, 16, 16)
    for flag in (c3d.CONV3D_F_PREACT, c3d.CONV3D_F_POSITIONS):
        d.flags = flag
        assert status(c3d.conv3d_plan, d) == BAD
