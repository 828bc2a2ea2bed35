"""Attention's C ABI on the host: planning, validation, error statuses.

Every argument check runs before the device is touched, so fake addresses that
are never dereferenced are enough to reach each status.
"""
import ctypes
import math

import pytest
import torch

import convolution_implicit_gemm_amd as c3d

BAD, UNSUP, WS = c3d.CONV3D_ERR_INVALID_ARG, c3d.CONV3D_ERR_UNSUPPORTED, c3d.CONV3D_ERR_WORKSPACE
A, B, C, D, E, F, G, H, I, J, K = ((i + 1) << 40 for i in range(11))  # far apart, aligned


def status(call, *args, **kw):
    with pytest.raises(c3d.Conv3dError) as e:
        call(*args, **kw)
    assert c3d.conv3d_last_error()
    return e.value.status


def desc(**kw):
    base = dict(n=2, tq=40, tk=50, heads_q=4, heads_k=2, head_dim=64)
    base.update(kw)
    return c3d.make_attention_desc(**base)


@pytest.mark.parametrize("bad,want", [
    (dict(n=-1), BAD), (dict(tq=-1), BAD), (dict(tk=-1), BAD), (dict(frame=-1), BAD), (dict(frame=4, window=-1), BAD),
    (dict(window=1), BAD), (dict(heads_q=0), BAD), (dict(heads_k=0), BAD), (dict(heads_q=3), BAD), (dict(heads_q=1), BAD),
    (dict(head_dim=0), BAD), (dict(head_dim=-8), BAD), (dict(scale=-1.0), BAD), (dict(scale=math.inf), BAD),
    (dict(scale=math.nan), BAD), (dict(flags=c3d.CONV3D_F_BIAS), BAD), (dict(flags=1 << 20), BAD),
    (dict(q_stride=(8, 4, 64)), BAD), (dict(k_stride=(-8, 128, 64)), BAD), (dict(v_stride=(0, 56, 64)), BAD),
    (dict(o_stride=(10240, 256, 60)), BAD), (dict(head_dim=60), UNSUP), (dict(head_dim=136), UNSUP),
    (dict(heads_q=16386), UNSUP), (dict(tk=1 << 30), UNSUP), (dict(tq=1 << 29), UNSUP),
    (dict(q_stride=(1 << 40, 256, 64)), UNSUP), (dict(k_stride=(0, (1 << 20) + 8, 64)), UNSUP),
    (dict(n=1 << 20, tq=256, k_stride=(8, 128, 64)), UNSUP), (dict(n=1 << 12, q_stride=((1 << 40) - 8, 256, 64)), UNSUP)])
def test_plan_refuses(bad, want):
    assert status(c3d.attention_plan, desc(**bad)) == want


@pytest.mark.parametrize("scale,ok", [(2.0 ** -64, True), (2.0 ** 64, True), (0.0, True), (2.0 ** -66, False), (1e-39, False),
                                      (2.0 ** 65, False)])
def test_scales_that_lse_can_be_divided_by(scale, ok):
    if ok:
        c3d.attention_plan(desc(scale=scale))
    else:
        assert status(c3d.attention_plan, desc(scale=scale)) == UNSUP


def test_null_pointers():
    lib = c3d.load_library()
    h, ws, d = ctypes.c_void_p(), ctypes.c_size_t(), desc()
    assert lib.attention_plan(None, ctypes.byref(h), ctypes.byref(ws)) == BAD
    assert lib.attention_plan(ctypes.byref(d), None, ctypes.byref(ws)) == BAD
    assert lib.attention_plan(ctypes.byref(d), ctypes.byref(h), None) == BAD
    assert lib.attention_plan_query(None, None) == BAD
    assert lib.attention_forward(None, *([A] * 6), 0, A, 0, None) == BAD
    assert lib.attention_backward(None, *([A] * 10), 0, A, 0, None) == BAD
    assert lib.attention_backward_workspace(None) == 0
    lib.attention_plan_destroy(None)


L = c3d.CONV3D_F_LENGTHS


@pytest.mark.parametrize("args,want", [
    ((None, B, C, D, E, F), BAD), ((A, None, C, D, E, F), BAD), ((A, B, None, D, E, F), BAD), ((A, B, C, None, E, F), BAD),
    ((A, B, C, D, E, None), BAD), ((A + 8, B, C, D, E, F), BAD), ((A, B, C + 2, D, E, F), BAD), ((A, B, C, D, E + 2, F), BAD),
    ((A, B, C, D, E, F + 1), BAD), ((A, B, C, A, E, F), BAD), ((A, B, C, B + 64, E, F), BAD), ((A, B, C, D, D, F), BAD),
    ((A, B, C, D, C, F), BAD), ((A, B, C, D, F, F), BAD)])
def test_forward_refuses(args, want):
    plan = c3d.attention_plan(desc(flags=L))
    assert status(c3d.attention_forward, plan, *args, 0, G, 1 << 30, stream=0) == want


def test_forward_refuses_offsets_and_workspaces():
    plan = c3d.attention_plan(desc())
    for off in ((1 << 30) + 1, -(1 << 30) - 1, 1 << 62):
        assert status(c3d.attention_forward, plan, A, B, C, D, None, None, off, G, 0, stream=0) == BAD
    split = c3d.attention_plan(desc(n=1, tq=1, tk=100000))
    assert split.info().splits > 1 and split.workspace_bytes > 0
    assert status(c3d.attention_forward, split, A, B, C, D, None, None, 0, None, 0, stream=0) == WS
    assert status(c3d.attention_forward, split, A, B, C, D, None, None, 0, G, split.workspace_bytes - 1, stream=0) == WS
    assert status(c3d.attention_forward, split, A, B, C, D, None, None, 0, G + 8, 1 << 40, stream=0) == BAD
    assert status(c3d.attention_forward, split, A, B, C, D, None, None, 0, B + 1024, split.workspace_bytes, stream=0) == BAD


def back(flags=L, wsb=1 << 30, q_offset=0, plan=None, **kw):
    a = dict(dout=A, q=B, k=C, v=D, o=E, lse=F, dq=G, dk=H, dv=I, lengths=J, ws=K)
    a.update(kw)
    plan = plan or c3d.attention_plan(desc(flags=flags))
    ws = a.pop("ws")
    c3d.attention_backward(plan, *a.values(), q_offset=q_offset, workspace=ws, workspace_bytes=wsb, stream=0)


@pytest.mark.parametrize("bad,want", [
    (dict(dout=None), BAD), (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(o=None), BAD),
    (dict(lse=None), BAD), (dict(lengths=None), BAD), (dict(dq=None, dk=None, dv=None), BAD), (dict(dq=G + 2), BAD),
    (dict(lse=F + 2), BAD), (dict(dq=B), BAD), (dict(dk=C), BAD), (dict(dv=C + 64), BAD), (dict(dq=A), BAD), (dict(dk=E), BAD),
    (dict(dk=I), BAD), (dict(dq=I + 64), BAD), (dict(dq=F), BAD), (dict(ws=G), BAD), (dict(ws=F), BAD), (dict(ws=B), BAD),
    (dict(ws=K + 4), BAD), (dict(q_offset=1 << 31), BAD), (dict(ws=None, wsb=0), WS), (dict(wsb=64), WS)])
def test_backward_refuses(bad, want):
    assert status(lambda: back(**bad)) == want


def test_outputs_that_fold_are_refused():
    plan = c3d.attention_plan(desc(o_stride=(10240, 256, 32)))
    assert status(c3d.attention_forward, plan, A, B, C, D, None, None, 0, None, 0, stream=0) == BAD
    plan = c3d.attention_plan(desc(k_stride=(0, 128, 64)))  # keys that all samples share are fine, their gradient is not
    assert status(lambda: back(plan=plan)) == BAD


def test_fused_projections_are_told_apart():
    # q, k and v side by side in a token's row, gradients too: refused only where they really meet
    row = 8 * 64
    st = (40 * row, row, 64)
    plan = c3d.attention_plan(desc(tk=40, q_stride=st, k_stride=st, v_stride=st))
    w = c3d.attention_backward_workspace(plan)
    args = dict(q=A, k=A + 4 * 128, v=A + 6 * 128, dout=B, o=C, dq=D, dk=D + 4 * 128, lse=F, lengths=None, plan=plan, wsb=w)
    assert status(lambda: back(dv=D + 5 * 128, **args)) == BAD
    assert "gradients overlap" in c3d.conv3d_last_error()


def test_workspace_sizes_and_kernels():
    one = c3d.attention_plan(desc(tq=1))
    many = c3d.attention_plan(desc(tq=1000))
    assert one.info().kernel_name == b"attention_few" and one.info().tile_rows == 32
    assert many.info().kernel_name in (b"attention_64x128", b"attention_128x128", b"attention_256x64")
    assert many.info().backward_workspace_bytes == c3d.attention_backward_workspace(many) >= 2 * 4 * 2 * 4 * 1000
    assert c3d.attention_plan(desc(n=0)).workspace_bytes == 0
    assert c3d.attention_plan(desc(tk=0)).workspace_bytes == 0


def test_binding_checks_tensors_before_the_call():
    plan = c3d.attention_plan(desc())
    cpu = torch.zeros((2, 40, 4, 64), dtype=torch.float16)
    with pytest.raises(c3d.Conv3dError, match="q is on cpu"):
        c3d.attention_forward(plan, cpu, B, C, D, stream=0)


def test_other_operators_refuse_attentions_flags():
    for flag in (c3d.CONV3D_F_LENGTHS, c3d.CONV3D_F_TAIL):
        assert status(c3d.linear_plan, c3d.make_linear_desc(8, 8, 8, flags=flag)) == BAD
        assert status(c3d.rope3d_plan, c3d.make_rope3d_desc(1, 1, 1, 1, 1, 1, 16, (16, 0, 0), flags=flag)) == BAD
        d = c3d.make_desc(1, 4, 8, 8, 16, 16)
        d.flags = flag
        assert status(c3d.conv3d_plan, d) == BAD
