"""The AdamW step's C ABI on the host: validation and error statuses, on fake addresses
that are never dereferenced."""
import ctypes
import math

import pytest
import torch

import convolution_implicit_gemm_amd as c3d

BAD, UNSUP = c3d.CONV3D_ERR_INVALID_ARG, c3d.CONV3D_ERR_UNSUPPORTED
A = [(i + 1) << 42 for i in range(16)]
S8, G32 = c3d.CONV3D_F_STATE8, c3d.CONV3D_F_GRAD32


def tensor(**kw):
    base = dict(param=A[0], master=A[1], grad=A[2], m=A[3], v=A[4], m_scale=A[5], v_scale=A[6], count=1000, decay=1.0)
    base.update(kw)
    return c3d.adamw_tensor(**base)


def plan(tensors, flags=0, count=None):
    h = ctypes.c_void_p()
    arr = (c3d.adamw_tensor * max(len(tensors), 1))(*tensors)
    lib = c3d.load_library()
    st = lib.adamw_plan(arr, len(tensors) if count is None else count, flags, ctypes.byref(h))
    if st == 0:
        lib.adamw_plan_destroy(h)
    return st


@pytest.mark.parametrize("bad,flags,want", [
    (dict(), 0, 0), (dict(), S8, 0), (dict(param=None), 0, 0), (dict(master=None), 0, 0), (dict(count=0, grad=None), 0, 0),
    (dict(m_scale=None, v_scale=None), 0, 0), (dict(param=None, master=None), 0, BAD), (dict(grad=None), 0, BAD),
    (dict(m=None), 0, BAD), (dict(v=None), 0, BAD), (dict(m_scale=None), S8, BAD), (dict(v_scale=None), S8, BAD),
    (dict(count=-1), 0, BAD), (dict(decay=-1.0), 0, BAD), (dict(decay=math.nan), 0, BAD), (dict(decay=math.inf), 0, BAD),
    (dict(param=A[0] + 2), 0, BAD), (dict(grad=A[2] + 4), 0, BAD), (dict(m=A[3] + 8), 0, BAD), (dict(m_scale=A[5] + 1), S8, 0),
    (dict(v=A[3]), 0, BAD), (dict(v=A[3] + 3984), 0, BAD), (dict(v=A[3] + 4000), 0, 0), (dict(grad=A[0]), 0, BAD),
    (dict(grad=A[1] + 3984), G32, BAD), (dict(v_scale=A[5] + 7), S8, BAD), (dict(v_scale=A[5] + 8), S8, 0),
    (dict(count=1 << 40), 0, UNSUP), (dict(), 1, BAD), (dict(), 1 << 20, BAD)])
def test_plan_checks_a_tensor(bad, flags, want):
    assert plan([tensor(**bad)], flags) == want


def test_plan_checks_tensors_against_each_other():
    shift = 1 << 30
    moved = {k: A[i] + shift for i, k in enumerate(("param", "master", "grad", "m", "v", "m_scale", "v_scale"))}
    assert plan([tensor(), tensor(**moved)]) == 0
    assert plan([tensor(), tensor(**dict(moved, grad=A[2]))]) == 0  # gradients are only read
    assert plan([tensor(), tensor(**dict(moved, grad=A[2] + 16))]) == 0
    for k in ("param", "master", "m", "v"):
        assert plan([tensor(), tensor(**dict(moved, **{k: getattr(tensor(), k)}))]) == BAD
    assert plan([tensor(), tensor(**dict(moved, grad=A[1]))]) == BAD
    assert plan([tensor(), tensor()]) == BAD
    # a long gradient over several tensors' outputs
    assert plan([tensor(grad=A[7], count=1 << 20), tensor(**dict(moved, m=A[7] + 4096))]) == BAD


def test_null_arguments():
    lib = c3d.load_library()
    h = ctypes.c_void_p()
    arr = (c3d.adamw_tensor * 1)(tensor())
    assert lib.adamw_plan(None, 1, 0, ctypes.byref(h)) == BAD
    assert lib.adamw_plan(arr, 1, 0, None) == BAD
    assert lib.adamw_plan(arr, -1, 0, ctypes.byref(h)) == BAD
    assert lib.adamw_plan(None, 0, 0, ctypes.byref(h)) == 0
    hyper = c3d.make_adamw_hyper(1e-3)
    assert lib.adamw_step(h, ctypes.byref(hyper), None, None) == 0  # nothing to do
    assert lib.adamw_step(h, None, None, None) == BAD
    lib.adamw_plan_destroy(h)
    assert lib.adamw_step(None, ctypes.byref(hyper), None, None) == BAD
    assert lib.adamw_hyper_pack(None, (ctypes.c_float * 9)()) == BAD
    assert lib.adamw_hyper_pack(ctypes.byref(hyper), None) == BAD
    lib.adamw_plan_destroy(None)


@pytest.mark.parametrize("bad", [
    dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=math.nan),
    dict(eps=-1e-8), dict(eps=math.inf), dict(weight_decay=-0.1), dict(grad_scale=math.nan), dict(step=0), dict(step=-5)])
def test_hyperparameters_are_checked(bad):
    with pytest.raises(c3d.Conv3dError) as e:
        c3d.adamw_hyper_pack(c3d.make_adamw_hyper(**dict(dict(lr=1e-3), **bad)))
    assert e.value.status == BAD


@pytest.mark.parametrize("bad", [dict(lr=1e39), dict(lr=1e38, beta1=0.999), dict(eps=1e39), dict(grad_scale=-1e39),
                                 dict(lr=1e20, weight_decay=1e20)])
def test_hyperparameters_past_fp32(bad):
    with pytest.raises(c3d.Conv3dError) as e:
        c3d.adamw_hyper_pack(c3d.make_adamw_hyper(**dict(dict(lr=1e-3), **bad)))
    assert e.value.status == BAD


def test_packed_numbers():
    h = c3d.make_adamw_hyper(1e-3, 0.9, 0.999, 1e-8, 0.1, 10, 0.5)
    want = [0.5, 0.9, 0.1, 0.999, 0.001, 1e-3 / (1 - 0.9 ** 10), (1 - 0.999 ** 10) ** -0.5, 1e-8, 1e-4]
    assert c3d.adamw_hyper_pack(h) == pytest.approx(want, rel=2.0 ** -24)
    far = c3d.adamw_hyper_pack(c3d.make_adamw_hyper(1e-3, 0.0, 1 - 2.0 ** -40, step=1))
    assert far[5] == pytest.approx(1e-3, rel=2.0 ** -24) and far[6] == pytest.approx(2.0 ** 20, rel=1e-6)


def test_device_hyperparameters_are_checked():
    lib = c3d.load_library()
    h = ctypes.c_void_p()
    assert lib.adamw_plan((c3d.adamw_tensor * 1)(tensor()), 1, 0, ctypes.byref(h)) == 0
    for at in (A[8] + 2, A[1], A[1] + 3996, A[3] - 4, A[0] + 1996):
        assert lib.adamw_step(h, None, at, None) == BAD
    lib.adamw_plan_destroy(h)


def test_binding_checks_the_lists():
    f = torch.zeros(16)
    for args in (([f], [f, f], [f], [f]), ([f], [f], [f], [f]), (None, [f.half()], [f], [f.half()]),
                 (None, [f], [f], [f])):
        with pytest.raises(c3d.Conv3dError):
            c3d.adamw_list(*args, master=[f])
    with pytest.raises(c3d.Conv3dError, match=r"grads\[1\] is missing"):
        c3d.adamw_list(None, [f, None], [f, f], [f, f], master=[f, f])


@pytest.mark.parametrize("eps,ok", [(0.0, True), (2.0 ** -126, True), (1e-30, True), (1.1e-38, False), (1e-39, False),
                                    (1e-45, False), (1e-60, False)])
def test_eps_is_a_normal_number_or_zero(eps, ok):
    hyper = c3d.make_adamw_hyper(1e-3, eps=eps)
    if ok:
        assert c3d.adamw_hyper_pack(hyper)[7] == eps or eps == 1e-30
    else:
        with pytest.raises(c3d.Conv3dError) as e:
            c3d.adamw_hyper_pack(hyper)
        assert e.value.status == BAD
        lib, h = c3d.load_library(), ctypes.c_void_p()
        assert lib.adamw_plan((c3d.adamw_tensor * 1)(tensor()), 1, 0, ctypes.byref(h)) == 0
        assert lib.adamw_step(h, ctypes.byref(hyper), None, None) == BAD
        lib.adamw_plan_destroy(h)
