"""What the Python binding checks and binds before it calls the library (no GPU needed)."""
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as c3d


def unset_while_tested_name_is_set(monkeypatch, bind, tested, others):
    """The names that another thread could find unset after `tested` is set, at any
    instruction of `bind` (a thread switch may come between any two)."""
    for name in (tested,) + others:
        monkeypatch.setattr(c3d, name, None)
    seen = set()

    def trace(frame, event, arg):
        frame.f_trace_opcodes = True
        if frame.f_code is bind.__code__ and getattr(c3d, tested) is not None:
            seen.update(n for n in others if getattr(c3d, n) is None)
        return trace

    old = sys.gettrace()
    sys.settrace(trace)
    try:
        bind()
    finally:
        sys.settrace(old)
    assert all(getattr(c3d, n) is not None for n in (tested,) + others)
    return seen


def test_first_use_from_two_threads_finds_every_element_type(monkeypatch):
    assert not unset_while_tested_name_is_set(monkeypatch, c3d._bind_torch, "_F16", ("_BF16", "_F32", "_I32"))


def test_first_use_from_two_threads_finds_the_device_with_the_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert not unset_while_tested_name_is_set(monkeypatch, c3d._bind_streams, "_raw_stream", ("_current_device",))


class OnGpu:
    """A host tensor that says it is on a GPU: the binding's checks read nothing else of it."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def rows_address(t, rows, cols, stride=0, dtype=torch.float16):
    return c3d._rows_addr(OnGpu(t), "x", rows, cols, stride, dtype)


def heads_address(t, n, tokens, heads, dim, strides):
    return c3d._strided_addr(OnGpu(t), "q", (n, tokens, heads, dim), tuple(strides) + (1,), torch.float16)


BUF = torch.zeros((64, 48), dtype=torch.float16)


@pytest.mark.parametrize("t,rows,cols,stride", [
    (BUF[:10], 11, 48, 0), (BUF[:10], 64, 48, 0), (BUF[:1], 2, 48, 0), (BUF[:10, :32], 11, 32, 48),
    (BUF[:10, :24], 10, 32, 48), (BUF[20:30, 8:40], 12, 32, 48), (BUF[:, :1], 64, 8, 48),
    (BUF.view(-1)[:480], 10, 48, 56), (BUF.view(-1)[:480], 11, 48, 0), (BUF[:10].view(2, 5, 48), 11, 48, 0),
    (BUF[:1].expand(10, 48), 10, 48, 0), (BUF[:10].t(), 10, 48, 0), (BUF[::2], 32, 48, 0), (BUF, 65, 48, 0)])
def test_rows_outside_the_tensor_are_refused(t, rows, cols, stride):
    # also where its storage goes on behind it
    with pytest.raises(c3d.Conv3dError) as e:
        rows_address(t, rows, cols, stride)
    assert e.value.status == c3d.CONV3D_ERR_INVALID_ARG


@pytest.mark.parametrize("t,rows,cols,stride", [
    (BUF, 64, 48, 0), (BUF, 10, 48, 0), (BUF[:10], 10, 48, 0), (BUF[5:6], 1, 48, 96), (BUF[:, 8:40], 64, 32, 48),
    (BUF, 64, 32, 48), (BUF.view(-1), 64, 48, 0), (BUF.view(-1)[:480], 10, 48, 0), (BUF.view(4, 16, 48), 64, 48, 0),
    (BUF.view(1, -1), 64, 48, 0), (BUF.view(-1)[:-16], 64, 32, 48), (BUF[::2, :16], 32, 16, 96), (BUF[:0], 0, 48, 0)])
def test_rows_inside_the_tensor_are_taken(t, rows, cols, stride):
    assert rows_address(t, rows, cols, stride) == (t.data_ptr() or None)


def test_heads_outside_the_tensor_are_refused():
    # the heads of q, k and v side by side in each token's row
    qkv = torch.zeros((2, 6, 12, 16), dtype=torch.float16)
    q = qkv[:, :, :4]
    assert heads_address(q, 2, 6, 4, 16, q.stride()[:3]) == q.data_ptr()
    for view in (qkv[:1, :, :4], qkv[:, :5, :4], qkv[:, :, :3], qkv[:, :, :4, :8]):
        with pytest.raises(c3d.Conv3dError):
            heads_address(view, 2, 6, 4, 16, q.stride()[:3])
