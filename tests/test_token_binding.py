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
