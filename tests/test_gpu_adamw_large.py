"""AdamW steps over more memory than the last-level cache holds (256 MiB), which go past the caches, in workgroups
of twice the elements: against the formula in 64 bits, and bit by bit against steps over the same tensors piece by piece."""
import pytest
import torch

import convolution_implicit_gemm_amd as c3d
from test_gpu_adamw import B, SIZES, Tensors

pytestmark = pytest.mark.gpu

CACHED = 256 << 20


def copies(t):
    """The lists that a step writes, and grads, as new tensors."""
    return {k: [None if x is None else x.clone() for x in getattr(t, k)]
            for k in ("params", "master", "grads", "m", "v", "ms", "vs")}


def pieces(sizes, most):
    """(index of the tensor, first and last element) of pieces of at most `most` elements."""
    for i, n in enumerate(sizes):
        for lo in range(0, n, most):
            yield i, lo, min(n, lo + most)


@pytest.mark.parametrize("state8", [False, True])
@pytest.mark.parametrize("dtype,master,param,grad32", [
    ("bf16", True, True, False), ("bf16", True, True, True), ("fp16", True, True, False), ("fp16", True, True, True),
    ("bf16", False, True, False), ("fp16", True, False, True)])
def test_steps_past_the_caches(dtype, master, param, grad32, state8):
    each = 2 * param + 4 * master + (4 if grad32 else 2) + (2 if state8 else 8)
    large = CACHED // each + 4099  # no multiple of anything
    sizes = SIZES[:6] + [large] + SIZES[6:]
    t = Tensors(sizes, dtype, master, param, grad32, state8, seed=21)
    assert sum(sizes) * each > CACHED
    before = copies(t)
    h = c3d.make_adamw_hyper(1e-3, 0.9, 0.98, 1e-8, 0.1, 10, grad_scale=0.25)
    want = [t.want(h, i) for i in range(len(sizes))]
    c3d.adamw_step(t.list(), h)
    t.check(want)
    del want
    most = large // 4 // B * B
    for i, lo, hi in pieces(sizes, most):
        def cut(k, block=1):
            x = before[k][i] if before[k] else None
            return None if x is None else [x[lo // block:-(-hi // block)]]

        names = ("params", "grads", "m", "v")
        got = [cut(k) for k in names]
        more = dict(master=cut("master"), decay=[t.decay[i]])
        if state8:
            more.update(m_scale=cut("ms", B), v_scale=cut("vs", B))
        c3d.adamw_step(c3d.adamw_list(*got, **more), h)
    for k, lists in before.items():
        for i, x in enumerate(lists):
            assert x is None or torch.equal(x, getattr(t, k)[i]), "%s[%d]" % (k, i)


@pytest.mark.parametrize("state8", [False, True])
def test_neighbours_of_large_tensors_are_left_alone(state8):
    n, at = CACHED // (10 if state8 else 14) + 1237, 64
    kind = torch.uint8 if state8 else torch.float32
    w = torch.full((n + 4 * at,), 3.0, device="cuda:0")
    m, v = (torch.full((n + 4 * at,), 17, dtype=kind, device="cuda:0") for _ in range(2))
    p = torch.full((n + 4 * at,), 3.0, dtype=torch.bfloat16, device="cuda:0")
    blocks = -(-n // B)
    ms, vs = (torch.full((blocks + 16,), 100, dtype=torch.uint8, device="cuda:0") for _ in range(2))
    g = torch.ones(n, device="cuda:0")
    lst = c3d.adamw_list([p[at:at + n]], [g], [m[at:at + n]], [v[at:at + n]], master=[w[at:at + n]],
                         m_scale=[ms[5:5 + blocks]] if state8 else None, v_scale=[vs[5:5 + blocks]] if state8 else None)
    c3d.adamw_step(lst, c3d.make_adamw_hyper(1e-1))
    for x, fill in ((w, 3.0), (p, 3.0), (m, 17), (v, 17)):
        assert bool((x[:at] == fill).all()) and bool((x[at + n:] == fill).all())
        assert not bool((x[at:at + n] == fill).any())
    if state8:
        for x in (ms, vs):
            assert bool((x[:5] == 100).all()) and bool((x[5 + blocks:] == 100).all())
