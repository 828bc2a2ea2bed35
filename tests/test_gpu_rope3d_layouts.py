"""rope3d on layouts that its overlap checks have to let through, against the 64-bit form."""
import pytest
import torch

import convolution_implicit_gemm_amd as c3d
from test_gpu_rope3d import grid_positions, rope64
from token_helpers import assert_within, gen, normal

pytestmark = pytest.mark.gpu

T, H, W, HQ, HK, D, DIMS = 2, 3, 5, 4, 2, 64, (16, 24, 24)
TOK = T * H * W


def check(x, got, n, what, inverse=False):
    ref, slack = rope64(x, grid_positions(n, T, H, W), DIMS, 10000.0, "adjacent", inverse)
    assert_within(got, ref, slack, what)


def plan(n, **strides):
    return c3d.rope3d_plan(c3d.make_rope3d_desc(n, T, H, W, HQ, HK, D, DIMS, **strides))


def views(layout, n):
    """q and k heads of one buffer in a layout of (sample, token, head, element)."""
    sizes = {"n": n, "t": TOK, "h": HQ + HK, "d": D}
    buf = normal(gen(7), tuple(sizes[a] for a in layout), torch.float16)
    v = buf.permute([layout.index(a) for a in "nthd"])
    return v[:, :, :HQ], v[:, :, HQ:]


@pytest.mark.parametrize("layout", ["nthd", "nhtd", "tnhd", "htnd", "hntd", "thnd"])
def test_queries_and_keys_of_one_buffer_in_place_in_any_order(layout):
    n = 3
    q, k = views(layout, n)
    oldq, oldk = q.clone(), k.clone()
    st = q.stride()[:3]
    assert k.stride()[:3] == st
    p = plan(n, q_stride=st, k_stride=st, q_out_stride=st, k_out_stride=st)
    c3d.rope3d_forward(p, q, k, q, k)
    torch.cuda.synchronize()
    check(oldq, q, n, "q")
    check(oldk, k, n, "k")
    # and back into another buffer of that order, the one's heads between the other's
    out_q, out_k = views(layout, n)
    c3d.rope3d_backward(p, q, k, out_q, out_k)
    torch.cuda.synchronize()
    check(q, out_q, n, "dq", True)
    check(k, out_k, n, "dk", True)


@pytest.mark.parametrize("n", [1, 3])
def test_inputs_that_repeat_their_elements(n):
    # one sample's queries and one key head for all, read through strides of 0
    q, k = normal(gen(1), (1, TOK, HQ, D), torch.float16), normal(gen(2), (n, TOK, 1, D), torch.float16)
    qb, kb = q.expand(n, -1, -1, -1), k.expand(-1, -1, HK, -1)
    qo = torch.empty((n, TOK, HQ, D), dtype=torch.float16, device="cuda:0")
    ko = torch.empty((n, TOK, HK, D), dtype=torch.float16, device="cuda:0")
    c3d.rope3d_forward(plan(n, q_stride=qb.stride()[:3], k_stride=kb.stride()[:3]), qb, kb, qo, ko)
    torch.cuda.synchronize()
    check(qb, qo, n, "q")
    check(kb, ko, n, "k")
    # a gradient that comes in broadcast, as that of a sum does
    p = plan(n, q_out_stride=qb.stride()[:3], k_out_stride=kb.stride()[:3])
    c3d.rope3d_backward(p, qb, kb, qo, ko)
    torch.cuda.synchronize()
    check(qb, qo, n, "dq", True)
    check(kb, ko, n, "dk", True)


def test_tensors_refused_before_the_call():
    n = 2
    q, k = normal(gen(1), (n, TOK, HQ, D), torch.float16), normal(gen(2), (n, TOK, HK, D), torch.float16)
    p = plan(n)
    buf = torch.empty((n * TOK * HQ * D,), dtype=torch.float16, device="cuda:0")
    qo, ko = buf.view(n, TOK, HQ, D), buf[D:D + n * TOK * HK * D].view(n, TOK, HK, D)
    for args in ((q, k, qo, ko), (q, k, qo, q.view(-1)[:n * TOK * HK * D].view(n, TOK, HK, D))):
        with pytest.raises(c3d.Conv3dError, match="overlaps the other"):
            c3d.rope3d_forward(p, *args)
