"""rope3d and its gradient against the 64-bit form (bounds: token_helpers.py)."""
import math

import pytest
import torch

import convolution_implicit_gemm_amd as c3d
from token_helpers import DTYPES, assert_within, gen, normal

pytestmark = pytest.mark.gpu

PAIRINGS = {"adjacent": c3d.ROPE3D_PAIR_ADJACENT, "halves": c3d.ROPE3D_PAIR_HALVES}


def grid_positions(n, t, h, w, t_offset=0):
    i = torch.arange(t * h * w, device="cuda:0")
    p = torch.stack([i // (h * w) + t_offset, i // w % h, i % w], 1)
    return p[None].expand(n, -1, -1)


def rope64(x, pos, dims, base, pairing, inverse=False):
    """(rotated x, slack); x [n, tokens, heads, d], pos [n, tokens, 3]."""
    x = x.double()
    pos = pos.double()
    ang, far = [], []
    for a, dim in enumerate(dims):
        for i in range(dim // 2):
            step = base ** (-2.0 * i / dim)
            ang.append(pos[:, :, a] * step)
            # the angle before reduction is exact to 2^-52 of it, on both sides
            far.append(pos[:, :, a].abs() * step * 2.0 ** -50)
    ang, far = torch.stack(ang, 2)[:, :, None], torch.stack(far, 2)[:, :, None]
    cos, sin = torch.cos(ang), torch.sin(ang) * (-1.0 if inverse else 1.0)
    r = sum(dims)
    y, slack = x.clone(), torch.zeros_like(x)
    iu, iv = (slice(0, r, 2), slice(1, r, 2)) if pairing == "adjacent" else (slice(0, r // 2), slice(r // 2, r))
    u, v = x[..., iu], x[..., iv]
    y[..., iu], y[..., iv] = u * cos - v * sin, u * sin + v * cos
    # turns to fp32 (2 pi 2^-25), sincospi and two products: below 2^-20 of |u| + |v|
    s = (u.abs() + v.abs()) * (2.0 ** -20 + far)
    slack[..., iu], slack[..., iv] = s, s
    return y, slack


CASES = [  # n, (t, h, w), heads_q, heads_k, head_dim, dims
    (1, (1, 1, 1), 1, 0, 8, (2, 2, 2)),
    (1, (1, 1, 1), 16, 4, 128, (44, 42, 42)),
    (2, (3, 5, 7), 4, 2, 64, (16, 24, 24)),
    (1, (2, 9, 11), 3, 1, 80, (16, 32, 32)),
    (3, (1, 4, 33), 5, 5, 96, (0, 48, 48)),
    (1, (5, 3, 3), 2, 1, 40, (16, 8, 8)),
    (1, (4, 16, 16), 9, 3, 128, (32, 48, 48)),
    (1, (2, 3, 4), 2, 2, 512, (64, 96, 96)),
    (1, (7, 1, 1), 17, 17, 48, (32, 0, 0)),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("pairing", sorted(PAIRINGS))
@pytest.mark.parametrize("case", CASES, ids=str)
def test_grid(case, pairing, dtype, inverse):
    n, (t, h, w), hq, hk, d, dims = case
    if pairing == "halves" and sum(dims) % 16:
        pytest.skip("dims of the two halves are multiples of 16 together")
    dt, tok = DTYPES[dtype], t * h * w
    q, k = normal(gen(1), (n, tok, hq, d), dt), normal(gen(2), (n, tok, max(hk, 1), d), dt)
    plan = c3d.rope3d_plan(c3d.make_rope3d_desc(n, t, h, w, hq, hk, d, dims, 10000.0, PAIRINGS[pairing],
                                                c3d.CONV3D_F_BF16 if dtype == "bf16" else 0))
    qo, ko = torch.full_like(q, 12.5), torch.full_like(k, 12.5)
    call = c3d.rope3d_backward if inverse else c3d.rope3d_forward
    call(plan, q, k if hk else None, qo, ko if hk else None, None, 5)
    torch.cuda.synchronize()
    pos = grid_positions(n, t, h, w, 5)
    ref, slack = rope64(q, pos, dims, 10000.0, pairing, inverse)
    assert_within(qo, ref, slack, "q")
    if hk:
        ref, slack = rope64(k, pos, dims, 10000.0, pairing, inverse)
        assert_within(ko, ref, slack, "k")
    else:
        assert bool((ko == 12.5).all())
    rot = sum(dims)
    assert torch.equal(qo[..., rot:], q[..., rot:])  # the other elements are copied


@pytest.mark.parametrize("pairing", sorted(PAIRINGS))
def test_given_positions_of_any_size(pairing):
    n, tok, hq, hk, d, dims = 2, 37, 3, 1, 64, (16, 24, 24)
    g = gen(3)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, tok, 3), generator=g, device="cuda:0").int()
    pos[0, :8] = torch.arange(-4, 4, device="cuda:0", dtype=torch.int32)[:, None]
    pos[1, 0] = torch.tensor([2 ** 31 - 1, -2 ** 31, 0], device="cuda:0").int()
    q, k = normal(g, (n, tok, hq, d), torch.float16), normal(g, (n, tok, hk, d), torch.float16)
    plan = c3d.rope3d_plan(c3d.make_rope3d_desc(n, 1, 1, tok, hq, hk, d, dims, 500.0, PAIRINGS[pairing],
                                                c3d.CONV3D_F_POSITIONS))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    c3d.rope3d_forward(plan, q, k, qo, ko, pos, 77)
    for x, y in ((q, qo), (k, ko)):
        ref, slack = rope64(x, pos, dims, 500.0, pairing)
        assert_within(y, ref, slack, "given positions")


@pytest.mark.parametrize("pairing", sorted(PAIRINGS))
def test_in_place_inside_a_fused_projection(pairing):
    n, t, h, w, hq, hk, d, dims = 2, 2, 5, 7, 4, 2, 64, (16, 16, 16)
    qkv = normal(gen(4), (n, t * h * w, hq + 2 * hk, d), torch.bfloat16)
    old = qkv.clone()
    q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    st = q.stride()[:3]
    plan = c3d.rope3d_plan(c3d.make_rope3d_desc(n, t, h, w, hq, hk, d, dims, 10000.0, PAIRINGS[pairing],
                                                c3d.CONV3D_F_BF16, st, st, st, st))
    c3d.rope3d_forward(plan, q, k, q, k)
    torch.cuda.synchronize()
    pos = grid_positions(n, t, h, w)
    ref, slack = rope64(old[:, :, :hq + hk], pos, dims, 10000.0, pairing)
    assert_within(qkv[:, :, :hq + hk], ref, slack, "rotated heads")
    assert torch.equal(qkv[:, :, hq + hk:], old[:, :, hq + hk:])  # the values are not touched


def test_heads_first_outputs():
    n, t, h, w, hq, hk, d, dims = 2, 2, 3, 5, 4, 2, 64, (16, 24, 24)
    tok = t * h * w
    q, k = normal(gen(5), (n, tok, hq, d), torch.float16), normal(gen(6), (n, tok, hk, d), torch.float16)
    qo = torch.empty((n, hq, tok, d), dtype=torch.float16, device="cuda:0")
    ko = torch.empty((n, hk, tok, d), dtype=torch.float16, device="cuda:0")
    plan = c3d.rope3d_plan(c3d.make_rope3d_desc(n, t, h, w, hq, hk, d, dims,
                                                q_out_stride=(hq * tok * d, d, tok * d),
                                                k_out_stride=(hk * tok * d, d, tok * d)))
    c3d.rope3d_forward(plan, q, k, qo.transpose(1, 2), ko.transpose(1, 2))
    torch.cuda.synchronize()
    for x, y in ((q, qo), (k, ko)):
        ref, slack = rope64(x, grid_positions(n, t, h, w), dims, 10000.0, "adjacent")
        assert_within(y.transpose(1, 2), ref, slack, "heads first")
    back_q, back_k = torch.empty_like(q), torch.empty_like(k)
    c3d.rope3d_backward(plan, qo.transpose(1, 2), ko.transpose(1, 2), back_q, back_k)
    torch.cuda.synchronize()
    # the turn back; each way rounds once (2^-11 of the pair's size each)
    for x, y in ((q, back_q), (k, back_k)):
        assert float((x.double() - y.double()).abs().max()) <= 2.0 ** -9 * float(x.abs().max()) * math.sqrt(2.0)


def test_backward_matches_differences():
    n, t, h, w, hq, d, dims = 1, 2, 3, 4, 2, 32, (8, 12, 12)
    g = gen(9)
    dy = normal(g, (n, t * h * w, hq, d), torch.float16)
    plan = c3d.rope3d_plan(c3d.make_rope3d_desc(n, t, h, w, hq, 0, d, dims))
    dx = torch.empty_like(dy)
    c3d.rope3d_backward(plan, dy, None, dx, None)
    pos = grid_positions(n, t, h, w)
    ref, slack = rope64(dy, pos, dims, 10000.0, "adjacent", True)
    x = torch.randn(dy.shape, generator=g, device="cuda:0", dtype=torch.float64)
    v = torch.randn(dy.shape, generator=g, device="cuda:0", dtype=torch.float64)
    f = [(dy.double() * rope64(x + s * 1e-4 * v, pos, dims, 10000.0, "adjacent")[0]).sum() for s in (1, -1)]
    diff = float((f[0] - f[1]) / 2e-4)
    bound = float(((slack + 2.0 ** -11 * ref.abs() + 2.0 ** -25) * v.abs()).sum()) + 1e-6 * abs(diff) + 1e-5
    assert abs(float((dx.double() * v).sum()) - diff) <= bound


def test_non_finite_values_stay_in_their_pairs():
    dims, d = (8, 12, 12), 40
    q = normal(gen(10), (1, 6, 1, d), torch.float16)
    q[0, 2, 0, 4] = float("inf")
    q[0, 3, 0, 35] = float("nan")  # not rotated
    plan = c3d.rope3d_plan(c3d.make_rope3d_desc(1, 1, 2, 3, 1, 0, d, dims))
    qo = torch.empty_like(q)
    c3d.rope3d_forward(plan, q, None, qo, None)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(qo)
    assert bad.nonzero()[:, 1:].tolist() in ([[2, 0, 4], [2, 0, 5], [3, 0, 35]], [[2, 0, 4], [3, 0, 35]])


def test_zero_tokens_and_long_offsets():
    e = torch.empty((0, 6, 1, 64), dtype=torch.float16, device="cuda:0")
    plan = c3d.rope3d_plan(c3d.make_rope3d_desc(0, 1, 2, 3, 1, 0, 64, (16, 24, 24)))
    c3d.rope3d_forward(plan, e, None, e, None)
    # tokens 2^20 elements apart: 2100 of them pass 4 GiB
    tok, d, dims = 2100, 64, (16, 24, 24)
    buf = torch.empty((tok, 1 << 20), dtype=torch.float16, device="cuda:0")
    q = buf.as_strided((1, tok, 1, d), (tok << 20, 1 << 20, d, 1))
    q.copy_(normal(gen(12), (1, tok, 1, d), torch.float16))
    old = q.clone()
    st = (tok << 20, 1 << 20, d)
    plan = c3d.rope3d_plan(c3d.make_rope3d_desc(1, 3, 70, 10, 1, 0, d, dims, q_stride=st, q_out_stride=st))
    c3d.rope3d_forward(plan, q, None, q, None)
    ref, slack = rope64(old, grid_positions(1, 3, 70, 10), dims, 10000.0, "adjacent")
    assert_within(q, ref, slack, "long offsets")


def test_other_stream_and_graph_replay():
    n, t, h, w, hq, hk, d, dims = 1, 3, 8, 8, 4, 2, 64, (16, 24, 24)
    q, k = normal(gen(1), (n, t * h * w, hq, d), torch.float16), normal(gen(2), (n, t * h * w, hk, d), torch.float16)
    pos = torch.randint(0, 999, (n, t * h * w, 3), device="cuda:0").int()
    plan = c3d.rope3d_plan(c3d.make_rope3d_desc(n, t, h, w, hq, hk, d, dims, flags=c3d.CONV3D_F_POSITIONS))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c3d.rope3d_forward(plan, q, k, qo, ko, pos)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c3d.rope3d_forward(plan, q, k, qo, ko, pos)
    for i in range(4):
        q.copy_(normal(gen(50 + i), tuple(q.shape), torch.float16))
        pos.copy_(torch.randint(0, 999, tuple(pos.shape), device="cuda:0").int())
        c3d.rope3d_forward(plan, q, k, qo, ko, pos)
        torch.cuda.synchronize()
        want = (qo.clone(), ko.clone())
        qo.zero_()
        ko.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
