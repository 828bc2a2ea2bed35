"""rope3d's checks of what its outputs share with each other and with its inputs.

Every check runs before the device is touched, so fake addresses that are never
dereferenced are enough; only refused calls are made.
"""
import itertools
import random

import pytest
import torch

import convolution_implicit_gemm_amd as c3d

BAD, UNSUP = c3d.CONV3D_ERR_INVALID_ARG, c3d.CONV3D_ERR_UNSUPPORTED
A, B, C, D, P = ((i + 1) << 40 for i in range(5))  # far apart, aligned
H, K, DIM, TOK = 4, 2, 64, 24                      # query and key heads, head size, tokens of a 2 x 3 x 4 grid
CALLS = [c3d.rope3d_forward, c3d.rope3d_backward]


def plan(n=1, flags=0, **strides):
    return c3d.rope3d_plan(c3d.make_rope3d_desc(n, 2, 3, 4, H, K, DIM, (16, 24, 24), flags=flags, **strides))


def refused(call, p, *args):
    with pytest.raises(c3d.Conv3dError) as e:
        call(p, *args, stream=0)
    return e.value.status == BAD and "overlap" in c3d.conv3d_last_error()


SPAN = TOK * H * DIM * 2  # bytes of contiguous q


@pytest.mark.parametrize("args", [
    (A, B, C, C), (A, B, C, C + SPAN - 128), (A, B, B, D), (A, B, B + 128, D), (A, B, C, A), (A, B, C, A + SPAN - 16),
    (A, B, C, C + 16)])
@pytest.mark.parametrize("call", CALLS)
def test_an_output_may_not_be_the_other_output_or_input(args, call):
    assert refused(call, plan(), *args)


@pytest.mark.parametrize("call", CALLS)
def test_heads_of_a_fused_row_may_lie_side_by_side_but_not_on_each_other(call):
    # q and k in place inside rows of 12 heads; k begins one head, half a head or 16 bytes too early
    st = (TOK * 12 * DIM, 12 * DIM, DIM)
    p = plan(2, q_stride=st, k_stride=st, q_out_stride=st, k_out_stride=st)
    for early in (DIM, DIM // 2, 8):
        k = A + (H * DIM - early) * 2
        assert refused(call, p, A, k, A, k)
    # behind the rows' last heads, on the next token's first
    k = A + (11 * DIM) * 2
    assert refused(call, p, A, k, A, k)
    # one token on, at the right place in the row but for 8 elements
    k = A + (12 * DIM * 3 + H * DIM - 8) * 2
    assert refused(call, p, A, k, A, k)


@pytest.mark.parametrize("stride", [(0, 256, 64), (6144, 0, 64), (6144, 256, 0), (6144, 256, 56), (6144, 248, 64),
                                    (6136, 256, 64), (256, 256, 64), (64, 256, 64)])
def test_outputs_on_their_own_elements_are_refused(stride):
    # forward writes with the outputs' strides, the gradient with the inputs'
    p = plan(2, q_out_stride=stride)
    assert refused(c3d.rope3d_forward, p, A, B, C, D)
    p = plan(2, q_stride=stride)
    assert refused(c3d.rope3d_backward, p, A, B, C, D)
    if stride[2] < 64 or stride[1] < 128 or stride[0] < 24 * 128:  # for the two key heads too
        assert refused(c3d.rope3d_backward, plan(2, k_stride=stride), A, B, C, D)


@pytest.mark.parametrize("call", CALLS)
def test_positions_may_not_be_written(call):
    p = plan(flags=c3d.CONV3D_F_POSITIONS)
    for pos in (C, C + SPAN - 4, D + 64, C - 12 * TOK + 4):
        assert refused(call, p, A, B, C, D, pos, 0)


def shared(a, sa, ea, b, sb, eb, dim):
    """Whether two layouts share an element, by their elements."""
    def elements(base, st, ext):
        return {base + sum(i * s for i, s in zip(ix, st)) + e for ix in itertools.product(*map(range, ext))
                for e in range(0, dim, 8)}
    return not elements(a, sa, ea).isdisjoint(elements(b, sb, eb))


def folded(st, ext, dim):
    """Whether a layout puts two heads on one element."""
    starts = [sum(i * s for i, s in zip(ix, st)) for ix in itertools.product(*map(range, ext))]
    starts.sort()
    return any(b - a < dim for a, b in zip(starts, starts[1:]))


def test_overlaps_found_are_the_ones_there_are():
    # random small layouts of q's and k's outputs in one buffer, one contiguous input each; a
    # call that passes the checks goes no further than to find that there is no device here
    rng = random.Random(3)
    found = passed = 0
    for _ in range(400):
        n, hq, hk, dim = rng.choice([1, 2]), rng.choice([1, 2, 3]), rng.choice([1, 2]), rng.choice([8, 16])
        row = (hq + hk + rng.choice([0, 1])) * dim
        st = (3 * row + rng.choice([0, 8]), row, dim) if rng.random() < 0.7 else (hq * 3 * dim, dim, 3 * dim)
        off = rng.randrange(0, 2 * row, 8)
        ext = (n, 3, hq), (n, 3, hk)
        p = c3d.rope3d_plan(c3d.make_rope3d_desc(n, 1, 1, 3, hq, hk, dim, (4, 2, 2), q_out_stride=st, k_out_stride=st))
        if shared(0, st, ext[0], off, st, ext[1], dim) or folded(st, ext[0], dim) or folded(st, ext[1], dim):
            found += 1
            assert refused(c3d.rope3d_forward, p, A, B, C, C + 2 * off)
        elif not torch.cuda.is_available():  # (with one, the addresses would be read)
            passed += 1
            with pytest.raises(c3d.Conv3dError) as e:
                c3d.rope3d_forward(p, A, B, C, C + 2 * off, stream=0)
            assert e.value.status == c3d.CONV3D_ERR_NO_DEVICE
    assert found > 100 and (passed > 100 or torch.cuda.is_available())


@pytest.mark.parametrize("bad", [
    dict(n=1 << 30, t=1, h=1, w=1, q_stride=(1 << 39, 256, 64)),
    dict(n=1 << 12, t=1 << 10, h=1 << 4, w=1, k_out_stride=(1 << 37, 128, 64)),
    dict(n=1, t=1 << 30, h=1, w=1, k_stride=(0, 1 << 30, 64)), dict(n=0, t=1 << 30, h=1 << 10, w=1 << 20),
    dict(n=0, t=2, h=1 << 15, w=1 << 15)])
def test_tensors_too_long_for_their_offsets_are_refused(bad):
    with pytest.raises(c3d.Conv3dError) as e:
        c3d.rope3d_plan(c3d.make_rope3d_desc(heads_q=H, heads_k=K, head_dim=DIM, dims=(16, 24, 24), **bad))
    assert e.value.status == UNSUP


def test_the_longest_tensors_are_planned():
    for good in (dict(n=1 << 8, t=1, h=1, w=1, q_stride=((1 << 40) - 64, 256, 64)), dict(n=0, t=1 << 10, h=1 << 10, w=1 << 10),
                 dict(n=1, t=1 << 10, h=1 << 10, w=(1 << 11) - 1)):
        c3d.rope3d_plan(c3d.make_rope3d_desc(heads_q=H, heads_k=K, head_dim=DIM, dims=(16, 24, 24), **good))


def test_empty_tensors_overlap_nothing():
    # views of no rows, wherever they point, and a workspace that is not used
    p = c3d.linear_plan(c3d.make_linear_desc(0, 64, 32, flags=c3d.CONV3D_F_BIAS))
    c3d.linear_forward(p, B + 64, B, C, None, B + 128, None, C + 16, stream=0)
    c3d.layernorm(A + 16, A, C, A + 32, None, 0, 64, 1e-6, stream=0)
    c3d.layernorm(A + 16, A, C, C + 64, A + 64, 0, 64, 1e-6, stream=0)
