"""Attention whose output is made by many weak keys beside a strong one with a value of zero.

The strong key's exponential sets the scale that the others are rounded at.  A weak key's probability p is rounded
half a step of its type (u p), and no finer than fp16's least steps reach: 2^-25 of 2^11, the lift that the kernel
gives the row's largest, so 2^-36 of that one's probability for each key.  The sums run in fp32, one 2^-24 for each
of their keys, and so do the scores (exact here: the queries are a unit vector).
"""
import math

import pytest
import torch

import convolution_implicit_gemm_amd as c3d
from token_helpers import DTYPES, U24, assert_within, gen, scratch

pytestmark = pytest.mark.gpu

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
LEAST = {torch.float16: 2.0 ** -36, torch.bfloat16: 2.0 ** -134}


def check(tq, tk, d, dtype, strong, at, spread=0.0):
    """Scores of 0 (or `spread` wide below it), one of `strong` at key `at`, whose value is 0."""
    dt, dev = DTYPES[dtype], "cuda:0"
    g = gen(3)
    q = torch.zeros((1, tq, 2, d), dtype=dt, device=dev)
    q[..., 0] = 1.0
    k = torch.zeros((1, tk, 1, d), dtype=dt, device=dev)
    if spread:
        k[0, :, 0, 0] = -(torch.rand(tk, generator=g, device=dev) * spread).to(dt)
    k[0, at, 0, 0] = strong
    v = (torch.rand((1, tk, 1, d), generator=g, device=dev) + 0.5).to(dt)
    v[0, at] = 0.0
    plan = c3d.attention_plan(c3d.make_attention_desc(1, tq, tk, 2, 1, d, scale=1.0,
                                                      flags=c3d.CONV3D_F_BF16 if dtype == "bf16" else 0))
    o, lse = torch.empty_like(q), torch.empty((1, 2, tq), device=dev)
    c3d.attention_forward(plan, q, k, v, o, lse, workspace=scratch(plan.workspace_bytes))
    s, vv = k[0, :, 0, 0].double(), v[0, :, 0].double()
    z = torch.logsumexp(s, 0)
    p = torch.exp(s - z)
    ref = p @ vv
    # the exponent's argument, product with log2(e) and sum, and the exponential
    arg = U24 * (4 * float(s.abs().max()) + 8)
    slack = ((UNIT[dt] + (tk + 8) * U24 + 2 * arg) * p + LEAST[dt] * p.max()) @ vv
    assert bool((ref > 2.0 ** -14).all())  # normal numbers in fp16: the result itself keeps its digits
    for h in range(2):
        assert_within(o[0, :, h], ref.expand(tq, d), slack.expand(tq, d), "o[:, %d]" % h)
        assert bool(((lse[0, h].double() - z).abs() <= arg + (tk + 16) * U24 + 4 * U24 * abs(float(z))).all())
    return plan


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("strong", [12.0, 17.5, 19.5])
@pytest.mark.parametrize("at", [0, 20000, 36863])
def test_one_token(strong, at, dtype):
    assert check(1, 36864, 64, dtype, strong, at).info().kernel_name == b"attention_few"


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("tile", ["attention_64x128", "attention_128x128", "attention_256x64"])
@pytest.mark.parametrize("strong,at,d", [(17.5, 0, 64), (17.5, 36863, 128), (19.5, 77, 96), (19.5, 20000, 32)])
def test_every_tile_and_pieces(strong, at, d, tile, splits, monkeypatch):
    monkeypatch.setenv("CONV3D_ATTENTION_TILE", tile)
    monkeypatch.setenv("CONV3D_ATTENTION_SPLITS", str(splits))
    check(40, 36864, d, "fp16", strong, at)


@pytest.mark.parametrize("tq", [1, 300])
def test_weak_keys_of_many_sizes(tq):
    check(tq, 36864, 64, "fp16", 16.0, 5, spread=2.0)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tq", [1, 40, 300])
@pytest.mark.parametrize("scale", [1.0, 13.0, 16.0])
@pytest.mark.parametrize("most", [241.0, 247.0, 251.0, 253.0])
def test_large_scores_do_not_overflow(most, scale, tq, dtype):
    # scores of up to 2^22 scale (2^26, where fp32 counts in steps of 8), far apart: the largest alone counts, and
    # its exponential, off by the rounding of such scores, still fits
    d, tk, dev, top = 64, 500, "cuda:0", 251.0 * most * 64 * scale
    g = gen(4)
    q = torch.full((1, tq, 2, d), 251.0, dtype=DTYPES[dtype], device=dev)
    k = (torch.randint(0, 4, (1, tk, 1, 1), generator=g, device=dev) * 64.0).to(DTYPES[dtype]).expand(1, tk, 1, d).contiguous()
    k[0, 123], k[0, 321] = most, 192.0
    v = torch.randn((1, tk, 1, d), generator=g, device=dev).to(DTYPES[dtype])
    plan = c3d.attention_plan(c3d.make_attention_desc(1, tq, tk, 2, 1, d, scale=scale,
                                                      flags=c3d.CONV3D_F_BF16 if dtype == "bf16" else 0))
    o, lse = torch.empty_like(q), torch.empty((1, 2, tq), device=dev)
    c3d.attention_forward(plan, q, k, v, o, lse, workspace=scratch(plan.workspace_bytes))
    want = v[0, 123, 0].double()
    # the largest's exponential rounds once as an operand, the result once
    assert_within(o[0], want.expand(tq, 2, d), (UNIT[o.dtype] + 16 * U24) * want.abs().expand(tq, 2, d), "o")
    assert bool(((lse.double() / top - 1.0).abs() <= 8 * U24).all()) and math.isfinite(float(lse.sum()))
