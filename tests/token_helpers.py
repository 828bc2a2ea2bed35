"""Plain 64-bit forms of the token operators, and the bounds the kernels are held to.

Every output is rounded once from fp32, so each bound is half an ulp of the
output's type plus what fp32 arithmetic may lose before that:
  sums of d terms one after the other err by at most d * 2^-24 of the sum of
  the absolute values; the kernels' other fp32 steps (activation, normalisation,
  rotation) by a few 2^-24 of the values they combine, bounded per operator.
"""
import math

import torch

import convolution_implicit_gemm_amd as c3d

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
ACTS = {"none": c3d.CONV3D_ACT_NONE, "silu": c3d.CONV3D_ACT_SILU, "gelu": c3d.CONV3D_ACT_GELU,
        "gelu_tanh": c3d.CONV3D_ACT_GELU_TANH}
U24 = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return g


def normal(g, shape, dtype, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g, device="cuda:0") * scale + shift).to(dtype)


def gapped(g, rows, cols, gap, dtype, scale=1.0):
    """[rows, cols] values in rows of cols + gap elements; the gaps hold NaN."""
    buf = torch.full((rows, cols + gap), float("nan"), dtype=dtype, device="cuda:0")
    buf[:, :cols] = normal(g, (rows, cols), dtype, scale)
    return buf[:, :cols]


def marked(rows, cols, gap, dtype):
    """(buffer, view) of an output whose gaps and surroundings hold a marker."""
    n = 64 + rows * (cols + gap) + 64
    buf = torch.full((n,), 12.5, dtype=dtype, device="cuda:0")
    return buf, buf[64:64 + rows * (cols + gap)].view(rows, cols + gap)[:, :cols]


def assert_unmarked_only(buf, rows, cols, gap):
    assert bool((buf[:64] == 12.5).all()) and bool((buf[-64:] == 12.5).all()), "write outside the tensor"
    if gap:
        inner = buf[64:-64].view(rows, cols + gap)[:, cols:]
        assert bool((inner == 12.5).all()), "write between the rows"


def half_ulp(v, dtype):
    """0.51 ulp of the element type at |v| (v: float64)."""
    low, bits = (-14, 10) if dtype == torch.float16 else (-126, 7)
    a = v.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.full_like(a, 2.0 ** low))))
    return 0.51 * torch.exp2(e.clamp(min=low) - bits)


def assert_within(got, ref, slack, what):
    """|got - ref| <= slack + half an ulp of the output's type."""
    got64 = got.double()
    tol = slack + (half_ulp(torch.maximum(ref.abs(), got64.abs()), got.dtype) if got.dtype != torch.float32 else 0.0)
    bad = ~((got64 - ref).abs() <= tol)
    if bool(bad.any()):
        i = int(torch.nonzero(bad.flatten())[0])
        raise AssertionError("%s: %d of %d outside the bound, first at %d: got %r, want %r, bound %r"
                             % (what, int(bad.sum()), bad.numel(), i, float(got64.flatten()[i]),
                                float(ref.flatten()[i]), float((tol + torch.zeros_like(ref)).flatten()[i])))


def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def slope64(z, act):
    if act == "none":
        return torch.ones_like(z)
    z = z.detach().requires_grad_(True)
    g, = torch.autograd.grad(act64(z, act).sum(), z)
    return g


def linear64(x, w, bias, residual, act):
    """(y, z, the sum of |x w| + |bias|)."""
    xd, wd = x.double(), w.double().t().contiguous()
    z, mag = xd @ wd, xd.abs() @ wd.abs()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    y = act64(z, act)
    return (y if residual is None else y + residual.double()), z, mag


def linear_slack(k, mag, z, y, act):
    # the product's sum, then the activation (slope below 1.2; its own fp32 steps
    # and the erf formula's 1.5e-7 stay below 4e-6 (1 + |z|)) and the residual's addition
    zs = k * U24 * mag
    return zs, 1.2 * zs + (0.0 if act == "none" else 4e-6 * (1.0 + z.abs())) + 2 * U24 * y.abs()


def scratch(nbytes):
    """Workspace whose old contents are NaN patterns."""
    return torch.full((max(int(nbytes), 16),), 0xFF, dtype=torch.uint8, device="cuda:0")
