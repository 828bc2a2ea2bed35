"""The token path of a video transformer over the VAE decoder's latent grid.

One pre-norm transformer block runs on the voxels of a latent video (one token
per voxel), forward and backward, through the library's token operators, an
AdamW step updates its weights, and the decoder's first causal convolution takes the result:

    layernorm -> q, k, v projection -> rope3d -> attention -> out projection + x
    layernorm -> up projection + GELU -> down projection + x -> conv3d

Each frame attends to itself.  Run it on a GPU:

    python examples/latent_block.py [--frames 5] [--size 16] [--channels 256] [--heads 4]

It prints the size of the error against the same block in fp64 torch autograd.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import convolution_implicit_gemm_amd as c3d  # noqa: E402

EPS = 1e-6


def frame_attention(q, k, v):
    """softmax(q k^T / sqrt(d)) v within each frame; [frames, voxels, heads, d] fp32."""
    s = torch.einsum("fqhd,fkhd->fhqk", q, k) / q.shape[-1] ** 0.5
    return torch.einsum("fhqk,fkhd->fqhd", torch.softmax(s, -1), v)


class LatentBlock:
    """Weights, plans, workspaces and buffers of one block on a [t, h, w] latent grid (bf16)."""

    def __init__(self, t, h, w, channels, heads, seed=0):
        self.grid, self.c, self.heads = (t, h, w), channels, heads
        self.m, self.d = t * h * w, channels // heads
        dev, dt = torch.device("cuda"), torch.bfloat16
        g = torch.Generator(device=dev)
        g.manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device=dev) * k ** -0.5).to(dt)

        c = channels
        self.p = {"g1": torch.ones(c), "b1": torch.zeros(c), "g2": torch.ones(c), "b2": torch.zeros(c),
                  "qkv": weight(3 * c, c), "qkv_b": torch.zeros(3 * c), "out": weight(c, c), "out_b": torch.zeros(c),
                  "up": weight(4 * c, c), "up_b": torch.zeros(4 * c), "down": weight(c, 4 * c),
                  "down_b": torch.zeros(c)}
        self.p = {n: v.to(dev, dt) for n, v in self.p.items()}
        bias, res = c3d.CONV3D_F_BF16 | c3d.CONV3D_F_BIAS, c3d.CONV3D_F_RESIDUAL
        m = self.m
        self.plans = {
            "qkv": c3d.linear_plan(c3d.make_linear_desc(m, 3 * c, c, flags=bias)),
            "out": c3d.linear_plan(c3d.make_linear_desc(m, c, c, flags=bias | res)),
            "up": c3d.linear_plan(c3d.make_linear_desc(m, 4 * c, c, c3d.CONV3D_ACT_GELU_TANH,
                                                       bias | c3d.CONV3D_F_PREACT)),
            "down": c3d.linear_plan(c3d.make_linear_desc(m, c, 4 * c, flags=bias | res))}
        # queries and keys are rotated in place, inside the rows of the fused projection
        stride = (m * 3 * c, 3 * c, self.d)
        rest = self.d // 16 * 6  # 3/8 of a head for height and width each, the rest for time
        self.rope = c3d.rope3d_plan(c3d.make_rope3d_desc(
            1, t, h, w, heads, heads, self.d, (self.d - 2 * rest, rest, rest), flags=c3d.CONV3D_F_BF16,
            q_stride=stride, k_stride=stride, q_out_stride=stride, k_out_stride=stride))
        # the frames are told apart by a mask over all tokens, one frame wide
        self.attention = c3d.attention_plan(c3d.make_attention_desc(
            1, m, m, heads, heads, self.d, frame=h * w, window=1, flags=c3d.CONV3D_F_BF16, q_stride=stride,
            k_stride=stride, v_stride=stride))
        need = max([p.workspace_bytes for p in self.plans.values()] +
                   [c3d.linear_backward_workspace(p) for p in self.plans.values()] +
                   [self.attention.workspace_bytes, c3d.attention_backward_workspace(self.attention),
                    c3d.layernorm_backward_workspace(m, c)])
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)

    def rows(self, n, dtype=torch.bfloat16):
        return torch.empty((self.m, n), dtype=dtype, device="cuda")

    def _qkv(self, qkv):
        return qkv.view(1, self.m, 3 * self.heads, self.d).split(self.heads, 2)

    def forward(self, x):
        """y, and what the backward pass needs."""
        m, c, p, ws = self.m, self.c, self.p, self.ws
        s = {"x": x, "n1": self.rows(c), "st1": self.rows(2, torch.float32), "qkv": self.rows(3 * c),
             "o": self.rows(c), "lse": torch.empty((1, self.heads, m), device="cuda"), "x1": self.rows(c), "n2": self.rows(c),
             "st2": self.rows(2, torch.float32), "up": self.rows(4 * c), "z": self.rows(4 * c)}
        y = self.rows(c)
        c3d.layernorm_bf16(x, p["g1"], p["b1"], s["n1"], s["st1"], m, c, EPS)
        c3d.linear_forward(self.plans["qkv"], s["n1"], p["qkv"], p["qkv_b"], None, s["qkv"], None, ws)
        q, k, v = self._qkv(s["qkv"])
        c3d.rope3d_forward(self.rope, q, k, q, k)
        c3d.attention_forward(self.attention, q, k, v, s["o"], s["lse"], workspace=ws)
        c3d.linear_forward(self.plans["out"], s["o"], p["out"], p["out_b"], x, s["x1"], None, ws)
        c3d.layernorm_bf16(s["x1"], p["g2"], p["b2"], s["n2"], s["st2"], m, c, EPS)
        c3d.linear_forward(self.plans["up"], s["n2"], p["up"], p["up_b"], None, s["up"], s["z"], ws)
        c3d.linear_forward(self.plans["down"], s["up"], p["down"], p["down_b"], s["x1"], y, None, ws)
        return y, s

    def backward(self, dy, s):
        """dx and the weights' gradients."""
        m, c, p, ws = self.m, self.c, self.p, self.ws
        g = {n: torch.empty_like(v) for n, v in p.items()}
        d_up, d_n, d_x1 = self.rows(4 * c), self.rows(c), self.rows(c)
        c3d.linear_backward(self.plans["down"], dy, s["up"], p["down"], None, d_up, g["down"], g["down_b"], ws)
        c3d.linear_backward(self.plans["up"], d_up, s["n2"], p["up"], s["z"], d_n, g["up"], g["up_b"], ws)
        # the residual path's gradient joins in the norm's
        c3d.layernorm_backward_bf16(d_n, s["x1"], p["g2"], s["st2"], dy, d_x1, g["g2"], g["b2"], m, c, ws)
        d_o, d_x = self.rows(c), self.rows(c)
        c3d.linear_backward(self.plans["out"], d_x1, s["o"], p["out"], None, d_o, g["out"], g["out_b"], ws)
        d_qkv = self.rows(3 * c)
        dq, dk, dv = self._qkv(d_qkv)
        c3d.attention_backward(self.attention, d_o, *self._qkv(s["qkv"]), s["o"], s["lse"], dq, dk, dv, workspace=ws)
        c3d.rope3d_backward(self.rope, dq, dk, dq, dk)
        c3d.linear_backward(self.plans["qkv"], d_qkv, s["n1"], p["qkv"], None, d_n, g["qkv"], g["qkv_b"], ws)
        c3d.layernorm_backward_bf16(d_n, s["x"], p["g1"], s["st1"], d_x1, d_x, g["g1"], g["b1"], m, c, ws)
        return d_x, g

    def optimizer(self, grads):
        """What steps over the block's weights need: fp32 copies of them and 8-bit states."""
        names = list(self.p)
        blocks = [-(-self.p[n].numel() // c3d.ADAMW_BLOCK) for n in names]

        def zeros(sizes):
            return [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes]

        sizes = [self.p[n].numel() for n in names]
        master = [self.p[n].float() for n in names]
        return master, c3d.adamw_list([self.p[n] for n in names], [grads[n] for n in names], zeros(sizes), zeros(sizes),
                                      master=master, m_scale=zeros(blocks), v_scale=zeros(blocks),
                                      decay=[float(self.p[n].dim() > 1) for n in names])


def decode_first_conv(tokens, grid, seed=1):
    """The VAE decoder's causal 3x3x3 convolution on the block's output (tokens are its NDHWC rows)."""
    (t, h, w), c = grid, tokens.shape[1]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    wt = (torch.randn(c, 3, 3, 3, c, generator=g, device="cuda") * (27 * c) ** -0.5).to(tokens.dtype)
    plan = c3d.conv3d_plan(c3d.make_desc(1, t, h, w, c, c, pad_t_front=2, pad_t_back=0,
                                         t_pad_mode=c3d.CONV3D_TPAD_REPLICATE, flags=c3d.CONV3D_F_BF16))
    y = torch.empty((1, t, h, w, c), dtype=tokens.dtype, device="cuda")
    ws = torch.empty(max(plan.workspace_bytes, 16), dtype=torch.uint8, device="cuda")
    c3d.conv3d_forward(plan, tokens.view(1, t, h, w, c), wt, None, None, y, ws)
    return y


def reference(block, x, dy):
    """The block in fp64 torch: y, dx and the weights' gradients."""
    (t, h, w), c, m, heads, d = block.grid, block.c, block.m, block.heads, block.d
    p = {n: v.double().requires_grad_(True) for n, v in block.p.items()}
    x = x.double().requires_grad_(True)

    def norm(v, g, b):
        return torch.nn.functional.layer_norm(v, (c,), p[g], p[b], EPS)

    rest = d // 16 * 6
    dims = (d - 2 * rest, rest, rest)
    i = torch.arange(m, device=x.device)
    pos = torch.stack([i // (h * w), i // w % h, i % w], 1).double()
    ang = torch.cat([pos[:, a:a + 1] * 10000.0 ** (-torch.arange(0, n, 2, device=x.device).double() / n)
                     for a, n in enumerate(dims) if n], 1)[:, None]
    cos, sin = torch.cos(ang), torch.sin(ang)

    def rotate(v):
        a, b = v[..., 0::2], v[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)

    qkv = (norm(x, "g1", "b1") @ p["qkv"].t() + p["qkv_b"]).view(m, 3, heads, d)
    f = [v.reshape(t, h * w, heads, d) for v in (rotate(qkv[:, 0]), rotate(qkv[:, 1]), qkv[:, 2])]
    x1 = frame_attention(*f).reshape(m, c) @ p["out"].t() + p["out_b"] + x
    up = torch.nn.functional.gelu(norm(x1, "g2", "b2") @ p["up"].t() + p["up_b"], approximate="tanh")
    y = up @ p["down"].t() + p["down_b"] + x1
    grads = torch.autograd.grad(y, [x] + list(p.values()), dy.double())
    return y.detach(), grads[0], dict(zip(p, grads[1:]))


def run(frames=5, size=16, channels=256, heads=4):
    """{name: relative L2 error against fp64} of the output, dx and every weight's gradient."""
    block = LatentBlock(frames, size, size, channels, heads)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(block.m, channels, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(block.m, channels, generator=g, device="cuda").to(torch.bfloat16)
    y, saved = block.forward(x)
    dx, grads = block.backward(dy, saved)
    frames_out = decode_first_conv(y, block.grid)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(frames_out.float()).all())
    ry, rdx, rg = reference(block, x, dy)

    def err(a, b):
        return float((a.double() - b).norm() / b.norm())

    errors = dict({"y": err(y, ry), "dx": err(dx, rdx)}, **{n: err(grads[n], rg[n]) for n in grads})
    # the first step on these gradients, against the formula: with new states m / (1 - beta1) = g, v / (1 - beta2) = g^2
    before = {n: v.double() for n, v in block.p.items()}
    master, tensors = block.optimizer(grads)
    hyper = c3d.make_adamw_hyper(1e-3, weight_decay=0.1)
    c3d.adamw_step(tensors, hyper)
    torch.cuda.synchronize()
    for w, (n, old) in zip(master, before.items()):
        gr = grads[n].double()
        want = old - hyper.lr * (hyper.weight_decay * (old.dim() > 1) * old + gr / (gr.abs() + hyper.eps))
        errors["step " + n] = err(w, want)
    return errors


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("frames", 5), ("size", 16), ("channels", 256), ("heads", 4)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    for name, e in run(a.frames, a.size, a.channels, a.heads).items():
        print("%-8s relative error %.2e" % (name, e))
