"""The operators of a video transformer's token path, as measured cases.

The tokens are the voxels of the latent grid that the VAE decoder of this
library takes (9 frames of 64 x 64 in the decoder's own benchmark), one row
each.  Three operators run on them in turn: a layer norm, a matrix product with
bias, activation and residual in its epilogue, and rotary positions over (time,
height, width); each also has its gradient.

``own`` selects what ``run`` computes: the plain form in elementary torch
operations (32 bits, rounded once at the end), or the library's kernels.
"""
import math

import torch

own = False

_DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
_ACTS = ("none", "silu", "gelu", "gelu_tanh")


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one row through the embedding of the time step: latency and the weights' bytes
        dict(name="linear_one_row", op="linear", m=1, n=4096, k=1024, act="silu", dtype="bf16", bias=True,
             residual=False, keep=False, gap=0),
        # a prompt's projection: an ordinary, odd number of rows
        dict(name="linear_prompt", op="linear", m=613, n=2048, k=2048, act="gelu", dtype="fp16", bias=True,
             residual=False, keep=True, gap=0),
        # the MLP's second product with the residual stream, an odd token count, rows inside wider ones
        dict(name="linear_down", op="linear", m=9217, n=2048, k=8192, act="none", dtype="fp16", bias=True,
             residual=True, keep=False, gap=64),
        # the MLP's first product over all tokens of 9 frames of 64 x 64
        dict(name="linear_up", op="linear", m=36864, n=8192, k=2048, act="gelu_tanh", dtype="bf16", bias=True,
             residual=False, keep=False, gap=0),
        # training: one frame and a token more through a narrow projection
        dict(name="linear_grad_frame", op="linear_grad", m=4097, n=2048, k=512, act="gelu_tanh", dtype="fp16",
             bias=True, gap=0),
        # training: the MLP's first product over all tokens
        dict(name="linear_grad_up", op="linear_grad", m=36864, n=8192, k=2048, act="gelu_tanh", dtype="bf16",
             bias=True, gap=0),
        # a single token's norm: latency
        dict(name="layernorm_one_row", op="layernorm", rows=1, c=1024, dtype="bf16", keep=False, gap=0),
        # the norm in front of the MLP over all tokens, statistics kept for the backward pass
        dict(name="layernorm_tokens", op="layernorm", rows=36864, c=2048, dtype="bf16", keep=True, gap=0),
        # training: an odd row count and an odd multiple of 8 channels
        dict(name="layernorm_grad_odd", op="layernorm_grad", rows=1543, c=1032, dtype="fp16", residual=False,
             gap=8),
        # training: all tokens, joined with the residual stream's gradient
        dict(name="layernorm_grad_tokens", op="layernorm_grad", rows=36864, c=2048, dtype="bf16", residual=True,
             gap=0),
        # single tokens of 16 samples at given positions, shared key heads
        dict(name="rope3d_single_tokens", op="rope3d", n=16, t=1, h=1, w=1, heads_q=16, heads_k=4, head_dim=128,
             dim_t=44, dim_h=42, dim_w=42, pairing="adjacent", dtype="bf16", given=True, grad=False, fused=False),
        # queries and keys of all tokens, rotated inside the fused projection's output rows
        dict(name="rope3d_tokens", op="rope3d", n=1, t=9, h=64, w=64, heads_q=16, heads_k=16, head_dim=128,
             dim_t=32, dim_h=48, dim_w=48, pairing="halves", dtype="fp16", given=False, grad=False, fused=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    v = max(lo, min(hi, int(round(v / step)) * step))
    return v + step if v == 3072 else v  # a size that none of the library's workloads has


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "layernorm", "layernorm_grad", "rope3d"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "linear":
        while True:
            m, n, k = _log(rng, 1, 36864), _log(rng, 64, 8192, 8), _log(rng, 64, 8192, 8)
            if m * n * k <= 36864 * 8192 * 2048:
                break
        return dict(op=op, m=m, n=n, k=k, act=rng.choice(_ACTS), dtype=dtype, bias=rng.random() < 0.8,
                    residual=rng.random() < 0.4, keep=rng.random() < 0.3, gap=rng.choice([0, 0, 8, 72]))
    if op == "linear_grad":
        while True:
            m, n, k = _log(rng, 1, 36864), _log(rng, 64, 8192, 8), _log(rng, 64, 8192, 8)
            if m * n * k <= 36864 * 8192 * 2048:
                break
        return dict(op=op, m=m, n=n, k=k, act=rng.choice(_ACTS), dtype=dtype, bias=rng.random() < 0.8,
                    gap=rng.choice([0, 0, 8, 72]))
    if op == "layernorm":
        return dict(op=op, rows=_log(rng, 1, 36864), c=_log(rng, 64, 8192, 8), dtype=dtype,
                    keep=rng.random() < 0.5, gap=rng.choice([0, 0, 8, 72]))
    if op == "layernorm_grad":
        return dict(op=op, rows=_log(rng, 1, 36864), c=_log(rng, 64, 8192, 8), dtype=dtype,
                    residual=rng.random() < 0.5, gap=rng.choice([0, 0, 8, 72]))
    head_dim = rng.choice([64, 80, 96, 128])
    part = rng.choice([1, 2, 3, 4]) * 8
    rest = (head_dim - part) // 4 * 2  # even; the head's last elements may stay as they are
    pairing = rng.choice(["adjacent", "halves"])
    odd = (part + 2 * rest) % 16  # the rotated part is two halves of whole 8-element groups
    heads_k = rng.choice([1, 2, 4, 8])
    given = rng.random() < 0.4
    if given and rng.random() < 0.4:
        n, t, h, w = _log(rng, 1, 64), 1, 1, 1
    else:
        n, t, h, w = rng.choice([1, 1, 2]), _log(rng, 1, 9), _log(rng, 4, 64), _log(rng, 4, 64)
    return dict(op=op, n=n, t=t, h=h, w=w, heads_q=heads_k * rng.choice([1, 2]), heads_k=heads_k,
                head_dim=head_dim, dim_t=part, dim_h=rest - odd, dim_w=rest, pairing=pairing, dtype=dtype, given=given,
                grad=rng.random() < 0.4, fused=rng.random() < 0.5)


def work(case):
    op = case["op"]
    if op in ("linear", "linear_grad"):
        m, n, k = case["m"], case["n"], case["k"]
        if op == "linear":
            elems = m * k + n * k + m * n * (1 + case["residual"] + case["keep"]) + n * case["bias"]
            return {"bytes": 2 * elems, "flops": 2 * m * n * k}
        elems = m * n * (1 + (case["act"] != "none")) + 2 * m * k + 2 * n * k + n * case["bias"]
        return {"bytes": 2 * elems, "flops": 4 * m * n * k}
    if op == "layernorm":
        rc = case["rows"] * case["c"]
        return {"bytes": 2 * (2 * rc + 2 * case["c"]) + 8 * case["rows"] * case["keep"], "flops": 8 * rc}
    if op == "layernorm_grad":
        rc = case["rows"] * case["c"]
        return {"bytes": 2 * (rc * (3 + case["residual"]) + 3 * case["c"]) + 8 * case["rows"], "flops": 16 * rc}
    tokens = case["n"] * case["t"] * case["h"] * case["w"]
    elems = tokens * (case["heads_q"] + case["heads_k"]) * case["head_dim"]
    return {"bytes": 4 * elems + 12 * tokens * case["given"], "flops": 3 * elems}


# --------------------------------------------------------------- the inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


class _Maker:
    """Seeded tensors of one case."""

    def __init__(self, seed, dtype):
        self.dev = _device()
        self.gen = torch.Generator(device=self.dev)
        self.gen.manual_seed(int(seed) % (1 << 62))
        self.dtype = dtype

    def normal(self, shape, scale=1.0, shift=0.0):
        v = torch.empty(shape, dtype=torch.float32, device=self.dev).normal_(0.0, 1.0, generator=self.gen)
        return v.mul_(scale).add_(shift).to(self.dtype)

    def rows(self, rows, cols, gap, scale=1.0):
        """[rows, cols] values, inside rows of cols + gap elements."""
        return self.normal((rows, cols + gap), scale)[:, :cols]


def _inputs(case, seed):
    mk = _Maker(seed, _DTYPES[case["dtype"]])
    op = case["op"]
    if op in ("linear", "linear_grad"):
        m, n, k = case["m"], case["n"], case["k"]
        s = {"x": mk.rows(m, k, case["gap"]), "w": mk.normal((n, k), 1.0 / math.sqrt(k)),
             "bias": mk.normal((n,), 0.1) if case["bias"] else None}
        if op == "linear":
            s["residual"] = mk.normal((m, n)) if case["residual"] else None
        else:
            s["dy"] = mk.normal((m, n), 0.1)
            # what the forward pass kept: its values before the activation
            s["z"] = mk.normal((m, n)) if case["act"] != "none" else None
        return s
    if op in ("layernorm", "layernorm_grad"):
        rows, c = case["rows"], case["c"]
        x = mk.rows(rows, c, case["gap"])
        # channels with an offset and a few of large scale, as residual streams have them
        x.mul_(1.0 + 8.0 * (torch.rand((c,), device=mk.dev, generator=mk.gen) > 0.99))
        x.add_(mk.normal((c,), 0.5))
        s = {"x": x, "gamma": mk.normal((c,), 0.1, 1.0)}
        if op == "layernorm":
            s["beta"] = mk.normal((c,), 0.1)
        else:
            s["dy"] = mk.normal((rows, c), 0.1)
            s["dres"] = mk.rows(rows, c, case["gap"], 0.1) if case["residual"] else None
            mean = x.float().mean(1)
            rstd = torch.rsqrt((x.float() - mean[:, None]).square().mean(1) + _EPS)
            s["stats"] = torch.stack([mean, rstd], 1).contiguous()
        return s
    n, tok, d = case["n"], case["t"] * case["h"] * case["w"], case["head_dim"]
    hq, hk = case["heads_q"], case["heads_k"]
    if case["fused"]:  # queries, keys and values of a token side by side
        qkv = mk.normal((n, tok, hq + 2 * hk, d))
        s = {"q": qkv[:, :, :hq], "k": qkv[:, :, hq:hq + hk]}
    else:
        s = {"q": mk.normal((n, tok, hq, d)), "k": mk.normal((n, tok, hk, d))}
    s["positions"] = torch.randint(0, 4096, (n, tok, 3), dtype=torch.int32, device=mk.dev,
                                   generator=mk.gen) if case["given"] else None
    return s


_EPS = 1e-6
_BASE = 10000.0


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    import convolution_implicit_gemm_amd as c3d

    case = s["case"]
    op, bf16 = case["op"], case["dtype"] == "bf16"
    ref = s["q"] if op == "rope3d" else s["x"]

    def out(*shape, dtype=None):
        return torch.empty(shape, dtype=dtype or ref.dtype, device=ref.device)

    def scratch(nbytes):
        return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=ref.device)

    if op in ("linear", "linear_grad"):
        m, n, k = case["m"], case["n"], case["k"]
        act = {"none": c3d.CONV3D_ACT_NONE, "silu": c3d.CONV3D_ACT_SILU, "gelu": c3d.CONV3D_ACT_GELU,
               "gelu_tanh": c3d.CONV3D_ACT_GELU_TANH}[case["act"]]
        flags = (c3d.CONV3D_F_BF16 if bf16 else 0) | (c3d.CONV3D_F_BIAS if case["bias"] else 0)
        if op == "linear":
            flags |= c3d.CONV3D_F_RESIDUAL if case["residual"] else 0
            flags |= c3d.CONV3D_F_PREACT if case["keep"] else 0
        s["plan"] = c3d.linear_plan(c3d.make_linear_desc(m, n, k, act=act, flags=flags, x_stride=k + case["gap"]))
        if op == "linear":
            s["y"] = out(m, n)
            s["zk"] = out(m, n) if case["keep"] else None
            s["ws"] = scratch(s["plan"].workspace_bytes)
        else:
            s["dx"] = out(m, k + case["gap"])[:, :k]
            s["dw"] = out(n, k)
            s["db"] = out(n) if case["bias"] else None
            s["ws"] = scratch(c3d.linear_backward_workspace(s["plan"]))
    elif op == "layernorm":
        s["y"] = out(case["rows"], case["c"])
        s["stats"] = out(case["rows"], 2, dtype=torch.float32) if case["keep"] else None
    elif op == "layernorm_grad":
        rows, c = case["rows"], case["c"]
        s["dx"] = out(rows, c + case["gap"])[:, :c]
        s["dgamma"], s["dbeta"] = out(c), out(c)
        s["ws"] = scratch(c3d.layernorm_backward_workspace(rows, c))
    else:
        flags = (c3d.CONV3D_F_BF16 if bf16 else 0) | (c3d.CONV3D_F_POSITIONS if case["given"] else 0)
        pairing = {"adjacent": c3d.ROPE3D_PAIR_ADJACENT, "halves": c3d.ROPE3D_PAIR_HALVES}[case["pairing"]]
        q, k = s["q"], s["k"]
        # the tensors given are a gradient's incoming side when the call is the gradient's
        side = ("q_out_stride", "k_out_stride") if case["grad"] else ("q_stride", "k_stride")
        strides = dict(zip(side, (q.stride()[:3], k.stride()[:3])))
        s["plan"] = c3d.rope3d_plan(c3d.make_rope3d_desc(
            case["n"], case["t"], case["h"], case["w"], case["heads_q"], case["heads_k"], case["head_dim"],
            _dims(case), base=_BASE, pairing=pairing, flags=flags, **strides))
        s["qo"], s["ko"] = out(*q.shape), out(*k.shape)


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import convolution_implicit_gemm_amd as c3d

    case = s["case"]
    op, bf16 = case["op"], case["dtype"] == "bf16"
    if op == "linear":
        c3d.linear_forward(s["plan"], s["x"], s["w"], s["bias"], s["residual"], s["y"], s["zk"], s["ws"])
        return [s["y"], s["zk"]] if case["keep"] else [s["y"]]
    if op == "linear_grad":
        c3d.linear_backward(s["plan"], s["dy"], s["x"], s["w"], s["z"], s["dx"], s["dw"], s["db"], s["ws"])
        return [s["dx"], s["dw"], s["db"]] if case["bias"] else [s["dx"], s["dw"]]
    if op == "layernorm":
        c3d.layernorm(s["x"], s["gamma"], s["beta"], s["y"], s["stats"], case["rows"], case["c"], _EPS,
                      x_stride=case["c"] + case["gap"], bf16=bf16)
        return [s["y"], s["stats"]] if case["keep"] else [s["y"]]
    if op == "layernorm_grad":
        c3d.layernorm_backward(s["dy"], s["x"], s["gamma"], s["stats"], s["dres"], s["dx"], s["dgamma"],
                               s["dbeta"], case["rows"], case["c"], s["ws"], x_stride=case["c"] + case["gap"],
                               bf16=bf16)
        return [s["dx"], s["dgamma"], s["dbeta"]]
    call = c3d.rope3d_backward if case["grad"] else c3d.rope3d_forward
    call(s["plan"], s["q"], s["k"], s["qo"], s["ko"], s["positions"])
    return [s["qo"], s["ko"]]


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    a = math.sqrt(2.0 / math.pi)
    th = torch.tanh(a * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * a * (1.0 + 3 * 0.044715 * z * z)


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], _DTYPES[case["dtype"]]
    if op == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return [y.to(dt), z.to(dt)] if case["keep"] else [y.to(dt)]
    if op == "linear_grad":
        dz = s["dy"].float()
        if case["act"] != "none":
            dz = dz * _act_slope(s["z"].float(), case["act"])
        dx = (dz @ s["w"].float()).to(dt)
        dw = (dz.t() @ s["x"].float()).to(dt)
        return [dx, dw, dz.sum(0).to(dt)] if case["bias"] else [dx, dw]
    if op == "layernorm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + _EPS)
        y = (d * rstd * s["gamma"].float() + s["beta"].float()).to(dt)
        return [y, torch.cat([mean, rstd], 1)] if case["keep"] else [y]
    if op == "layernorm_grad":
        dy = s["dy"].float()
        mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
        xh = (s["x"].float() - mean) * rstd
        g = dy * s["gamma"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return [dx.to(dt), (dy * xh).sum(0).to(dt), dy.sum(0).to(dt)]
    cos, sin = _rotations(s, torch.float32)
    return [_rotate(s["q"].float(), cos, sin, case).to(dt), _rotate(s["k"].float(), cos, sin, case).to(dt)]


def _dims(case):
    return [case["dim_t"], case["dim_h"], case["dim_w"]]


def _positions(case, given, device):
    """[n, tokens, 3] positions in (time, height, width)."""
    if given is not None:
        return given
    t, h, w = case["t"], case["h"], case["w"]
    i = torch.arange(t * h * w, device=device)
    return torch.stack([i // (h * w), i // w % h, i % w], 1)[None].expand(case["n"], -1, -1)


def _rotations(s, dtype):
    """cos and sin of every (sample, token, pair), [n, tokens, 1, pairs]."""
    case = s["case"]
    pos = _positions(case, s["positions"], s["q"].device)
    parts = []
    for axis, dim in enumerate(_dims(case)):
        i = torch.arange(dim // 2, device=pos.device, dtype=torch.float64)
        step = torch.exp(i * (-2.0 * math.log(_BASE) / max(dim, 1)))
        # whole turns are dropped in 64 bits, as tables made at load time do
        angle = pos[:, :, axis, None].to(torch.float64) * step
        parts.append(torch.remainder(angle, 2.0 * math.pi).to(dtype))
    angle = torch.cat(parts, 2)[:, :, None]
    sin = torch.sin(angle)
    return torch.cos(angle), (-sin if case["grad"] else sin)


def _rotate(x, cos, sin, case):
    r = sum(_dims(case))
    y = x.clone()
    if case["pairing"] == "adjacent":
        u, v = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2] = u * cos - v * sin
        y[..., 1:r:2] = u * sin + v * cos
    else:
        u, v = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2] = u * cos - v * sin
        y[..., r // 2:r] = u * sin + v * cos
    return y


# ---------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    d = {key: v.double() if v is not None and v.is_floating_point() else v for key, v in s.items()}
    op = case["op"]
    if op == "linear":
        z = torch.matmul(d["x"], d["w"].transpose(0, 1))
        z += 0.0 if d["bias"] is None else d["bias"]
        y = _act64(z, case["act"])[0]
        if d["residual"] is not None:
            y = y + d["residual"]
        return [y, z] if case["keep"] else [y]
    if op == "linear_grad":
        dz = d["dy"] if d["z"] is None else d["dy"] * _act64(d["z"], case["act"])[1]
        grads = [torch.matmul(dz, d["w"]), torch.matmul(dz.transpose(0, 1).contiguous(), d["x"])]
        return grads + [dz.sum(dim=0)] if case["bias"] else grads
    if op == "layernorm":
        mean = d["x"].sum(dim=1) / case["c"]
        var = (d["x"] - mean[:, None]).pow(2).sum(dim=1) / case["c"]
        rstd = (var + _EPS).pow(-0.5)
        y = torch.addcmul(d["beta"], (d["x"] - mean[:, None]) * rstd[:, None], d["gamma"])
        return [y, torch.stack((mean, rstd), dim=1)] if case["keep"] else [y]
    if op == "layernorm_grad":
        c = case["c"]
        r = d["stats"][:, 1].unsqueeze(1)
        xh = (d["x"] - d["stats"][:, 0].unsqueeze(1)) * r
        dxh = d["dy"] * d["gamma"]
        dx = (r / c) * (c * dxh - dxh.sum(1, keepdim=True) - xh * (dxh * xh).sum(1, keepdim=True))
        return [dx if d["dres"] is None else dx + d["dres"], torch.mul(d["dy"], xh).sum(0), d["dy"].sum(0)]
    # rotations as products of complex numbers
    pos = _positions(case, d["positions"], d["q"].device).double()
    turn = []
    for axis, dim in enumerate(_dims(case)):
        for i in range(dim // 2):
            turn.append(pos[:, :, axis] * _BASE ** (-2.0 * i / dim))
    unit = torch.polar(torch.ones_like(pos[:, :, :1]), torch.stack(turn, dim=2))[:, :, None, :]
    if case["grad"]:
        unit = unit.conj()
    half, outs = len(turn), []
    for x in (d["q"], d["k"]):
        r, rest = x[..., :2 * half], x[..., 2 * half:]
        if case["pairing"] == "adjacent":
            c = torch.complex(r[..., 0::2].contiguous(), r[..., 1::2].contiguous()) * unit
            r = torch.stack((c.real, c.imag), dim=-1).flatten(-2)
        else:
            c = torch.complex(r[..., :half].contiguous(), r[..., half:].contiguous()) * unit
            r = torch.cat((c.real, c.imag), dim=-1)
        outs.append(torch.cat((r, rest), dim=-1))
    return outs


def _act64(z, act):
    """The activation and its derivative."""
    if act == "silu":
        sg = torch.sigmoid(z)
        return z * sg, sg + z * sg * (1 - sg)
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / 2 ** 0.5)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
    if act == "gelu_tanh":
        a, b = (2 / math.pi) ** 0.5, 0.044715
        sg = torch.sigmoid(2 * a * (z + b * z ** 3))
        return z * sg, sg + z * sg * (1 - sg) * 2 * a * (1 + 3 * b * z ** 2)
    return z, torch.ones_like(z)
