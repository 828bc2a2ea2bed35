"""The operators that complete a training step of the transformer over the
latent grid, as measured cases.

Attention over the grid's tokens (within frames, causal by frames, against a
cache, against a padded prompt), its gradient, and the AdamW step over all
weights of such blocks.  Tokens are the voxels of the latent video, as in
operators.py beside this file.

``own`` selects what ``run`` computes: the plain form in elementary torch
operations (32 bits, rounded once at the end), or the library's kernels.
"""
import math

import torch

own = False

_DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def _att(op="attention", n=1, tq=1, tk=0, hq=16, hk=16, d=128, frame=0, window=0, q_offset=0, ragged=False, tail=False,
         layout="tokens", dtype="bf16", keep=False, **more):
    """frame: tokens of a frame, 0 for no mask; window: frames that a query sees, 0 for all before its own;
    ragged: samples of different lengths; tail: the queries are a sample's last tokens;
    layout: tokens [n, t, h, d], heads [n, h, t, d], or fused, q, k and v side by side in a token's row."""
    return dict(more, op=op, n=n, tq=tq, tk=tk or tq, hq=hq, hk=hk, d=d, frame=frame, window=window, q_offset=q_offset,
                ragged=ragged, tail=tail, layout=layout, dtype=dtype, keep=keep)


def _adam(tensors="block", size=256, count=1, dtype="bf16", master=True, grad32=False, state8=False, **more):
    """tensors: block, `count` transformer blocks of `size` channels; or mixed, `count` tensors of odd sizes up to `size`."""
    return dict(more, op="adamw", tensors=tensors, size=size, count=count, dtype=dtype, master=master, grad32=grad32,
                state8=state8)


def listed():
    return [
        # one query over a short sequence: latency
        _att(name="attention_one_token", tq=1, tk=257, hk=4),
        # serving: one token for each of 16 samples against caches of different lengths, shared key heads
        _att(name="attention_cache_tokens", n=16, tq=1, tk=36864, hk=4, ragged=True, tail=True),
        # one frame and a token against padded prompts of different lengths
        _att(name="attention_prompt", n=2, tq=4097, tk=613, hq=12, hk=12, d=80, ragged=True, layout="heads", dtype="fp16"),
        # chunked decoding: the next frame against the frames before it and itself
        _att(name="attention_next_frame", tq=4096, tk=20480, hk=4, d=64, frame=4096, q_offset=16384, dtype="fp16"),
        # each of 9 frames of 32 x 32 by itself, inside the fused projection's rows
        _att(name="attention_frames", tq=9216, frame=1024, window=1, layout="fused", keep=True),
        # 5 frames of 64 x 64, a frame sees itself and those before it
        _att(name="attention_causal_frames", tq=20480, frame=4096, layout="fused", keep=True),
        # training: a few tokens, latency
        _att(name="attention_grad_small", op="attention_grad", tq=64, hq=2, hk=2, d=64, layout="fused", dtype="fp16"),
        # training: token by token, padded samples of an odd length, shared key heads
        _att(name="attention_grad_ragged", op="attention_grad", n=3, tq=1543, hq=12, hk=4, d=80, frame=1, ragged=True),
        # training: 5 frames of 64 x 64, causal by frames
        _att(name="attention_grad_causal_frames", op="attention_grad", tq=20480, frame=4096, layout="fused"),
        # a block of 256 channels, fp32 states
        _adam(name="adamw_small_block"),
        # many odd tensors without a master copy, 32-bit gradients, 8-bit states
        _adam(name="adamw_mixed", tensors="mixed", size=2359297, count=61, dtype="fp16", master=False, grad32=True,
              state8=True),
        # four blocks of 2048 channels, 201 million weights, 8-bit states
        _adam(name="adamw_blocks", size=2048, count=4, state8=True),
    ]


_MOST_SCORES = 16 * 20480 * 20480  # of the largest listed case, seen or not
_MOST_FLOPS = {"attention": 4 * 16 * 128 * 15 * 4096 ** 2, "attention_grad": 10 * 16 * 128 * 15 * 4096 ** 2}
_MOST_WEIGHTS = 4 * 12 * 2048 * 2048


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "attention_grad", "attention_grad", "adamw"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "adamw":
        if rng.random() < 0.5:
            tensors, size, count = "block", _log(rng, 64, 2048) // 8 * 8, rng.randint(1, 4)
        else:
            tensors, size, count = "mixed", _log(rng, 1, 1 << 24), _log(rng, 1, 200)
            while size * count > _MOST_WEIGHTS:
                count = (count + 1) // 2
        return _adam(tensors, size, count, dtype, rng.random() < 0.6, rng.random() < 0.3, rng.random() < 0.5)
    d = rng.choice([32, 40, 64, 64, 72, 80, 96, 128, 128, 128])
    hk = rng.choice([1, 2, 4, 8, 16])
    hq = hk * rng.choice([1, 1, 1, 2, 4])
    layout, keep = rng.choice(["tokens", "heads", "fused"]), rng.random() < 0.5
    ragged = rng.random() < 0.3
    kind = rng.choice(["self", "self", "frames", "cross", "cache"])
    if kind == "cache" and op == "attention":  # single tokens, or a few
        n, tq, tk = _log(rng, 1, 32), rng.choice([1, 1, 1, 2, 7, 33]), _log(rng, 1, 36864)
        tk = max(tk, tq)
        while n * hk * tk * d > 16 * 4 * 36864 * 128:
            n = (n + 1) // 2 if n > 1 else n
            hk, hq = (hk // 2, hq // 2) if n == 1 else (hk, hq)
        return _att(op, n, tq, tk, hq, hk, d, frame=1, ragged=ragged, tail=True, dtype=dtype, keep=keep,
                    window=rng.choice([0, 0, 4096]), layout=rng.choice(["tokens", "heads"]))
    if kind == "cross":
        n, tq, tk, frame, window = rng.choice([1, 1, 2, 4]), _log(rng, 1, 20480), _log(rng, 1, 4096), 0, 0
        layout = "tokens" if layout == "fused" else layout
    elif kind == "frames":
        n, side, frames = 1, _log(rng, 3, 64), rng.randint(1, 9)
        frame, window = side * side, rng.choice([0, 0, 1, 2, 3])
        tq = tk = min(frame * frames, 20480)
    else:
        n, tq, frame, window = rng.choice([1, 1, 2, 3]), _log(rng, 1, 20480), rng.choice([0, 1]), 0
        tk = tq
        if frame:
            window = rng.choice([0, 0, 100, 1024])
    # some queries stand before the first key, or past the last
    offset = rng.choice([0, 0, 0, -17, 300]) if frame and layout != "fused" else 0
    while True:
        case = _att(op, n, tq, tk, hq, hk, d, frame, window, offset, ragged, False, layout, dtype, keep)
        if n * hq * tq * tk <= _MOST_SCORES and work(case)["flops"] <= _MOST_FLOPS[op]:
            return case
        if n > 1:
            n -= 1
        elif hk > 1:
            hk, hq = hk // 2, hq // 2
        else:
            hq = hk


def _lengths(case):
    """(queries, keys) of each sample; the case alone decides."""
    n, tq, tk = case["n"], case["tq"], case["tk"]
    if not case["ragged"]:
        return [(tq, tk)] * n
    keys = [tk - (i * 7919 + 131) % (tk // 2 + 1) for i in range(n)]
    if case["tail"]:
        return [(min(tq, kl), kl) for kl in keys]
    if tq == tk:
        return [(kl, kl) for kl in keys]
    return [(tq - (i * 104729) % (tq // 2 + 1), kl) for i, kl in enumerate(keys)]


def _adam_sizes(case):
    c, k = case["size"], case["count"]
    if case["tensors"] == "block":
        return [3 * c * c, 3 * c, c * c, c, 4 * c * c, 4 * c, 4 * c * c, c, c, c, c, c] * k
    return [max(1, int(c ** (((i * 37) % k + 1) / k))) for i in range(k)]


def _pairs(case):
    """Pairs of a query and a key that it sees, over the samples (of one head)."""
    total = 0
    for ql, kl in _lengths(case):
        pos = torch.arange(ql, dtype=torch.int64) + case["q_offset"] + (kl - ql if case["tail"] else 0)
        if not case["frame"]:
            total += ql * kl
            continue
        f = torch.div(pos, case["frame"], rounding_mode="floor")
        hi = ((f + 1) * case["frame"]).clamp(0, kl)
        lo = ((f + 1 - case["window"]) * case["frame"]).clamp(0, kl) if case["window"] else torch.zeros_like(hi)
        total += int((hi - lo).clamp(min=0).sum())
    return total


def work(case):
    if case["op"] == "adamw":
        count = sum(_adam_sizes(case))
        state = 2.0 + 2.0 / 128 if case["state8"] else 8.0
        weight = 6.0 if case["master"] else 2.0
        read = weight - (2.0 if case["master"] else 0.0) + (4.0 if case["grad32"] else 2.0) + state
        return {"bytes": count * (read + weight + state), "flops": 14 * count}
    rows = sum(ql for ql, _ in _lengths(case)) * case["hq"]
    keys = sum(kl for _, kl in _lengths(case)) * case["hk"]
    all_q, all_k = case["n"] * case["tq"] * case["hq"], case["n"] * case["tk"] * case["hk"]
    d, pairs = case["d"], _pairs(case) * case["hq"]
    if case["op"] == "attention":
        return {"bytes": 2 * d * (rows + all_q + 2 * keys) + 4 * all_q * case["keep"], "flops": 4 * d * pairs}
    return {"bytes": 2 * d * (3 * rows + all_q + 2 * keys + 2 * all_k) + 4 * rows, "flops": 10 * d * pairs}


# --------------------------------------------------------------- the inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


class _Maker:
    """Seeded values of one case."""

    def __init__(self, seed):
        self.dev = _device()
        self.gen = torch.Generator(device=self.dev)
        self.gen.manual_seed(int(seed) % (1 << 62))

    def normal(self, shape, scale=1.0, shift=0.0, dtype=torch.float32):
        v = torch.empty(shape, dtype=torch.float32, device=self.dev).normal_(0.0, 1.0, generator=self.gen)
        return v.mul_(scale).add_(shift).to(dtype)


_BLOCK = 128  # elements that share a scale of 8-bit states
_HYPER = dict(lr=3e-4, beta1=0.9, beta2=0.98, eps=1e-8, weight_decay=0.05, step=12, grad_scale=0.5)


def _attention_inputs(case, seed):
    mk, dt = _Maker(seed), _DTYPES[case["dtype"]]
    n, tq, tk, hq, hk, d = (case[x] for x in ("n", "tq", "tk", "hq", "hk", "d"))

    def heads(t, h, scale, shift=0.0):
        if case["layout"] == "heads":
            return mk.normal((n, h, t, d), scale, shift, dt).transpose(1, 2)
        return mk.normal((n, t, h, d), scale, shift, dt)

    if case["layout"] == "fused":
        qkv = mk.normal((n, tq, hq + 2 * hk, d), 1.0, 0.0, dt)
        qkv[:, :, :hq] *= 1.5
        s = {"qkv": qkv, "q": qkv[:, :, :hq], "k": qkv[:, :, hq:hq + hk], "v": qkv[:, :, hq + hk:]}
    else:
        s = {"q": heads(tq, hq, 1.5), "k": heads(tk, hk, 1.0, 0.1), "v": heads(tk, hk, 1.0)}
    s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=mk.dev) if case["ragged"] else None
    if case["op"] == "attention_grad":
        s["do"] = heads(tq, hq, 0.05)
    return s


def _encode(x):
    """Blocks [b, 128] of values as e4m3 numbers and the power of two of each block."""
    f, e = torch.frexp(x.abs().amax(1, keepdim=True))  # f in [1/2, 1); 448 = 7/8 * 2^9
    e = (e - 9 + (f > 0.875)).clamp(min=-126)
    x = torch.ldexp(x, -e)
    step = torch.ldexp(torch.ones_like(x), (torch.frexp(x)[1] - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step, e


def _encode_root(v):
    """The same of square roots: a positive one never becomes 0."""
    root = torch.sqrt(v)
    c, e = _encode(root)
    return torch.where((c == 0) & (root > 0), torch.full_like(c, 2.0 ** -9), c), e


def _adam_inputs(case, seed):
    mk, dt, sizes = _Maker(seed), _DTYPES[case["dtype"]], _adam_sizes(case)
    # all tensors lie in one buffer of each kind, every one from a multiple of 128 on
    blocks = [-(-v // _BLOCK) for v in sizes]
    first = [0]
    for b in blocks:
        first.append(first[-1] + b)
    used = torch.ones((first[-1], _BLOCK), dtype=torch.bool, device=mk.dev)
    at = torch.tensor([f - 1 for f in first[1:]], device=mk.dev)
    last = torch.tensor([v - (b - 1) * _BLOCK for v, b in zip(sizes, blocks)], device=mk.dev)
    used[at] = torch.arange(_BLOCK, device=mk.dev)[None] < last[:, None]
    shape = (first[-1], _BLOCK)
    w = mk.normal(shape, 0.02).mul_(used)
    # gradients and states whose size differs from row to row
    size = torch.exp(mk.normal((first[-1], 1), 2.0)) * 1e-3
    g = (mk.normal(shape) * size).mul_(used)
    m = (mk.normal(shape, 0.3) * size).mul_(used)
    v = (mk.normal(shape).square() * size.square() * 0.2).mul_(used)
    s = {"sizes": sizes, "first": first, "grad": g if case["grad32"] else g.to(dt), "param": w.to(dt),
         "master": w if case["master"] else None}
    # weights decay, biases and norms (the odd places of a block's list) do not
    decay = [float(v >= 4096) for v in sizes]
    s["decay"] = decay
    s["decay_rows"] = torch.repeat_interleave(torch.tensor(decay, device=mk.dev), torch.tensor(blocks, device=mk.dev))
    if case["state8"]:
        for key, (c, e) in (("m", _encode(m)), ("v", _encode_root(v))):
            s[key] = c.to(torch.float8_e4m3fn)
            s[key + "_scale"] = (e + 127).to(torch.uint8).flatten()
    else:
        s["m"], s["v"] = m, v
    return s


def _inputs(case, seed):
    return _adam_inputs(case, seed) if case["op"] == "adamw" else _attention_inputs(case, seed)


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if case["op"] == "attention_grad":  # what the forward pass left
        o, lse = _attention_plain(s, _DTYPES[case["dtype"]])
        s["o"] = torch.empty_like(s["do"]).copy_(o)
        s["lse"] = lse
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    import convolution_implicit_gemm_amd as c3d

    case = s["case"]
    bf16 = c3d.CONV3D_F_BF16 if case["dtype"] == "bf16" else 0
    if case["op"] == "adamw":
        def parts(key):
            flat = s[key].view(-1)
            return [flat[f * _BLOCK:f * _BLOCK + v] for f, v in zip(s["first"], s["sizes"])]

        def scales(key):
            return [s[key][a:b] for a, b in zip(s["first"], s["first"][1:])]

        s["list"] = c3d.adamw_list(parts("param"), parts("grad"), parts("m"), parts("v"),
                                   master=parts("master") if case["master"] else None,
                                   m_scale=scales("m_scale") if case["state8"] else None,
                                   v_scale=scales("v_scale") if case["state8"] else None, decay=s["decay"])
        s["hyper"] = c3d.make_adamw_hyper(**_HYPER)
        return
    flags = bf16 | (c3d.CONV3D_F_LENGTHS if case["ragged"] else 0) | (c3d.CONV3D_F_TAIL if case["tail"] else 0)
    if case["layout"] == "heads":
        o = torch.empty((case["n"], case["hq"], case["tq"], case["d"]), dtype=s["q"].dtype,
                        device=s["q"].device).transpose(1, 2)
    else:
        o = torch.empty((case["n"], case["tq"], case["hq"], case["d"]), dtype=s["q"].dtype, device=s["q"].device)
    s["plan"] = plan = c3d.attention_plan(c3d.make_attention_desc(
        case["n"], case["tq"], case["tk"], case["hq"], case["hk"], case["d"], frame=case["frame"], window=case["window"],
        flags=flags, q_stride=s["q"].stride()[:3], k_stride=s["k"].stride()[:3], v_stride=s["v"].stride()[:3],
        o_stride=o.stride()[:3]))
    if case["op"] == "attention":
        need = plan.workspace_bytes
        s["o"] = o
        s["lse"] = torch.empty((case["n"], case["hq"], case["tq"]), dtype=torch.float32,
                               device=o.device) if case["keep"] else None
    else:
        need = c3d.attention_backward_workspace(plan)
        if case["layout"] == "fused":
            hq, hk = case["hq"], case["hk"]
            g = torch.empty_like(s["qkv"])
            s["dq"], s["dk"], s["dv"] = g[:, :, :hq], g[:, :, hq:hq + hk], g[:, :, hq + hk:]
        else:
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in ("q", "k", "v"))
    s["ws"] = torch.empty(max(int(need), 16), dtype=torch.uint8, device=o.device)


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _adam_outputs(s):
    out = {x: s[x] for x in ("param", "master", "m", "v") if s[x] is not None}
    if s["case"]["state8"]:  # powers of two
        out["m_scale"], out["v_scale"] = (s[x].view(torch.float8_e8m0fnu) for x in ("m_scale", "v_scale"))
    return out


def _run_own(s):
    import convolution_implicit_gemm_amd as c3d

    case = s["case"]
    if case["op"] == "adamw":
        c3d.adamw_step(s["list"], s["hyper"])
        return _adam_outputs(s)
    if case["op"] == "attention":
        c3d.attention_forward(s["plan"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["lengths"], case["q_offset"], s["ws"])
        return [s["o"], s["lse"]] if case["keep"] else [s["o"]]
    c3d.attention_backward(s["plan"], s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["dq"], s["dk"], s["dv"],
                           s["lengths"], case["q_offset"], s["ws"])
    return [s["dq"], s["dk"], s["dv"]]


def _hidden(s):
    """(scores that are not seen [n, 1, 1, tq, tk], queries behind a sample's last [n, 1, 1, tq, 1]); None: none."""
    case, dev = s["case"], s["q"].device
    tq, tk, frame = case["tq"], case["tk"], case["frame"]
    if not frame and s["lengths"] is None:
        return None, None
    i, j = torch.arange(tq, device=dev), torch.arange(tk, device=dev)
    ql = kl = None
    pos = (i + case["q_offset"])[None]
    if s["lengths"] is not None:
        ql, kl = s["lengths"][:, :1].long(), s["lengths"][:, 1:].long()
    if case["tail"]:
        pos = pos + (kl - ql if kl is not None else tk - tq)
    # the range of keys that each query sees
    lo, hi = torch.zeros_like(pos), torch.full_like(pos, tk)
    if frame:
        f = torch.div(pos, frame, rounding_mode="floor")
        hi = (f + 1) * frame
        if case["window"]:
            lo = (f + 1 - case["window"]) * frame
    past = None
    if kl is not None:
        hi = torch.minimum(hi, kl)
        past = i[None] >= ql
        hi = torch.where(past, torch.zeros_like(hi), hi)
        past = past[:, None, None, :, None]
    hidden = (j >= hi[:, :, None]) | (j < lo[:, :, None])
    return hidden[:, None, None], past


def _by_key_head(s, key):
    """[n, hk, queries of all heads that share a key head, d] or [n, hk, tk, d], in 32 bits."""
    case, x = s["case"], s[key].float().transpose(1, 2)
    return x.reshape(case["n"], case["hk"], -1, case["d"])


def _scores(s, q, k, hidden):
    case = s["case"]
    x = torch.matmul(q, k.transpose(2, 3)).mul_(case["d"] ** -0.5)
    if hidden is not None:
        x.view(case["n"], case["hk"], -1, case["tq"], case["tk"]).masked_fill_(hidden, -math.inf)
    return x


def _rows_of(case, x):
    """[n, hk, queries of a group, d] as [n, tq, hq, d]."""
    return x.reshape(case["n"], case["hq"], case["tq"], case["d"]).transpose(1, 2)


def _clean(s, key):
    """Keys and values with zeros behind the sample's last one."""
    x = _by_key_head(s, key)
    if s["lengths"] is None:
        return x
    behind = torch.arange(s["case"]["tk"], device=x.device) >= s["lengths"][:, 1:]
    return x.masked_fill(behind[:, None, :, None], 0.0)


def _attention_plain(s, dt):
    case = s["case"]
    hidden, _ = _hidden(s)
    x = _scores(s, _by_key_head(s, "q"), _clean(s, "k"), hidden)
    top = x.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x.sub_(top).exp_()
    total = x.sum(3, keepdim=True)
    o = torch.matmul(x, _clean(s, "v")) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).reshape(case["n"], case["hq"], case["tq"])
    return _rows_of(case, o).to(dt), lse


def _run_plain(s):
    case = s["case"]
    if case["op"] == "adamw":
        return _adam_plain(s)
    dt = _DTYPES[case["dtype"]]
    if case["op"] == "attention":
        o, lse = _attention_plain(s, dt)
        return [o, lse] if case["keep"] else [o]
    hidden, past = _hidden(s)
    q, k, do = _by_key_head(s, "q"), _clean(s, "k"), _by_key_head(s, "do")
    if past is not None:  # rows behind the last query give nothing, whatever they hold
        for x in (q, do):
            x.view(case["n"], case["hk"], -1, case["tq"], case["d"]).masked_fill_(past, 0.0)
    p = _scores(s, q, k, hidden)
    lse = s["lse"].reshape(case["n"], case["hk"], -1, 1)
    p.sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)).exp_()
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, _clean(s, "v").transpose(2, 3))
    ds.sub_((ds * p).sum(3, keepdim=True)).mul_(p).mul_(case["d"] ** -0.5)
    del p
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)
    return [_rows_of(case, dq).to(dt), dk.transpose(1, 2).to(dt), dv.transpose(1, 2).to(dt)]


def _adam_plain(s):
    case, h = s["case"], _HYPER
    c1, c2 = 1.0 - h["beta1"] ** h["step"], 1.0 - h["beta2"] ** h["step"]
    g = s["grad"].float() * h["grad_scale"]
    m, v = s["m"].float(), s["v"].float()
    if case["state8"]:
        m = torch.ldexp(m, s["m_scale"].to(torch.int32)[:, None] - 127)
        v = torch.ldexp(v, s["v_scale"].to(torch.int32)[:, None] - 127).square()
    m = m * h["beta1"] + g * (1.0 - h["beta1"])
    v = v * h["beta2"] + g * g * (1.0 - h["beta2"])
    w = s["master"] if case["master"] else s["param"].float()
    w = w * (1.0 - h["lr"] * h["weight_decay"] * s["decay_rows"][:, None]) \
        - h["lr"] * ((m / c1) / (torch.sqrt(v / c2) + h["eps"]))
    if case["master"]:
        s["master"].copy_(w)
    s["param"].copy_(w)
    if case["state8"]:
        m, em = _encode(m)
        v, ev = _encode_root(v)
        s["m_scale"].copy_(em.flatten() + 127)
        s["v_scale"].copy_(ev.flatten() + 127)
    s["m"].copy_(m)
    s["v"].copy_(v)
    return _adam_outputs(s)


# ---------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    if case["op"] == "adamw":
        return _adam_exact(case, seed)
    s = _attention_inputs(case, seed)
    dev, grad = s["q"].device, case["op"] == "attention_grad"
    n, tq, tk, hq, hk, d = (case[x] for x in ("n", "tq", "tk", "hq", "hk", "d"))

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.float64, device=dev)

    o, lse = zeros(n, tq, hq, d), torch.full((n, hq, tq), -math.inf, dtype=torch.float64, device=dev)
    dq, dk, dv = (zeros(n, tq, hq, d), zeros(n, tk, hk, d), zeros(n, tk, hk, d)) if grad else (None, None, None)
    step = max(1, (1 << 27) // tk)  # rows at a time
    for b, (ql, kl) in enumerate(_lengths(case)):
        fk = torch.arange(kl, device=dev)
        for h in range(hq):
            k, v = (s[x][b, :kl, h // (hq // hk)].double() for x in ("k", "v"))
            for r0 in range(0, ql, step):
                r1 = min(ql, r0 + step)
                q = s["q"][b, r0:r1, h].double()
                x = torch.matmul(q, k.t()) / math.sqrt(d)
                if case["frame"]:
                    at = torch.arange(r0, r1, device=dev) + case["q_offset"] + (kl - ql) * case["tail"]
                    ahead = torch.floor_divide(fk, case["frame"])[None] - torch.floor_divide(at, case["frame"])[:, None]
                    seen = ahead <= 0
                    if case["window"]:
                        seen &= ahead > -case["window"]
                    x = torch.where(seen, x, torch.full_like(x, -math.inf))
                z = torch.logsumexp(x, dim=1)
                p = torch.where(x == -math.inf, torch.zeros_like(x), torch.exp(x - z[:, None]))
                if not grad:
                    o[b, r0:r1, h], lse[b, h, r0:r1] = torch.matmul(p, v), z
                    continue
                go = s["do"][b, r0:r1, h].double()
                gp = torch.matmul(go, v.t())
                gx = (p * gp - p * torch.linalg.vecdot(p, gp)[:, None]) / math.sqrt(d)
                dq[b, r0:r1, h] = torch.matmul(gx, k)
                dk[b, :kl, h // (hq // hk)] += torch.matmul(gx.t(), q)
                dv[b, :kl, h // (hq // hk)] += torch.matmul(p.t(), go)
    if grad:
        return [dq, dk, dv]
    return [o, lse] if case["keep"] else [o]


def _adam_exact(case, seed):
    s, h = _adam_inputs(case, seed), _HYPER
    g = s["grad"].double().mul(h["grad_scale"])
    m, v = s["m"].double(), s["v"].double()
    if case["state8"]:
        m = m * 2.0 ** (s["m_scale"].double().unsqueeze(1) - 127)
        v = (v * 2.0 ** (s["v_scale"].double().unsqueeze(1) - 127)).pow(2)
    m.lerp_(g, 1 - h["beta1"])
    v.lerp_(g.pow(2), 1 - h["beta2"])
    w = s["master"].double() if case["master"] else s["param"].double()
    denominator = v.div(1 - h["beta2"] ** h["step"]).sqrt_().add_(h["eps"])
    w = w - h["lr"] * h["weight_decay"] * s["decay_rows"].double().unsqueeze(1) * w
    w.addcdiv_(m, denominator, value=-h["lr"] / (1 - h["beta1"] ** h["step"]))
    out = {"param": w}
    if case["master"]:
        out["master"] = w
    if not case["state8"]:
        return dict(out, m=m, v=v)
    for key, x in (("m", m), ("v", v.sqrt())):
        top = x.abs().amax(dim=1).clamp(min=448 * 2.0 ** -126)
        # the least power of two that brings the block's largest value to 448 or below
        e = torch.ceil(torch.log2(top / 448))
        e = torch.where(448 * 2.0 ** e < top, e + 1, torch.where(448 * 2.0 ** (e - 1) >= top, e - 1, e)).clamp(min=-126)
        y = x / (2.0 ** e).unsqueeze(1)
        unit = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        code = torch.round(y / unit).mul(unit)
        out[key] = code.clamp(min=2.0 ** -9).where(x > 0, code) if key == "v" else code
        out[key + "_scale"] = 2.0 ** e
    return out
