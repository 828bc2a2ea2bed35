"""Attention and its gradient against the definition in 64 bits.

Bounds.  A probability p is rounded to the element type before the product with v
(half a step, u relative, u = 2^-11 fp16 and 2^-8 bf16), so o errs by at most u sum_j p_j |v_j| / 1 from
that, plus half a step of o itself; fp32 arithmetic adds (d + 16) 2^-24 of the scores' absolute sums,
exponentiated.  In the gradients P and dS are rounded once each as operands:
  dv: u sum_i P |dout|;  dq: scale u sum_j |dS| |k|;  dk: scale u sum_i |dS| |q|,
and dS carries fp32 errors of P (the scores', as above), of dP (d 2^-24 sum |dout||v|) and of delta, which is taken
of the rounded o: |delta| errs by u sum_d |dout o|, so dS by P times that.
"""
import math

import pytest
import torch

import convolution_implicit_gemm_amd as c3d
from token_helpers import DTYPES, U24, assert_within, gen, normal, scratch

pytestmark = pytest.mark.gpu

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half of the least step


def seen_mask(tq, tk, ql, kl, frame, window, q_offset, tail):
    """[tq, tk] bool, by the definition, one pair at a time in spirit."""
    i = torch.arange(tq, device="cuda:0")[:, None]
    j = torch.arange(tk, device="cuda:0")[None]
    m = (i < ql) & (j < kl)
    if frame:
        p = q_offset + i + (kl - ql if tail else 0)
        fq, fk = torch.floor_divide(p, frame), torch.floor_divide(j, frame)
        m = m & (fk <= fq)
        if window:
            m = m & (fk > fq - window)
    return m


class Case:
    def __init__(self, n=1, tq=64, tk=64, hq=2, hk=2, d=64, frame=0, window=0, q_offset=0, lengths=None, tail=False,
                 layout="tokens", dtype="bf16", scale=0.0, seed=1, spread=1.0):
        self.__dict__.update(locals())
        self.dt = DTYPES[dtype]
        g = gen(seed)

        def heads(t, h, s):
            if layout == "heads":
                return normal(g, (n, h, t, d), self.dt, s).transpose(1, 2)
            if layout == "gaps":
                buf = torch.full((n, t, h + 1, d + 8), float("nan"), dtype=self.dt, device="cuda:0")
                buf[:, :, :h, :d] = normal(g, (n, t, h, d), self.dt, s)
                return buf[:, :, :h, :d]
            return normal(g, (n, t, h, d), self.dt, s)

        if layout == "fused":
            qkv = normal(g, (n, tq, hq + 2 * hk, d), self.dt, spread)
            self.q, self.k, self.v = qkv[:, :, :hq], qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:]
        else:
            self.q, self.k, self.v = heads(tq, hq, spread), heads(tk, hk, spread), heads(tk, hk, 1.0)
        self.do = heads(tq, hq, 0.1) if layout != "fused" else normal(g, (n, tq, hq, d), self.dt, 0.1)
        self.len = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda:0")
        if lengths is not None:  # what lies behind the lengths is never read
            for b, (ql, kl) in enumerate(lengths):
                self.q[b, max(ql, 0):] = float("nan")
                self.do[b, max(ql, 0):] = float("inf")
                self.k[b, max(kl, 0):] = float("nan")
                self.v[b, max(kl, 0):] = float("inf")
        flags = (c3d.CONV3D_F_BF16 if dtype == "bf16" else 0) | (c3d.CONV3D_F_LENGTHS if lengths is not None else 0) | \
            (c3d.CONV3D_F_TAIL if tail else 0)
        self.o = torch.empty_strided(self.do.shape, self.do.stride(), dtype=self.dt, device="cuda:0").fill_(9.0)
        self.plan = c3d.attention_plan(c3d.make_attention_desc(
            n, tq, tk, hq, hk, d, frame=frame, window=window, scale=scale, flags=flags, q_stride=self.q.stride()[:3],
            k_stride=self.k.stride()[:3], v_stride=self.v.stride()[:3], o_stride=self.o.stride()[:3]))
        self.lse = torch.full((n, hq, tq), 7.0, device="cuda:0")
        self.s = scale or 1.0 / math.sqrt(d)

    def forward(self):
        c3d.attention_forward(self.plan, self.q, self.k, self.v, self.o, self.lse, self.len, self.q_offset,
                              scratch(self.plan.workspace_bytes))

    def backward(self, dq=True, dk=True, dv=True):
        def like(x, on):
            return torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=x.device).fill_(5.0) if on else None

        if self.layout == "fused":
            buf = torch.full((self.n, self.tq, self.hq + 2 * self.hk, self.d), 5.0, dtype=self.dt, device="cuda:0")
            parts = buf[:, :, :self.hq], buf[:, :, self.hq:self.hq + self.hk], buf[:, :, self.hq + self.hk:]
            outs = [x if on else None for x, on in zip(parts, (dq, dk, dv))]
        else:
            outs = [like(x, on) for x, on in ((self.q, dq), (self.k, dk), (self.v, dv))]
        c3d.attention_backward(self.plan, self.do, self.q, self.k, self.v, self.o, self.lse, *outs, self.len,
                               self.q_offset, scratch(c3d.attention_backward_workspace(self.plan)))
        return outs

    def lens(self, b):
        if self.lengths is None:
            return self.tq, self.tk
        ql, kl = self.lengths[b]
        return min(max(ql, 0), self.tq), min(max(kl, 0), self.tk)

    def one(self, b, h):
        """(q, k, v, do, mask, P, lse, the scores' fp32 error) of a head in 64 bits."""
        ql, kl = self.lens(b)

        def part(x, hh, live):
            x = x[b, :, hh].double().clone()
            x[live:] = 0.0
            return x

        hk = h // (self.hq // self.hk)
        q, do = part(self.q, h, ql), part(self.do, h, ql)
        k, v = part(self.k, hk, kl), part(self.v, hk, kl)
        m = seen_mask(self.tq, self.tk, ql, kl, self.frame, self.window, self.q_offset, self.tail)
        x = (q @ k.t()) * self.s
        # the product's sum, the scaling, the exponent's argument and the exponential itself
        err = U24 * ((self.d + 4) * self.s * (q.abs() @ k.abs().t()) + 4 * x.abs() + 8)
        x = x.masked_fill(~m, -math.inf)
        lse = torch.logsumexp(x, 1)
        p = torch.where(m, torch.exp(x - lse[:, None]), torch.zeros_like(x))
        err = torch.where(m, err, torch.zeros_like(x))
        return q, k, v, do, m, p, lse, err

    def check_forward(self):
        u = UNIT[self.dt]
        for b in range(self.n):
            for h in range(self.hq):
                q, k, v, do, m, p, lse, err = self.one(b, h)
                o = p @ v
                worst = err.amax(1, keepdim=True)  # of the row's scores, in the sum as well
                # fp16 has fixed steps below 2^-14: a small probability (as a share of the largest, which may be up
                # to 2^8 above the running maximum) loses up to half of one
                top = p.amax(1, keepdim=True)
                slack = (u * p + (2.2 * worst + (self.tk + 8) * U24) * p + TINY[self.dt] * top * m) @ v.abs()
                assert_within(self.o[b, :, h], o, slack, "o[%d, :, %d]" % (b, h))
                got = self.lse[b, h].double()
                none = ~m.any(1)
                assert bool((got[none] == -math.inf).all()) and bool((self.o[b, none, h] == 0).all())
                off = (got - lse)[~none].abs()
                bound = (worst[:, 0] + (self.tk + 16) * U24 + 4 * U24 * lse.abs())[~none]
                assert bool((off <= bound).all()), "lse: off by %g of %g" % tuple(
                    float(x) for x in ((off / bound).max(), bound.max()))

    def check_backward(self, outs):
        u, t = UNIT[self.dt], TINY[self.dt]
        for b in range(self.n):
            for hk in range(self.hk):
                sums = [torch.zeros((self.tk, self.d), dtype=torch.float64, device="cuda:0") for _ in range(4)]
                for h in range(hk * (self.hq // self.hk), (hk + 1) * (self.hq // self.hk)):
                    q, k, v, do, m, p, lse, err = self.one(b, h)
                    dp = do @ v.t()
                    delta = (p * dp).sum(1, keepdim=True)
                    ds = p * (dp - delta)
                    o = p @ v
                    worst = err.amax(1, keepdim=True) + (self.tk + 16) * U24
                    # what o, as the forward pass rounds it and its probabilities, is off by
                    off = u * (p @ v.abs()) + u * o.abs() + 4 * worst * (p @ v.abs()) + t
                    ddelta = (do.abs() * off).sum(1, keepdim=True)
                    mag = do.abs() @ v.abs().t()
                    pe = (2 * worst + 4 * U24) * p
                    de = pe * (dp - delta).abs() + p * (ddelta + (self.d + 8) * U24 * (mag + (do.abs() * o.abs()).sum(1, keepdim=True)))
                    if outs[0] is not None:
                        slack = self.s * (((u + (self.tk + 8) * U24) * ds.abs() + de + t * m) @ k.abs())
                        assert_within(outs[0][b, :, h], self.s * (ds @ k), slack, "dq[%d, :, %d]" % (b, h))
                    n = (self.tq * (self.hq // self.hk) + 8) * U24
                    sums[0] += self.s * (ds.t() @ q)
                    sums[1] += self.s * (((u + n) * ds.abs() + de + t * m).t() @ q.abs())
                    sums[2] += p.t() @ do
                    sums[3] += ((u + n) * p + pe + t * m).t() @ do.abs()
                if outs[1] is not None:
                    assert_within(outs[1][b, :, hk], sums[0], sums[1], "dk[%d, :, %d]" % (b, hk))
                if outs[2] is not None:
                    assert_within(outs[2][b, :, hk], sums[2], sums[3], "dv[%d, :, %d]" % (b, hk))


CASES = [
    dict(tq=1, tk=1), dict(tq=1, tk=1, dtype="fp16", d=8), dict(tq=1, tk=257, hq=4, hk=1, d=128),
    dict(n=3, tq=1, tk=1000, hq=8, hk=2, d=80, dtype="fp16"), dict(tq=7, tk=33, hq=2, hk=1, d=40),
    dict(tq=33, tk=31, d=32), dict(tq=64, tk=64, dtype="fp16"), dict(tq=65, tk=129, d=96),
    dict(tq=257, tk=255, d=128, hq=4, hk=2), dict(tq=300, tk=300, d=72, frame=1, dtype="fp16"),
    dict(tq=300, tk=300, d=128, frame=1, layout="fused"), dict(tq=320, tk=320, frame=64, d=64),
    dict(tq=250, tk=250, frame=25, window=1, layout="heads"), dict(tq=250, tk=250, frame=25, window=3, d=128, dtype="fp16"),
    dict(tq=600, tk=600, frame=1, window=100, hq=4, hk=1, d=64), dict(tq=100, tk=400, frame=50, q_offset=300),
    dict(tq=100, tk=400, frame=1, tail=True, d=24), dict(tq=100, tk=100, frame=1, q_offset=-30),
    dict(tq=90, tk=60, frame=7, q_offset=200, window=2), dict(tq=90, tk=60, frame=1000000, q_offset=1 << 30),
    dict(n=4, tq=130, tk=200, lengths=[(130, 200), (0, 77), (61, 0), (128, 64)], d=80),
    dict(n=3, tq=300, tk=300, lengths=[(300, 300), (1, 1), (177, 177)], frame=1, hq=6, hk=2, dtype="fp16", layout="heads"),
    dict(n=3, tq=40, tk=500, lengths=[(40, 500), (40, 20), (9, 333)], frame=1, tail=True, d=128),
    dict(n=5, tq=1, tk=900, lengths=[(1, 900), (1, 0), (0, 5), (1, 1), (1, 513)], frame=1, tail=True, hq=8, hk=2, d=128),
    dict(n=2, tq=50, tk=70, lengths=[(1000, 1000), (-3, -5)], d=64),
    dict(tq=70, tk=90, layout="gaps", hq=3, hk=3, d=56), dict(tq=200, tk=200, spread=4.0, d=64, dtype="fp16"),
    dict(tq=200, tk=200, spread=6.0, d=128), dict(tq=64, tk=100, scale=0.5, d=16),
    dict(tq=5, tk=4000, hq=1, hk=1, d=128, dtype="fp16"), dict(tq=40, tk=5000, hq=1, hk=1, d=64),
    dict(tq=700, tk=3, hq=2, hk=1, d=64), dict(tq=2100, tk=2000, hq=1, hk=1, d=128, frame=333),
]


def ident(c):
    return "-".join("%s=%s" % (k, v if k != "lengths" else "given") for k, v in c.items())


@pytest.mark.parametrize("splits,together", [(1, 0), (3, 0), (1, 1), (4, 1)])
@pytest.mark.parametrize("tile", ["attention_64x128", "attention_128x128", "attention_256x64"])
@pytest.mark.parametrize("case", [c for c in CASES if c.get("tq", 64) > 1 and c.get("tk", 64) > 40], ids=ident)
def test_every_tile_and_pieces(case, tile, splits, together, monkeypatch):
    monkeypatch.setenv("CONV3D_ATTENTION_TOGETHER", str(together))
    monkeypatch.setenv("CONV3D_ATTENTION_TILE", tile)
    monkeypatch.setenv("CONV3D_ATTENTION_SPLITS", str(splits))
    c = Case(**case)
    assert c.plan.info().kernel_name.decode() == tile
    c.forward()
    c.check_forward()
    c.check_backward(c.backward())


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_forward_and_gradients(case):
    c = Case(**case)
    c.forward()
    c.check_forward()
    outs = c.backward()
    c.check_backward(outs)


@pytest.mark.parametrize("scale", [2.0 ** -64, 2.0 ** -10, 2.0])
@pytest.mark.parametrize("d,tk", [(64, 90), (128, 300)])
def test_scales_far_from_the_usual(d, tk, scale):
    c = Case(tq=80, tk=tk, hq=4, hk=2, d=d, scale=scale)
    c.forward()
    c.check_forward()
    c.check_backward(c.backward())


def l2(a, b):
    """Relative, beyond what the result's own rounding below fp16's normal numbers allows: half of 2^-24 for each
    element (dk of the first case below is 1e-5, where fp16's steps are 2^-24 = 6e-8)."""
    return max(0.0, float((a.double() - b).norm()) - 2.0 ** -25 * a.numel() ** 0.5) / float(b.norm())


@pytest.mark.parametrize("tile", ["attention_64x128", "attention_128x128", "attention_256x64"])
@pytest.mark.parametrize("dout,vs,ks", [(0.05, 0.05, 8.0), (200.0, 4.0, 1.0), (0.05, 1.0, 1.0)])
def test_fp16_gradients_of_any_size_keep_their_digits(dout, vs, ks, tile, monkeypatch):
    # dS between 1e-7 (below fp16's normal numbers) and 1e4 (their products' scales overflow them): P and dS round
    # once each, and the result once; three roundings of at most 2^-11
    monkeypatch.setenv("CONV3D_ATTENTION_TILE", tile)
    c = Case(tq=4096, tk=4096, hq=1, hk=1, d=64, dtype="fp16", seed=5)
    g = gen(77)
    c.k, c.v, c.do = (normal(g, x.shape, c.dt, s) for x, s in ((c.k, ks), (c.v, vs), (c.do, dout)))
    c.q = normal(g, c.q.shape, c.dt, 1.0 / ks)
    c.forward()
    dq, dk, dv = c.backward()
    q, k, v, do, m, p, lse, err = c.one(0, 0)
    dp = do @ v.t()
    ds = p * (dp - (p * dp).sum(1, keepdim=True))
    want = c.s * (ds @ k), c.s * (ds.t() @ q), p.t() @ do
    for name, got, ref in zip(("dq", "dk", "dv"), (dq, dk, dv), want):
        ref = torch.where(ref.abs() > 65504.0, torch.full_like(ref, math.inf) * ref.sign(), ref)
        fits = torch.isfinite(ref)
        assert l2(got[0, :, 0][fits], ref[fits]) < 3 * 2.0 ** -11, name


def test_fp16_gradients_whose_size_grows_on_the_way():
    # the last keys' and queries' dS are 2^20 times the first ones': sums so far are scaled down, nothing overflows
    c = Case(tq=700, tk=900, hq=2, hk=1, d=64, dtype="fp16", seed=6)
    ramp = torch.exp2(torch.arange(900, device="cuda:0") / 900 * 10).half()
    c.v = (c.v * ramp[None, :, None, None]).contiguous()
    c.do = (c.do * 0.1 * ramp[None, :700, None, None]).contiguous()
    c.forward()
    dq, dk, dv = c.backward()
    sums = [0.0] * 2
    for h in range(2):
        q, k, v, do, m, p, lse, err = c.one(0, h)
        dp = do @ v.t()
        ds = p * (dp - (p * dp).sum(1, keepdim=True))
        # row by row: each has a scale of its own
        ref = c.s * (ds @ k)
        assert float(((dq[0, :, h].double() - ref).norm(dim=1) / ref.norm(dim=1)).max()) < 2.0 ** -7
        sums[0] = sums[0] + c.s * (ds.t() @ q)
        sums[1] = sums[1] + p.t() @ do
    assert l2(dk[0, :, 0], sums[0]) < 4 * 2.0 ** -11 and l2(dv[0, :, 0], sums[1]) < 3 * 2.0 ** -11
