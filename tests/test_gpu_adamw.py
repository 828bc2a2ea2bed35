"""The AdamW step against its formula in 64 bits, fp32 and 8-bit states.

Bounds: every fp32 coefficient and operation is off by 2^-24 of its value; m is a sum of
two products (at most four such steps to each), v of two with a square (six), the update's quotient
adds the square root's half of v's error and six steps.  A 16-bit weight rounds once
more.  An 8-bit state is off by at most half a step of e4m3 at its block's scale.
"""
import pytest
import torch

import convolution_implicit_gemm_amd as c3d
from token_helpers import DTYPES, U24, assert_within, gen

pytestmark = pytest.mark.gpu

B = c3d.ADAMW_BLOCK


def decode(codes, scale):
    """Values of 8-bit states in 64 bits (of sqrt(v), for v)."""
    n = codes.numel()
    x = codes.view(torch.float8_e4m3fn).to(torch.float32).double()
    s = torch.exp2(scale.double() - 127).repeat_interleave(B)[:n]
    return x * s


def half_step(y):
    """Half an e4m3 step at y (a value over its block's power of two)."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e - 4)


class Tensors:
    def __init__(self, sizes, dtype="bf16", master=True, param=True, grad32=False, state8=False, seed=1, spread=2.0):
        g = gen(seed)
        dt = DTYPES[dtype]

        def normal(n, s=1.0):
            return torch.randn(n, generator=g, device="cuda:0") * s

        self.state8, self.sizes = state8, sizes
        self.grads, self.params, self.master, self.m, self.v, self.ms, self.vs = [], [], [], [], [], [], []
        for n in sizes:
            size = torch.exp(normal(1) * spread) * 1e-2
            w = normal(n, 0.1)
            self.grads.append((normal(n) * size).to(torch.float32 if grad32 else dt))
            self.params.append(w.to(dt) if param else None)
            self.master.append(w.clone() if master else None)
            if state8:
                # codes of every kind but NaN; scales that give m and sqrt(v) of the gradient's size
                blocks = -(-n // B)
                code = torch.randint(0, 127, (n,), generator=g, device="cuda:0")
                sign = torch.randint(0, 2, (n,), generator=g, device="cuda:0") * 128
                self.m.append((code + sign).to(torch.uint8))
                self.v.append(torch.randint(0, 127, (n,), generator=g, device="cuda:0").to(torch.uint8))
                self.ms.append(torch.randint(108, 114, (blocks,), generator=g, device="cuda:0").to(torch.uint8))
                self.vs.append(torch.randint(108, 114, (blocks,), generator=g, device="cuda:0").to(torch.uint8))
            else:
                self.m.append(normal(n) * size)
                self.v.append(normal(n).square() * size.square())
        self.decay = [float(i % 2) for i in range(len(sizes))]

    def list(self):
        return c3d.adamw_list(self.params if any(x is not None for x in self.params) else None, self.grads, self.m, self.v,
                              master=self.master, m_scale=self.ms if self.state8 else None,
                              v_scale=self.vs if self.state8 else None, decay=self.decay)

    def want(self, h, i):
        """(w, m, v or sqrt(v), their fp32 slacks) of tensor i in 64 bits, from the state as it is now."""
        x = self.grads[i].double() * h.grad_scale
        if self.state8:
            m, v = decode(self.m[i], self.ms[i]), decode(self.v[i], self.vs[i]).square()
        else:
            m, v = self.m[i].double(), self.v[i].double()
        a, b = h.beta1 * m, (1 - h.beta1) * x
        m, dm = a + b, 4 * U24 * (a.abs() + b.abs())
        v, dv = h.beta2 * v + (1 - h.beta2) * x * x, 6 * U24 * (h.beta2 * v + (1 - h.beta2) * x * x)
        w = (self.master[i] if self.master[i] is not None else self.params[i]).double()
        c1, c2 = 1 - h.beta1 ** h.step, 1 - h.beta2 ** h.step
        scale = h.lr / c1 / (torch.sqrt(v / c2) + h.eps)
        up = m * scale
        dw = 4 * U24 * (w.abs() + up.abs()) + dm * scale + up.abs() * 10 * U24
        w = w * (1 - h.lr * h.weight_decay * self.decay[i]) - up
        if self.state8:
            v = torch.sqrt(v)
            dv = 5 * U24 * v
        return w, m, v, dw, dm, dv

    def check(self, want, before=None):
        for i, (w, m, v, dw, dm, dv) in enumerate(want):
            if self.master[i] is not None:
                assert_within(self.master[i], w, dw, "master[%d]" % i)
            if self.params[i] is not None:
                assert_within(self.params[i], w, dw, "params[%d]" % i)
                if self.master[i] is not None:
                    assert torch.equal(self.params[i], self.master[i].to(self.params[i].dtype))
            if not self.state8:
                assert_within(self.m[i], m, dm, "m[%d]" % i)
                assert_within(self.v[i], v, dv, "v[%d]" % i)
                continue
            for what, codes, scale, x, dx in (("m", self.m[i], self.ms[i], m, dm), ("v", self.v[i], self.vs[i], v, dv)):
                n = x.numel()
                pad = -n % B
                top = torch.nn.functional.pad(x.abs(), (0, pad)).view(-1, B).amax(1)
                slack = torch.nn.functional.pad(dx, (0, pad)).view(-1, B).amax(1)
                unit = torch.exp2(scale.double() - 127)
                assert bool((top - slack <= 448 * unit).all()), "%s[%d]: a scale is too small" % (what, i)
                least = scale == 1  # 2^-126
                assert bool(((top + slack > 224 * unit) | least).all()), "%s[%d]: a scale is too large" % (what, i)
                u = unit.repeat_interleave(B)[:n]
                got = decode(codes, scale)
                tol = half_step(torch.maximum(x.abs(), got.abs()) / u) * u + dx
                if what == "v":
                    assert bool((got[x > 0] > 0).all()), "a positive sqrt(v) became 0"
                    tol = torch.where(got == 2.0 ** -9 * u, torch.maximum(tol, 2.0 ** -9 * u), tol)
                bad = (got - x).abs() > tol
                assert not bool(bad.any()), "%s[%d]: %d codes outside half a step" % (what, i, int(bad.sum()))


SIZES = [1, 7, 8, 9, 127, 128, 129, 1000, 2047, 2048, 2049, 5001, 70000]


@pytest.mark.parametrize("state8", [False, True])
@pytest.mark.parametrize("dtype,master,param,grad32", [
    ("bf16", True, True, False), ("fp16", True, True, True), ("bf16", False, True, False), ("fp16", False, True, True),
    ("bf16", True, False, True), ("fp16", True, False, False)])
def test_two_steps_match_the_formula(dtype, master, param, grad32, state8):
    t = Tensors(SIZES, dtype, master, param, grad32, state8)
    lst = t.list()
    for step in (1, 1000):
        h = c3d.make_adamw_hyper(1e-3, 0.9, 0.98, 1e-8, 0.1, step, grad_scale=0.25)
        want = [t.want(h, i) for i in range(len(SIZES))]
        c3d.adamw_step(lst, h)
        t.check(want)


@pytest.mark.parametrize("state8", [False, True])
def test_many_tensors_take_several_launches(state8):
    sizes = [(i * 7919) % 3001 + 1 for i in range(131)] + [0, 300000]
    t = Tensors(sizes, state8=state8)
    h = c3d.make_adamw_hyper(1e-2, step=3)
    want = [t.want(h, i) for i in range(len(sizes) - 2)]
    last = t.want(h, len(sizes) - 1)
    c3d.adamw_step(t.list(), h)
    for x in (t.params, t.master, t.m, t.v, t.ms, t.vs):
        del x[len(sizes) - 2:len(sizes) - 1]
    t.check(want + [last])


def test_one_large_tensor_takes_several_units_to_a_workgroup():
    t = Tensors([4096 * 2048 * 2 + 12345], state8=True)
    h = c3d.make_adamw_hyper(1e-3, step=7)
    want = [t.want(h, 0)]
    c3d.adamw_step(t.list(), h)
    t.check(want)


def test_neighbours_are_left_alone():
    # a tensor inside a larger buffer, its count no multiple of anything
    buf = torch.full((4096,), 3.0, device="cuda:0")
    code = torch.full((4096,), 17, dtype=torch.uint8, device="cuda:0")
    n, at = 333, 64
    g = torch.ones(n, device="cuda:0")
    m, v = (code.clone() for _ in range(2))
    ms, vs = (torch.full((16,), 100, dtype=torch.uint8, device="cuda:0") for _ in range(2))
    lst = c3d.adamw_list(None, [g], [m[at:at + n]], [v[at:at + n]], master=[buf[at:at + n]], m_scale=[ms[5:8]],
                         v_scale=[vs[5:8]])
    c3d.adamw_step(lst, c3d.make_adamw_hyper(1e-3))
    assert bool((buf[:at] == 3.0).all()) and bool((buf[at + n:] == 3.0).all()) and not bool((buf[at:at + n] == 3.0).any())
    for x in (m, v):
        assert bool((x[:at] == 17).all()) and bool((x[at + n:] == 17).all())
    for x in (ms, vs):
        assert bool((x[:5] == 100).all()) and bool((x[8:] == 100).all()) and not bool((x[5:8] == 100).any())


def test_zero_states_and_zero_gradients():
    n = 1000
    z8 = [torch.zeros(n, dtype=torch.uint8, device="cuda:0") for _ in range(2)]
    sc = [torch.zeros(8, dtype=torch.uint8, device="cuda:0") for _ in range(2)]
    w = torch.ones(n, device="cuda:0")
    lst = c3d.adamw_list(None, [torch.zeros(n, device="cuda:0")], z8[:1], z8[1:], master=[w], m_scale=sc[:1], v_scale=sc[1:])
    c3d.adamw_step(lst, c3d.make_adamw_hyper(0.5, weight_decay=0.0))
    assert bool((w == 1.0).all()) and bool((z8[0] == 0).all()) and bool((z8[1] == 0).all())


def test_a_gradient_that_is_not_finite_stays_with_its_element():
    n = 512
    g = torch.full((n,), 0.5, device="cuda:0")
    g[3], g[200], g[201] = float("nan"), float("inf"), float("-inf")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda:0") for _ in range(2))
    ms, vs = (torch.zeros(4, dtype=torch.uint8, device="cuda:0") for _ in range(2))
    w = torch.ones(n, device="cuda:0")
    c3d.adamw_step(c3d.adamw_list(None, [g], [m], [v], master=[w], m_scale=[ms], v_scale=[vs]), c3d.make_adamw_hyper(1e-2))
    bad = ~torch.isfinite(g)
    for x, s in ((m, ms), (v, vs)):
        got = decode(x, s)
        assert bool(torch.isnan(got[bad]).all()) and bool(torch.isfinite(got[~bad]).all()) and bool((got[~bad] > 0).all())
    assert not bool(torch.isfinite(w[bad]).any()) and bool(torch.isfinite(w[~bad]).all())


def test_hyperparameters_on_the_device_and_replays():
    a, b = Tensors([5000, 77], seed=3), Tensors([5000, 77], seed=3)
    la, lb = a.list(), b.list()
    hyper = torch.zeros(c3d.ADAMW_DEVICE_HYPER, device="cuda:0")
    steps = [c3d.make_adamw_hyper(1e-3 * k, step=k, grad_scale=1.0 / k) for k in range(1, 6)]
    hyper.copy_(torch.tensor(c3d.adamw_hyper_pack(steps[0])))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            c3d.adamw_step(la, hyper)
    torch.cuda.current_stream().wait_stream(s)
    for h in steps:
        hyper.copy_(torch.tensor(c3d.adamw_hyper_pack(h)))
        graph.replay()
        c3d.adamw_step(lb, h)
        torch.cuda.synchronize()
        for x, y in zip(a.params + a.master + a.m + a.v, b.params + b.master + b.m + b.v):
            assert torch.equal(x, y)


@pytest.mark.parametrize("state8", [False, True])
def test_states_have_the_bits_of_the_formula_in_fp32(state8):
    # products, sums and the root rounded one by one, as elementwise operations in fp32 round them
    t = Tensors([300000], state8=state8, grad32=True, seed=8)
    h = c3d.make_adamw_hyper(1e-3, 0.9, 0.98, 1e-8, 0.1, 5, grad_scale=0.3)
    x = t.grads[0] * h.grad_scale
    if state8:
        m, root = decode(t.m[0], t.ms[0]).float(), decode(t.v[0], t.vs[0]).float()
        v = root * root
    else:
        m, v = t.m[0].clone(), t.v[0].clone()
    m = m * h.beta1 + x * (1.0 - h.beta1)
    v = v * h.beta2 + x * x * (1.0 - h.beta2)
    c3d.adamw_step(t.list(), h)
    if not state8:
        assert torch.equal(t.m[0], m) and torch.equal(t.v[0], v)
        return
    for codes, scale, want in ((t.m[0], t.ms[0], m), (t.v[0], t.vs[0], torch.sqrt(v))):
        pad = torch.nn.functional.pad(want, (0, -len(want) % B)).view(-1, B)
        f, e = torch.frexp(pad.abs().amax(1))
        e = (e - 9 + (f > 0.875).int()).clamp(min=-126)  # 448 = 0.875 * 2^9
        assert torch.equal(scale.int(), e + 127)
        y = torch.ldexp(pad, -e[:, None]).flatten()[:len(want)]
        code = y.to(torch.float8_e4m3fn).float()
        if want is not m:
            code = torch.where((code == 0) & (y > 0), torch.full_like(code, 2.0 ** -9), code)
        assert torch.equal(codes.view(torch.float8_e4m3fn).float(), code)


@pytest.mark.parametrize("state8", [False, True])
def test_the_least_eps_divides_nothing_by_it(state8):
    n = 300
    kind = torch.uint8 if state8 else torch.float32
    m, v = (torch.zeros(n, dtype=kind, device="cuda:0") for _ in range(2))
    ms, vs = (torch.zeros(3, dtype=torch.uint8, device="cuda:0") for _ in range(2))
    w = torch.full((n,), 0.75, device="cuda:0")
    lst = c3d.adamw_list(None, [torch.zeros(n, device="cuda:0")], [m], [v], master=[w], m_scale=[ms] if state8 else None,
                         v_scale=[vs] if state8 else None)
    c3d.adamw_step(lst, c3d.make_adamw_hyper(1e-3, weight_decay=0.0, eps=2.0 ** -126))
    assert bool((w == 0.75).all())
