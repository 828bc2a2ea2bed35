"""Attention as programs use it: captured and replayed, on several streams, token by token and frame by frame
against a cache, inside larger buffers, over offsets past 2^31 elements; its gradients against differences."""
import math

import pytest
import torch

import convolution_implicit_gemm_amd as c3d
from test_gpu_attention import Case
from token_helpers import gen, normal, scratch

pytestmark = pytest.mark.gpu


def workspace(plan):
    return scratch(max(plan.workspace_bytes, c3d.attention_backward_workspace(plan)))


@pytest.mark.parametrize("case", [
    dict(n=2, tq=150, tk=150, hq=4, hk=2, frame=30, lengths=[(150, 150), (77, 77)]),
    dict(n=2, tq=1, tk=3000, hq=8, hk=2, d=128, frame=1, tail=True, lengths=[(1, 3000), (1, 1)], dtype="fp16"),
    dict(tq=60, tk=2500, hq=2, hk=1, d=80)])
def test_captured_and_replayed(case):
    c = Case(**case)
    ws = workspace(c.plan)
    grads = [torch.empty_like(x) for x in (c.q, c.k, c.v)]

    def both(o, lse, g):
        c3d.attention_forward(c.plan, c.q, c.k, c.v, o, lse, c.len, 0, ws)
        c3d.attention_backward(c.plan, c.do, c.q, c.k, c.v, o, lse, *g, c.len, 0, ws)

    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        both(c.o, c.lse, grads)
    torch.cuda.current_stream().wait_stream(s)
    for step in range(4):
        eager_o, eager_lse, eager = torch.empty_like(c.o), torch.empty_like(c.lse), [torch.empty_like(x) for x in grads]
        graph.replay()
        torch.cuda.synchronize()
        both(eager_o, eager_lse, eager)
        for x, y in zip([c.o, c.lse] + grads, [eager_o, eager_lse] + eager):
            assert torch.equal(x, y), "replay %d" % step
        c.q.mul_(0.5)
        c.k[:, :1].add_(0.25)
        if c.len is not None:  # the lengths are read when the graph runs
            c.len[0, 1] -= 7


def test_streams_with_workspaces_of_their_own():
    a, b = Case(tq=1, tk=20000, hq=8, hk=2, d=128, seed=1), Case(tq=400, tk=400, hq=4, hk=4, d=64, frame=1, seed=2)
    want = []
    for c in (a, b):
        c.forward()
        want.append((c.o.clone(), c.lse.clone(), [x.clone() for x in c.backward()]))
        c.o.fill_(3.0)
        c.lse.fill_(3.0)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [workspace(c.plan) for c in (a, b)]
    outs = [[torch.empty_like(x) for x in (c.q, c.k, c.v)] for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, ws, g in zip((a, b), streams, spaces, outs):
            c3d.attention_forward(c.plan, c.q, c.k, c.v, c.o, c.lse, workspace=ws, stream=s)
            c3d.attention_backward(c.plan, c.do, c.q, c.k, c.v, c.o, c.lse, *g, workspace=ws, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for c, g, (o, lse, grads) in zip((a, b), outs, want):
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse) and all(torch.equal(x, y) for x, y in zip(g, grads))


def test_results_do_not_vary_from_call_to_call():
    c = Case(n=2, tq=900, tk=900, hq=6, hk=2, d=96, frame=1)
    first = None
    for _ in range(4):
        c.forward()
        now = [c.o.clone(), c.lse.clone()] + [x.clone() for x in c.backward()]
        first = first or now
        assert all(torch.equal(x, y) for x, y in zip(first, now))


@pytest.mark.parametrize("skip", [(0,), (1,), (2,), (1, 2), (0, 1), (0, 2)])
def test_gradients_that_are_not_asked_for(skip):
    c = Case(tq=130, tk=170, hq=4, hk=2, d=64)
    c.forward()
    whole = c.backward()
    part = c.backward(*[i not in skip for i in range(3)])
    for i, (x, y) in enumerate(zip(whole, part)):
        assert y is None if i in skip else torch.equal(x, y)


def test_tokens_one_by_one_and_frames_one_by_one():
    hq, hk, d, frame, frames = 8, 2, 64, 24, 5
    t = frame * frames
    g = gen(4)
    q, k, v = normal(g, (1, t, hq, d), torch.bfloat16), normal(g, (1, t, hk, d), torch.bfloat16), normal(g, (1, t, hk, d), torch.bfloat16)

    def run(tq, tk, fr, qq, offset, o):
        p = c3d.attention_plan(c3d.make_attention_desc(1, tq, tk, hq, hk, d, frame=fr, flags=c3d.CONV3D_F_BF16))
        c3d.attention_forward(p, qq, k[:, :tk].contiguous(), v[:, :tk].contiguous(), o, q_offset=offset,
                              workspace=scratch(p.workspace_bytes))

    whole, parts = torch.empty_like(q), torch.empty_like(q)
    for fr in (1, frame):
        run(t, t, fr, q, 0, whole)
        for i in range(0, t, fr):
            o = torch.empty((1, fr, hq, d), dtype=q.dtype, device=q.device)
            run(fr, i + fr, fr, q[:, i:i + fr].contiguous(), i, o)
            parts[:, i:i + fr] = o
        # both round probabilities and the result: four halves of a step, of values up to the largest |v|
        assert float((whole.double() - parts.double()).abs().max()) <= 4 * 2.0 ** -8 * float(v.abs().max())


def test_ragged_cache_buffers_longer_than_their_samples():
    # serving: room for 512 tokens a sample, fewer in use, the new token at each sample's end; what the room holds
    # behind them is never read
    n, hq, hk, d, room = 3, 8, 2, 128, 512
    g = gen(9)
    used = [1, 300, 512]
    k, v = (torch.full((n, room, hk, d), float("nan"), dtype=torch.float16, device="cuda:0") for _ in range(2))
    for b, u in enumerate(used):
        k[b, :u], v[b, :u] = normal(g, (u, hk, d), torch.float16), normal(g, (u, hk, d), torch.float16)
    q, o = normal(g, (n, 1, hq, d), torch.float16), torch.empty((n, 1, hq, d), dtype=torch.float16, device="cuda:0")
    p = c3d.attention_plan(c3d.make_attention_desc(n, 1, room, hq, hk, d, frame=1,
                                                   flags=c3d.CONV3D_F_LENGTHS | c3d.CONV3D_F_TAIL))
    lens = torch.tensor([[1, u] for u in used], dtype=torch.int32, device="cuda:0")
    c3d.attention_forward(p, q, k, v, o, None, lens, 0, scratch(p.workspace_bytes))
    for b, u in enumerate(used):
        for h in range(hq):
            kk, vv = k[b, :u, h // 4].double(), v[b, :u, h // 4].double()
            ref = torch.softmax(q[b, 0, h].double() @ kk.t() / math.sqrt(d), 0) @ vv
            # probabilities and the result round once each, 2^-11 of values up to the largest |v|
            assert float((o[b, 0, h].double() - ref).abs().max()) <= 3 * 2.0 ** -11 * float(vv.abs().max())


@pytest.mark.parametrize("frame, window", [(1, 0), (1, 40), (7, 0)])
@pytest.mark.parametrize("kind", ["", "attention_64x128", "attention_128x128", "attention_256x64"])
@pytest.mark.parametrize("tq, room, at", [(1, 300, 0), (1, 3000, 1777), (5, 300, 41), (70, 517, 130), (300, 700, 100)])
def test_caches_hold_anything_behind_what_the_call_sees(tq, room, at, kind, frame, window, monkeypatch):
    if kind:
        monkeypatch.setenv("CONV3D_ATTENTION_TILE", kind)
    hq, hk, d = 4, 2, 64
    seen = min(((at + tq - 1) // frame + 1) * frame, room)
    g = gen(13)
    q, k, v = (normal(g, (1, t, h, d), torch.bfloat16) for t, h in ((tq, hq), (room, hk), (room, hk)))
    desc = c3d.make_attention_desc(1, tq, room, hq, hk, d, frame=frame, window=window, flags=c3d.CONV3D_F_BF16)
    p = c3d.attention_plan(desc)
    outs = []
    for fill in (0.0, float("nan"), float("inf")):
        k[:, seen:] = v[:, seen:] = fill
        outs.append(torch.empty_like(q))
        c3d.attention_forward(p, q, k, v, outs[-1], q_offset=at, workspace=scratch(p.workspace_bytes))
    assert not torch.isnan(outs[0]).any()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_outputs_leave_what_lies_around_them():
    n, t, hq, hk, d = 2, 70, 3, 1, 40
    g = gen(5)
    q, k, v, do = (normal(g, (n, t, h, d), torch.bfloat16) for h in (hq, hk, hk, hq))

    def room(h):
        buf = torch.full((n, t + 3, h + 2, d + 16), 12.5, dtype=torch.bfloat16, device="cuda:0")
        return buf, buf[:, 1:t + 1, 1:h + 1, 8:d + 8]

    bufs, views = zip(*(room(h) for h in (hq, hq, hk, hk)))
    o, dq, dk, dv = views
    st = {"o": o.stride()[:3], "q": dq.stride()[:3], "k": dk.stride()[:3]}

    def plan(**kw):
        return c3d.attention_plan(c3d.make_attention_desc(n, t, t, hq, hk, d, frame=7, flags=c3d.CONV3D_F_BF16, **kw))

    p = plan(o_stride=st["o"])
    lse = torch.full((n * hq * t + 16,), 12.5, device="cuda:0")
    c3d.attention_forward(p, q, k, v, o, lse[8:-8], workspace=scratch(p.workspace_bytes))
    assert bool((lse[:8] == 12.5).all()) and bool((lse[-8:] == 12.5).all())
    # the gradients take the strides of q, k and v: inputs laid out like them
    qq, kk, vv = (room(h)[1].copy_(x) for h, x in ((hq, q), (hk, k), (hk, v)))
    p2 = plan(q_stride=st["q"], k_stride=st["k"], v_stride=st["k"], o_stride=st["o"])
    dd = room(hq)[1].copy_(do)
    c3d.attention_backward(p2, dd, qq, kk, vv, o, lse[8:-8], dq, dk, dv, workspace=scratch(c3d.attention_backward_workspace(p2)))
    for buf, view in zip(bufs, views):
        assert bool(torch.isfinite(view.float()).all())
        inside = torch.zeros_like(buf, dtype=torch.bool)
        inside[:, 1:t + 1, 1:view.shape[2] + 1, 8:d + 8] = True
        assert bool((buf[~inside] == 12.5).all())


def test_offsets_past_32_bits():
    # rows 2^20 elements apart, 2200 of them: 2.3e9 elements from the first to the last
    d, tk, stride = 64, 2200, 1 << 20
    g = gen(6)
    buf = torch.empty(((tk - 1) * stride + 256,), dtype=torch.float16, device="cuda:0")

    def at(o):
        return buf.as_strided((1, tk, 1, d), (tk * stride, stride, d, 1), o)

    k, v = normal(g, (1, tk, 1, d), torch.float16), normal(g, (1, tk, 1, d), torch.float16)
    q, do = normal(g, (1, 300, 2, d), torch.float16), normal(g, (1, 300, 2, d), torch.float16)
    st = (tk * stride, stride, d)
    far = c3d.attention_plan(c3d.make_attention_desc(1, 300, tk, 2, 1, d, frame=1, k_stride=st, v_stride=st))
    near = c3d.attention_plan(c3d.make_attention_desc(1, 300, tk, 2, 1, d, frame=1))
    ws = scratch(max(far.workspace_bytes, c3d.attention_backward_workspace(far)))
    at(0).copy_(k)
    at(64).copy_(v)
    o, o2, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((1, 2, 300), device="cuda:0")
    one = c3d.attention_plan(c3d.make_attention_desc(1, 1, tk, 2, 1, d, frame=1, k_stride=st, v_stride=st))
    ones = [torch.empty((1, 1, 2, d), dtype=q.dtype, device=q.device) for _ in range(2)]
    off = tk - 300
    c3d.attention_forward(far, q, at(0), at(64), o, lse, None, off, ws)
    c3d.attention_forward(near, q, k, v, o2, lse, None, off, ws)
    assert torch.equal(o, o2)
    c3d.attention_forward(one, q[:, -1:].contiguous(), at(0), at(64), ones[0], None, None, tk - 1, scratch(one.workspace_bytes))
    assert float((ones[0].float() - o[:, -1:].float()).abs().max()) <= 4 * 2.0 ** -11 * float(v.abs().max())
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    c3d.attention_backward(near, do, q, k, v, o, lse, dq, dk, dv, None, off, ws)
    dq2 = torch.empty_like(q)
    c3d.attention_backward(far, do, q, at(0), at(64), o, lse, dq2, at(128), at(192), None, off, ws)
    assert torch.equal(dq, dq2) and torch.equal(at(128), dk) and torch.equal(at(192), dv)


@pytest.mark.parametrize("case", [dict(tq=90, tk=110, hq=4, hk=2, d=40), dict(tq=128, tk=128, frame=16, window=2, d=64)])
def test_gradients_against_differences(case):
    c = Case(dtype="fp16", **case)
    c.forward()
    grads = c.backward()
    g = gen(31)
    rep = c.hq // c.hk
    mask = None
    if c.frame:
        from test_gpu_attention import seen_mask
        mask = seen_mask(c.tq, c.tk, c.tq, c.tk, c.frame, c.window, 0, False)

    def loss(q, k, v):
        x = q.transpose(1, 2) @ k.repeat_interleave(rep, 2).permute(0, 2, 3, 1) * c.s
        if mask is not None:
            x = x.masked_fill(~mask, -math.inf)
        return (torch.softmax(x, -1) @ v.repeat_interleave(rep, 2).transpose(1, 2)).transpose(1, 2).mul(c.do.double()).sum()

    x = [t.double() for t in (c.q, c.k, c.v)]
    for i in range(3):
        u = torch.randn(x[i].shape, generator=g, device="cuda:0", dtype=torch.float64)
        h = 1e-4
        up, down = ([t + (sign * h * u if j == i else 0.0) for j, t in enumerate(x)] for sign in (1, -1))
        slope = float(loss(*up) - loss(*down)) / (2 * h)
        got = float((grads[i].double() * u).sum())
        # each element of the gradient is off by about 2^-10 of the gradients' size, in any direction; 6 deviations
        size = float(grads[i].double().norm())
        assert abs(got - slope) <= 6 * 2.0 ** -10 * size + 1e-6
