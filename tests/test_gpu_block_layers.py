"""A conditioned block of a video transformer as its parts are used together:
norm and modulation, the projections, cross attention to a text, the gated
residual and the next norm; forward, backward, and captured into a graph."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

B, N, C, H, D, M, CT = 2, 336, 256, 4, 64, 77, 192


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


def inputs(dt=torch.bfloat16):
    g = torch.Generator().manual_seed(0)

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()

    p = dict(x=normal(B, N, C), text=normal(B, M, CT), mod=normal(B, 6 * C, std=0.3),
             wq=normal(H * D, C, std=C ** -0.5), wkv=normal(2 * H * D, CT, std=CT ** -0.5), wo=normal(C, H * D, std=(H * D) ** -0.5),
             w3=normal(C, std=0.1, dtype=torch.float32) + 1)
    p["len"] = torch.tensor([77, 20], dtype=torch.int32, device="cuda")
    return p


def forward(p):
    """(out of the next norm, the residual stream, what the backward pass needs)."""
    fw = _fw()
    shift1, scale1, gate, shift2, scale2, _ = p["mod"].split(C, -1)
    y1, _ = fw.wsattn_block_norm(p["x"], scale=scale1, shift=shift1)
    q = fw.wsattn_linear(y1, p["wq"]).view(B, N, H, D).transpose(1, 2)
    kv = fw.wsattn_linear(p["text"], p["wkv"]).view(B, M, 2, H, D).permute(2, 0, 3, 1, 4)
    lse = torch.empty((B, H, N), device="cuda")
    att = fw.wsattn_cross(q, kv[0], kv[1], k_lengths=p["len"], lse=lse)
    o = fw.wsattn_linear(att.transpose(1, 2).flatten(2), p["wo"])
    y2, h = fw.wsattn_block_norm(o, p["x"], gate=gate, scale=scale2, shift=shift2, weight=p["w3"], norm="rms")
    return y2, h, (y1, q, kv, lse, att, o)


def backward(p, saved, h, dy):
    fw = _fw()
    y1, q, kv, lse, att, o = saved
    _, scale1, gate, _, scale2, _ = p["mod"].split(C, -1)
    g2 = fw.wsattn_block_norm_backward(dy, h, o, gate=gate, scale=scale2, weight=p["w3"], norm="rms")
    datt, dwo, _ = fw.wsattn_linear_backward(g2.dx, att.transpose(1, 2).flatten(2), p["wo"], need_db=False)
    dkv = torch.empty((B, M, 2, H, D), dtype=dy.dtype, device="cuda")
    t = dkv.permute(2, 0, 3, 1, 4)
    dq, _, _ = fw.wsattn_cross_backward(datt.view(B, N, H, D).transpose(1, 2), q, kv[0], kv[1], att, lse, k_lengths=p["len"], dk=t[0], dv=t[1])
    dy1, dwq, _ = fw.wsattn_linear_backward(dq.transpose(1, 2).flatten(2), y1, p["wq"], need_db=False)
    dtext, dwkv, _ = fw.wsattn_linear_backward(dkv.flatten(2), p["text"], p["wkv"], need_db=False)
    g1 = fw.wsattn_block_norm_backward(dy1, p["x"], dhidden=g2.dresidual, scale=scale1)
    return dict(x=g1.dx, text=dtext, wq=dwq, wkv=dwkv, wo=dwo, w3=g2.dweight,
                mod=torch.cat((g1.dshift, g1.dscale, g2.dgate, g2.dshift, g2.dscale), -1))


def plain(p):
    """The same block in 64 bits; (out, residual stream)."""
    x, text, mod = p["x"], p["text"], p["mod"]
    shift1, scale1, gate, shift2, scale2, _ = (t[:, None] for t in mod.split(C, -1))
    n = (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, correction=0, keepdim=True) + 1e-6)
    q = ((n * (1 + scale1) + shift1) @ p["wq"].T).view(B, N, H, D).transpose(1, 2)
    k, v = (text @ p["wkv"].T).view(B, M, 2, H, D).permute(2, 0, 3, 1, 4)
    s = (q @ k.transpose(2, 3) / math.sqrt(D)).masked_fill(torch.arange(M, device="cuda") >= p["len"][:, None, None, None], -math.inf)
    o = (torch.softmax(s, -1) @ v).transpose(1, 2).flatten(2) @ p["wo"].T
    h = x + gate * o
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * p["w3"] * (1 + scale2) + shift2, h


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def check(p, y, h, grads, dy):
    d = {k: v.double().requires_grad_() if k != "len" else v for k, v in p.items()}
    wy, wh = plain(d)
    # a result passes through at most eight roundings to bf16 (half a step, 2^-8 relative, each) before its own, and their errors
    # are not aligned: 2^-8 sqrt(9) would be typical for the largest, 2^-6 is above it
    assert rel(y, wy) < 2.0 ** -6 and rel(h, wh) < 2.0 ** -6
    names = [k for k in grads]
    want = torch.autograd.grad(wy, [d[k] for k in names], dy.double())
    for k, w in zip(names, want):
        if k == "mod":
            w = w[:, :5 * C]
        assert grads[k].shape == w.shape and rel(grads[k], w) < 2.0 ** -5, (k, rel(grads[k], w))


def test_block_forward_and_backward():
    p = inputs()
    y, h, saved = forward(p)
    dy = torch.randn(y.shape, generator=torch.Generator().manual_seed(1)).to(y.dtype).cuda()
    check(p, y, h, backward(p, saved, h, dy), dy)
    assert _fw().wsattn_op_status() == 0


def test_block_in_a_graph():
    p = inputs()
    dy = torch.randn(B, N, C, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm-up, as a capture wants it
        y, h, saved = forward(p)
        backward(p, saved, h, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h, saved = forward(p)
        grads = backward(p, saved, h, dy)
    for seed in range(2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        p["x"].normal_(generator=g)
        p["text"].normal_(generator=g)
        p["len"].copy_(torch.tensor([33, 77 - seed]))
        dy.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        check(p, y, h, grads, dy)
    assert _fw().wsattn_op_status() == 0


def test_two_streams_at_once():
    # the same calls on two streams, each with outputs and scratch of its own
    p, r = inputs(), inputs()
    dy = torch.randn(B, N, C, device="cuda").to(torch.bfloat16)
    y, h, saved = forward(p)
    want = backward(p, saved, h, dy)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for s, t in zip(streams, (p, r)):
        with torch.cuda.stream(s):
            for _ in range(3):
                y, h, saved = forward(t)
                got.append(backward(t, saved, h, dy))
    torch.cuda.synchronize()
    for g in got:
        for k in want:
            assert torch.equal(g[k], want[k]), k
