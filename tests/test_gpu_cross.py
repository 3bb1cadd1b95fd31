"""Attention to an encoder's states against the 64-bit definition: types, head
widths and layouts, lengths from none to many, what lies behind a length, other
streams, graphs; and its gradients, against the formulas and against differences."""
import pytest
import torch

import _block_ref as ref
from _ops_ref import assert_close

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


def make(seed, dt, b, h, hk, n, m, d, std=1.5, layout="packed"):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(dt).cuda()

    if layout == "packed":  # heads of projections
        q = normal(b, n, h, d, std=std).transpose(1, 2)
        kv = normal(b, m, 2 * hk, d).transpose(1, 2)
        return q, kv[:, :hk], kv[:, hk:]
    return normal(b, h, n, d, std=std), normal(b, hk, m, d), normal(b, hk, m, d)


def lens(values):
    return None if values is None else torch.tensor(values, dtype=torch.int32, device="cuda")


def spoil(k, v, lengths, m):
    """What lies behind a length must not matter."""
    if lengths is not None:
        for i, n in enumerate(lengths):
            n = max(0, min(n, m))
            k[i, :, n:] = float("nan")
            v[i, :, n:] = float("inf")
            v[i, :, n::2] = float("nan")


def check_forward(q, k, v, lengths, out, lse, scale=None):
    scale = q.shape[3] ** -0.5 if scale is None else scale
    o, tol, l, ltol = ref.cross_forward(q, k, v, lengths, scale)
    assert_close(out, o.cpu(), ref.rounded(tol, o, out.dtype).cpu(), "out")
    gone = torch.isinf(l)
    assert torch.equal(torch.isinf(lse) & (lse < 0), gone)
    zero = torch.zeros(())
    assert_close(lse.masked_fill(gone, 0), l.masked_fill(gone, 0).cpu(), ltol.cpu() + zero, "lse")


def check_backward(dout, q, k, v, out, lse, lengths, grads, scale=None):
    scale = q.shape[3] ** -0.5 if scale is None else scale
    want = ref.cross_backward(dout, q, k, v, out, lse, lengths, scale)
    for name, got in zip(("dq", "dk", "dv"), grads):
        if got is not None:
            w, tol = want[name]
            assert_close(got, w.cpu(), ref.rounded(tol, w, got.dtype).cpu(), name)


CASES = [
    # type, batch, heads, key heads, queries, keys, D, lengths, layout
    ("bf16", 1, 1, 1, 1, 1, 128, None, "packed"),
    ("bf16", 1, 8, 8, 1, 512, 128, None, "packed"),
    ("fp16", 1, 2, 2, 240, 77, 64, [41], "packed"),
    ("bf16", 2, 2, 1, 128, 128, 128, [128, 1], "plain"),
    ("bf16", 2, 2, 2, 129, 129, 64, [129, 128], "packed"),
    ("fp16", 3, 6, 2, 199, 333, 96, [0, 333, 17], "packed"),
    ("bf16", 2, 4, 4, 257, 512, 128, [511, 513], "packed"),
    ("bf16", 4, 3, 1, 65, 250, 16, [-3, 16, 240, 250], "plain"),
    ("fp16", 1, 5, 5, 300, 1000, 80, None, "plain"),
    ("bf16", 1, 3, 3, 700, 96, 32, [95], "packed"),
    ("bf16", 2, 16, 2, 7, 700, 128, [700, 300], "packed"),
    ("fp16", 1, 2, 1, 513, 384, 112, [257], "packed"),
    ("bf16", 1, 1, 1, 1500, 1, 48, None, "packed"),
    ("bf16", 1, 2, 2, 40, 6000, 128, [5555], "packed"),
    ("fp16", 1, 12, 3, 3, 9000, 64, None, "plain"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_cross(i):
    dt, b, h, hk, n, m, d, lengths, layout = CASES[i]
    q, k, v = make(i, T[dt], b, h, hk, n, m, d, layout=layout)
    spoil(k, v, lengths, m)
    lse = torch.empty((b, h, n), device="cuda")
    out = _fw().wsattn_cross(q, k, v, k_lengths=lens(lengths), lse=lse)
    assert out.transpose(1, 2).is_contiguous() and out.shape == q.shape
    check_forward(q, k, v, lens(lengths), out, lse)
    assert torch.equal(_fw().wsattn_cross(q, k, v, k_lengths=lens(lengths)), out)
    assert _fw().wsattn_op_status() == 0


@pytest.mark.parametrize("i", range(len(CASES)))
def test_cross_backward(i):
    dt, b, h, hk, n, m, d, lengths, layout = CASES[i]
    q, k, v = make(i + 50, T[dt], b, h, hk, n, m, d, layout=layout)
    spoil(k, v, lengths, m)
    lse = torch.empty((b, h, n), device="cuda")
    out = _fw().wsattn_cross(q, k, v, k_lengths=lens(lengths), lse=lse)
    dout = (torch.randn(b, n, h, d, generator=torch.Generator().manual_seed(i)) * 0.5).to(T[dt]).cuda().transpose(1, 2)
    args = (dout, q, k, v, out, lse)
    grads = _fw().wsattn_cross_backward(*args, k_lengths=lens(lengths))
    check_backward(*args, lens(lengths), grads)
    assert _fw().wsattn_op_status() == 0
    for x, y in zip(grads, _fw().wsattn_cross_backward(*args, k_lengths=lens(lengths))):
        assert torch.equal(x, y)  # fixed order of sums
    # one at a time
    for j in range(3):
        need = dict(need_dq=j == 0, need_dk=j == 1, need_dv=j == 2)
        got = _fw().wsattn_cross_backward(*args, k_lengths=lens(lengths), **need)
        assert [t is None for t in got] == [x != j for x in range(3)]
        assert torch.equal(got[j], grads[j])


def test_nothing_to_read_or_write():
    fw = _fw()
    for n, m in ((0, 5), (5, 0), (0, 0)):
        q, k, v = make(1, torch.bfloat16, 2, 4, 2, n, m, 64, layout="plain")
        lse = torch.full((2, 4, n), 3.0, device="cuda")
        out = fw.wsattn_cross(q, k, v, lse=lse)
        assert out.shape == q.shape and (out == 0).all() and torch.isinf(lse).all()
        dq, dk, dv = fw.wsattn_cross_backward(out, q, k, v, out, lse)
        assert (dq == 0).all() and (dk == 0).all() and (dv == 0).all() and dk.shape == k.shape
    q, k, v = make(1, torch.bfloat16, 0, 4, 2, 3, 3, 64, layout="plain")
    assert fw.wsattn_cross(q, k, v).shape == (0, 4, 3, 64)
    assert fw.wsattn_op_status() == 0


def test_logits_far_apart_and_scales():
    # maxima that grow from key to key, rows that one key takes, and a scale of the caller's
    fw = _fw()
    for std, scale in ((30.0, None), (0.01, None), (2.0, 1.0), (4.0, 0.003)):
        q, k, v = make(2, torch.bfloat16, 1, 2, 2, 150, 400, 64, std=std)
        k.mul_(torch.linspace(0.02, 3.0, 400, device="cuda", dtype=torch.bfloat16)[None, None, :, None])
        lse = torch.empty((1, 2, 150), device="cuda")
        out = fw.wsattn_cross(q, k, v, scale=scale, lse=lse)
        check_forward(q, k, v, None, out, lse, scale)
        dout = torch.randn_like(q)
        grads = fw.wsattn_cross_backward(dout, q, k, v, out, lse, scale=scale)
        check_backward(dout, q, k, v, out, lse, None, grads, scale)


def test_views_and_rows_beside_them():
    # slices of wider rows, a batch that shares its keys, outputs inside larger buffers
    fw = _fw()
    b, h, hk, n, m, d = 3, 4, 2, 140, 200, 64
    big = torch.randn(b, n + 9, 3 * h, d, device="cuda").to(torch.bfloat16)
    q = big[:, 4:4 + n, h:2 * h].transpose(1, 2)
    kv = torch.randn(1, m, 2 * hk, d, device="cuda").to(torch.bfloat16).transpose(1, 2)
    k, v = kv[:, :hk].expand(b, -1, -1, -1), kv[:, hk:].expand(b, -1, -1, -1)
    lse = torch.empty((b, h, n), device="cuda")
    buf = torch.full((b, h + 1, n + 30, d + 8), 7.0, device="cuda", dtype=torch.bfloat16)
    out = buf[:, 1:, 10:10 + n, :d]
    assert fw.wsattn_cross(q, k, v, lse=lse, out=out) is out
    check_forward(q, k, v, None, out, lse)
    rest = torch.ones(buf.shape, dtype=torch.bool, device="cuda")
    rest[:, 1:, 10:10 + n, :d] = False
    assert (buf[rest] == 7).all()
    dout = torch.randn(b, h, n, d, device="cuda").to(torch.bfloat16)
    bufs = [torch.full((b, x + 1, y + 30, d + 8), 7.0, device="cuda", dtype=torch.bfloat16) for x, y in ((h, n), (hk, m), (hk, m))]
    views = [t[:, 1:, 10:10 + y, :d] for t, y in zip(bufs, (n, m, m))]
    grads = fw.wsattn_cross_backward(dout, q, k, v, out, lse, dq=views[0], dk=views[1], dv=views[2])
    check_backward(dout, q, k, v, out, lse, None, grads)
    for t, y in zip(bufs, (n, m, m)):
        rest = torch.ones(t.shape, dtype=torch.bool, device="cuda")
        rest[:, 1:, 10:10 + y, :d] = False
        assert (t[rest] == 7).all()


def test_gradients_against_differences():
    fw = _fw()
    q, k, v = make(4, torch.bfloat16, 2, 4, 2, 37, 150, 32)
    lengths = lens([150, 40])
    lse = torch.empty((2, 4, 37), device="cuda")
    out = fw.wsattn_cross(q, k, v, k_lengths=lengths, lse=lse)
    g = torch.Generator().manual_seed(1)
    dout = torch.randn(2, 4, 37, 32, generator=g).to(torch.bfloat16).cuda()
    grads = fw.wsattn_cross_backward(dout, q, k, v, out, lse, k_lengths=lengths)

    def loss(a):  # in 64 bits
        return float((ref.cross_forward(a[0], a[1], a[2], lengths, 32 ** -0.5)[0] * dout.double()).sum())

    for i in range(3):
        d = torch.randn(grads[i].shape, generator=g).double().cuda()
        d /= d.norm()
        step, sides = 1e-4, []
        for sign in (1, -1):
            a = [t.double() for t in (q, k, v)]
            a[i] = a[i] + sign * step * d
            sides.append(loss(a))
        want, got = (sides[0] - sides[1]) / (2 * step), float((grads[i].double() * d).sum())
        # roundings of p, ds, out and of the gradient itself: a few half steps of 2^-9, spread over a random direction
        assert abs(got - want) <= 2.0 ** -6 * float(grads[i].double().norm()), (i, got, want)


def test_streams_graphs_and_workspaces():
    fw = _fw()
    q, k, v = make(6, torch.bfloat16, 2, 4, 4, 60, 5000, 128)
    lengths = lens([5000, 3000])
    lse = torch.empty((2, 4, 60), device="cuda")
    out = fw.wsattn_cross(q, k, v, k_lengths=lengths, lse=lse)
    dout = torch.randn_like(q)
    want = fw.wsattn_cross_backward(dout, q, k, v, out, lse, k_lengths=lengths)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lse2 = torch.empty_like(lse)
    out2 = fw.wsattn_cross(q, k, v, k_lengths=lengths, lse=lse2, stream=side)
    got = fw.wsattn_cross_backward(dout, q, k, v, out2, lse2, k_lengths=lengths, stream=side)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    # captured with workspaces of the caller's, and replayed on other values and lengths
    ws = torch.empty(max(fw.wsattn_cross_workspace(q, k, v), 16), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(max(fw.wsattn_cross_backward_workspace(dout, q, k, v, out, lse), 16), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out3 = fw.wsattn_cross(q, k, v, k_lengths=lengths, lse=lse2, workspace=ws)
        got = fw.wsattn_cross_backward(dout, q, k, v, out3, lse2, k_lengths=lengths, workspace=ws2)
    for values in ([5000, 3000], [0, 77], [4999, 128]):
        lengths.copy_(torch.tensor(values))
        q.normal_()
        ws.random_()
        ws2.random_()
        graph.replay()
        torch.cuda.synchronize()
        check_forward(q, k, v, lengths, out3, lse2)
        check_backward(dout, q, k, v, out3, lse2, lengths, got)
    assert fw.wsattn_op_status() == 0


@pytest.mark.parametrize("shape", [(2, 24, 24, 2500, 226, 128), (1, 40, 40, 3000, 512, 128), (3, 8, 2, 4000, 1100, 64), (1, 64, 8, 9, 3000, 128)])
def test_many_tiles(shape):
    # several work items a CTA, and keys in many steps
    b, h, hk, n, m, d = shape
    q, k, v = make(8, torch.bfloat16, b, h, hk, n, m, d)
    lengths = lens([m - 37 * i for i in range(b)])
    lse = torch.empty((b, h, n), device="cuda")
    out = _fw().wsattn_cross(q, k, v, k_lengths=lengths, lse=lse)
    check_forward(q, k, v, lengths, out, lse)
    dout = torch.randn(b, n, h, d, device="cuda").to(torch.bfloat16).transpose(1, 2)
    grads = _fw().wsattn_cross_backward(dout, q, k, v, out, lse, k_lengths=lengths)
    check_backward(dout, q, k, v, out, lse, lengths, grads)
    assert _fw().wsattn_op_status() == 0
