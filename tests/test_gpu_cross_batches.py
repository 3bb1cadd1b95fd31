"""Cross attention over many batch elements whose lengths leave gaps: the
gradients' work is shared by the keys that count, so shares begin and end
anywhere among the batch elements, and runs of them have no keys at all."""
import pytest
import torch

from test_gpu_cross import check_backward, check_forward, lens, make, spoil

pytestmark = pytest.mark.gpu


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


def _lengths(kind, b, m):
    g = torch.Generator().manual_seed(b)
    t = torch.randint(0, m + 1, (b,), generator=g)
    if kind == "gaps":    # runs without keys, at both ends too
        t[torch.arange(b) % 97 < 60] = 0
        t[-40:] = 0
    elif kind == "none":
        t[:] = 0
    elif kind == "last":  # one element has all the keys there are
        t[:] = 0
        t[-1] = m
    elif kind == "first":
        t[1:] = 0
        t[0] = m
    return None if kind == "all" else t.tolist()


@pytest.mark.parametrize("kind", ["gaps", "none", "last", "first", "random", "all"])
@pytest.mark.parametrize("shape", [(1300, 2, 1, 5, 40, 64), (300, 3, 3, 140, 300, 32), (37, 4, 2, 300, 520, 128)])
def test_many_batch_elements(shape, kind):
    fw = _fw()
    b, h, hk, n, m, d = shape
    lengths = _lengths(kind, b, m)
    q, k, v = make(b + n, torch.bfloat16, b, h, hk, n, m, d)
    spoil(k, v, lengths, m)
    lse = torch.empty((b, h, n), device="cuda")
    out = fw.wsattn_cross(q, k, v, lens(lengths), lse=lse)
    check_forward(q, k, v, lens(lengths), out, lse)
    dout = torch.randn(b, h, n, d, device="cuda").to(torch.bfloat16)
    # what lies in the scratch and in the outputs before does not matter
    ws = torch.full((fw.wsattn_cross_backward_workspace(dout, q, k, v, out, lse),), 255, dtype=torch.uint8, device="cuda")
    old = [torch.full((b, x, y, d), float("nan"), device="cuda", dtype=torch.bfloat16) for x, y in ((h, n), (hk, m), (hk, m))]
    grads = fw.wsattn_cross_backward(dout, q, k, v, out, lse, lens(lengths), dq=old[0], dk=old[1], dv=old[2], workspace=ws)
    check_backward(dout, q, k, v, out, lse, lens(lengths), grads)
    if lengths is not None:
        for i, count in enumerate(lengths):
            assert not grads[1][i, :, count:].any() and not grads[2][i, :, count:].any()
    alone = fw.wsattn_cross_backward(dout, q, k, v, out, lse, lens(lengths), need_dq=False)
    assert alone[0] is None and torch.equal(alone[1], grads[1]) and torch.equal(alone[2], grads[2])
    again = fw.wsattn_cross_backward(dout, q, k, v, out, lse, lens(lengths), need_dk=False)
    assert again[1] is None and torch.equal(again[0], grads[0]) and torch.equal(again[2], grads[2])


def test_gradients_of_no_queries_are_zeros_over_many_tiles():
    fw = _fw()
    b, h, m, d = 3, 2, 3000, 80
    q = torch.empty(b, h, 0, d, device="cuda", dtype=torch.float16)
    k, v = (torch.full((b, h, m, d), float("nan"), device="cuda", dtype=torch.float16) for _ in range(2))
    lse = torch.empty(b, h, 0, device="cuda")
    dk, dv = (torch.full((b, h, m, d), float("nan"), device="cuda", dtype=torch.float16) for _ in range(2))
    fw.wsattn_cross_backward(q, q, k, v, q, lse, dk=dk, dv=dv)
    assert not dk.any() and not dv.any()


def test_norm_gradients_of_no_rows_on_a_stream():
    fw = _fw()
    x = torch.empty(0, 5, 24, dtype=torch.bfloat16, device="cuda")
    scale = torch.ones(24, device="cuda")
    gate = torch.empty(0, 24, device="cuda")
    stream = torch.cuda.Stream()
    g = fw.wsattn_block_norm_backward(x, x, scale=scale, weight=scale, stream=stream)
    stream.synchronize()
    assert (g.dscale == 0).all() and (g.dweight == 0).all()
    out, hidden = fw.wsattn_block_norm(x, x, gate=gate)
    assert out.shape == x.shape and hidden.shape == x.shape
    assert fw.wsattn_block_norm_backward(x, hidden, x, gate=gate).dgate.shape == gate.shape
