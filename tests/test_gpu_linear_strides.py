"""wsattn_linear_backward on rows inside wider buffers, and past 2^31 elements
(GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


def _ints(shape, most, g, dtype):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


@pytest.mark.parametrize("pad", [3, 8])
@pytest.mark.parametrize("shape", [(40, 264, 72), (333, 257, 131), (1030, 520, 200), (20, 96, 40)],
                         ids=lambda c: "x".join(map(str, c)))
def test_linear_backward_strided_rows(shape, pad):
    # rows inside wider buffers: the inputs' gaps are not read, the outputs' not written
    fw = _fw()
    m, n, k = shape
    dt = torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(7)

    def wide(rows, cols, fill):
        buf = torch.full((rows, cols + pad), fill, dtype=dt, device="cuda")
        buf[:, :cols] = torch.randn((rows, cols), generator=g, device="cuda").to(dt)
        return buf
    nan = float("nan")
    dyb, xb, wb, zb = wide(m, n, nan), wide(m, k, nan), wide(n, k, nan), wide(m, n, nan)
    dy, x, w, z = dyb[:, :n], xb[:, :k], wb[:, :k], zb[:, :n]
    want = fw.wsattn_linear_backward(*(t.contiguous() for t in (dy, x, w, z)), "gelu")
    dxb, dwb = wide(m, k, 5.0), wide(n, k, 5.0)
    dx, dw, db = fw.wsattn_linear_backward(dy, x, w, z, "gelu", dx=dxb[:, :k], dw=dwb[:, :k])
    for a, b in zip((dx, dw, db), want):
        assert torch.equal(a, b) and torch.isfinite(a).all()
    assert (dxb[:, k:] == 5.0).all() and (dwb[:, k:] == 5.0).all()
    # without an activation dout itself is the operand
    want = fw.wsattn_linear_backward(dy.contiguous(), x.contiguous(), w.contiguous())
    for a, b in zip(fw.wsattn_linear_backward(dy, x, w, dx=dxb[:, :k], dw=dwb[:, :k]), want):
        assert torch.equal(a, b)
    # no rows: dw is zeroed row by row, db too
    _, dw, db = fw.wsattn_linear_backward(dy[:0], x[:0], w, z[:0], "gelu", dw=dwb[:, :k])
    assert (dwb[:, :k] == 0).all() and (dwb[:, k:] == 5.0).all() and (db == 0).all()
    assert fw.wsattn_op_status() == 0


def test_linear_backward_sums_past_2_to_31_elements():
    # dw and db of a slope pass and a product whose offsets pass 32 bits, in
    # whole and half numbers: every sum is exact, and so are all three gradients
    fw = _fw()
    m, n, k = 540000, 4104, 64
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB")
    dt = torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(3)
    dy, x, w = _ints((m, n), 2, g, dt), _ints((m, k), 2, g, dt), _ints((n, k), 2, g, dt)
    z = 300 * _ints((m, n), 1, g, dt)
    assert dy.numel() > 1 << 31
    dx, dw, db = fw.wsattn_linear_backward(dy, x, w, z, "silu")
    assert fw.wsattn_op_status() == 0
    dw64 = torch.zeros((n, k), dtype=torch.float64, device="cuda")
    db64 = torch.zeros(n, dtype=torch.float64, device="cuda")
    for i in range(0, m, 20000):
        rows = slice(i, min(i + 20000, m))
        dz = dy[rows].double() * (z[rows].double().sign() + 1) / 2
        dw64 += dz.t() @ x[rows].double()
        db64 += dz.sum(0)
        assert torch.equal(dx[rows], (dz @ w.double()).to(dt)), i
    assert float(dw64.abs().max()) < 2 ** 23 and torch.equal(dw, dw64.to(dt))
    assert torch.equal(db, db64.float())
