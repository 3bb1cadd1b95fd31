"""Outputs whose rows start on 16 bytes and whose last column does not end on
them (GPU): the columns behind it belong to someone else."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _ints(shape, most, g, dtype):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


def _wide(rows, cols, ld, dtype):
    buf = torch.full((rows, ld), 5.0, dtype=dtype, device="cuda")
    return buf, buf[:, :cols]


# every remainder of 8 columns; pairs of 128 and of 256 columns, a split last round, single CTAs
@pytest.mark.parametrize("shape", [(3000, 64 + r, 64) for r in range(1, 9)]
                         + [(300, 4900, 72), (301, 4903, 72), (261, 501, 66001), (33, 77, 64)],
                         ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32], ids=str)
def test_linear_leaves_the_columns_behind_its_own(shape, odt):
    import frame_aligned_window_gb300 as fw
    m, n, k = shape
    dt = torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(n)
    ld = (n + 15) // 8 * 8
    x, w, r = _ints((m, k), 2, g, dt), _ints((n, k), 1, g, dt), _ints((m, n), 9, g, odt)
    z = x.double() @ w.double().t()
    buf, out = _wide(m, n, ld, odt)
    assert out.stride(0) * out.element_size() % 16 == 0
    fw.wsattn_linear(x, w, out=out)
    assert torch.equal(out, z.to(odt)) and (buf[:, n:] == 5.0).all()
    # with a residual in place and a pre-activation
    out.copy_(r)
    pbuf, pre = _wide(m, n, ld, dt)
    fw.wsattn_linear(x, w, residual=out, out=out, preact=pre)
    assert torch.equal(out, (z + r.double()).to(odt)) and (buf[:, n:] == 5.0).all()
    assert torch.equal(pre, z.to(dt)) and (pbuf[:, n:] == 5.0).all()
    assert fw.wsattn_op_status() == 0


@pytest.mark.parametrize("shape", [(1, 5, 79), (1, 264, 133), (640, 1288, 1157), (3000, 128, 67), (9000, 20, 33),
                                   (6575, 1340, 971), (57601, 300, 499)], ids=lambda c: "x".join(map(str, c)))
def test_linear_backward_leaves_the_columns_behind_its_own(shape):
    import frame_aligned_window_gb300 as fw
    m, n, k = shape
    dt = torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(k)
    ld = (k + 15) // 8 * 8
    dy, x, w = _ints((m, n), 2, g, dt), _ints((m, k), 1, g, dt), _ints((n, k), 1, g, dt)
    want = ((dy.double() @ w.double()).to(dt), (dy.double().t() @ x.double()).to(dt))
    for need in ((True, True), (True, False), (False, True)):
        dxb, dx = _wide(m, k, ld, dt)
        dwb, dw = _wide(n, k, ld, dt)
        fw.wsattn_linear_backward(dy, x, w, dx=dx if need[0] else None, dw=dw if need[1] else None,
                                  need_dx=need[0], need_dw=need[1], need_db=False)
        for on, buf, got, exact in ((need[0], dxb, dx, want[0]), (need[1], dwb, dw, want[1])):
            assert torch.equal(got, exact) if on else (got == 5.0).all()
            assert (buf[:, k:] == 5.0).all()
    assert fw.wsattn_op_status() == 0
