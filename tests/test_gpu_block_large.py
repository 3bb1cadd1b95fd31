"""Cross attention and a block's norms where element offsets pass 2^31: whole
numbers, whose results are known without a second implementation of the size."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


def test_a_memory_past_2_31_elements():
    # one key far from all others takes every query's probability: 40 in the exponent leaves 2^-57 for the rest
    fw = _fw()
    h, m, d = 2, (1 << 31) // 128 // 2 + 4099, 128
    kv = torch.zeros((1, m, 2 * h, d), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    k, v = kv[:, :h], kv[:, h:]
    assert (k.stride(2)) * (m - 1) > 1 << 31
    q = torch.zeros((1, h, 3, d), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    for at in (m - 1, m // 2, 5):
        k[:, :, at, 0], v[:, :, at] = 40, torch.arange(d, device="cuda", dtype=torch.bfloat16)
        lse = torch.empty((1, h, 3), device="cuda")
        out = fw.wsattn_cross(q, k, v, scale=1.0, lse=lse)
        assert torch.equal(out.float(), torch.arange(d, device="cuda").float().expand_as(out)) and (lse - 40).abs().max() < 1e-4
        dout = torch.ones_like(q)
        dq, dk, dv = fw.wsattn_cross_backward(dout, q, k, v, out, lse, scale=1.0)
        # p is 1 there: dv is the sum over the three queries; ds is 0 to the products' rounding
        assert torch.equal(dv[:, :, at].float(), torch.full((1, h, d), 3.0, device="cuda"))
        assert dq.abs().max() < 1 and dk.abs().max() < 1e-1
        del dk, dv
        k[:, :, at], v[:, :, at] = 0, 0
    assert fw.wsattn_op_status() == 0


def test_queries_past_2_31_elements():
    # every row sees one key: out is its value, whatever the query
    fw = _fw()
    h, n, d = 40, (1 << 31) // 128 // 40 + 1000, 128
    q = torch.ones((1, h, n, d), dtype=torch.bfloat16, device="cuda")
    assert q.numel() > 1 << 31
    k = torch.ones((1, h, 1, d), dtype=torch.bfloat16, device="cuda")
    v = (torch.arange(h, device="cuda")[None, :, None, None] + torch.arange(d, device="cuda")).to(torch.bfloat16)
    lse = torch.empty((1, h, n), device="cuda")
    out = fw.wsattn_cross(q, k, v, lse=lse, out=torch.empty_like(q))
    assert torch.equal(out, v.expand_as(out))
    assert (lse - d ** 0.5).abs().max() < 1e-4
    dq, _, dv = fw.wsattn_cross_backward(q, q, k, v, out, lse, dq=torch.empty_like(q), need_dk=False)
    # ds = p (dout v - dout out) = 0 in whole numbers
    assert not dq.any()
    assert torch.equal(dv, torch.full_like(dv, n).to(torch.bfloat16))
    assert fw.wsattn_op_status() == 0


def test_rows_past_2_31_elements():
    # rows of +-a: mean 0, deviation a, so the norm is +-1 (eps 0)
    fw = _fw()
    n, m = 4096, (1 << 31) // 4096 + 77
    sign = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    sign[1::2] = -1
    x = (torch.arange(m, device="cuda") % 7 + 1).to(torch.bfloat16)[:, None] * sign
    scale = torch.full((m // 11 if m % 11 == 0 else 1, n), 2.0, device="cuda")
    out, hidden = fw.wsattn_block_norm(x, x, scale=scale, eps=0.0)
    assert torch.equal(hidden, 2 * x)
    assert (out - 3 * sign).abs().max() <= 2.0 ** -7
    del out
    dout = torch.ones_like(x)
    g = fw.wsattn_block_norm_backward(dout, hidden, dhidden=x, scale=scale, eps=0.0)
    # out does not move with a row's mean: its gradient for equal dout is 0, and dhidden comes through
    assert (g.dx - x).abs().max() <= 2.0 ** -8
    assert torch.equal(g.dshift, torch.full_like(g.dshift, m / g.dshift.shape[0]))
    assert fw.wsattn_op_status() == 0
