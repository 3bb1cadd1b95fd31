"""The operators around the attention at sizes whose rows or offsets pass 32
bits (GPU).  Whole numbers make the linear products exact; what needs more
memory than is free is skipped."""
import pytest
import torch

from _ops_ref import NORM, TURN, angles, assert_close, half_step, normed, tiny, turn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


@pytest.fixture(autouse=True)
def _give_back():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _needs(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB")


def _ints(shape, most, g, dtype):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


def _chunks(rows, step):
    return [slice(i, min(i + step, rows)) for i in range(0, rows, step)]


def test_rotary_in_place_over_more_than_2_to_31_rows():
    fw = _fw()
    _needs(90)
    B, N, D = 2, 1_100_000_000, 16
    x = torch.ones((B, 1, N, D), dtype=BF, device="cuda")
    x[1] = 2
    pos = (torch.arange(N, device="cuda", dtype=torch.int32) % 1009).float()[:, None].contiguous()
    rot = fw.wsattn_rotary_plan(D, (8,))
    assert fw.wsattn_rotary(rot, x, pos, out=x) is x and fw.wsattn_op_status() == 0
    for b in range(B):
        for first in (0, N // 2, N - 1000):
            rows = slice(first, first + 1000)
            one = torch.full((1, 1, 1000, D), 1.0 + b, dtype=torch.float64)
            want = turn(one, angles(pos[rows], (8,), D), True)
            assert_close(x[b:b + 1, :, rows], want,
                         half_step(BF) * want.abs() + TURN * 2 * (1 + b) + tiny(BF), (b, first))


def test_qknorm_backward_of_more_than_2_to_31_elements():
    fw = _fw()
    _needs(40)
    H, N, D, eps = 34, 500000, 128, 1e-6
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.empty((1, H, N, D), dtype=BF, device="cuda").normal_(generator=g)
    up = torch.empty((1, H, N, D), dtype=BF, device="cuda").normal_(generator=g)
    assert q.numel() > 1 << 31
    pos = torch.arange(N, device="cuda", dtype=torch.float32)[:, None].contiguous()
    rot = fw.wsattn_rotary_plan(D, (64,))
    w = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
    dq, dk, _, dwq, dwk = fw.wsattn_qknorm_backward(rot, up, up[:, 3:4], q, q[:, 5:6], pos, w, w, eps)
    assert fw.wsattn_op_status() == 0
    ang, wd = angles(pos, (64,), D).cuda(), w.double()
    dw, terms = (torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(2))
    for i, (x, u, got) in enumerate([(q[:, h:h + 1], up[:, h:h + 1], dq[:, h:h + 1]) for h in range(H)]
                                    + [(q[:, 5:6], up[:, 3:4], dk)]):
        xh, _, r = normed(x.double(), None, eps)
        t = turn(u.double(), ang, True, -1)
        v = t * wd
        want = r * (v - xh * (v * xh).mean(-1, keepdim=True))
        pair = (t.abs()[..., 0::2] + t.abs()[..., 1::2]).repeat_interleave(2, -1)
        mag = r * (pair * wd.abs() + xh.abs() * (v * xh).abs().mean(-1, keepdim=True))
        bad = ~((got.double() - want).abs() <= half_step(BF) * want.abs() + (TURN + 4 * NORM) * mag + tiny(BF))
        assert not bad.any(), (i, int(bad.sum()))
        if i < H:
            dw += (t * xh).sum((0, 1, 2))
            terms += (pair * xh.abs()).sum((0, 1, 2))
        else:
            # rows of 8 warps a CTA, two halves of a warp each: at most N / 304 / 16
            # items of a head, and the sums over warps and CTAs
            tol = (TURN + 2 * NORM + (N / 4000 + 64) * 2.0 ** -24) * (pair * xh.abs()).sum((0, 1, 2))
            assert_close(dwk, (t * xh).sum((0, 1, 2)).cpu(), tol.cpu())
    assert_close(dwq, dw.cpu(), ((TURN + 2 * NORM + (H * N / 4000 + 64) * 2.0 ** -24) * terms).cpu())


def test_linear_of_attention_output_past_2_to_31_elements():
    fw = _fw()
    _needs(40)
    B, H, N, D = 2, 40, 220000, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    a = _ints((B, H, N, D), 2, g, torch.float32)
    assert a.numel() > 1 << 31
    w = _ints((24, H * D), 1, g, BF)
    got = fw.wsattn_linear(a, w, out_dtype=torch.float32)
    assert fw.wsattn_op_status() == 0
    for b in range(B):
        for rows in _chunks(N, 20000):
            x = a[b, :, rows].transpose(0, 1).reshape(-1, H * D).double()
            assert torch.equal(got[b, rows], (x @ w.double().t()).float()), (b, rows)


@pytest.mark.parametrize("n,k", [(64, 4101), (4101, 64)])
def test_linear_of_odd_rows_past_2_to_31_elements(n, k):
    # operands copied to aligned rows, outputs stored row by row
    fw = _fw()
    _needs(60)
    m = 540000
    g = torch.Generator(device="cuda").manual_seed(4)
    x, w = _ints((m, k), 2, g, BF), _ints((n, k), 1, g, BF)
    assert m * max(n, k) > 1 << 31
    out, pre = _ints((m, n), 9, g, torch.float32), torch.empty((m, n), dtype=BF, device="cuda")
    keep = out.to(torch.int8)
    fw.wsattn_linear(x, w, residual=out, out=out, preact=pre)
    assert fw.wsattn_op_status() == 0
    for rows in _chunks(m, 20000):
        z = x[rows].double() @ w.double().t()
        assert torch.equal(out[rows], (z + keep[rows].double()).float()), rows
        assert torch.equal(pre[rows], z.to(BF)), rows


def test_linear_over_as_many_rows_as_it_takes():
    fw = _fw()
    _needs(160)
    m, n, k = (1 << 31) - 512, 8, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w = _ints((m, k), 2, g, BF), _ints((n, k), 2, g, BF)
    y = fw.wsattn_linear(x, w)
    dx, _, _ = fw.wsattn_linear_backward(y, x, w, need_dw=False, need_db=False)
    assert fw.wsattn_op_status() == 0
    for rows in _chunks(m, 1 << 26):   # sums of at most 32, and of 8 x 32 x 2, are exact
        assert torch.equal(y[rows].float(), x[rows].float() @ w.float().t()), rows
        assert torch.equal(dx[rows], (y[rows].float() @ w.float()).to(BF)), rows
