"""wsattn_qknorm_backward with many more work items than CTAs (GPU): gain
gradients summed over several items of a CTA, shares that run from one head
group into the next and from q's items into k's, where the registers' sums are
flushed, the gain is loaded anew and the ring of asynchronous loads runs on."""
import pytest
import torch

from _ops_ref import NORM, TURN, angles, assert_close, half_step, normed, sections_for, tiny, turn

pytestmark = pytest.mark.gpu


def _cdiv(a, b):
    return -(-a // b)


def _shares(heads, kv, rows, dim):
    """How the pass deals out its items: (most items of a CTA, heads of q's and
    k's groups, CTAs whose share spans two groups, and q and k)."""
    lanes = 1
    while 16 * lanes < dim:
        lanes *= 2
    blocks = _cdiv(rows, 8 * (32 // lanes))
    ctas = min(2 * torch.cuda.get_device_properties(0).multi_processor_count, 1024)
    io, gh = (heads, kv), [heads, kv]
    while True:
        i = 1 if gh[1] > gh[0] else 0
        want = (32 if gh[i] > 12 else 8) * ctas
        if blocks * sum(map(_cdiv, io, gh)) >= want or gh[i] <= 4:
            break
        gh[i] = (gh[i] + 1) // 2
    groups = [_cdiv(h, x) for h, x in zip(io, gh)]
    ctas = min(ctas, blocks * sum(groups))
    nq, wq, wk = groups[0] * blocks, 2 * gh[0] + 3, 2 * gh[1] + 3
    weight = nq * wq + groups[1] * blocks * wk
    at = [_cdiv(x, wq) if x <= nq * wq else nq + _cdiv(x - nq * wq, wk)
          for x in (weight * c // ctas for c in range(ctas + 1))]
    own = list(zip(at, at[1:]))
    return (max(b - a for a, b in own), gh, sum(b > a and a // blocks != (b - 1) // blocks for a, b in own),
            sum(a < nq < b for a, b in own))


def _pairs(x, interleaved):
    """|a| + |b| of each element's pair."""
    m = x.abs()
    if interleaved:
        return (m[..., 0::2] + m[..., 1::2]).repeat_interleave(2, -1)
    half = x.shape[-1] // 2
    s = m[..., :half] + m[..., half:]
    return torch.cat((s, s), -1)


CASES = [
    # batch, heads, key heads, tokens, dim, interleaved, shares that span groups
    (2, 24, 24, 10007, 64, True, False),
    (2, 6, 2, 10007, 64, False, True),
    (3, 9, 3, 10007, 80, True, True),      # five lanes of eight
    (2, 5, 3, 10007, 128, False, True),
]


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_qknorm_backward_shares_of_several_items(case, dt, pad):
    import frame_aligned_window_gb300 as fw
    B, H, K, N, D, inter, spans = case
    most, gh, two_groups, two_parts = _shares(H, K, B * N, D)
    assert most >= 4 and (not spans or (two_groups and two_parts))
    eps = 1e-5
    g = torch.Generator(device="cuda").manual_seed(61)

    def rows(heads, std):
        # [B, heads, N, D] views of token rows that start on 16 bytes, or off them
        buf = std * torch.randn((B, N, heads * D + pad), generator=g, device="cuda")
        return buf.to(dt)[..., :heads * D].unflatten(-1, (heads, D)).transpose(1, 2)
    packed = rows(H + 2 * K, 2.0)
    q, k, v = packed[:, :H], packed[:, H:H + K], packed[:, H + K:]
    up = [rows(h, 1.0) for h in (H, K, K)]
    w = [1 + 0.3 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    pos = torch.randint(0, 300, (N, 2), generator=g, device="cuda").float()
    sec = sections_for(D, 2)
    rot = fw.wsattn_rotary_plan(D, sec, interleaved=inter)
    d = torch.full((B, N, (H + 2 * K) * D + pad), 7.0, dtype=dt, device="cuda")
    dv = d[..., :(H + 2 * K) * D].unflatten(-1, (H + 2 * K, D)).transpose(1, 2)
    out = fw.wsattn_qknorm_backward(rot, up[0], up[1], q, k, pos, w[0], w[1], eps, dv_out=up[2],
                                    dq=dv[:, :H], dk=dv[:, H:H + K], dv=dv[:, H + K:])
    assert fw.wsattn_op_status() == 0
    assert (d[..., (H + 2 * K) * D:] == 7.0).all() and torch.equal(out[2], up[2])
    ang = angles(pos, sec, D).cuda()
    for i, x in enumerate((q, k)):
        x, wi = x.double(), w[i].double()
        xh, _, r = normed(x, wi, eps)
        h = turn(up[i].double(), ang, inter, -1)
        u = h * wi
        want = r * (u - xh * (u * xh).mean(-1, keepdim=True))
        # errors of h (TURN on its pair), of r and of the mean, on the magnitudes
        mag = r * (_pairs(h, inter) * wi.abs() + xh.abs() * (u * xh).abs().mean(-1, keepdim=True))
        assert_close(out[i], want.cpu(),
                     (half_step(dt) * want.abs() + (TURN + 4 * NORM) * mag + tiny(dt)).cpu(), f"part {i}")
        # a register adds the heads of its CTA's items one after the other, then 5
        # steps over a warp, 8 warps, and the CTAs' rows in up to 16 + 32 additions
        terms = (_pairs(h, inter) * xh.abs()).sum((0, 1, 2))
        tol = (TURN + 2 * NORM + (most * gh[i] + 64) * 2.0 ** -24) * terms
        assert_close(out[3 + i], (h * xh).sum((0, 1, 2)).cpu(), tol.cpu(), f"gain {i}")
