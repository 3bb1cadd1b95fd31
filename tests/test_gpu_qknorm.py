"""wsattn_rotary, wsattn_qknorm and wsattn_qknorm_backward against their 64-bit
definitions (GPU).  Tolerances: half a step of the stored type plus the fp32
error bounds in _ops_ref, on the magnitudes that enter each sum."""
import pytest
import torch

from _ops_ref import (NORM, TURN, angles, assert_close, half_step, normed, sections_for, tiny, turn)

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _positions(n, axes, g, far=0, batch=None):
    shape = (n, axes) if batch is None else (batch, n, axes)
    return (torch.randint(0, 300, shape, generator=g) + far).float()


def _pairmax(x, interleaved):
    """|a| + |b| of each element's pair."""
    m = x.abs()
    if interleaved:
        s = m[..., 0::2] + m[..., 1::2]
        return s.repeat_interleave(2, -1)
    half = x.shape[-1] // 2
    s = m[..., :half] + m[..., half:]
    return torch.cat((s, s), -1)


def _turn_tol(x, want, interleaved, dt):
    return half_step(dt) * want.abs() + TURN * _pairmax(x, interleaved) + tiny(dt)


ROTARY = [
    # batch, heads, tokens, dim, axes, far
    (1, 1, 1, 128, 1, 0),
    (2, 3, 37, 64, 3, 0),
    (1, 8, 1, 128, 3, 70000),      # one new token, far from the start
    (3, 5, 130, 96, 2, 0),         # six lanes of eight
    (1, 2, 70, 16, 4, 5),          # one lane a row
    (2, 1, 33, 256, 3, 1000000),
    (1, 7, 9, 80, 1, 16000000),    # five lanes of eight, at the edge of fp32 integers
]


@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("case", ROTARY, ids=lambda c: "x".join(map(str, c)))
def test_rotary(case, interleaved, dt):
    fw = _fw()
    B, H, N, D, axes, far = case
    g = _gen(B * 1000 + N)
    x = torch.randn((B, H, N, D), generator=g).to(dt)
    pos = _positions(N, axes, g, far)
    sec = sections_for(D, axes)
    rot = fw.wsattn_rotary_plan(D, sec, interleaved=interleaved)
    ang = angles(pos, sec, D)
    for inverse in (False, True):
        got = fw.wsattn_rotary(rot, x.cuda(), pos.cuda(), inverse=inverse)
        assert got.is_contiguous() and got.dtype == dt
        want = turn(x.double(), ang, interleaved, -1 if inverse else 1)
        assert_close(got, want, _turn_tol(x.double(), want, interleaved, dt))
    # pairs behind the sections are left exactly alone
    last = [D - 2, D - 1] if interleaved else [D // 2 - 1, D - 1]
    assert torch.equal(got.cpu()[..., last], x[..., last])


@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_rotary_strides_batch_positions_and_in_place(dt):
    fw = _fw()
    B, H, N, D = 2, 3, 41, 64
    g = _gen(7)
    pos = _positions(N, 3, g, batch=B)
    sec = sections_for(D, 3)
    rot = fw.wsattn_rotary_plan(D, sec)
    ang = angles(pos, sec, D)
    # rows of an odd stride: nothing starts on 16 bytes; the gaps stay as they were
    buf = torch.randn((B, N, H * (D + 3) + 1), generator=g).to(dt).cuda()
    view = buf[..., 1:].as_strided((B, H, N, D), (buf.stride(0), D + 3, buf.stride(1), 1),
                                   storage_offset=1)
    x = view.cpu().double()
    before = buf.clone()
    out = fw.wsattn_rotary(rot, view, pos.cuda())
    want = turn(x, ang, True)
    assert_close(out, want, _turn_tol(x, want, True, dt))
    assert torch.equal(buf, before)
    # in place
    got = fw.wsattn_rotary(rot, view, pos.cuda(), out=view)
    assert got is view
    assert torch.equal(view, out)
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask.as_strided((B, H, N, D), view.stride(), view.storage_offset()).fill_(False)
    assert torch.equal(buf[mask], before[mask])
    # an expanded (broadcast) input reads one head for all
    one = torch.randn((B, 1, N, D), generator=g).to(dt)
    got = fw.wsattn_rotary(rot, one.cuda().expand(B, 4, N, D), pos.cuda())
    want = turn(one.double(), ang, True).expand(B, 4, N, D)
    assert_close(got, want, _turn_tol(one.double(), turn(one.double(), ang, True), True, dt)
                 .expand(B, 4, N, D))


def test_rotary_matches_the_producers_table():
    # the grid of workloads.rope_table, as positions on three axes
    import oracle  # noqa: F401  (the table's consumer)
    from workloads import WORKLOADS, rope_table
    fw = _fw()
    wl = WORKLOADS["small"]
    cos, sin = rope_table(wl.n_tokens, wl.tokens_per_frame, wl.grid_w, wl.head_dim)
    n = torch.arange(wl.n_tokens)
    t = wl.tokens_per_frame
    pos = torch.stack((n // t, n % t // wl.grid_w, n % wl.grid_w), 1).float()
    half = wl.head_dim // 2
    rot = fw.wsattn_rotary_plan(wl.head_dim, (half - 2 * (half // 3), half // 3, half // 3))
    x = torch.zeros((1, 1, wl.n_tokens, wl.head_dim))
    x[..., 0::2] = 1
    y = fw.wsattn_rotary(rot, x.cuda(), pos.cuda()).cpu()
    assert (y[0, 0, :, 0::2] - cos).abs().max() <= 2 * TURN
    assert (y[0, 0, :, 1::2] - sin).abs().max() <= 2 * TURN


QK = [
    # batch, heads, key heads, tokens, dim, interleaved, gain
    (1, 2, 2, 240, 64, True, "same"),
    (2, 6, 2, 33, 128, False, "fp32"),     # shared key heads
    (1, 1, 1, 1, 16, True, "none"),
    (3, 5, 5, 77, 96, True, "fp32"),
    (1, 12, 3, 130, 256, False, "same"),
    (2, 9, 1, 257, 80, True, "none"),
]


def _qk_case(case, dt, seed):
    B, H, K, N, D, inter, gain = case
    g = _gen(seed)
    rows = (2 * torch.randn((B, N, H + 2 * K, D), generator=g)).to(dt)
    rows[0, 0, 0] = 0                      # a row of zeros
    t = rows.transpose(1, 2)
    q, k, v = t[:, :H], t[:, H:H + K], t[:, H + K:]
    w = [None, None]
    if gain != "none":
        w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dt if gain == "same" else torch.float32)
             for _ in range(2)]
    pos = _positions(N, 3, g, 100)
    return rows, (q, k, v), w, pos, sections_for(D, 3)


@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("case", QK, ids=lambda c: "x".join(map(str, c)))
def test_qknorm(case, dt):
    fw = _fw()
    B, H, K, N, D, inter, gain = case
    eps = 1e-5
    rows, parts, w, pos, sec = _qk_case(case, dt, 11)
    rot = fw.wsattn_rotary_plan(D, sec, interleaved=inter)
    dev = rows.cuda().transpose(1, 2)
    dq, dk, dv = dev[:, :H], dev[:, H:H + K], dev[:, H + K:]
    wd = [None if x is None else x.cuda() for x in w]
    got = fw.wsattn_qknorm(rot, dq, dk, pos.cuda(), wd[0], wd[1], eps, v=dv)
    ang = angles(pos, sec, D)
    for i in range(2):
        _, y, _ = normed(parts[i].double(), None if w[i] is None else w[i].double(), eps)
        want = turn(y, ang, inter)
        tol = half_step(dt) * want.abs() + (TURN + 2 * NORM) * _pairmax(y, inter) + tiny(dt)
        assert got[i].is_contiguous()
        assert_close(got[i], want, tol, f"part {i}")
    assert torch.equal(got[2].cpu(), parts[2]) and got[2].is_contiguous()
    # without v, in place: the same values, v's rows untouched
    two = fw.wsattn_qknorm(rot, dq, dk, pos.cuda(), wd[0], wd[1], eps, q_out=dq, k_out=dk)
    assert two[0] is dq and torch.equal(dq, got[0]) and torch.equal(dk, got[1])
    assert torch.equal(dv.cpu(), parts[2])


@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("case", QK, ids=lambda c: "x".join(map(str, c)))
def test_qknorm_backward(case, dt):
    fw = _fw()
    B, H, K, N, D, inter, gain = case
    eps = 1e-5
    rows, parts, w, pos, sec = _qk_case(case, dt, 23)
    g = _gen(5)
    up = [torch.randn((B, n, N, D), generator=g).to(dt) for n in (H, K, K)]
    rot = fw.wsattn_rotary_plan(D, sec, interleaved=inter)
    dev = rows.cuda().transpose(1, 2)
    wd = [None if x is None else x.cuda() for x in w]
    packed = torch.full((B, N, H + 2 * K, D), 7.0, dtype=dt, device="cuda")
    d = packed.transpose(1, 2)
    out = fw.wsattn_qknorm_backward(rot, up[0].cuda(), up[1].cuda(), dev[:, :H], dev[:, H:H + K],
                                    pos.cuda(), wd[0], wd[1], eps, dv_out=up[2].cuda(),
                                    dq=d[:, :H], dk=d[:, H:H + K], dv=d[:, H + K:])
    again = fw.wsattn_qknorm_backward(rot, up[0].cuda(), up[1].cuda(), dev[:, :H],
                                      dev[:, H:H + K], pos.cuda(), wd[0], wd[1], eps)
    ang = angles(pos, sec, D)
    for i in range(2):
        x = parts[i].double()
        wi = None if w[i] is None else w[i].double()
        xh, _, r = normed(x, wi, eps)
        h = turn(up[i].double(), ang, inter, -1)
        u = h if wi is None else h * wi
        mean = (u * xh).mean(-1, keepdim=True)
        want = r * (u - xh * mean)
        # errors of h (TURN on its pair), of r and of the mean, on the magnitudes
        mag = r * ((_pairmax(u, inter) if wi is None else _pairmax(h, inter) * wi.abs())
                   + xh.abs() * (u * xh).abs().mean(-1, keepdim=True))
        tol = half_step(dt) * want.abs() + (TURN + 4 * NORM) * mag + tiny(dt)
        assert_close(out[i], want, tol, f"part {i}")
        if wi is not None:
            dw = (h * xh).sum((0, 1, 2))
            terms = (_pairmax(h, inter) * xh.abs()).sum((0, 1, 2))
            n = B * N * x.shape[1]
            # each term as above; sums of n terms in registers (at most n / 8 in a row)
            assert_close(out[3 + i], dw, (TURN + 2 * NORM + (n / 8 + 64) * 2.0 ** -24) * terms)
            assert torch.equal(again[3 + i], out[3 + i])   # a fixed order
        else:
            assert out[3 + i] is None
        assert torch.equal(again[i], out[i])
    assert torch.equal(out[2].cpu(), up[2]) and again[2] is None


def test_qknorm_backward_matches_differences():
    # directional difference of the forward in fp32 against the gradient
    fw = _fw()
    B, H, N, D, eps = 1, 2, 9, 64, 1e-3
    g = _gen(3)
    q, k = (torch.randn((B, H, N, D), generator=g).cuda() for _ in range(2))
    w = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    pos = _positions(N, 3, g).cuda()
    rot = fw.wsattn_rotary_plan(D, sections_for(D, 3))
    gq, gk, dirq, dirk = (torch.randn((B, H, N, D), generator=g).cuda() for _ in range(4))
    dirw = torch.randn(D, generator=g).cuda()
    dq, dk, _, dwq, _ = fw.wsattn_qknorm_backward(rot, gq, gk, q, k, pos, w, None, eps)

    def loss(t):
        a, b = fw.wsattn_qknorm(rot, q + t * dirq, k + t * dirk, pos, w + t * dirw, None, eps)
        return float((a.double() * gq.double()).sum() + (b.double() * gk.double()).sum())

    t = 1e-2
    # central difference: its own error is t^2 / 6 of the third derivative,
    # and fp32 outputs give 2^-23 * |loss terms| / t
    diff = (loss(t) - loss(-t)) / (2 * t)
    grad = float((dq.double() * dirq.double()).sum() + (dk.double() * dirk.double()).sum()
                 + (dwq.double() * dirw.double()).sum())
    scale = float(dq.abs().double().sum() + dk.abs().double().sum() + dwq.abs().double().sum())
    assert abs(diff - grad) <= 1e-3 * scale


def test_empty_and_single():
    fw = _fw()
    rot = fw.wsattn_rotary_plan(64, (32,))
    for B, N in ((0, 5), (2, 0)):
        x = torch.empty((B, 3, N, 64), dtype=torch.bfloat16, device="cuda")
        pos = torch.zeros((N, 1), device="cuda")
        assert fw.wsattn_rotary(rot, x, pos).shape == x.shape
        w = torch.ones(64, device="cuda")
        q, k, v = fw.wsattn_qknorm(rot, x, x, pos, w, w, v=x)
        assert q.shape == x.shape
        *_, dwq, dwk = fw.wsattn_qknorm_backward(rot, x, x, x, x, pos, w, w)
        assert torch.equal(dwq, torch.zeros_like(w)) and torch.equal(dwk, torch.zeros_like(w))


def test_nonfinite_rows_stay_their_own():
    # an infinity or NaN in one head row reaches that row only
    fw = _fw()
    g = _gen(9)
    x = torch.randn((1, 4, 20, 128), generator=g).to(torch.bfloat16)
    pos = _positions(20, 1, g)
    rot = fw.wsattn_rotary_plan(128, (64,), interleaved=False)
    clean = fw.wsattn_qknorm(rot, x.cuda(), x.cuda(), pos.cuda())[0].cpu()
    bad = x.clone()
    bad[0, 1, 3, 5] = float("inf")
    bad[0, 2, 7, 0] = float("nan")
    got = fw.wsattn_qknorm(rot, bad.cuda(), bad.cuda(), pos.cuda())[0].cpu()
    hit = torch.zeros((1, 4, 20), dtype=torch.bool)
    hit[0, 1, 3] = hit[0, 2, 7] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert got[0, 2, 7].isnan().all()


def test_capture_and_other_stream():
    fw = _fw()
    g = _gen(13)
    B, H, N, D = 1, 4, 100, 128
    q = torch.randn((B, H, N, D), generator=g).to(torch.bfloat16).cuda()
    up = torch.randn((B, H, N, D), generator=g).to(torch.bfloat16).cuda()
    w = torch.ones(D, device="cuda")
    pos = _positions(N, 3, g).cuda()
    rot = fw.wsattn_rotary_plan(D, sections_for(D, 3))
    fwd = fw.wsattn_qknorm(rot, q, q, pos, w, w)
    bwd = fw.wsattn_qknorm_backward(rot, up, up, q, q, pos, w, w)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a = fw.wsattn_qknorm(rot, q, q, pos, w, w)
            b = fw.wsattn_qknorm_backward(rot, up, up, q, q, pos, w, w)
        graphs.append((graph, a, b))
    # both graphs at once on two streams: neither shares scratch with the other
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (graph, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, a, b in graphs:
        assert torch.equal(a[0], fwd[0]) and torch.equal(a[1], fwd[1])
        for i in (0, 1, 3, 4):
            assert torch.equal(b[i], bwd[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = fw.wsattn_qknorm_backward(rot, up, up, q, q, pos, w, w, stream=side)
    side.synchronize()
    assert torch.equal(c[0], bwd[0]) and torch.equal(c[3], bwd[3])


@pytest.mark.parametrize("heads,kv", [(2, 1), (24, 24)])
def test_qknorm_many_tokens(heads, kv):
    # enough tokens for several rounds of CTAs, with few heads (one warp walks
    # q, k and v of its tokens) and with many (head groups of their own)
    fw = _fw()
    B, N, D, eps = 2, 10007, 32, 1e-6
    g = _gen(31)
    rows = torch.randn((B, N, heads + 2 * kv, D), generator=g).to(torch.bfloat16)
    t = rows.transpose(1, 2)
    parts = t[:, :heads], t[:, heads:heads + kv], t[:, heads + kv:]
    w = [(1 + 0.3 * torch.randn(D + 1, generator=g))[1:] for _ in range(2)]
    pos = _positions(N, 2, g, batch=B)
    sec = sections_for(D, 2)
    rot = fw.wsattn_rotary_plan(D, sec)
    dev = rows.cuda().transpose(1, 2)
    wd = [torch.empty(D + 1, device="cuda")[1:].copy_(x) for x in w]   # gains off 16 bytes
    got = fw.wsattn_qknorm(rot, dev[:, :heads], dev[:, heads:heads + kv], pos.cuda(), wd[0], wd[1],
                           eps, v=dev[:, heads + kv:])
    ang = angles(pos, sec, D)
    for i in range(2):
        _, y, _ = normed(parts[i].double(), w[i].double(), eps)
        want = turn(y, ang, True)
        tol = half_step(torch.bfloat16) * want.abs() + (TURN + 2 * NORM) * _pairmax(y, True)
        assert_close(got[i], want, tol + tiny(torch.bfloat16), f"part {i}")
    assert torch.equal(got[2].cpu(), parts[2])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("pad", [0, 3])
def test_qknorm_backward_in_place(dt, pad):
    # gradients over the incoming ones, and over the forward's inputs; rows on
    # 16 bytes (the asynchronous ring) and off them
    fw = _fw()
    B, H, N, D, eps = 2, 5, 700, 64, 1e-5
    g = _gen(41)

    def heads():
        buf = torch.randn((B, H, N, D + pad), generator=g).to(dt).cuda()
        return buf[..., :D]
    q, k, gq, gk = heads(), heads(), heads(), heads()
    w = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    pos = _positions(N, 1, g).cuda()
    rot = fw.wsattn_rotary_plan(D, (32,))
    dq, dk, _, dwq, dwk = fw.wsattn_qknorm_backward(rot, gq, gk, q, k, pos, w, w, eps)
    over = [t.clone() for t in (gq, gk, q, k)]  # clone of a view: contiguous rows of D
    a = fw.wsattn_qknorm_backward(rot, over[0], over[1], q, k, pos, w, w, eps, dq=over[0], dk=over[1])
    assert a[0] is over[0] and torch.equal(over[0], dq) and torch.equal(over[1], dk)
    a = fw.wsattn_qknorm_backward(rot, gq, gk, over[2], over[3], pos, w, w, eps, dq=over[2], dk=over[3])
    assert torch.equal(over[2], dq) and torch.equal(over[3], dk)
    assert torch.equal(a[3], dwq) and torch.equal(a[4], dwk)


def test_binding_refusals():
    fw = _fw()
    rot = fw.wsattn_rotary_plan(64, (16, 16))
    x = torch.zeros((2, 3, 5, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((5, 2), device="cuda")
    ok = fw.wsattn_rotary(rot, x, pos)
    for bad, err in (
            (lambda: fw.wsattn_rotary(rot, x[..., :32], pos), ValueError),
            (lambda: fw.wsattn_rotary(rot, x.transpose(2, 3), pos), ValueError),
            (lambda: fw.wsattn_rotary(rot, x[:, :, ::2, ::1].transpose(0, 1)[..., ::1], pos), ValueError),
            (lambda: fw.wsattn_rotary(rot, x, pos.double()), TypeError),
            (lambda: fw.wsattn_rotary(rot, x, pos[:, :1]), ValueError),
            (lambda: fw.wsattn_rotary(rot, x, torch.zeros((2, 5), device="cuda").t()), ValueError),
            (lambda: fw.wsattn_rotary(rot, x, pos.cpu()), TypeError),
            (lambda: fw.wsattn_rotary(rot, x.to(torch.int16), pos), TypeError),
            (lambda: fw.wsattn_rotary(rot, x, pos, out=ok.float()), TypeError),
            (lambda: fw.wsattn_rotary(rot, x, pos, out=ok[:1]), ValueError),
            (lambda: fw.wsattn_rotary(rot, x, pos, out=ok[:, :1].expand(2, 3, 5, 64)), fw.WsattnError),
            (lambda: fw.wsattn_qknorm(rot, x, x.half(), pos), TypeError),
            (lambda: fw.wsattn_qknorm(rot, x, x[:1], pos), ValueError),
            (lambda: fw.wsattn_qknorm(rot, x, x, pos, q_weight=pos[:, 0]), ValueError),
            (lambda: fw.wsattn_qknorm(rot, x, x, pos, eps=-1.0), fw.WsattnError),
            (lambda: fw.wsattn_qknorm(rot, x, x, pos, v_out=ok), ValueError),
            (lambda: fw.wsattn_qknorm(rot, x, x, pos, torch.ones(64, device="cuda"),
                                      torch.ones(64, device="cuda").bfloat16()), TypeError),
            (lambda: fw.wsattn_qknorm_backward(rot, x, x, x, x, pos, dv=ok), ValueError),
            (lambda: fw.wsattn_qknorm_backward(rot, x, x, x, x, pos, torch.ones(64, device="cuda"),
                                               workspace=torch.empty(8, device="cuda")), fw.WsattnError)):
        with pytest.raises(err):
            bad()


def test_rates_given_pair_by_pair():
    # any axis for any pair, any rate, one column of the positions not used
    fw = _fw()
    g = _gen(51)
    D, N = 32, 50
    axis = torch.randint(0, 2, (16,), generator=g)
    freq = torch.randn(16, generator=g, dtype=torch.float64)
    freq[3] = 0
    rot = fw.wsattn_rotary_plan(D, pair_axis=axis.tolist(), pair_freq=freq.tolist(), axes=3,
                                interleaved=False)
    pos = 40 * torch.randn((N, 3), generator=g)
    x = torch.randn((1, 2, N, D), generator=g)
    want = turn(x.double(), pos.double()[:, axis] * freq, False)
    got = fw.wsattn_rotary(rot, x.cuda(), pos.cuda())
    assert_close(got, want, _turn_tol(x.double(), want, False, torch.float32))


def test_more_than_2_to_31_elements():
    # the last heads and tokens of a tensor whose offsets pass 32 bits
    fw = _fw()
    H, N, D = 34, 500000, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    x = torch.empty((1, H, N, D), dtype=torch.bfloat16, device="cuda").normal_()
    assert x.numel() > 1 << 31
    pos = torch.arange(N, device="cuda", dtype=torch.float32)[:, None].contiguous()
    rot = fw.wsattn_rotary_plan(D, (64,))
    w = torch.full((D,), 1.5, device="cuda")
    for y, gain in ((fw.wsattn_rotary(rot, x, pos), None),
                    (fw.wsattn_qknorm(rot, x, x[:, :1], pos, w, w, 1e-6)[0], 1.5)):
        for h, n0 in ((0, 0), (H - 1, N - 300), (H - 2, N // 2)):
            part = x[:, h:h + 1, n0:n0 + 300].cpu().double()
            if gain:
                part = gain * normed(part, None, 1e-6)[0]
            want = turn(part, angles(pos[n0:n0 + 300], (64,), D), True)
            tol = _turn_tol(part, want, True, torch.bfloat16) + 2 * NORM * _pairmax(part, True)
            assert_close(y[:, h:h + 1, n0:n0 + 300], want, tol)
        del y
