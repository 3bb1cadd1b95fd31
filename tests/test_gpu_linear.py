"""wsattn_linear and wsattn_linear_backward against their 64-bit definitions
(GPU).  Tolerances: half a step of the stored type, the tensor cores' fp32
error on the sum of magnitudes (_ops_ref.product_tol), 2^-20 relative for the
activation (its slope is at most 1.13); the gradients' products read a dz that
was itself rounded by half a step."""
import pytest
import torch

from _ops_ref import act, assert_close, half_step, product_tol, tiny

pytestmark = pytest.mark.gpu


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


def _case(m, n, k, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, k), generator=g).to(dt)
    w = (torch.randn((n, k), generator=g) / k ** 0.5).to(dt)
    b = (0.5 * torch.randn(n, generator=g)).to(dt)
    r = torch.randn((m, n), generator=g)
    return x, w, b, r


SHAPES = [
    # m, n, k
    (1, 1, 1), (1, 256, 320), (3, 130, 64), (1, 1000, 1500), (17, 96, 520),
    (33, 333, 77), (100, 1024, 1024), (129, 257, 65), (240, 384, 128), (256, 256, 256),
    (300, 511, 999), (700, 640, 200), (2080, 1024, 1024), (5000, 384, 64), (1, 8, 4096),
    (4100, 2304, 192), (20000, 20, 40), (70000, 9, 24),
]


def _check_forward(fw, x, w, b, r, name, dt, odt, want_pre=True):
    m, n = x.shape[0], w.shape[0]
    xd, wd = x.double(), w.double()
    z = xd @ wd.t() + (0 if b is None else b.double())
    s = xd.abs() @ wd.abs().t() + (0 if b is None else b.double().abs())
    ztol = product_tol(s, x.shape[1])
    want = act(z, name) + (0 if r is None else r.to(odt).double())
    pre = torch.full((m, n), 9.0, dtype=dt, device="cuda") if want_pre else None
    got = fw.wsattn_linear(x.cuda(), w.cuda(), None if b is None else b.cuda(),
                           None if r is None else r.to(odt).cuda(), name, preact=pre,
                           out_dtype=odt)
    torch.cuda.synchronize()
    assert fw.wsattn_op_status() == 0
    tol = 1.13 * ztol + 2.0 ** -20 * z.abs() + half_step(odt) * want.abs() + tiny(odt)
    assert_close(got, want, tol, "out")
    if want_pre:
        assert_close(pre, z, ztol + half_step(dt) * z.abs() + tiny(dt), "preact")
    return got


@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=str)
def test_linear_shapes(shape, dt):
    m, n, k = shape
    x, w, b, r = _case(m, n, k, dt, m + n + k)
    _check_forward(_fw(), x, w, b, r, "silu", dt, dt)
    _check_forward(_fw(), x, w, None, None, "none", dt, dt, want_pre=False)


@pytest.mark.parametrize("odt", [torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("shape", [(300, 512, 57600), (261, 501, 66001)], ids=lambda c: "x".join(map(str, c)))
def test_linear_split_contraction(shape, odt):
    # four tiles of 256 x 256 and a long contraction: 16 parts each, added by
    # a second kernel with the epilogue
    fw = _fw()
    m, n, k = shape
    x, w, b, r = _case(m, n, k, torch.float16, 12)
    x, w = x.cuda(), w.cuda()
    assert fw.wsattn_linear_workspace(x, w) >= 4 * 16 * 256 * 256 * 4
    z = (x.double() @ w.double().t()).cpu() + b.double()
    ztol = product_tol((x.double().abs() @ w.double().abs().t()).cpu() + b.double().abs(), k)
    pre = torch.empty((m, n), dtype=torch.float16, device="cuda")
    got = fw.wsattn_linear(x, w, b.cuda(), r.to(odt).cuda(), "gelu_tanh", preact=pre, out_dtype=odt)
    torch.cuda.synchronize()
    assert fw.wsattn_op_status() == 0
    want = act(z, "gelu_tanh") + r.to(odt).double()
    assert_close(got, want, 1.13 * ztol + 2.0 ** -20 * z.abs() + half_step(odt) * want.abs() + tiny(odt))
    assert_close(pre, z, ztol + half_step(torch.float16) * z.abs() + tiny(torch.float16))
    buf = r.to(odt).cuda()     # the residual in place: the same values
    fw.wsattn_linear(x, w, b.cuda(), buf, "gelu_tanh", out=buf)
    assert torch.equal(buf, got)


def test_linear_backward_split_contraction():
    # dw [300, 500] over 57601 rows is split, dx is not; one after the other
    fw = _fw()
    m, n, k = 57601, 300, 500
    dt = torch.bfloat16
    x, w, _, _ = _case(m, n, k, dt, 21)
    dy = (0.3 * torch.randn((m, n), generator=torch.Generator().manual_seed(1))).to(dt)
    args = (dy.cuda(), x.cuda(), w.cuda())
    assert fw.wsattn_linear_backward_workspace(*args, need_db=False) >= 4 * 16 * 256 * 256 * 4
    dx, dw, _ = fw.wsattn_linear_backward(*args, need_db=False)
    torch.cuda.synchronize()
    assert fw.wsattn_op_status() == 0
    d, xd, wd = (t.double() for t in args)
    for got, want, mag, kk in ((dx, d @ wd, d.abs() @ wd.abs(), n),
                               (dw, d.t() @ xd, d.abs().t() @ xd.abs(), m)):
        want, mag = want.cpu(), mag.cpu()
        assert_close(got, want, product_tol(mag, kk) + half_step(dt) * want.abs() + tiny(dt))
    again = fw.wsattn_linear_backward(*args, need_db=False)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("name", ["none", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("shape", [(5, 200, 136), (600, 700, 264), (1100, 2056, 72), (513, 131, 72)],
                         ids=lambda c: "x".join(map(str, c)))
def test_linear_activations_and_types(shape, odt, name):
    m, n, k = shape
    x, w, b, r = _case(m, n, k, torch.bfloat16, 5)
    _check_forward(_fw(), x, w, b, r, name, torch.bfloat16, odt)
    _check_forward(_fw(), x, w, b, None, name, torch.bfloat16, odt, want_pre=False)


@pytest.mark.parametrize("shape", [(40, 264, 72), (900, 520, 200)], ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("pad", [3, 8])
def test_linear_strided_rows_and_residual_in_place(shape, pad):
    # rows inside wider buffers (odd and 16-byte strides): the gaps stay as they were
    fw = _fw()
    dt = torch.bfloat16
    m, n, k = shape
    x, w, b, r = _case(m, n, k, dt, 77)

    def wide(t):
        buf = torch.full((t.shape[0], t.shape[1] + pad), 5.0, dtype=dt, device="cuda")
        buf[:, :t.shape[1]] = t.to(dt).cuda()
        return buf
    xb, wb, ob, pb = wide(x), wide(w), wide(r), wide(r)
    want = fw.wsattn_linear(x.cuda(), w.cuda(), b.cuda(), r.to(dt).cuda(), "gelu")
    out = fw.wsattn_linear(xb[:, :k], wb[:, :k], b.cuda(), ob[:, :n], "gelu", preact=pb[:, :n],
                           out=ob[:, :n])
    assert torch.equal(out, want)
    for buf, c in ((ob, n), (pb, n), (xb, k), (wb, k)):
        assert (buf[:, c:] == 5.0).all()
    # leading dimensions fold into rows
    if m % 4 == 0:
        y = fw.wsattn_linear(x.cuda().view(2, m // 4, 2, k), w.cuda(), b.cuda(),
                             r.to(dt).cuda().view(2, m // 4, 2, n), "gelu")
        assert torch.equal(y.view(m, n), want)


@pytest.mark.parametrize("dims", [(1, 2, 48, 64), (2, 3, 100, 128), (1, 5, 1, 8)])
def test_linear_of_attention_output(dims):
    # fp32 [B, H, N, D]: heads merged, rounded once
    fw = _fw()
    B, H, N, D = dims
    g = torch.Generator().manual_seed(4)
    a = torch.randn(dims, generator=g)
    w = (torch.randn((72, H * D), generator=g) / (H * D) ** 0.5).to(torch.bfloat16)
    got = fw.wsattn_linear(a.cuda(), w.cuda())
    rows = a.transpose(1, 2).reshape(B, N, H * D).to(torch.bfloat16)
    want = fw.wsattn_linear(rows.cuda(), w.cuda())
    assert got.shape == (B, N, 72) and torch.equal(got, want)


def _slope64(z, name):
    z = z.clone().requires_grad_(True)
    act(z, name).sum().backward()
    return z.grad


@pytest.mark.parametrize("name", ["none", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 264, 136), (37, 77, 33), (130, 200, 72), (333, 256, 512),
                                   (1030, 515, 90), (3000, 128, 64), (640, 1288, 1160), (9000, 20, 36)],
                         ids=lambda c: "x".join(map(str, c)))
def test_linear_backward(shape, dt, name):
    fw = _fw()
    m, n, k = shape
    x, w, _, r = _case(m, n, k, dt, 3 * m + n)
    g = torch.Generator().manual_seed(1)
    dy = (0.3 * torch.randn((m, n), generator=g)).to(dt)
    z = None if name == "none" else (1.5 * r).to(dt)
    args = (dy.cuda(), x.cuda(), w.cuda(), None if z is None else z.cuda(), name)
    dx, dw, db = fw.wsattn_linear_backward(*args)
    torch.cuda.synchronize()
    assert fw.wsattn_op_status() == 0
    dz = dy.double() * (1 if z is None else _slope64(z.double(), name))
    # of dz: half a step where it is rounded, 2^-19 relative to dout for the slope
    dztol = (0 if z is None else half_step(dt) * dz.abs() + 2.0 ** -19 * dy.double().abs() + tiny(dt))
    wa, xa = w.double().abs(), x.double().abs()
    # each gradient by itself too (its product may be tiled, and so summed, another way)
    only_dx = fw.wsattn_linear_backward(*args, need_dw=False, need_db=False)
    only_dw = fw.wsattn_linear_backward(*args, need_dx=False, need_db=False)
    only_db = fw.wsattn_linear_backward(*args, need_dx=False, need_dw=False)
    assert only_dx[1:] == (None, None) and only_dw[::2] == (None, None)
    assert only_db[:2] == (None, None) and torch.equal(only_db[2], db)
    for got, want, mag, extra, kk in (
            ((dx, only_dx[0]), dz @ w.double(), dz.abs() @ wa, dztol @ wa if z is not None else 0, n),
            ((dw, only_dw[1]), dz.t() @ x.double(), dz.abs().t() @ xa,
             dztol.t() @ xa if z is not None else 0, m)):
        tol = 1.01 * extra + product_tol(mag, kk) + half_step(dt) * want.abs() + tiny(dt)
        for t in got:
            assert_close(t, want, tol)
    sums = dz.abs().sum(0)
    assert_close(db, dz.sum(0), (2.0 ** -19 + (m / 64 + 32) * 2.0 ** -24) * (sums + dy.double().abs().sum(0)))
    again = fw.wsattn_linear_backward(*args)
    for a, b in zip(again, (dx, dw, db)):
        assert torch.equal(a, b)


def test_linear_empty():
    fw = _fw()
    w = torch.ones((5, 7), dtype=torch.bfloat16, device="cuda")
    x = torch.empty((0, 7), dtype=torch.bfloat16, device="cuda")
    assert fw.wsattn_linear(x, w).shape == (0, 5)
    dx, dw, db = fw.wsattn_linear_backward(torch.empty((0, 5), dtype=torch.bfloat16, device="cuda"), x, w)
    assert dx.shape == (0, 7) and torch.equal(dw, torch.zeros_like(w)) and (db == 0).all()


def test_linear_extreme_values():
    # activations at the ends of bf16's range; rows of infinities reach their own rows only
    fw = _fw()
    dt = torch.bfloat16
    x = torch.zeros((300, 64), dtype=dt)
    x[:, 0] = 1
    w = torch.zeros((8, 64), dtype=dt)
    w[:, 0] = torch.tensor([1e30, -1e30, 100.0, -100.0, 0.0, -0.0, 3e38, -3e38])
    for name in ("gelu", "gelu_tanh", "silu"):
        y = fw.wsattn_linear(x.cuda(), w.cuda(), activation=name).cpu().float()
        want = torch.relu(w[:, 0].float())
        assert torch.equal(y, want.expand(300, 8)), name
        z = w[:, 0].expand(300, 8).contiguous()
        one = torch.ones((300, 8), dtype=dt)
        _, _, db = fw.wsattn_linear_backward(one.cuda(), x.cuda(), w.cuda(), z.cuda(), name)
        assert torch.equal(db.cpu(), 300 * torch.tensor([1, 0, 1, 0, 0.5, 0.5, 1, 0])), name
    x[7, 3] = float("inf")
    w[:, 3] = 1
    y = fw.wsattn_linear(x.cuda(), w.cuda()).cpu()
    assert y[7].isinf().all() and torch.isfinite(y[:7]).all() and torch.isfinite(y[8:]).all()


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_activations_keep_their_relative_precision(name):
    """Every bf16 value up to 12, the far negative side too: value and slope.
    The exponential's argument T has up to six roundings of 2^-24 on its way
    (2^-21 T relative in the result); the reciprocal, the exponential, the fit
    of the normal distribution and the products are below 2^-18 together, and
    a logistic or exponential below 2^-126 may be flushed to zero, which the
    value multiplies by |z| and the slope by |z| u'(z), up to 12 * 33."""
    fw = _fw()
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    z = bits.view(torch.bfloat16)
    z = z[z.float().abs() <= 12]
    z = z[: z.numel() // 8 * 8]
    zd = z.double()
    phi = torch.exp(-zd * zd / 2) / (2 * torch.pi) ** 0.5
    if name == "gelu":
        s = 0.5 * torch.special.erfc(-zd / 2 ** 0.5)
        arg, slope, mag, du = zd * zd / 2, s + zd * phi, s + zd.abs() * phi, 1
    else:
        u = zd if name == "silu" else (8 / torch.pi) ** 0.5 * (zd + 0.044715 * zd ** 3)
        du = torch.ones_like(zd) if name == "silu" else (8 / torch.pi) ** 0.5 * (1 + 0.134145 * zd ** 2)
        s, other = 1 / (1 + torch.exp(-u)), 1 / (1 + torch.exp(u))
        # the slope's 1 - s is rounded at the size of s
        arg, slope, mag = u.abs(), s + zd * s * other * du, s * (1 + zd.abs() * du)
    rel = 2.0 ** -18 + 2.0 ** -21 * arg
    # value: one product with 1, so that the activation's argument is z itself
    x = torch.zeros((z.numel(), 8), dtype=torch.bfloat16)
    x[:, 0] = z
    w = torch.zeros((8, 8), dtype=torch.bfloat16)
    w[:, 0] = 1
    got = fw.wsattn_linear(x.cuda(), w.cuda(), activation=name, out_dtype=torch.float32)
    want = (zd * s)[:, None].expand(-1, 8)
    flush = 2.0 ** -125 * (1 + zd.abs())
    assert_close(got, want, (rel * want[:, 0].abs() + flush)[:, None].expand(-1, 8), "value")
    # slope: the bias gradient of one row is dz itself
    one = torch.ones((1, z.numel()), dtype=torch.bfloat16)
    wide = torch.zeros((z.numel(), 8), dtype=torch.bfloat16)
    _, _, db = fw.wsattn_linear_backward(one.cuda(), one[:, :8].contiguous().cuda(), wide.cuda(),
                                         z[None].contiguous().cuda(), name, need_dx=False, need_dw=False)
    # z = -10.0625 in the tanh form: u = -88.8, logistic 2.7e-39 (flushed), |z| u' = 224
    assert_close(db, slope, rel * mag + 2.0 ** -125 * (1 + zd.abs() * du), "slope")
    assert fw.wsattn_op_status() == 0


def test_linear_capture_and_streams():
    fw = _fw()
    dt = torch.bfloat16
    x, w, b, r = _case(300, 257, 77, dt, 8)   # odd widths: operands go through the workspace
    x, w, b, r = x.cuda(), w.cuda(), b.cuda(), r.to(dt).cuda()
    want = fw.wsattn_linear(x, w, b, r, "gelu")
    grads = fw.wsattn_linear_backward(r, x, w, r, "silu")
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = fw.wsattn_linear(x, w, b, r, "gelu")
            d = fw.wsattn_linear_backward(r, x, w, r, "silu")
        graphs.append((graph, y, d))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (graph, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, y, d in graphs:
        assert torch.equal(y, want)
        for a, c in zip(d, grads):
            assert torch.equal(a, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = fw.wsattn_linear(x, w, b, r, "gelu", stream=side)
    side.synchronize()
    assert torch.equal(y, want)


def test_linear_more_than_2_to_31_elements():
    # outputs, pre-activations and residuals whose offsets pass 32 bits
    fw = _fw()
    m, n, k = 540000, 4104, 64
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    dt = torch.bfloat16
    x = torch.empty((m, k), dtype=dt, device="cuda").normal_()
    w = (torch.empty((n, k), device="cuda").normal_() / 8).to(dt)
    r = torch.empty((m, n), dtype=dt, device="cuda").normal_()
    assert r.numel() > 1 << 31
    z = torch.empty_like(r)
    y = fw.wsattn_linear(x, w, residual=r, activation="silu", preact=z)
    dx, dw, db = fw.wsattn_linear_backward(r, x, w, preact=z, activation="silu")
    torch.cuda.synchronize()
    assert fw.wsattn_op_status() == 0
    for rows in (slice(0, 300), slice(m // 2, m // 2 + 300), slice(m - 300, m)):
        zz = x[rows].double() @ w.double().t()
        ztol = product_tol(x[rows].double().abs() @ w.double().abs().t(), k)
        assert_close(z[rows], zz.cpu(), (ztol + half_step(dt) * zz.abs() + tiny(dt)).cpu())
        want = act(zz, "silu") + r[rows].double()
        assert_close(y[rows], want.cpu(),
                     (1.13 * ztol + 2.0 ** -20 * zz.abs() + half_step(dt) * want.abs()).cpu())
        dz = r[rows].double() * _slope64(z[rows].double(), "silu")
        want = dz @ w.double()
        tol = (1.01 * half_step(dt) + 2.0 ** -19) * (dz.abs() + r[rows].double().abs() * 2.0 ** -10) @ w.double().abs()
        tol = tol + product_tol(dz.abs() @ w.double().abs(), n) + half_step(dt) * want.abs()
        assert_close(dx[rows], want.cpu(), tol.cpu())


def test_first_call_may_be_captured():
    # a fresh process whose first call of each operator is inside a capture
    import subprocess
    import sys
    code = """
import torch, frame_aligned_window_gb300 as fw
x = torch.randn(300, 77, device="cuda").bfloat16(); w = torch.randn(40, 77, device="cuda").bfloat16()
q = torch.randn(1, 2, 9, 64, device="cuda"); pos = torch.zeros(9, 1, device="cuda")
rot = fw.wsattn_rotary_plan(64, (32,))
def run():
    y = fw.wsattn_linear(x, w, activation="silu")
    d = fw.wsattn_linear_backward(y, x, w, preact=y, activation="silu")
    a = fw.wsattn_qknorm(rot, q, q, pos)
    b = fw.wsattn_qknorm_backward(rot, q, q, q, q, pos, q[0, 0, 0], q[0, 0, 1])
    return [y, *d, *a, b[0], b[3], fw.wsattn_rotary(rot, q, pos)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = run()
g.replay()
torch.cuda.synchronize()
want = run()
assert all(torch.equal(a, b) for a, b in zip(out, want)) and fw.wsattn_op_status() == 0
print("captured")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_binding_refusals():
    fw = _fw()
    x = torch.zeros((6, 24), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((16, 24), dtype=torch.bfloat16, device="cuda")
    y = fw.wsattn_linear(x, w)
    for bad, err in (
            (lambda: fw.wsattn_linear(x[:, :23], w), ValueError),
            (lambda: fw.wsattn_linear(x.half(), w), TypeError),
            (lambda: fw.wsattn_linear(x.float(), w.float()), TypeError),
            (lambda: fw.wsattn_linear(x, w.t()), ValueError),
            (lambda: fw.wsattn_linear(x.t().contiguous().t(), w), ValueError),
            (lambda: fw.wsattn_linear(x[:1].expand(6, 24), w), ValueError),
            (lambda: fw.wsattn_linear(x, w, activation="relu"), ValueError),
            (lambda: fw.wsattn_linear(x, w, bias=torch.zeros(15, dtype=x.dtype, device="cuda")), ValueError),
            (lambda: fw.wsattn_linear(x, w, bias=torch.zeros(16, device="cuda")), TypeError),
            (lambda: fw.wsattn_linear(x, w, residual=y.float()), TypeError),
            (lambda: fw.wsattn_linear(x, w, residual=y[:5]), ValueError),
            (lambda: fw.wsattn_linear(x, w, residual=y[:1].expand(6, 16)), ValueError),
            (lambda: fw.wsattn_linear(x, w, out=y, out_dtype=torch.float32), TypeError),
            (lambda: fw.wsattn_linear(x, w, out_dtype=torch.float16), TypeError),
            (lambda: fw.wsattn_linear(x, w, preact=y.float()), TypeError),
            (lambda: fw.wsattn_linear(x.cpu(), w), TypeError),
            (lambda: fw.wsattn_linear(torch.zeros((1, 3, 2, 7), device="cuda"), w), ValueError),
            (lambda: fw.wsattn_linear(torch.zeros((1, 6, 2, 4), device="cuda"), w), fw.WsattnError),
            (lambda: fw.wsattn_linear(x[:, :23].contiguous(), w[:, :23].contiguous(),
                                      workspace=torch.empty(16, device="cuda")), fw.WsattnError),
            (lambda: fw.wsattn_linear_backward(y, x, w, activation="gelu"), ValueError),
            (lambda: fw.wsattn_linear_backward(y[:5], x, w), ValueError),
            (lambda: fw.wsattn_linear_backward(y, x, w, dw=w.float()), TypeError),
            (lambda: fw.wsattn_linear_backward(y, x, w, db=torch.zeros(16, dtype=x.dtype, device="cuda")),
             TypeError)):
        with pytest.raises(err):
            bad()
    assert fw.wsattn_op_status() == 0
