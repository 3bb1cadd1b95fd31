"""A transformer block through the library (GPU): projection with bias ->
qknorm (norms, three-axis rotary, packing) -> prepare -> forward -> output
projection with residual (reads the attention's fp32 heads) -> feed-forward
with gelu -> second product with residual, and the feed-forward's backward
pass.  Every stage is checked against its 64-bit definition on the values that
entered it, so each stage's own tolerance holds; the chain is then captured
into a graph and replayed."""
import pytest
import torch

import oracle
from _helpers import TOL_MAX_ABS, TOL_REL_L2, rel_l2
from _ops_ref import NORM, TURN, act, angles, assert_close, half_step, normed, product_tol, turn
from workloads import WORKLOADS

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _weights(c, wide, seed):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std):
        return (std * torch.randn(shape, generator=g)).to(BF).cuda()
    return dict(wqkv=normal(3 * c, c, std=c ** -0.5), bqkv=normal(3 * c, std=0.1),
                wo=normal(c, c, std=c ** -0.5), bo=normal(c, std=0.1),
                w1=normal(wide, c, std=c ** -0.5), b1=normal(wide, std=0.1),
                w2=normal(c, wide, std=wide ** -0.5), b2=normal(c, std=0.1),
                gain=1 + normal(128, std=0.1))


def _grid(wl):
    n = torch.arange(wl.n_tokens)
    t = wl.tokens_per_frame
    return torch.stack((n // t, n % t // wl.grid_w, n % wl.grid_w), 1).float()


def _product(x, w, b, r=None):
    """64-bit x w^T + b (+ r) and the fp32 error allowed to it."""
    x, w = x.double().cpu(), w.double().cpu()
    s = x.abs() @ w.abs().t() + b.double().cpu().abs()
    want = x @ w.t() + b.double().cpu()
    return (want if r is None else want + r.double().cpu()), product_tol(s, x.shape[-1])


def _close(got, want, tol):
    assert_close(got, want, tol + half_step(got.dtype) * want.abs())


@pytest.mark.parametrize("name,batch", [("tiny", 1), ("tiny", 2), ("small", 1)])
def test_block_forward_backward_and_capture(name, batch):
    import frame_aligned_window_gb300 as fw
    wl = WORKLOADS[name]
    B, H, D, N = batch, wl.heads, wl.head_dim, wl.n_tokens
    C, wide, eps = H * D, 3 * H * D, 1e-6
    w = _weights(C, wide, 17)
    gain = w["gain"][:D].contiguous()
    g = torch.Generator().manual_seed(23)
    x = torch.randn((B, N, C), generator=g).to(BF).cuda()
    plan = fw.wsattn_plan(wl.frames, wl.tokens_per_frame, wl.window, wl.ref_frames, H, D)
    half = D // 2
    sec = (half - 2 * (half // 3), half // 3, half // 3)
    rot = fw.wsattn_rotary_plan(D, sec)
    pos = _grid(wl).cuda()
    pre = torch.empty((B, N, wide), dtype=BF, device="cuda")

    def run():
        qkv = fw.wsattn_linear(x, w["wqkv"], w["bqkv"])
        q, k, v = (t for t in qkv.view(B, N, 3, H, D).permute(2, 0, 3, 1, 4))
        q2, k2, v2 = fw.wsattn_qknorm(rot, q, k, pos, gain, gain, eps, v=v)
        fw.wsattn_prepare(plan, q2, k2)
        att = fw.wsattn_forward(plan, q2, k2, v2)
        y = fw.wsattn_linear(att, w["wo"], w["bo"], residual=x)
        h = fw.wsattn_linear(y, w["w1"], w["b1"], activation="gelu", preact=pre)
        z = fw.wsattn_linear(h, w["w2"], w["b2"], residual=y)
        # backward of the feed-forward part, for dout = z
        dh, dw2, db2 = fw.wsattn_linear_backward(z, h, w["w2"])
        dy, dw1, db1 = fw.wsattn_linear_backward(dh, y, w["w1"], preact=pre, activation="gelu")
        return dict(qkv=qkv, q=q2, k=k2, v=v2, att=att, y=y, h=h, z=z, dh=dh, dw2=dw2, db2=db2,
                    dy=dy, dw1=dw1, db1=db1)

    o = run()
    torch.cuda.synchronize()
    assert fw.wsattn_op_status() == 0 and fw.wsattn_device_status(plan) == 0
    want, tol = _product(x, w["wqkv"], w["bqkv"])
    _close(o["qkv"], want, tol)
    heads = o["qkv"].cpu().view(B, N, 3, H, D).permute(2, 0, 3, 1, 4)
    ang = angles(pos, sec, D)
    for i, key in enumerate("qk"):
        _, t, _ = normed(heads[i].double(), gain.double().cpu(), eps)
        m = t[..., 0::2].abs() + t[..., 1::2].abs()
        _close(o[key], turn(t, ang, True), (TURN + 2 * NORM) * m.repeat_interleave(2, -1))
    assert torch.equal(o["v"].cpu(), heads[2])
    if name == "tiny":  # every row against the oracle
        att = oracle.attention_full(o["q"].cpu(), o["k"].cpu(), o["v"].cpu(), wl.frames,
                                    wl.tokens_per_frame, wl.window, wl.ref_frames, wl.scale)
        got = o["att"].double().cpu().numpy().reshape(-1, N, D)
        assert abs(got - att).max() <= TOL_MAX_ABS and rel_l2(got, att) <= TOL_REL_L2
    rows = o["att"].cpu().transpose(1, 2).reshape(B, N, C).to(BF)   # merged, rounded once
    want, tol = _product(rows, w["wo"], w["bo"], x)
    _close(o["y"], want, tol)
    zz, tol = _product(o["y"], w["w1"], w["b1"])
    _close(pre, zz, tol)
    want = act(zz, "gelu")
    _close(o["h"], want, 1.13 * tol + 2.0 ** -20 * zz.abs())
    want, tol = _product(o["h"], w["w2"], w["b2"], o["y"])
    _close(o["z"], want, tol)

    zd, hd = o["z"].double().cpu().view(-1, C), o["h"].double().cpu().view(-1, wide)
    w2 = w["w2"].double().cpu()
    _close(o["dh"].view(-1, wide), zd @ w2, product_tol(zd.abs() @ w2.abs(), C))
    _close(o["dw2"], zd.t() @ hd, product_tol(zd.abs().t() @ hd.abs(), B * N))
    assert_close(o["db2"], zd.sum(0), (B * N / 64 + 40) * 2.0 ** -24 * zd.abs().sum(0))
    p = pre.double().cpu().view(-1, wide).requires_grad_(True)
    act(p, "gelu").sum().backward()
    dh = o["dh"].double().cpu().view(-1, wide)
    dz = dh * p.grad
    ztol = half_step(BF) * dz.abs() + 2.0 ** -19 * dh.abs()
    w1, yd = w["w1"].double().cpu(), o["y"].double().cpu().view(-1, C)
    _close(o["dy"].view(-1, C), dz @ w1, 1.01 * ztol @ w1.abs() + product_tol(dz.abs() @ w1.abs(), wide))
    _close(o["dw1"], dz.t() @ yd,
           1.01 * ztol.t() @ yd.abs() + product_tol(dz.abs().t() @ yd.abs(), B * N))

    # captured, and replayed twice
    keep = {k: t.clone() for k, t in o.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = run()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert fw.wsattn_op_status() == 0 and fw.wsattn_device_status(plan) == 0
    for key, t in keep.items():
        assert torch.equal(c[key], t), key


def test_early_start_waits_for_the_results_before():
    # every kernel may be set up while the one before it still runs: a long
    # chain in which each call reads what the last one wrote, many times over
    import frame_aligned_window_gb300 as fw
    g = torch.Generator().manual_seed(2)
    rot = fw.wsattn_rotary_plan(64, (16, 16))
    pos = torch.randint(0, 50, (700, 2), generator=g).float().cuda()
    w = (torch.randn((256, 256), generator=g) / 16).to(BF).cuda()
    x0 = torch.randn((1, 700, 256), generator=g).to(BF).cuda()

    def step(x, sync):
        t = x.view(1, 700, 4, 64).transpose(1, 2)
        q, k = fw.wsattn_qknorm(rot, t, t, pos)
        if sync:
            torch.cuda.synchronize()
        r = fw.wsattn_rotary(rot, q, pos, inverse=True)
        if sync:
            torch.cuda.synchronize()
        rows = r.transpose(1, 2).reshape(1, 700, 256)
        y = fw.wsattn_linear(rows, w, residual=x, activation="silu")
        if sync:
            torch.cuda.synchronize()
        dx, dw, db = fw.wsattn_linear_backward(y, rows, w, preact=y, activation="silu")
        if sync:
            torch.cuda.synchronize()
        return fw.wsattn_linear(dx, dw, residual=y)

    def chain(sync):
        x = x0
        for _ in range(12):
            x = step(x, sync)
            x = (x / x.float().abs().amax()).to(BF)
        return x
    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False), want)


RERUN = ["tests/test_gpu_linear.py::test_linear_shapes", "tests/test_gpu_linear.py::test_linear_backward",
         "tests/test_gpu_linear.py::test_linear_split_contraction",
         "tests/test_gpu_linear.py::test_linear_backward_split_contraction",
         "tests/test_gpu_linear.py::test_linear_strided_rows_and_residual_in_place",
         "tests/test_gpu_linear.py::test_linear_of_attention_output",
         "tests/test_gpu_qknorm.py::test_rotary", "tests/test_gpu_qknorm.py::test_qknorm",
         "tests/test_gpu_qknorm.py::test_qknorm_backward",
         "tests/test_gpu_block.py::test_status_in_the_bounds_checking_build"]


def test_operators_pass_bounds_checks():
    # the same parity tests in a child that loads the bounds-checking build
    import os
    import subprocess
    import sys

    import frame_aligned_window_gb300 as fw
    if os.environ.get("WSATTN_EXPECT_DEBUG") == "1":
        pytest.skip("runs in the parent process only")
    assert os.path.exists(fw.DEBUG_LIB_PATH)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, WSATTN_LIBRARY=fw.DEBUG_LIB_PATH, WSATTN_EXPECT_DEBUG="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *RERUN]
    r = subprocess.run(cmd, cwd=root, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-2000:])
    assert " passed" in r.stdout and "skipped" not in r.stdout.splitlines()[-1], r.stdout[-500:]


def test_status_in_the_bounds_checking_build():
    # last of the child's list: no check failed in any test before it
    import os

    import frame_aligned_window_gb300 as fw
    if os.environ.get("WSATTN_EXPECT_DEBUG") == "1":
        assert fw.wsattn_build_flags() & fw.BUILD_DEBUG
    assert fw.wsattn_op_status() == 0
