"""wsattn_linear and wsattn_linear_backward under every tiling that the library
chooses.  The first test runs on the CPU: it asks the library for the tiling
of each shape below, so that a shape whose tiling changes is noticed.  The
others compare the products with their 64-bit definitions (GPU; tolerances as
in test_gpu_linear.py)."""
import ctypes

import pytest
import torch

from _ops_ref import act, assert_close, half_step, product_tol, tiny

# m, n, k of x [m, k], w [n, k]
FORWARD = [
    (20, 96, 40), (17, 92, 201), (17, 97, 453), (756, 145, 592), (289, 136, 272),       # 16 rows a tile
    (1549, 129, 967), (18, 4776, 354), (17, 2560, 400), (17, 1048, 520),                # 32
    (3029, 130, 2681), (2485, 148, 1511), (33, 4103, 675), (36, 3612, 977),             # 64
    (530, 3233, 7873), (4962, 144, 4080), (69, 4672, 4315), (66, 3140, 2349),           # 128
    (1353, 133, 42), (301, 4904, 72),                                                   # pairs
    (239, 4256, 8448), (1549, 2783, 2014), (2080, 2304, 2056),                          # a split last round
]
BACKWARD = [
    (1108, 2445, 44), (798, 95, 42), (1267, 1952, 40), (2985, 2992, 135), (7515, 2656, 40),
    (8070, 280, 5224), (4132, 4945, 142), (2007, 96, 6704), (20, 96, 40), (66, 264, 4880),
    (18, 205, 41), (17, 476, 42), (636, 257, 42), (1506, 592, 48), (3117, 1056, 40), (17, 448, 2440),
    (33, 710, 4518), (67, 2526, 3395), (6400, 2862, 42), (17, 337, 4935), (33, 999, 3106), (33, 1316, 4801),
    (65, 1619, 6821), (4936, 4136, 136), (17, 616, 1048), (2472, 111, 40), (270, 91, 4885),
    (6575, 1340, 975), (3577, 4968, 512), (1708, 1008, 5000), (6430, 2456, 544),
]


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


class Shape(ctypes.Structure):  # GemmShape of csrc/ops.h
    _fields_ = [(n, ctypes.c_int) for n in ("pair_cols", "bn", "split", "whole")]


def _tilings():
    """(rows, columns, contraction, rows lie along the contraction?) -> (tiling,
    nanoseconds), and the time of both gradients in one launch."""
    lib = ctypes.CDLL(_fw().LIB_PATH)   # internal functions, by their C++ names
    choose = lib._ZN6wsattn11choose_gemmEliibPd
    choose.restype = Shape
    choose.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_bool,
                       ctypes.POINTER(ctypes.c_double)]
    two = lib._ZN6wsattn16pair_time_of_twoEliilii
    two.restype = ctypes.c_double
    two.argtypes = 2 * [ctypes.c_int64, ctypes.c_int, ctypes.c_int]

    def tiling(rows, cols, k, mn):
        ns = ctypes.c_double()
        s = choose(rows, cols, k, mn, ctypes.byref(ns))
        if s.pair_cols:
            return (s.pair_cols, s.split > 1, s.whole > 0), ns.value
        return (s.bn, s.split), ns.value
    return tiling, two


def test_shapes_cover_every_tiling():
    tiling, two = _tilings()
    fwd = {tiling(m, n, k, False)[0] for m, n, k in FORWARD}
    dw, dx, together = set(), set(), set()
    for m, n, k in BACKWARD:
        (a, ta), (b, tb) = tiling(n, k, m, True), tiling(m, k, n, False)
        dw.add(a)
        dx.add(b)
        together.add(two(n, k, m, m, k, n) < ta + tb)
    pairs = {(128, False, False), (256, False, False), (256, True, False), (256, True, True)}
    few = {(16, s) for s in (1, 2, 3, 4, 8)} | {(32, s) for s in (2, 3, 4, 8)} | {(64, s) for s in (2, 3, 4, 8)}
    assert fwd == pairs | few | {(128, s) for s in (2, 3, 4, 8)}
    # (the operand with the rows side by side needs 64 of them)
    assert dw == pairs | {(r, s) for r in (64, 128) for s in (2, 3, 4, 8)}
    assert dx == pairs | few | {(128, s) for s in (3, 4, 8)}
    assert together == {False, True}


def _ints(shape, most, g, dtype):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("odt", [torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("shape", FORWARD, ids=lambda c: "x".join(map(str, c)))
def test_linear_under_every_tiling(shape, odt):
    fw = _fw()
    m, n, k = shape
    dt = torch.float16
    g = torch.Generator(device="cuda").manual_seed(m + n + k)

    def normal(*s, std=1.0, dtype=dt):
        return (std * torch.randn(s, generator=g, device="cuda")).to(dtype)
    x, w, b, r = normal(m, k), normal(n, k, std=k ** -0.5), normal(n, std=0.5), normal(m, n, dtype=odt)
    z = x.double() @ w.double().t() + b.double()
    ztol = product_tol(x.double().abs() @ w.double().abs().t() + b.double().abs(), k)
    want = act(z, "silu") + r.double()
    pre = torch.full((m, n), 9.0, dtype=dt, device="cuda")
    got = fw.wsattn_linear(x, w, b, r, "silu", preact=pre, out_dtype=odt)
    assert fw.wsattn_op_status() == 0
    tol = 1.13 * ztol + 2.0 ** -20 * z.abs() + half_step(odt) * want.abs() + tiny(odt)
    assert_close(got, want.cpu(), tol.cpu(), "out")
    assert_close(pre, z.cpu(), (ztol + half_step(dt) * z.abs() + tiny(dt)).cpu(), "preact")
    buf = r.clone()
    fw.wsattn_linear(x, w, b, buf, "silu", out=buf)
    assert torch.equal(buf, got)
    # small whole numbers: every sum is exact, so is the result
    x, w, r = _ints((m, k), 2, g, dt), _ints((n, k), 1, g, dt), _ints((m, n), 9, g, odt)
    want = x.double() @ w.double().t() + r.double()
    assert torch.equal(fw.wsattn_linear(x, w, residual=r, out_dtype=odt), want.to(odt))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", BACKWARD, ids=lambda c: "x".join(map(str, c)))
def test_linear_backward_under_every_tiling(shape):
    fw = _fw()
    m, n, k = shape
    dt = torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    # small whole numbers, and slopes that are 0, 1/2 and 1: every sum is exact
    dy, x, w = _ints((m, n), 2, g, dt), _ints((m, k), 2, g, dt), _ints((n, k), 2, g, dt)
    z = 300 * _ints((m, n), 1, g, dt)
    dz = dy.double() * (z.double().sign() + 1) / 2
    want = ((dz @ w.double()).to(dt), (dz.t() @ x.double()).to(dt), dz.sum(0).float())
    got = fw.wsattn_linear_backward(dy, x, w, z, "silu")
    only_dx = fw.wsattn_linear_backward(dy, x, w, z, "silu", need_dw=False)
    only_dw = fw.wsattn_linear_backward(dy, x, w, z, "silu", need_dx=False)
    assert fw.wsattn_op_status() == 0
    for i, t in enumerate((got, only_dx, only_dw)):
        for j, name in enumerate(("dx", "dw", "db")):
            if t[j] is not None:
                assert torch.equal(t[j], want[j]), (name, i)
    assert only_dx[1] is None and only_dw[0] is None
    # the two orders of the products' operands with values of every size
    dy, x, w = (torch.randn(t.shape, generator=g, device="cuda").to(dt) for t in (dy, x, w))
    for need_dx, need_dw in ((True, True), (True, False), (False, True)):
        dx, dw, _ = fw.wsattn_linear_backward(dy, x, w, need_dx=need_dx, need_dw=need_dw, need_db=False)
        d, xd, wd = dy.double(), x.double(), w.double()
        for t, a, b, kk in ((dx, d, wd, n), (dw, d.t(), xd, m)):
            if t is not None:
                v, mag = a @ b, a.abs() @ b.abs()
                assert_close(t, v.cpu(), (product_tol(mag, kk) + half_step(dt) * v.abs() + tiny(dt)).cpu())
