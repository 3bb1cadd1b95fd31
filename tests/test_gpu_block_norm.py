"""A block's norms against the 64-bit definition: types, widths, groups, odd
strides, in place, on other streams and in graphs; and their gradients, against
the formulas and against differences."""
import pytest
import torch

import _block_ref as ref
from _ops_ref import assert_close

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


def make(seed, lead, n, dt, rt, vt, mod, affine, post, norm, residual=True, spread=1.0, offset=0.0):
    """Operands of one call; mod: leading dimensions of gate, scale and shift, or None."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, dtype=dt, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, dtype=torch.float32) * std + mean).to(dtype).cuda()

    a = dict(x=normal(*lead, n, std=spread, mean=offset), residual=normal(*lead, n, dtype=rt, std=2.0, mean=offset) if residual else None)
    a["gate"] = a["scale"] = a["shift"] = a["weight"] = a["bias"] = a["post_weight"] = None
    if mod is not None:
        a["gate"], a["scale"], a["shift"] = normal(*mod, 3 * n, dtype=vt, std=0.5).split(n, -1)
    if affine:
        a["weight"] = normal(n, dtype=vt, std=0.2, mean=1.0)
        a["bias"] = normal(n, dtype=vt, std=0.2)
    if post:
        a["post_weight"] = normal(n, dtype=vt, std=0.2, mean=1.0)
    a.update(norm=norm, post_norm=post)
    return a


def check_forward(a, out, hidden, res_scale=1.0):
    y, dy, h, dh = ref.norm_forward(a["x"], a["residual"], a["gate"], a["scale"], a["shift"], a["weight"], a["bias"], a["norm"], EPS,
                                    a["post_norm"], a["post_weight"], res_scale)
    assert_close(out.reshape(y.shape), y, ref.rounded(dy, y, out.dtype), "out")
    if hidden is not None:
        assert_close(hidden.reshape(h.shape), h, ref.rounded(dh, h, hidden.dtype), "hidden")


def check_backward(a, dout, hidden, dhidden, grads, res_scale=1.0):
    want = ref.norm_backward(dout, hidden, a["x"], dhidden, a["gate"], a["scale"], a["shift"], a["weight"], a["bias"], a["norm"], EPS,
                             a["post_norm"], a["post_weight"], res_scale)
    for name, got in grads._asdict().items():
        if got is None:
            continue
        w, tol = want[name]
        assert_close(got.reshape(w.shape), w, ref.rounded(tol, w, got.dtype), name)
    return want


def back(a, dout, hidden, dhidden, **more):
    vectors = {i: a[i] for i in ("gate", "scale", "shift", "weight", "bias", "post_weight", "norm", "post_norm")}
    return _fw().wsattn_block_norm_backward(dout, hidden, a["x"], dhidden=dhidden, eps=EPS, **vectors, **more)


CASES = [
    # lead, n, x, residual, vectors, modulation, affine, post, norm
    ((1, 1), 1, "fp32", "fp32", "fp32", None, True, None, "rms"),
    ((1, 1), 5120, "bf16", "bf16", "bf16", (1,), False, None, "layer"),
    ((2, 3), 7, "fp16", "fp32", "fp16", (2,), True, "layer", "layer"),
    ((1, 5), 8, "bf16", "bf16", "fp32", (1, 5), True, "rms", "rms"),
    ((3, 37), 255, "fp32", "fp32", "fp32", (3,), False, "layer", "rms"),
    ((2, 48), 264, "bf16", "fp32", "bf16", (2, 6), True, None, "layer"),
    ((3, 111), 779, "fp16", "fp32", "fp32", None, True, "rms", "rms"),
    ((2, 130), 1024, "fp16", "fp16", "fp16", (2, 130), False, None, "layer"),
    ((1, 61), 2048, "fp32", "fp32", "fp32", (1,), True, "rms", "layer"),
    ((1, 40), 2056, "bf16", "bf16", "fp32", (1, 4), True, "layer", "layer"),
    ((1, 33), 4096, "bf16", "bf16", "bf16", (1, 1), False, "rms", "rms"),
    ((2, 19), 4103, "fp16", "fp16", "fp16", (2,), True, None, "layer"),
    ((1, 700), 5120, "bf16", "bf16", "bf16", (1,), False, None, "layer"),
    ((1, 9), 12288, "fp32", "fp32", "fp32", (1, 3), True, "layer", "layer"),
    ((1, 6), 12285, "bf16", "fp32", "fp32", (1,), True, "rms", "layer"),
    ((4, 700), 64, "bf16", "bf16", "bf16", (4,), True, None, "layer"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_block_norm_and_its_gradients(i):
    lead, n, dt, rt, vt, mod, affine, post, norm = CASES[i]
    a = make(i, lead, n, T[dt], T[rt], T[vt], mod, affine, post, norm)
    out, hidden = _fw().wsattn_block_norm(**a, eps=EPS, residual_scale=0.75)
    check_forward(a, out, hidden, 0.75)
    g = torch.Generator().manual_seed(i + 1000)
    dout = (torch.randn(*lead, n, generator=g) * 0.3).to(T[dt]).cuda()
    dhidden = (torch.randn(*lead, n, generator=g) * 0.3).to(T[rt]).cuda()
    grads = back(a, dout, hidden, dhidden, residual_scale=0.75)
    check_backward(a, dout, hidden, dhidden, grads, 0.75)
    for name in ("dgate", "dscale", "dshift"):
        assert (getattr(grads, name) is None) == (mod is None)
    assert (grads.dweight is None) != affine and (grads.dpost_weight is None) == (not post)
    assert _fw().wsattn_op_status() == 0


@pytest.mark.parametrize("dt,lead,n,mod", [("bf16", (3, 1000), 520, (3,)), ("fp32", (1, 2500), 96, (1, 50)), ("fp16", (2, 900), 301, (2, 900)),
                                           ("bf16", (5, 611), 2304, (5, 13)), ("bf16", (1, 3000), 4352, None)])
def test_gradients_of_groups_that_shares_split(dt, lead, n, mod):
    # groups inside a share, over several, and of single rows
    a = make(7, lead, n, T[dt], T[dt], torch.float32, mod, True, "rms", "layer")
    _, hidden = _fw().wsattn_block_norm(**a, eps=EPS)
    dout = torch.randn(*lead, n, device="cuda").to(T[dt])
    grads = back(a, dout, hidden, None)
    check_backward(a, dout, hidden, None, grads)
    again = back(a, dout, hidden, None)
    for x, y in zip(grads, again):
        assert x is None and y is None or torch.equal(x, y)  # fixed order of sums


def test_rows_far_from_zero_keep_their_precision():
    # deviations of 1 around a mean of 300, of 1e-3 around 0, and rows that do not vary
    for offset, spread in ((300.0, 1.0), (0.0, 1e-3), (50.0, 0.0)):
        a = make(3, (2, 20), 1000, torch.float32, torch.float32, torch.float32, (2,), False, "layer", "layer", residual=False, spread=spread,
                 offset=offset)
        out, hidden = _fw().wsattn_block_norm(**a, eps=EPS)
        check_forward(a, out, hidden)
        dout = torch.randn(2, 20, 1000, device="cuda")
        check_backward(a, dout, hidden, None, back(a, dout, hidden, None))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_strided_rows_and_odd_alignment(dt):
    # rows one element apart from their neighbours' alignment, columns behind them untouched
    lead, n = (2, 50), 333
    for ld, off in ((333, 1), (400, 0), (341, 3)):
        a = make(5, lead, n, T[dt], T[dt], torch.float32, (2, 10), True, None, "layer")

        def strided(t):
            buf = torch.full((off + 100 * ld,), 7.0, dtype=t.dtype, device="cuda")
            v = buf[off:].view(2, 50, ld)[..., :n]
            return v, buf

        x, _ = strided(a["x"])
        x.copy_(a["x"])
        residual, _ = strided(a["residual"])
        residual.copy_(a["residual"])
        out, buf_o = strided(a["x"])
        hidden, buf_h = strided(a["residual"])
        b = dict(a, x=x, residual=residual)
        got = _fw().wsattn_block_norm(**b, eps=EPS, out=out, hidden=hidden)
        assert got[0] is out and got[1] is hidden
        check_forward(a, out, hidden)
        for buf in (buf_o, buf_h):
            rest = torch.ones(buf.shape, dtype=torch.bool, device="cuda")
            rest[off:].view(2, 50, ld)[..., :n] = False
            assert (buf[rest] == 7).all()
        dx, buf_x = strided(a["x"])
        dout = torch.randn(2, 50, n, device="cuda").to(T[dt])
        grads = back(b, dout, hidden, residual, dx=dx)
        check_backward(b, dout, hidden, residual, grads)
        assert (buf_x[:off] == 7).all() and (buf_x[off:].view(2, 50, ld)[..., n:] == 7).all()


def test_in_place_and_parts_left_out():
    fw = _fw()
    a = make(11, (2, 64), 640, torch.bfloat16, torch.bfloat16, torch.bfloat16, (2,), False, None, "layer")
    out, hidden = fw.wsattn_block_norm(**a, eps=EPS)
    b = dict(a, x=a["x"].clone(), residual=a["residual"].clone())
    o2, h2 = fw.wsattn_block_norm(**b, eps=EPS, out=b["x"], hidden=b["residual"])
    assert o2 is b["x"] and torch.equal(o2, out) and h2 is b["residual"] and torch.equal(h2, hidden)
    # the residual alone, and the norm alone
    none, h3 = fw.wsattn_block_norm(**a, eps=EPS, need_out=False)
    assert none is None and torch.equal(h3, hidden)
    o4, h4 = fw.wsattn_block_norm(a["x"], scale=a["scale"], shift=a["shift"], eps=EPS)
    assert h4 is None
    check_forward(dict(a, gate=None, residual=None), o4, None)
    dout = torch.randn_like(a["x"])
    grads = fw.wsattn_block_norm_backward(dout, a["x"], scale=a["scale"], shift=a["shift"], eps=EPS)
    assert grads.dx is grads.dresidual  # one tensor where they are equal
    want = ref.norm_backward(dout, a["x"], a["x"], None, None, a["scale"], a["shift"], None, None, "layer", EPS, None, None, 1.0)
    for name in ("dx", "dscale", "dshift"):
        w, tol = want[name]
        assert_close(getattr(grads, name).reshape(w.shape), w, ref.rounded(tol, w, getattr(grads, name).dtype), name)
    # only dhidden: no norm behind it
    g2 = back(a, None, hidden, dout)
    check_backward(a, None, hidden, dout, g2)
    assert (g2.dscale == 0).all() and (g2.dshift == 0).all()
    # gradients in place
    g3 = back(a, dout, hidden, a["residual"])
    d, h = dout.clone(), hidden.clone()
    g4 = back(a, d, h, a["residual"], dx=d, dresidual=h)
    assert torch.equal(g3.dx, g4.dx) and torch.equal(g3.dresidual, g4.dresidual) and torch.equal(g3.dgate, g4.dgate)
    g5 = back(a, dout, hidden, None, need_vectors=False, need_dresidual=False)
    assert g5.dgate is None and g5.dresidual is None and g5.dx is not None


def test_no_rows():
    fw = _fw()
    x = torch.empty(2, 0, 24, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(24, device="cuda")
    out, hidden = fw.wsattn_block_norm(x, x, weight=w)
    assert out.shape == x.shape and hidden.shape == x.shape
    g = fw.wsattn_block_norm_backward(x, x, weight=w, bias=w, scale=torch.ones(2, 24, device="cuda"))
    assert (g.dweight == 0).all() and (g.dbias == 0).all() and (g.dscale == 0).all() and (g.dshift == 0).all()


def test_a_rows_infinities_stay_in_it():
    a = make(13, (1, 40), 200, torch.float32, torch.float32, torch.float32, (1, 40), False, "rms", "layer")
    _, clean_h = _fw().wsattn_block_norm(**a, eps=EPS)
    clean_o, _ = _fw().wsattn_block_norm(**a, eps=EPS)
    a["x"][0, 3, 5], a["residual"][0, 17, 0] = float("inf"), float("nan")
    out, hidden = _fw().wsattn_block_norm(**a, eps=EPS)
    keep = [i for i in range(40) if i not in (3, 17)]
    assert torch.equal(out[0, keep], clean_o[0, keep]) and torch.equal(hidden[0, keep], clean_h[0, keep])
    assert out[0, 3].isnan().any() and out[0, 17].isnan().all()
    dout = torch.randn_like(a["x"])
    g = back(a, dout, hidden, None)
    assert g.dx[0, keep].isfinite().all() and g.dgate[0, keep].isfinite().all() and not g.dx[0, 17].isfinite().any()


def test_gradients_against_differences():
    fw = _fw()
    a = make(17, (2, 6), 48, torch.float32, torch.float32, torch.float32, (2, 3), True, "layer", "layer")
    a["x"] *= 2
    wo, wh = (torch.randn(2, 6, 48, generator=torch.Generator().manual_seed(i)).cuda() for i in (1, 2))

    def loss(b):
        o, h = fw.wsattn_block_norm(**b, eps=1e-2, residual_scale=0.5)
        return float((o.double() * wo).sum() + (h.double() * wh).sum())

    _, hidden = fw.wsattn_block_norm(**a, eps=1e-2, residual_scale=0.5)
    vectors = {i: a[i] for i in ("gate", "scale", "shift", "weight", "bias", "post_weight", "norm", "post_norm")}
    g = fw.wsattn_block_norm_backward(wo, hidden, a["x"], dhidden=wh, eps=1e-2, residual_scale=0.5, **vectors)
    gen = torch.Generator().manual_seed(5)
    for name, grad in (("x", g.dx), ("residual", g.dresidual), ("gate", g.dgate), ("scale", g.dscale), ("shift", g.dshift),
                       ("weight", g.dweight), ("bias", g.dbias), ("post_weight", g.dpost_weight)):
        d = torch.randn(grad.shape, generator=gen).cuda()
        d /= d.norm()
        step = 2.0 ** -6
        up, down = (loss(dict(a, **{name: a[name] + k * step * d})) for k in (1, -1))
        want, got = (up - down) / (2 * step), float((grad.double() * d).sum())
        # the third derivative's step^2 / 6 is below 2^-12 of the gradient's size here, the sums' fp32 error below 2^-16
        # of |loss terms| / step
        assert abs(got - want) <= 2e-3 * float(grad.norm()) + 2e-3, (name, got, want)


def test_streams_graphs_and_workspaces():
    fw = _fw()
    a = make(19, (3, 500), 1040, torch.bfloat16, torch.float32, torch.float32, (3,), True, "rms", "layer")
    out, hidden = fw.wsattn_block_norm(**a, eps=EPS)
    dout = torch.randn(3, 500, 1040, device="cuda", dtype=torch.bfloat16)
    want = back(a, dout, hidden, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, h2 = fw.wsattn_block_norm(**a, eps=EPS, stream=side)
    g2 = back(a, dout, h2, None, stream=side)
    side.synchronize()
    assert torch.equal(out, o2) and torch.equal(hidden, h2)
    for x, y in zip(want, g2):
        assert torch.equal(x, y)
    # captured, and replayed on other values
    vec = {i: a[i] for i in ("gate", "scale", "shift", "weight", "bias", "post_weight", "norm", "post_norm")}
    need = fw.wsattn_block_norm_backward_workspace(dout, hidden, a["x"], **{k: v for k, v in vec.items()})
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, h3 = fw.wsattn_block_norm(**a, eps=EPS)
        g3 = back(a, dout, h3, None, workspace=ws)
    a["x"].normal_()
    dout.normal_()
    graph.replay()
    torch.cuda.synchronize()
    check_forward(a, o3, h3)
    check_backward(a, dout, h3, None, g3)
    with pytest.raises(fw.WsattnError):
        back(a, dout, hidden, None, workspace=ws[:need - 16])
