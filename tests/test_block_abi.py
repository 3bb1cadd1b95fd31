"""Cross attention and a block's norms on the CPU: the packed structs, argument
checks of the C ABI and of the Python binding (every refusal comes before any
device work), and workspace sizes, which need no GPU."""
import ctypes
import math

import pytest
import torch

BAD, UNSUPPORTED, CUDA = 1, 3, 6
BF16, FP16, FP32 = 0, 1, 2
P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
A = 1 << 20                # an aligned address that is never dereferenced


class Heads(ctypes.Structure):
    _fields_ = [("data", P), ("heads", I), ("stride_b", I64), ("stride_h", I64), ("stride_n", I64)]


class Cross(ctypes.Structure):
    _fields_ = [("dtype", I), ("head_dim", I), ("batch", I), ("n_tokens", I64), ("n_keys", I64), ("q", Heads), ("k", Heads),
                ("v", Heads), ("out", Heads), ("k_lengths", P), ("scale", F), ("lse", P)]


class CrossGrad(ctypes.Structure):
    _fields_ = [("dtype", I), ("head_dim", I), ("batch", I), ("n_tokens", I64), ("n_keys", I64), ("dout", Heads), ("q", Heads),
                ("k", Heads), ("v", Heads), ("out", Heads), ("lse", P), ("k_lengths", P), ("scale", F), ("dq", Heads), ("dk", Heads),
                ("dv", Heads)]


_HEAD = [("dtype", I), ("stream_dtype", I), ("mod_dtype", I), ("weight_dtype", I), ("m", I64), ("n", I), ("norm", I), ("post_norm", I),
         ("eps", F), ("residual_scale", F), ("group", I64)]


def _rows(*names):
    return [f for name, ld in names for f in ((name, P), (ld, I64))]


class Norm(ctypes.Structure):
    _fields_ = _HEAD + _rows(("x", "ldx"), ("residual", "ldr"), ("gate", "ldg"), ("scale", "lds"), ("shift", "ldf")) + \
        [("weight", P), ("bias", P), ("post_weight", P)] + _rows(("hidden", "ldh"), ("out", "ldo"))


class NormGrad(ctypes.Structure):
    _fields_ = _HEAD + _rows(("dout", "ldo"), ("dhidden", "lddh"), ("hidden", "ldh"), ("x", "ldx"), ("gate", "ldg"), ("scale", "lds")) + \
        [("weight", P), ("bias", P), ("post_weight", P)] + _rows(("dx", "lddx"), ("dresidual", "lddr")) + \
        [(i, P) for i in ("dgate", "dscale", "dshift", "dweight", "dbias", "dpost_weight")]


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


def _flat(kind):
    """The struct's fields one after another, and the struct itself, from 1, 2, 3, ..."""
    vals, s, n = [], kind(), 0
    for name, ty in kind._fields_:
        if ty is Heads:
            v = [n + 1 + i for i in range(5)]
            setattr(s, name, Heads(*v))
            vals += v
            n += 5
        else:
            n += 1
            vals.append(float(n) if ty is F else n)
            setattr(s, name, vals[-1])
    return vals, s


def test_packed_structs_match_the_header():
    fw = _fw()
    for pack, kind in ((fw._CROSS, Cross), (fw._CROSS_GRAD, CrossGrad), (fw._BLOCK_NORM, Norm), (fw._BLOCK_NORM_GRAD, NormGrad)):
        vals, s = _flat(kind)
        assert pack(*vals) == bytes(s), kind


def cross(**kw):
    n, m, b, h, e, d = (kw.pop(i, j) for i, j in (("n", 5), ("m", 7), ("b", 2), ("h", 4), ("e", 2), ("d", 64)))

    def view(heads, rows):
        return Heads(A, heads, rows * heads * d, d, heads * d)

    a = Cross(kw.pop("dtype", BF16), d, b, n, m, view(h, n), view(e, m), view(e, m), view(h, n), None, kw.pop("scale", 0.125), None)
    for name, value in kw.items():
        obj, field = name.split("_", 1) if name.split("_")[0] in ("q", "k", "v", "out") and name != "k_lengths" else (None, name)
        setattr(a if obj is None else getattr(a, obj), field, value)
    return a


def test_cross_refusals_come_before_device_work():
    fw = _fw()
    fn = fw.raw_call("wsattn_cross")

    def call(**kw):
        return fn(ctypes.byref(cross(**kw)), None, 0, None)

    assert fn(None, None, 0, None) == BAD
    for bad in (dict(b=-1), dict(n=-1), dict(m=-1), dict(n=(1 << 31) - 500), dict(m=1 << 31), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=math.nan), dict(scale=math.inf), dict(e=3), dict(h=0), dict(e=0), dict(v_heads=4),
                dict(q_data=A + 2), dict(k_data=A + 8), dict(out_data=A + 2), dict(q_stride_n=260), dict(k_stride_b=-8), dict(v_stride_h=4),
                dict(q_stride_b=1 << 39), dict(q_data=None), dict(k_data=None), dict(v_data=None), dict(out_data=None),
                dict(out_stride_h=0), dict(out_stride_n=64), dict(out_stride_b=0), dict(k_lengths=A + 2), dict(lse=A + 2)):
        assert call(**bad) == BAD, bad
    for bad in (dict(dtype=FP32), dict(d=8), dict(d=72), dict(d=144), dict(d=0)):
        assert call(**bad) == UNSUPPORTED, bad
    # nothing to do is no error
    assert call(b=0) == 0 and call(n=0, q_data=None, out_data=None) == 0
    if not torch.cuda.is_available():
        assert call() == CUDA and call(m=0, k_data=None, v_data=None) == CUDA
        # broadcast inputs, and strides of dimensions of one element, are no reason to refuse
        assert call(k_stride_b=0, v_stride_b=0, k_stride_h=0) == CUDA and call(b=1, q_stride_b=3) == CUDA


def test_cross_workspaces():
    fw = _fw()
    n = ctypes.c_size_t()
    ask = fw.raw_call("wsattn_cross_workspace")
    assert ask(ctypes.byref(cross()), None) == BAD and ask(None, ctypes.byref(n)) == BAD
    assert ask(ctypes.byref(cross(d=24)), ctypes.byref(n)) == UNSUPPORTED
    assert ask(ctypes.byref(cross()), ctypes.byref(n)) == 0 and n.value == 0
    # many tiles: nothing to join; few and long: fp32 rows and their sums, of one to 152 parts
    assert ask(ctypes.byref(cross(n=20000, m=4096, h=16, e=16)), ctypes.byref(n)) == 0 and n.value == 0
    big = cross(b=1, n=1, m=1 << 20, h=8, e=8, d=128)
    assert ask(ctypes.byref(big), ctypes.byref(n)) == 0 and n.value % (8 * 129 * 4) == 0 and 1 < n.value // (8 * 129 * 4) <= 152
    assert fw.raw_call("wsattn_cross")(ctypes.byref(big), A, n.value - 16, None) == BAD
    assert fw.raw_call("wsattn_cross")(ctypes.byref(big), A + 8, n.value, None) == BAD
    assert fw.raw_call("wsattn_cross")(ctypes.byref(big), None, n.value, None) == BAD


def grad(**kw):
    skip = kw.pop("skip", ())
    c = cross(**{i: j for i, j in kw.items() if i in ("n", "m", "b", "h", "e", "d", "dtype", "scale")})
    a = CrossGrad(c.dtype, c.head_dim, c.batch, c.n_tokens, c.n_keys, c.out, c.q, c.k, c.v, c.out, A, None, c.scale, c.q, c.k, c.v)
    for i in skip:
        getattr(a, i).data = None
    for name, value in kw.items():
        if name in ("lse", "k_lengths"):
            setattr(a, name, value)
        elif "_" in name:
            obj, field = name.split("_", 1)
            setattr(getattr(a, obj), field, value)
    return a


def test_cross_backward_refusals_and_workspaces():
    fw = _fw()
    fn, ask, n = fw.raw_call("wsattn_cross_backward"), fw.raw_call("wsattn_cross_backward_workspace"), ctypes.c_size_t()
    assert ask(ctypes.byref(grad()), ctypes.byref(n)) == 0 and n.value > 0
    need = n.value

    def call(ws=A, size=None, **kw):
        return fn(ctypes.byref(grad(**kw)), ws, need if size is None else size, None)

    assert fn(None, A, need, None) == BAD
    for bad in (dict(ws=None), dict(ws=A + 4), dict(size=need - 1), dict(lse=None), dict(lse=A + 1), dict(dout_data=None), dict(out_data=None),
                dict(k_data=None), dict(dk_stride_n=60), dict(dv_stride_h=0), dict(dq_stride_b=0), dict(dq_heads=2), dict(dk_heads=4),
                dict(dk_data=A + 2), dict(scale=-0.5), dict(b=-1), dict(dout_heads=3)):
        assert call(**bad) == BAD, bad
    assert call(d=40) == UNSUPPORTED and call(dtype=FP32) == UNSUPPORTED
    assert call(b=0) == 0 and call(skip=("dq", "dk", "dv")) == 0
    # dq alone needs no scratch
    assert ask(ctypes.byref(grad(skip=("dk", "dv"))), ctypes.byref(n)) == 0 and n.value == 0
    if not torch.cuda.is_available():
        assert call() == CUDA and call(ws=None, size=0, skip=("dk", "dv")) == CUDA


def norm(kind=Norm, **kw):
    a = kind()
    a.m, a.n, a.norm, a.group, a.eps, a.residual_scale = 6, 16, 2, 3, 1e-6, 1.0
    for name, _ in kind._fields_:
        if name.startswith("ld"):
            setattr(a, name, 16)
    for name in ("x", "residual", "gate", "scale", "shift", "out") if kind is Norm else ("dout", "hidden", "x", "gate", "scale", "dx", "dgate"):
        setattr(a, name, A)
    if kind is Norm:
        a.hidden = 2 * A
    for name, value in kw.items():
        setattr(a, name, value)
    return a


COMMON_BAD = [dict(dtype=3), dict(dtype=-1), dict(stream_dtype=FP16), dict(mod_dtype=FP16), dict(weight_dtype=FP16), dict(dtype=FP32), dict(m=-1),
              dict(m=(1 << 31) - 500), dict(n=0), dict(group=0), dict(norm=0), dict(norm=3), dict(post_norm=-1), dict(post_norm=3), dict(eps=-1.0),
              dict(eps=math.nan), dict(residual_scale=math.inf), dict(ldx=15), dict(ldg=8), dict(lds=15), dict(gate=A + 1), dict(weight=A + 1),
              dict(post_weight=A), dict(x=A + 1)]


def test_block_norm_refusals_come_before_device_work():
    fw = _fw()
    fn = fw.raw_call("wsattn_block_norm")

    def call(**kw):
        return fn(ctypes.byref(norm(**kw)), None)

    assert fn(None, None) == BAD
    for bad in COMMON_BAD + [dict(x=None), dict(ldr=15), dict(ldf=1), dict(ldo=3), dict(ldh=3), dict(out=A + 1), dict(hidden=A, out=A),
                             dict(stream_dtype=FP32, residual=A + 2)]:
        assert call(**bad) == BAD, bad
    wide = {i: 12289 for i in ("n", "ldx", "ldr", "ldg", "lds", "ldf", "ldh", "ldo")}
    assert call(**wide) == UNSUPPORTED
    assert call(m=0, x=None) == 0 and call(hidden=None, out=None, x=None) == 0
    if not torch.cuda.is_available():
        assert call() == CUDA and call(weight=A, weight_dtype=FP32, post_norm=1, post_weight=A) == CUDA


def test_block_norm_backward_refusals_and_workspaces():
    fw = _fw()
    fn, ask, n = fw.raw_call("wsattn_block_norm_backward"), fw.raw_call("wsattn_block_norm_backward_workspace"), ctypes.c_size_t()

    def size(**kw):
        assert ask(ctypes.byref(norm(NormGrad, **kw)), ctypes.byref(n)) == 0
        return n.value

    def call(ws=A, nbytes=1 << 30, **kw):
        return fn(ctypes.byref(norm(NormGrad, **kw)), ws, nbytes, None)

    assert fn(None, A, 0, None) == BAD and ask(None, ctypes.byref(n)) == BAD and ask(ctypes.byref(norm(NormGrad)), None) == BAD
    for bad in COMMON_BAD + [dict(dout=None), dict(hidden=None), dict(x=None), dict(dout=A + 1), dict(lddx=15), dict(dx=A, dresidual=A),
                             dict(dgate=A + 2), dict(dweight=A + 1), dict(x=None, dgate=None, dx=A, post_norm=1)]:
        assert call(**bad) == BAD, bad
    assert size(m=0) == 0 and size(dgate=None) == 0
    big = dict(m=4000, group=1000)
    assert size(**big) > 0 and size(**big, dgate=None) == 0      # groups that shares split
    assert size(m=4000, group=1) == 0                            # every group in one share
    assert size(**big, dweight=A) > size(**big)
    assert call(ws=None, **big) == BAD and call(ws=A + 8, **big) == BAD and call(nbytes=size(**big) - 1, **big) == BAD
    wide = {i: 12289 for i in ("n", "ldo", "lddh", "ldh", "ldx", "ldg", "lds", "lddx", "lddr")}
    assert call(**wide) == UNSUPPORTED
    if not torch.cuda.is_available():
        assert call() == CUDA and call(x=None, dgate=None) == CUDA


def test_vectors_serve_rows_of_the_same_leading_dimensions():
    fw = _fw()

    def groups(shape, lead):
        return fw._groups_of(torch.empty(shape, device="meta"), "gate", torch.Size(lead), 8)

    assert groups((8,), (2, 6)) == 1 and groups((1, 8), (2, 6)) == 1 and groups((1, 1, 8), (2, 6)) == 1
    assert groups((2, 8), (2, 6)) == 2 and groups((2, 1, 8), (2, 6)) == 2
    assert groups((2, 3, 8), (2, 6)) == 6 and groups((2, 6, 8), (2, 6)) == 12
    assert groups((4, 8), (12,)) == 4 and groups((1, 3, 8), (1, 6)) == 3
    # a vector a token of both clips, or of other leading dimensions, would be taken for something else
    for shape in ((6, 8), (1, 6, 8), (2, 4, 8), (3, 8), (2, 6, 2, 8), (2, 7), ()):
        with pytest.raises(ValueError):
            groups(shape, (2, 6))


@pytest.mark.parametrize("call", ["cross", "norm", "cross_back", "norm_back"])
def test_tensors_on_the_cpu_are_refused(call):
    fw = _fw()
    t = torch.zeros(1, 2, 3, 16)
    with pytest.raises(TypeError):
        {"cross": lambda: fw.wsattn_cross(t, t, t), "norm": lambda: fw.wsattn_block_norm(t),
         "cross_back": lambda: fw.wsattn_cross_backward(t, t, t, t, t, t[..., 0]),
         "norm_back": lambda: fw.wsattn_block_norm_backward(t, t)}[call]()
