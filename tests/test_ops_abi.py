"""The operators around the attention on the CPU: argument checks of the C ABI
and of the Python binding (every refusal comes before any device work), and
the workspace sizes, which need no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

BAD, UNSUPPORTED, CUDA = 1, 3, 6
BF16, FP16, FP32 = 0, 1, 2
P = ctypes.c_void_p
A = 1 << 20                # an aligned address that is never dereferenced


class Heads(ctypes.Structure):
    _fields_ = [("data", P), ("heads", ctypes.c_int), ("stride_b", ctypes.c_int64),
                ("stride_h", ctypes.c_int64), ("stride_n", ctypes.c_int64)]


class Linear(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("m", ctypes.c_int64),
                ("n", ctypes.c_int), ("k", ctypes.c_int), ("x", P), ("ldx", ctypes.c_int64),
                ("x_heads", ctypes.c_int), ("x_tokens", ctypes.c_int64), ("w", P),
                ("ldw", ctypes.c_int64), ("bias", P), ("residual", P), ("ldr", ctypes.c_int64),
                ("out", P), ("ldo", ctypes.c_int64), ("preact", P), ("ldp", ctypes.c_int64),
                ("activation", ctypes.c_int)]


class Grad(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("m", ctypes.c_int64), ("n", ctypes.c_int),
                ("k", ctypes.c_int), ("dout", P), ("ldd", ctypes.c_int64), ("x", P),
                ("ldx", ctypes.c_int64), ("w", P), ("ldw", ctypes.c_int64), ("preact", P),
                ("ldp", ctypes.c_int64), ("activation", ctypes.c_int), ("dx", P),
                ("lddx", ctypes.c_int64), ("dw", P), ("lddw", ctypes.c_int64), ("db", P)]


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


def _ref(x):
    return None if x is None else ctypes.byref(x)


def test_packed_structs_match_the_header():
    # the binding packs the structs itself: same fields, same bytes
    fw = _fw()
    v = Heads(1, 2, 3, 4, 5)
    assert fw._HEADS(1, 2, 3, 4, 5) == bytes(v)
    vals = [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 17, 18, 19]
    assert fw._LINEAR(*vals) == bytes(Linear(*vals))
    assert fw._LINEAR_GRAD(*vals[:18]) == bytes(Grad(*vals[:18]))


def test_rotary_plan_errors():
    fw = _fw()
    fn = fw.raw_call("wsattn_rotary_plan")

    def call(dim=64, axes=2, axis=None, freq=None, inter=1, out=True):
        half = max(dim, 0) // 2
        ax = np.zeros(half, np.int32) if axis is None else np.asarray(axis, np.int32)
        fr = np.ones(half) if freq is None else np.asarray(freq, np.float64)
        h = P()
        rc = fn(dim, axes, ax.ctypes.data, fr.ctypes.data, inter, ctypes.byref(h) if out else None)
        assert (rc == 0) == bool(h.value)
        if rc == 0:
            fw.raw_call("wsattn_rotary_destroy")(h)
        return rc

    assert call() == 0 and call(256) == 0 and call(16) == 0
    for dim in (0, 8, 40, 272, -16):
        assert call(dim) == UNSUPPORTED, dim
    assert call(axes=0) == BAD and call(axes=5) == BAD
    assert call(inter=2) == BAD and call(out=False) == BAD
    assert call(axis=[2] * 32) == BAD and call(axis=[-1] * 32) == BAD
    for bad in (math.nan, math.inf, 1e31):
        assert call(freq=[bad] * 32) == BAD
    h = P()
    assert fn(64, 1, None, None, 1, ctypes.byref(h)) == BAD
    assert fw.raw_call("wsattn_rotary_destroy")(None) == 0
    # the binding's own forms
    with pytest.raises(ValueError):
        fw.wsattn_rotary_plan(64)
    with pytest.raises(ValueError):
        fw.wsattn_rotary_plan(64, (20, 13))          # 33 pairs of 32
    with pytest.raises(ValueError):
        fw.wsattn_rotary_plan(64, (32,), base=0.0)
    with pytest.raises(ValueError):
        fw.wsattn_rotary_plan(64, pair_axis=[0] * 32, pair_freq=[1.0] * 31)
    with pytest.raises(fw.WsattnError) as e:
        fw.wsattn_rotary_plan(40, (20,))
    assert e.value.code == UNSUPPORTED
    rot = fw.wsattn_rotary_plan(64, (32,))
    fw.wsattn_rotary_destroy(rot)
    with pytest.raises(ValueError):
        rot.handle


def _rot(dim=64):
    return _fw().wsattn_rotary_plan(dim, (dim // 2,))


def test_rotary_errors_without_device_work():
    fw = _fw()
    fn, rot = fw.raw_call("wsattn_rotary"), _rot()
    view = lambda data=A, heads=2, sb=0, sh=64, sn=128: Heads(data, heads, sb, sh, sn)  # noqa: E731

    def call(r=rot.handle, dt=BF16, b=1, n=3, x=view(), pos=A, pb=0, inv=0, y=view()):
        return fn(r, dt, b, n, _ref(x), pos, pb, inv, _ref(y), None)

    assert call(r=None) == BAD
    assert call(dt=3) == BAD and call(dt=-1) == BAD
    assert call(b=-1) == BAD and call(n=-1) == BAD and call(inv=2) == BAD
    assert call(x=None) == BAD and call(y=None) == BAD
    assert call(x=view(None)) == BAD and call(y=view(None)) == BAD and call(pos=None) == BAD
    assert call(x=view(A + 1)) == BAD and call(dt=FP32, x=view(A + 2)) == BAD
    assert call(pos=A + 2) == BAD and call(pb=-1) == BAD
    assert call(x=view(heads=1)) == BAD and call(y=view(heads=0), x=view(heads=0)) == BAD
    assert call(x=view(sh=-64)) == BAD
    # outputs whose elements would meet: equal heads, rows closer than a head, equal batches
    assert call(y=view(sh=0)) == BAD and call(y=view(sn=100)) == BAD and call(b=2) == BAD
    # nothing to do is not an error, whatever the pointers
    assert call(b=0, x=view(None), y=view(None), pos=None) == 0
    assert call(n=0, x=view(None), y=view(None), pos=None) == 0
    if not torch.cuda.is_available():
        assert call() == CUDA


def test_sizes_past_64_bits_are_refused():
    # 4 x 2^62 tokens are 0 in 64 bits, and a stride times a size may wrap round
    fw = _fw()
    fn, rot = fw.raw_call("wsattn_rotary"), _rot()
    for b, n in ((4, 1 << 62), (1, 1 << 31), (0, 1 << 31)):
        v = Heads(A, 1, 1 << 40, 0, 64)
        assert fn(rot.handle, BF16, b, n, _ref(v), A, 0, 0, _ref(v), None) == BAD
        assert fw.raw_call("wsattn_qknorm")(
            rot.handle, BF16, b, n, _ref(v), _ref(v), None, A, A, BF16, ctypes.c_float(1e-6), A, 0,
            _ref(v), _ref(v), None, None) == BAD
        assert fw.raw_call("wsattn_qknorm_backward")(
            rot.handle, BF16, b, n, _ref(v), _ref(v), None, _ref(v), _ref(v), A, A, BF16,
            ctypes.c_float(1e-6), A, 0, _ref(v), _ref(v), None, A, A, A, 1 << 40, None) == BAD
    x, y = Heads(A, 4, 0, 64, 256), Heads(A, 4, 0, 1 << 62, 256)
    assert fn(rot.handle, BF16, 1, 3, _ref(x), A, 0, 0, _ref(y), None) == BAD


def test_qknorm_errors_without_device_work():
    fw = _fw()
    fwd, bwd, rot = fw.raw_call("wsattn_qknorm"), fw.raw_call("wsattn_qknorm_backward"), _rot()
    view = lambda data=A, heads=2, sh=64, sn=512: Heads(data, heads, 0, sh, sn)  # noqa: E731

    def call(q=view(), k=view(), v=view(), wq=A, wk=A, wdt=BF16, eps=1e-6, qo=view(), ko=view(),
             vo=view(), dt=BF16, n=3, r=rot.handle):
        return fwd(r, dt, 1, n, _ref(q), _ref(k), _ref(v), wq, wk, wdt, ctypes.c_float(eps), A, 0,
                   _ref(qo), _ref(ko), _ref(vo), None)

    for key in ("q", "k", "qo", "ko"):
        assert call(**{key: None}) == BAD
        assert call(**{key: view(None)}) == BAD
        assert call(**{key: view(heads=3)}) == BAD
    assert call(v=None) == BAD and call(vo=None) == BAD
    assert call(eps=-1.0) == BAD and call(eps=math.nan) == BAD and call(eps=math.inf) == BAD
    assert call(wdt=FP16) == BAD and call(wq=A + 1) == BAD and call(wdt=FP32, wk=A + 2) == BAD
    assert call(r=None) == BAD and call(dt=7) == BAD
    assert call(n=0, q=view(None), k=view(None), v=None, qo=view(None), ko=view(None), vo=None) == 0

    need = ctypes.c_size_t()
    size = fw.raw_call("wsattn_qknorm_backward_workspace")
    assert size(None, ctypes.byref(need)) == BAD and size(rot.handle, None) == BAD
    assert size(rot.handle, ctypes.byref(need)) == 0 and need.value > 0

    def back(dq=view(), dk=view(), dv=view(), gq=view(), gk=view(), gv=view(), q=view(), k=view(),
             dwq=A, dwk=A, ws=A, nb=need.value, wq=A, wdt=BF16):
        return bwd(rot.handle, BF16, 1, 3, _ref(gq), _ref(gk), _ref(gv), _ref(q), _ref(k), wq, A,
                   wdt, ctypes.c_float(1e-6), A, 0, _ref(dq), _ref(dk), _ref(dv), dwq, dwk, ws, nb,
                   None)

    for key in ("dq", "dk", "gq", "gk", "q", "k"):
        assert back(**{key: None}) == BAD
        assert back(**{key: view(heads=5)}) == BAD
    assert back(dv=None) == BAD and back(gv=None) == BAD
    assert back(ws=None) == BAD and back(ws=A + 8) == BAD and back(nb=need.value - 1) == BAD
    assert back(dwq=A + 2) == BAD and back(wq=A + 1) == BAD and back(wdt=FP16) == BAD
    if not torch.cuda.is_available():
        assert call() == CUDA and back() == CUDA
        assert back(dwq=None, dwk=None, ws=None, nb=0) == CUDA


def test_linear_errors_without_device_work():
    fw = _fw()
    fn, size = fw.raw_call("wsattn_linear"), fw.raw_call("wsattn_linear_workspace")

    def args(**over):
        a = Linear(BF16, BF16, 4, 16, 32, A, 32, 0, 0, A, 32, A, A, 16, A, 16, A, 16, 1)
        for key, val in over.items():
            setattr(a, key, val)
        return a

    def call(ws=None, nb=0, **over):
        return fn(ctypes.byref(args(**over)), ws, nb, None)

    assert fn(None, None, 0, None) == BAD
    for over in (dict(m=-1), dict(n=0), dict(k=0), dict(ldx=31), dict(ldw=31), dict(ldo=15),
                 dict(ldr=15), dict(ldp=15), dict(activation=4), dict(activation=-1),
                 dict(m=1 << 31), dict(x=None), dict(w=None), dict(out=None), dict(x=A + 1),
                 dict(w=A + 1), dict(bias=A + 1), dict(residual=A + 1), dict(out=A + 1),
                 dict(preact=A + 1), dict(out_dtype=FP32, out=A + 2), dict(x_heads=-1),
                 dict(x_heads=3), dict(x_heads=8), dict(x_heads=2, x_tokens=0),
                 dict(x_heads=2, x_tokens=3), dict(x_heads=2, x_tokens=4, x=A + 4)):
        assert call(**over) == BAD, over
    for over in (dict(dtype=FP32), dict(dtype=9), dict(out_dtype=FP16), dict(out_dtype=5)):
        assert call(**over) == UNSUPPORTED, over
    assert call(m=0, x=None, out=None) == 0

    need = ctypes.c_size_t()

    def bytes_of(**over):
        assert size(ctypes.byref(args(**over)), ctypes.byref(need)) == 0
        return need.value
    assert size(None, ctypes.byref(need)) == BAD and size(ctypes.byref(args()), None) == BAD
    assert bytes_of() == 0
    assert bytes_of(ldx=33) >= 4 * 32 * 2 and bytes_of(w=A + 2) >= 16 * 32 * 2
    assert bytes_of(x_heads=2, x_tokens=2) >= 4 * 32 * 2
    assert bytes_of(m=1, ldx=33) == 0            # a single row has no stride
    assert bytes_of(m=0, ldx=33) == 0
    # a workspace that is missing, too small or not aligned
    n = bytes_of(ldx=33)
    assert call(ldx=33) == BAD and call(ws=A, nb=n - 1, ldx=33) == BAD
    assert call(ws=A + 8, nb=n, ldx=33) == BAD
    if not torch.cuda.is_available():
        assert call() == CUDA and call(ws=A, nb=n, ldx=33) == CUDA


def test_linear_backward_errors_without_device_work():
    fw = _fw()
    fn, size = fw.raw_call("wsattn_linear_backward"), fw.raw_call("wsattn_linear_backward_workspace")

    def args(**over):
        a = Grad(FP16, 40, 16, 32, A, 16, A, 32, A, 32, A, 16, 1, A, 32, A, 32, A)
        for key, val in over.items():
            setattr(a, key, val)
        return a
    need = ctypes.c_size_t()

    def bytes_of(**over):
        assert size(ctypes.byref(args(**over)), ctypes.byref(need)) == 0
        return need.value

    def call(ws=A, nb=1 << 40, **over):
        return fn(ctypes.byref(args(**over)), ws, nb, None)

    assert fn(None, None, 0, None) == BAD
    for over in (dict(m=-1), dict(n=0), dict(k=0), dict(ldd=15), dict(ldx=31), dict(ldw=31),
                 dict(ldp=15), dict(lddx=31), dict(lddw=31), dict(activation=4),
                 dict(preact=None), dict(dout=None), dict(x=None), dict(w=None), dict(dout=A + 1),
                 dict(x=A + 1), dict(w=A + 1), dict(preact=A + 1), dict(dx=A + 1), dict(dw=A + 1),
                 dict(db=A + 2)):
        assert call(**over) == BAD, over
    for dt in (FP32, 4, -1):
        assert call(dtype=dt) == UNSUPPORTED
    total = bytes_of()
    assert total >= 40 * 16 * 2 + 16 * 4         # dz and one row of partial sums
    assert bytes_of(activation=0, preact=None, db=None) == 0
    assert bytes_of(activation=0, dx=None, dw=None) < total and bytes_of(m=0) == 0
    assert call(nb=total - 1) == BAD and call(ws=None) == BAD and call(ws=A + 4) == BAD
    if not torch.cuda.is_available():
        assert call(nb=total) == CUDA
        assert fw.raw_call("wsattn_op_status")(None) == CUDA


def test_binding_refuses_cpu_tensors_and_wrong_kinds():
    fw = _fw()
    rot = _rot()
    x, pos = torch.zeros(1, 2, 3, 64), torch.zeros(3, 1)
    for call in (lambda: fw.wsattn_rotary(rot, x, pos),
                 lambda: fw.wsattn_rotary(rot, None, pos),
                 lambda: fw.wsattn_qknorm(rot, x, x, pos),
                 lambda: fw.wsattn_qknorm_backward(rot, x, x, x, x, pos),
                 lambda: fw.wsattn_linear(torch.zeros(2, 4), torch.zeros(3, 4)),
                 lambda: fw.wsattn_linear(np.zeros((2, 4)), np.zeros((3, 4))),
                 lambda: fw.wsattn_linear_backward(torch.zeros(2, 3), torch.zeros(2, 4),
                                                   torch.zeros(3, 4))):
        with pytest.raises(TypeError):
            call()
    assert fw.ACTIVATIONS == {"none": 0, "gelu": 1, "gelu_tanh": 2, "silu": 3}
