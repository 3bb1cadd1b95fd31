"""Cross attention and a block's norms on the CPU: which shapes ask for no
workspace, views that are refused, vectors for no rows."""
import ctypes
import itertools

import torch

from test_block_abi import A, BAD, Cross, Heads, _fw


def _args(b, h, hk, n, m, d, **kw):
    def view(heads, rows):
        return Heads(A, heads, rows * heads * d, d, heads * d)

    return Cross(0, d, b, n, m, view(h, n), view(hk, m), view(hk, m), view(h, n), kw.get("k_lengths"), 1.0, None)


def test_shapes_without_a_workspace():
    """The binding asks for none where the library takes none."""
    fw = _fw()
    ask, size = fw.raw_call("wsattn_cross_workspace"), ctypes.c_size_t()
    some = none = 0
    for b, (h, hk), n, m in itertools.product((1, 2, 5, 30, 77, 400), ((1, 1), (4, 1), (6, 2), (8, 8), (40, 40), (76, 76), (77, 77)),
                                              (1, 3, 64, 128, 129, 256, 257, 512, 4000, 9729, 19457, 40000), (0, 1, 128, 129, 512, 5000, 10**6)):
        assert ask(ctypes.byref(_args(b, h, hk, n, m, 64)), ctypes.byref(size)) == 0
        if fw._keys_stay_whole((b, h, n, 64), (b, hk, m, 64)):
            none += 1
            assert size.value == 0, (b, h, hk, n, m)
        else:
            some += 1
    assert some and none


def test_rows_without_a_stride_are_refused():
    fw = _fw()
    fn = fw.raw_call("wsattn_cross")
    for name in ("q", "k", "v"):
        a = _args(2, 4, 2, 40, 50, 64)
        getattr(a, name).stride_n = 0
        assert fn(ctypes.byref(a), A, 1 << 40, None) == BAD


def test_vectors_for_no_rows():
    fw = _fw()

    def groups(shape, lead):
        return fw._groups_of(torch.empty(shape, device="meta"), "gate", torch.Size(lead), 8)

    assert groups((0, 8), (0, 6)) == 0 and groups((0, 6, 8), (0, 6)) == 0 and groups((8,), (0, 6)) == 1
    for shape, lead in (((0, 8), (2, 6)), ((2, 0, 8), (2, 6)), ((3, 0, 8), (2, 0))):
        try:
            groups(shape, lead)
        except ValueError:
            continue
        raise AssertionError((shape, lead))
