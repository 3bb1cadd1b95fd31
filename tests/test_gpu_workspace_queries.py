"""Asking for a workspace's size takes no memory of its own (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_size_queries_allocate_nothing():
    # (the product's output would be 4 TB)
    import frame_aligned_window_gb300 as fw
    dt = torch.bfloat16
    x = torch.zeros((1 << 21, 8), dtype=dt, device="cuda")
    w = torch.zeros((1 << 20, 8), dtype=dt, device="cuda")
    thin = torch.zeros((8, 1 << 21), dtype=dt, device="cuda")
    dy = torch.zeros((8, 8), dtype=dt, device="cuda")
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    fw.wsattn_linear_workspace(x, w)
    fw.wsattn_linear_backward_workspace(dy, thin, thin)
    assert torch.cuda.max_memory_allocated() == before


@pytest.mark.parametrize("shape", [(300, 512, 57600), (333, 257, 131), (2080, 4096, 1024), (64, 64, 64)],
                         ids=lambda c: "x".join(map(str, c)))
def test_the_size_asked_for_is_the_size_needed(shape):
    import frame_aligned_window_gb300 as fw
    m, n, k = shape
    dt = torch.float16
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w, dy = (torch.randn(s, generator=g, device="cuda").to(dt) for s in ((m, k), (n, k), (m, n)))

    def check(size, call):
        want = call(None)
        exact = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
        for a, b in zip(call(exact), want):
            assert (a is None and b is None) or torch.equal(a, b)
        if size:
            with pytest.raises(fw.WsattnError):
                call(exact[:size - 1])
    check(fw.wsattn_linear_workspace(x, w), lambda ws: [fw.wsattn_linear(x, w, workspace=ws)])
    for act in ("none", "silu"):
        for i in range(1, 8):
            need = dict(zip(("need_dx", "need_dw", "need_db"), (i & 1 != 0, i & 2 != 0, i & 4 != 0)))
            check(fw.wsattn_linear_backward_workspace(dy, x, w, dy, act, **need),
                  lambda ws: fw.wsattn_linear_backward(dy, x, w, dy, act, workspace=ws, **need))
    assert fw.wsattn_op_status() == 0
