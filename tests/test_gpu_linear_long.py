"""wsattn_linear_backward over as many rows as it takes (GPU): the wait for an
accumulator spans the whole contraction."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_weight_gradient_over_2_to_31_rows():
    # a single output value: 2^25 steps of 64 rows over the 8 CTAs of a cluster,
    # more than a second of matrix instructions.  1000 ones among zeros, the
    # first and the last row among them: the sum is exact
    import frame_aligned_window_gb300 as fw
    m = (1 << 31) - 512
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 110 GB")
    dt = torch.bfloat16
    rows = torch.arange(1000, device="cuda", dtype=torch.int64) * ((m - 1) // 999)
    rows[-1] = m - 1
    x = torch.zeros((m, 1), dtype=dt, device="cuda")
    x[rows] = 1
    dy = torch.full((m, 1), 0.5, dtype=dt, device="cuda")
    w = torch.ones((1, 1), dtype=dt, device="cuda")
    _, dw, db = fw.wsattn_linear_backward(dy, x, w, need_dx=False)
    assert fw.wsattn_op_status() == 0
    assert dw.item() == 500
    # 608 partial sums of 441,000 rows a warp, all of whole and half numbers
    assert db.item() == m / 2
    del x, dy
    torch.cuda.empty_cache()
