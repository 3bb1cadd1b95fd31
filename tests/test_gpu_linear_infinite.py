"""Gradients behind pre-activations that rounding made infinite (GPU): past
65504 fp16 holds an infinity where the product and the activation were finite.
The slope is 0 on the negative side and 1 on the positive one, exactly."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [2, 300])
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_gradients_behind_infinite_preactivations(name, rows):
    import frame_aligned_window_gb300 as fw
    dt = torch.float16
    x = torch.zeros((rows, 8), dtype=dt, device="cuda")
    x[:, 0] = 280
    w = torch.zeros((8, 8), dtype=dt, device="cuda")
    w[:, 0] = torch.tensor([250, -250, 1, -1, 0, 2, -250, 250])
    z = torch.empty((rows, 8), dtype=dt, device="cuda")
    y = fw.wsattn_linear(x, w, activation=name, preact=z, out_dtype=torch.float32)
    assert torch.equal(y, torch.relu(280 * w[:, 0].float()).expand(rows, 8))
    assert z.isinf().sum() == 4 * rows
    dx, dw, db = fw.wsattn_linear_backward(torch.ones_like(z), x, w, z, name)
    slope = torch.tensor([1, 0, 1, 0, 0.5, 1, 0, 1], device="cuda")
    assert torch.equal(db, rows * slope)
    assert torch.equal(dx[:, 0].float(), (slope * w[:, 0].float()).sum().expand(rows))
    # 280 a row, past fp16's range with 300 of them
    assert torch.equal(dw[:, 0], (280 * rows * slope).to(dt)) and (dw[:, 1:] == 0).all()


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_slopes_at_the_ends_of_the_types(name, dt):
    # and a NaN stays one
    import frame_aligned_window_gb300 as fw
    inf, most = float("inf"), torch.finfo(dt).max
    z = torch.tensor([inf, -inf, most, -most, 1000, -1000, 1e4, -1e4, float("nan"), 0], dtype=dt, device="cuda")
    one = torch.ones((1, 10), dtype=dt, device="cuda")
    wide = torch.zeros((10, 8), dtype=dt, device="cuda")
    _, _, db = fw.wsattn_linear_backward(one, one[:, :8].contiguous(), wide, z[None], name, need_dx=False,
                                         need_dw=False)
    assert torch.equal(db[:8], torch.tensor([1, 0, 1, 0, 1, 0, 1, 0.0], device="cuda"))
    assert db[8].isnan() and db[9] == 0.5
