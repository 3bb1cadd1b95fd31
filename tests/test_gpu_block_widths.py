"""Block norms at the widths where a row's layout changes, forward and back."""
import pytest
import torch

from test_gpu_block_norm import EPS, T, _fw, back, check_backward, check_forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,rt", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("n", [1024, 1025, 2048, 2056, 2560, 2561, 4096, 4100, 6152])
def test_widths(n, dt, rt):
    lead = (2, 301)
    a = make(n, lead, n, T[dt], T[rt], torch.float32, (2, 7), True, "layer", "layer")
    out, hidden = _fw().wsattn_block_norm(**a, eps=EPS)
    check_forward(a, out, hidden)
    dout = torch.randn(*lead, n, device="cuda").to(T[dt])
    check_backward(a, dout, hidden, None, back(a, dout, hidden, None))
    assert _fw().wsattn_op_status() == 0
