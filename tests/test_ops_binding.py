"""The binding of the operators around the attention on the CPU: what it
refuses or passes on before any tensor is read (shapes alone, on the meta
device)."""
import pytest
import torch


def _fw():
    import frame_aligned_window_gb300 as fw
    return fw


@pytest.mark.parametrize("shape", [((1 << 32) + 1, 1, 1, 16), (1 << 31, 1, 3, 16), (1, 1 << 31, 1, 16)])
def test_sizes_past_an_int_are_refused(shape):
    # 2^32 + 1 batch elements would be one of the C call's
    fw = _fw()
    rot = fw.wsattn_rotary_plan(16, (8,))
    big = torch.empty((1, 1, 1, 16), device="meta").expand(shape)
    one = torch.empty((1, 1, 1, 16), device="meta")
    with pytest.raises(ValueError):
        fw._heads_shape(big, "x", rot)
    with pytest.raises(ValueError):
        fw._qkv_shapes(rot, big, big, None)
    most = torch.empty((1, 1, 1, 16), device="meta").expand((1 << 31) - 1, 1, 1, 16)
    assert fw._heads_shape(most, "x", rot)[0] == (1 << 31) - 1
    assert fw._qkv_shapes(rot, one, one, one)[2] == one.shape


@pytest.mark.gpu
def test_batches_past_an_int_are_refused_before_any_memory_is_taken():
    fw = _fw()
    rot = fw.wsattn_rotary_plan(16, (8,))
    x = torch.zeros((1, 1, 1, 16), dtype=torch.bfloat16, device="cuda").expand((1 << 32) + 1, 1, 1, 16)
    pos = torch.zeros((1, 1), device="cuda")
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    for call in (lambda: fw.wsattn_rotary(rot, x, pos), lambda: fw.wsattn_qknorm(rot, x, x, pos),
                 lambda: fw.wsattn_qknorm_backward(rot, x, x, x, x, pos)):
        with pytest.raises(ValueError):
            call()
    assert torch.cuda.max_memory_allocated() == before


def test_status_is_asked_on_the_streams_device(monkeypatch):
    from types import SimpleNamespace
    fw = _fw()
    assert fw.torch.cuda is torch.cuda
    now, asked = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(fw, "_current_device", lambda: now[0])
    monkeypatch.setattr(fw._lib, "wsattn_op_status", lambda raw: asked.append((now[0], getattr(raw, "value", raw))) or 7)
    stream = SimpleNamespace(device=SimpleNamespace(index=3), cuda_stream=77)
    assert fw.wsattn_op_status(stream) == 7
    stream.device.index = 0
    assert fw.wsattn_op_status(stream) == 7
    assert asked == [(3, 77), (0, 77)] and now == [0]


@pytest.mark.parametrize("missing", [False, True])
def test_host_only_calls_do_without_torch(missing):
    # plans and their readers start without torch, where there is none too; a
    # call on tensors imports it
    import os
    import subprocess
    import sys
    code = f"""
import sys
if {missing}:
    sys.modules["torch"] = None            # any import of it fails
import frame_aligned_window_gb300 as fw
plan = fw.wsattn_plan(4, 48, 1, 1, 2, 64)
fw.wsattn_get_block_map(plan), fw.wsattn_get_csr(plan), fw.wsattn_get_tiles(plan), fw.wsattn_plan_info(plan)
rot = fw.wsattn_rotary_plan(64, (16, 16))
fw.wsattn_qknorm_backward_workspace(rot), fw.wsattn_build_flags(), fw.wsattn_status_string(0)
assert sys.modules.get("torch") is None
try:
    fw.wsattn_rotary(rot, 1, 2)
except TypeError:
    assert not {missing} and "torch" in sys.modules and fw.torch is sys.modules["torch"]
except ImportError:
    assert {missing}
print("done")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]
