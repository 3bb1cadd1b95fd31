"""The bounds-checking build (libwsattn_debug.so) under every tiling of the
linear products, strided gradients and the norms' gradients with several work
items a CTA: the parity tests again in a child process that loads it.  Each of
them asks for the operators' status, so a failed check fails the run."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
IN_CHILD = os.environ.get("WSATTN_EXPECT_DEBUG") == "1"

RERUN = [
    "tests/test_gpu_tilings.py::test_linear_under_every_tiling",
    "tests/test_gpu_tilings.py::test_linear_backward_under_every_tiling",
    "tests/test_gpu_linear_strides.py::test_linear_backward_strided_rows",
    "tests/test_gpu_linear_infinite.py::test_gradients_behind_infinite_preactivations",
    "tests/test_gpu_qknorm_shares.py::test_qknorm_backward_shares_of_several_items",
    "tests/test_gpu_zx_debug_operators.py::test_library_is_debug_build",
]


@pytest.mark.skipif(IN_CHILD, reason="runs in the parent process only")
def test_operators_pass_bounds_checks_under_every_tiling():
    import frame_aligned_window_gb300 as fw
    lib = fw.DEBUG_LIB_PATH
    assert os.path.exists(lib), "build it with `python frame_aligned_window_gb300/build.py --debug`"
    env = dict(os.environ, WSATTN_LIBRARY=lib, WSATTN_EXPECT_DEBUG="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *RERUN]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-2000:])
    assert " passed" in r.stdout and "skipped" not in r.stdout.splitlines()[-1], r.stdout[-500:]


@pytest.mark.skipif(not IN_CHILD, reason="runs only in the child process of the test above")
def test_library_is_debug_build():
    import frame_aligned_window_gb300 as fw
    assert os.path.samefile(fw.LIB_PATH, fw.DEBUG_LIB_PATH)
    assert fw.wsattn_build_flags() & fw.BUILD_DEBUG
    assert fw.wsattn_op_status() == 0
