"""The operators' status word (GPU): what sets it here is the library's
self-test kernel, whose wait runs out after a few microseconds."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

TIMEOUT = 7


def _library():
    """The binding, and internal functions by their C++ names: the word's
    address, the self-test kernel on a word, and the clearing of bits."""
    import frame_aligned_window_gb300 as fw
    lib = ctypes.CDLL(fw.LIB_PATH)
    word = lib._ZN6wsattn13op_status_ptrEv
    word.restype, word.argtypes = ctypes.c_void_p, []
    expire = lib._ZN6wsattn23launch_timeout_selftestExPiP11CUstream_st
    expire.argtypes = [ctypes.c_longlong, ctypes.c_void_p, ctypes.c_void_p]
    clear = lib._ZN6wsattn19launch_clear_statusEPiiP11CUstream_st
    clear.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
    return fw, word(), expire, clear


def test_an_expired_wait_is_reported_once():
    fw, word, expire, _ = _library()
    assert fw.wsattn_op_status() == 0
    side = torch.cuda.Stream()
    assert expire(1000, word, side.cuda_stream) == 0
    assert fw.wsattn_op_status(side) == TIMEOUT and fw.wsattn_op_status(side) == 0
    # the word is the device's: any stream is told
    assert expire(1000, word, side.cuda_stream) == 0
    side.synchronize()
    assert fw.wsattn_op_status() == TIMEOUT and fw.wsattn_op_status(side) == 0


def test_only_reported_bits_are_cleared():
    fw, word, expire, clear = _library()
    stream = torch.cuda.current_stream().cuda_stream
    assert fw.wsattn_op_status() == 0
    assert expire(1000, word, stream) == 0         # bit 8
    assert clear(word, 1 | 2 | 4 | 16, stream) == 0
    assert fw.wsattn_op_status() == TIMEOUT and fw.wsattn_op_status() == 0


def test_a_query_waits_for_its_own_stream_only():
    fw, word, expire, _ = _library()
    side = torch.cuda.Stream()
    assert expire(1000, word, side.cuda_stream) == 0
    done = torch.cuda.Event()
    torch.cuda._sleep(1 << 30)                     # about half a second on the default stream
    done.record()
    assert fw.wsattn_op_status(side) == TIMEOUT and fw.wsattn_op_status(side) == 0
    assert not done.query()
    torch.cuda.synchronize()


def test_queries_from_two_threads_lose_nothing():
    # expired waits and queries at once: each wait is reported by a query that
    # began before or after it, never by none
    import threading
    fw, word, expire, _ = _library()
    assert fw.wsattn_op_status() == 0
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    seen, stop = [0], threading.Event()

    def poll():
        while not stop.is_set():
            seen[0] += fw.wsattn_op_status(other) == TIMEOUT
    thread = threading.Thread(target=poll)
    thread.start()
    try:
        for _ in range(200):
            before = seen[0]
            assert expire(1000, word, side.cuda_stream) == 0
            side.synchronize()
            for _ in range(100000):                # the other thread's next reports
                if seen[0] > before:
                    break
                torch.cuda.synchronize()
            assert seen[0] > before
    finally:
        stop.set()
        thread.join()
    assert fw.wsattn_op_status() == 0
