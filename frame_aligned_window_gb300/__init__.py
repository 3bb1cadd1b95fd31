"""Python binding of libwsattn (frame-aligned window-sparse attention, GB300).

Argument marshalling only: every step of the computation runs in the CUDA
library (include/wsattn.h documents each call).  Tensors are torch tensors
used as device memory; the current torch CUDA stream is passed to the
library.  If libwsattn.so is missing or fails to load, importing this
package raises: there is no fallback implementation.  The environment
variable WSATTN_LIBRARY names another build of the same library to load
instead (the tests use it for the bounds-checking libwsattn_debug.so).

The names mirror the C ABI:
    wsattn_plan, wsattn_plan_ex, wsattn_plan_destroy, wsattn_prepare, wsattn_forward,
    wsattn_plan_info, wsattn_get_tiles, wsattn_get_block_map, wsattn_get_csr, wsattn_get_stats,
    wsattn_plan_set_debug, wsattn_plan_set_bound, wsattn_device_status,
    wsattn_selftest_timeout, wsattn_status_string, wsattn_prepare_static, wsattn_produce,
    wsattn_build_flags,
    wsattn_rotary_plan, wsattn_rotary_destroy, wsattn_rotary, wsattn_qknorm,
    wsattn_qknorm_backward, wsattn_qknorm_backward_workspace, wsattn_linear,
    wsattn_linear_workspace, wsattn_linear_backward, wsattn_linear_backward_workspace,
    wsattn_op_status
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np


class _Deferred:
    """Stands for torch until a call first uses it: plans, block maps and the
    other host-only calls do without it, and without its start-up."""

    def __getattr__(self, name):
        global torch, _raw_current_stream, _current_device
        import torch
        _DTYPES.update({torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32})
        # the raw handle of a device's current stream without a Stream object
        _raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        return getattr(torch, name)


torch = _Deferred()

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("WSATTN_LIBRARY") or os.path.join(_HERE, "libwsattn.so")
DEBUG_LIB_PATH = os.path.join(_HERE, "libwsattn_debug.so")

# C ABI entry points declared in include/wsattn.h
EXPORTS = (
    "wsattn_plan", "wsattn_plan_ex", "wsattn_plan_destroy", "wsattn_prepare", "wsattn_forward",
    "wsattn_plan_info", "wsattn_get_tiles", "wsattn_get_block_map", "wsattn_get_csr",
    "wsattn_get_stats",
    "wsattn_plan_set_debug", "wsattn_plan_set_bound", "wsattn_device_status",
    "wsattn_selftest_timeout", "wsattn_status_string", "wsattn_prepare_static",
    "wsattn_produce", "wsattn_build_flags",
    "wsattn_rotary_plan", "wsattn_rotary_destroy", "wsattn_rotary", "wsattn_qknorm",
    "wsattn_qknorm_backward", "wsattn_qknorm_backward_workspace", "wsattn_linear",
    "wsattn_linear_workspace", "wsattn_linear_backward", "wsattn_linear_backward_workspace",
    "wsattn_op_status",
)

# wsattn_bound
BOUND_GLOBAL = 0
BOUND_WINDOW = 1

# wsattn_mask_flags (or-ed)
MASK_CAUSAL = 1
MASK_REF_SUFFIX = 2
MASK_REF_LOCAL = 4

# wsattn_dtype
BF16, FP16, FP32 = 0, 1, 2

# wsattn_activation, by the name the linear products take
ACTIVATIONS = {"none": 0, "gelu": 1, "gelu_tanh": 2, "silu": 3}

STATUS = {0: "OK", 1: "BAD_ARG", 2: "BAD_BLOCK", 3: "UNSUPPORTED", 4: "NOT_PREPARED",
          5: "BATCH_MISMATCH", 6: "CUDA", 7: "TIMEOUT", 8: "NO_MEMORY", 9: "BOUNDS"}

# wsattn_build_flags bits
BUILD_DEBUG = 1


class WsattnError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)} ({status_text(code)})")


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python frame_aligned_window_gb300/build.py`"
                      + (" --debug" if LIB_PATH == DEBUG_LIB_PATH else ""))
_lib = ctypes.CDLL(LIB_PATH)

_P, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_lib.wsattn_plan.argtypes = [_I, _I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_P)]
_lib.wsattn_plan_ex.argtypes = [_I, _I, _I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_P)]
_lib.wsattn_plan_destroy.argtypes = [_P]
_lib.wsattn_prepare.argtypes = [_P, _I, _P, _P, _P]
_lib.wsattn_forward.argtypes = [_P, _I, _P, _P, _P, _P, _P]
_lib.wsattn_plan_info.argtypes = [_P, _P, _I]
_lib.wsattn_get_block_map.argtypes = [_P, _P, _SZ]
_lib.wsattn_get_csr.argtypes = [_P, _P, _P, _SZ, _SZ]
_lib.wsattn_get_tiles.argtypes = [_P, _P, _SZ, _P, _SZ]
_lib.wsattn_get_stats.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P]
_lib.wsattn_plan_set_debug.argtypes = [_P, _I, _F]
_lib.wsattn_plan_set_bound.argtypes = [_P, _I]
_lib.wsattn_device_status.argtypes = [_P, _P]
_lib.wsattn_selftest_timeout.argtypes = [_I, ctypes.POINTER(_I), _P]
_lib.wsattn_status_string.argtypes = [_I]
_lib.wsattn_prepare_static.argtypes = [_I, _I, _I, _I, _F, _P, _P, _P, _P, _P, _P, _P, _P, _P]
_lib.wsattn_produce.argtypes = [_P, _I, _P, _I, _P, _P, _P, _F, _P, _P, _P, _P]
_lib.wsattn_build_flags.argtypes = []


# The argument structs of include/wsattn.h, in the C layout ("@": native sizes
# and alignment; "0q" pads the end).  They are packed rather than built as
# ctypes structures: the smallest calls are bound by the host.
_HEADS = struct.Struct("@Piqqq0q").pack  # wsattn_heads: data, heads, strides b, h, n
# wsattn_linear_args: dtype, out_dtype, m, n, k, x, ldx, x_heads, x_tokens, w,
# ldw, bias, residual, ldr, out, ldo, preact, ldp, activation
_LINEAR = struct.Struct("@iiqiiPqiqPqPPqPqPqi0q").pack
# wsattn_linear_grad_args: dtype, m, n, k, dout, ldd, x, ldx, w, ldw, preact,
# ldp, activation, dx, lddx, dw, lddw, db
_LINEAR_GRAD = struct.Struct("@iqiiPqPqPqPqiPqPqP0q").pack

_I64, _SZP = ctypes.c_int64, ctypes.POINTER(_SZ)
_lib.wsattn_rotary_plan.argtypes = [_I, _I, _P, _P, _I, ctypes.POINTER(_P)]
_lib.wsattn_rotary_destroy.argtypes = [_P]
_lib.wsattn_rotary.argtypes = [_P, _I, _I, _I64, _P, _P, _I64, _I, _P, _P]
_lib.wsattn_qknorm.argtypes = [_P, _I, _I, _I64, _P, _P, _P, _P, _P, _I, _F, _P, _I64, _P,
                               _P, _P, _P]
_lib.wsattn_qknorm_backward.argtypes = [_P, _I, _I, _I64, _P, _P, _P, _P, _P, _P, _P, _I, _F,
                                        _P, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]
_lib.wsattn_qknorm_backward_workspace.argtypes = [_P, _SZP]
_lib.wsattn_linear.argtypes = [_P, _P, _SZ, _P]
_lib.wsattn_linear_workspace.argtypes = [_P, _SZP]
_lib.wsattn_linear_backward.argtypes = [_P, _P, _SZ, _P]
_lib.wsattn_linear_backward_workspace.argtypes = [_P, _SZP]
_lib.wsattn_op_status.argtypes = [_P]
_lib.wsattn_status_string.restype = ctypes.c_char_p
for _name in EXPORTS:
    if _name != "wsattn_status_string":
        getattr(_lib, _name).restype = _I


def wsattn_build_flags() -> int:
    """BUILD_DEBUG when the loaded library checks bounds in its kernels."""
    return int(_lib.wsattn_build_flags())


def status_text(code: int) -> str:
    return _lib.wsattn_status_string(int(code)).decode()


def wsattn_status_string(code: int) -> str:
    return status_text(code)


def _check(rc: int, what: str):
    if rc != 0:
        raise WsattnError(rc, what)


class Plan:
    """Owns a wsattn_plan_t handle (released by destroy() or on collection)."""

    def __init__(self, handle, args):
        self._h = handle
        self.args = args
        info = np.zeros(10, dtype=np.int64)
        _check(_lib.wsattn_plan_info(self._h, info.ctypes.data, 10), "wsattn_plan_info")
        (self.n_tokens, self.block_q, self.block_k, self.n_qblocks, self.n_kblocks, self.nnz,
         self.tiles_per_head, self.head_dim, self.heads, self.active_pairs) = (int(x) for x in info)
        self.frames, self.tokens_per_frame, self.window, self.ref_frames = args[:4]

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("plan was destroyed")
        return self._h

    def destroy(self):
        if self._h is not None:
            _lib.wsattn_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def _stream_ptr(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev_ptr(t, name, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _check_shape(plan: Plan, t, name):
    if t.dim() != 4 or t.shape[1] != plan.heads or t.shape[2] != plan.n_tokens \
            or t.shape[3] != plan.head_dim:
        raise ValueError(f"{name} must be [B, {plan.heads}, {plan.n_tokens}, {plan.head_dim}], "
                         f"got {tuple(t.shape)}")


def wsattn_plan(frames, tokens_per_frame, window, ref_frames, heads, head_dim, block_q=0,
                block_k=0, mask_flags=0) -> Plan:
    """wsattn_plan_ex when mask_flags != 0 (MASK_* or-ed), else wsattn_plan."""
    h = _P()
    args = (frames, tokens_per_frame, window, ref_frames, heads, head_dim, block_q, block_k)
    if mask_flags:
        _check(_lib.wsattn_plan_ex(*args, int(mask_flags), ctypes.byref(h)), "wsattn_plan_ex")
    else:
        _check(_lib.wsattn_plan(*args, ctypes.byref(h)), "wsattn_plan")
    plan = Plan(h, args)
    plan.mask_flags = int(mask_flags)
    return plan


def wsattn_plan_ex(frames, tokens_per_frame, window, ref_frames, heads, head_dim, block_q,
                   block_k, mask_flags) -> Plan:
    return wsattn_plan(frames, tokens_per_frame, window, ref_frames, heads, head_dim, block_q,
                       block_k, mask_flags)


def wsattn_plan_destroy(plan: Plan):
    plan.destroy()


def wsattn_prepare(plan: Plan, q, k, stream=None):
    """Key mean, row bounds, row fixed max and per-head eligibility (q, k read only)."""
    _check_shape(plan, q, "q")
    _check_shape(plan, k, "k")
    if q.shape[0] != k.shape[0]:
        raise ValueError("q and k batch differ")
    _check(_lib.wsattn_prepare(plan.handle, q.shape[0], _dev_ptr(q, "q", torch.bfloat16),
                               _dev_ptr(k, "k", torch.bfloat16), _stream_ptr(stream)),
           "wsattn_prepare")


def wsattn_produce(plan: Plan, x, w_qkv, rope_cos, rope_sin, eps: float = 1e-6, q=None, k=None,
                   v=None, stream=None):
    """Pre-attention producer: x [B, N, C] bf16, w_qkv [3HD, C] bf16, rope
    tables fp32 [N, D/2] -> (q, k, v) bf16 [B, H, N, D]; the plan's
    statistics are then ready for wsattn_forward, as after wsattn_prepare."""
    if x.dim() != 3 or x.shape[1] != plan.n_tokens:
        raise ValueError(f"x must be [B, {plan.n_tokens}, C], got {tuple(x.shape)}")
    B, _, C = x.shape
    hd = plan.heads * plan.head_dim
    if tuple(w_qkv.shape) != (3 * hd, C):
        raise ValueError(f"w_qkv must be [{3 * hd}, {C}], got {tuple(w_qkv.shape)}")
    for t, n in ((rope_cos, "rope_cos"), (rope_sin, "rope_sin")):
        if tuple(t.shape) != (plan.n_tokens, plan.head_dim // 2):
            raise ValueError(f"{n} must be [{plan.n_tokens}, {plan.head_dim // 2}]")
    shape = (B, plan.heads, plan.n_tokens, plan.head_dim)
    q = torch.empty(shape, dtype=torch.bfloat16, device=x.device) if q is None else q
    k = torch.empty(shape, dtype=torch.bfloat16, device=x.device) if k is None else k
    v = torch.empty(shape, dtype=torch.bfloat16, device=x.device) if v is None else v
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_shape(plan, t, n)
        if t.shape[0] != B:
            raise ValueError(f"{n} batch differs from x")
    _check(_lib.wsattn_produce(plan.handle, B, _dev_ptr(x, "x", torch.bfloat16), C,
                               _dev_ptr(w_qkv, "w_qkv", torch.bfloat16),
                               _dev_ptr(rope_cos, "rope_cos", torch.float32),
                               _dev_ptr(rope_sin, "rope_sin", torch.float32), float(eps),
                               _dev_ptr(q, "q", torch.bfloat16), _dev_ptr(k, "k", torch.bfloat16),
                               _dev_ptr(v, "v", torch.bfloat16), _stream_ptr(stream)),
           "wsattn_produce")
    return q, k, v


def wsattn_forward(plan: Plan, q, k, v, out=None, stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_shape(plan, t, n)
    if not (q.shape[0] == k.shape[0] == v.shape[0]):
        raise ValueError("q, k, v batch differ")
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    _check_shape(plan, out, "out")
    _check(_lib.wsattn_forward(plan.handle, q.shape[0], _dev_ptr(q, "q", torch.bfloat16),
                               _dev_ptr(k, "k", torch.bfloat16), _dev_ptr(v, "v", torch.bfloat16),
                               _dev_ptr(out, "out", torch.float32), _stream_ptr(stream)),
           "wsattn_forward")
    return out


def wsattn_plan_info(plan: Plan) -> dict:
    return {"n_tokens": plan.n_tokens, "block_q": plan.block_q, "block_k": plan.block_k,
            "n_qblocks": plan.n_qblocks, "n_kblocks": plan.n_kblocks, "nnz": plan.nnz,
            "tiles_per_head": plan.tiles_per_head, "head_dim": plan.head_dim,
            "heads": plan.heads, "active_pairs": plan.active_pairs}


def wsattn_get_block_map(plan: Plan) -> np.ndarray:
    out = np.zeros((plan.n_qblocks, plan.n_kblocks), dtype=np.uint8)
    _check(_lib.wsattn_get_block_map(plan.handle, out.ctypes.data, out.size),
           "wsattn_get_block_map")
    return out


def wsattn_get_tiles(plan: Plan):
    """The forward work list: int32 [tiles, 10] {row0, nvalid, nblk, run0, len0,
    run1, nstep, kbeg, gsz, gtab} and the merged tails' group table int32
    [groups, 4] {run0, len0, run1, len1}."""
    tiles = np.zeros((plan.tiles_per_head, 10), dtype=np.int32)
    # each merged tile holds at most 8 row groups (tails of at least 16 rows)
    groups = np.zeros((8 * plan.tiles_per_head, 4), dtype=np.int32)
    _check(_lib.wsattn_get_tiles(plan.handle, tiles.ctypes.data, tiles.size, groups.ctypes.data,
                                 groups.size), "wsattn_get_tiles")
    merged = tiles[:, 8] > 0
    n_groups = int((tiles[merged, 1] // tiles[merged, 8]).sum())  # nvalid = groups x gsz
    return tiles, groups[:n_groups]


def wsattn_get_csr(plan: Plan):
    row_ptr = np.zeros(plan.n_qblocks + 1, dtype=np.int32)
    col = np.zeros(max(plan.nnz, 1), dtype=np.int32)
    _check(_lib.wsattn_get_csr(plan.handle, row_ptr.ctypes.data, col.ctypes.data, row_ptr.size,
                               col.size), "wsattn_get_csr")
    return row_ptr, col[:plan.nnz]


def wsattn_get_stats(plan: Plan, batch: int, stream=None) -> dict:
    bh = batch * plan.heads
    b = np.zeros((bh, plan.n_tokens), dtype=np.float32)
    m = np.zeros((bh, plan.n_tokens), dtype=np.float32)
    mu = np.zeros((bh, plan.head_dim), dtype=np.float32)
    kmax = np.zeros(bh, dtype=np.float32)
    bmax = np.zeros(bh, dtype=np.float32)
    elig = np.zeros(bh, dtype=np.uint8)
    _check(_lib.wsattn_get_stats(plan.handle, b.ctypes.data, m.ctypes.data, mu.ctypes.data,
                                 kmax.ctypes.data, bmax.ctypes.data, elig.ctypes.data,
                                 _stream_ptr(stream)), "wsattn_get_stats")
    return {"b": b, "m": m, "mu": mu, "kmax": kmax, "bmax": bmax, "elig": elig}


def wsattn_plan_set_debug(plan: Plan, force_path: int = -1, tau: float = 0.0):
    _check(_lib.wsattn_plan_set_debug(plan.handle, int(force_path), float(tau)),
           "wsattn_plan_set_debug")


def wsattn_plan_set_bound(plan: Plan, mode: int):
    """BOUND_GLOBAL (default) or BOUND_WINDOW: the key-norm maximum of the row
    bounds; prepare again before the next forward."""
    _check(_lib.wsattn_plan_set_bound(plan.handle, int(mode)), "wsattn_plan_set_bound")


def wsattn_device_status(plan: Plan, stream=None) -> int:
    return int(_lib.wsattn_device_status(plan.handle, _stream_ptr(stream)))


def wsattn_selftest_timeout(limit_ms: int = 50, stream=None) -> int:
    st = _I(-1)
    _check(_lib.wsattn_selftest_timeout(int(limit_ms), ctypes.byref(st), _stream_ptr(stream)),
           "wsattn_selftest_timeout")
    return int(st.value)


def wsattn_prepare_static(q, k, out: dict, tau: float = 40.0, stream=None):
    """No-allocation prepare: statistics into the caller's tensors in `out`
    (keys b, m, mu, kmax, bmax, elig, shaped as wsattn_prepare_static_outputs
    makes them).  For callers that must not let the library allocate."""
    B, H, N, D = q.shape
    if k.shape != q.shape:
        raise ValueError("q and k shapes differ")
    _check(_lib.wsattn_prepare_static(
        B, H, N, D, float(tau), _dev_ptr(q, "q", torch.bfloat16), _dev_ptr(k, "k", torch.bfloat16),
        _dev_ptr(out["b"], "b", torch.float32), _dev_ptr(out["m"], "m", torch.float32),
        _dev_ptr(out["mu"], "mu", torch.float32), _dev_ptr(out["kmax"], "kmax", torch.float32),
        _dev_ptr(out["bmax"], "bmax", torch.float32), _dev_ptr(out["elig"], "elig", torch.uint8),
        _stream_ptr(stream)), "wsattn_prepare_static")
    return out


def wsattn_prepare_static_outputs(batch, heads, n_tokens, head_dim, device="cuda"):
    """Caller-owned output tensors for wsattn_prepare_static."""
    bh = batch * heads
    f = dict(dtype=torch.float32, device=device)
    return {"b": torch.empty(bh, n_tokens, **f), "m": torch.empty(bh, n_tokens, **f),
            "mu": torch.empty(bh, head_dim, **f), "kmax": torch.empty(bh, **f),
            "bmax": torch.empty(bh, **f),
            "elig": torch.empty(bh, dtype=torch.uint8, device=device)}


# ------------------------------------------------ operators around the attention

# filled and replaced by faster ones when torch is imported
_DTYPES = {}
_raw_current_stream = None


def _current_device():
    return torch.cuda.current_device()


def _dtype_code(t, name, allowed=(BF16, FP16, FP32)):
    code = _DTYPES.get(t.dtype)
    if code not in allowed:
        raise TypeError(f"{name} must not be {t.dtype}")
    return code


def _device_of(t, name):
    """Index of the CUDA device a call's tensors live on, from its first one."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _check_tensor(t, name, dev, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _raw_stream(dev, stream):
    """The stream a call on tensors of device `dev` goes to (default: that
    device's current one)."""
    if stream is None:
        if _raw_current_stream is not None:
            return _raw_current_stream(dev)
        return torch.cuda.current_stream(dev).cuda_stream
    if stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{dev}")
    return stream.cuda_stream


def _empty(shape, dtype, like, stream):
    """Memory on the device of `like`, from `stream`'s own pool, so that its reuse is ordered with the
    work the call enqueues there (and, in a capture, belongs to the graph)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _run(dev, what, fn, *args):
    """The C call, with the tensors' device current."""
    if _current_device() == dev:
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc:
        raise WsattnError(rc, what)


class RotaryPlan:
    """Owns a wsattn_rotary_t handle (host memory only)."""

    def __init__(self, handle, head_dim, axes):
        self._h = handle
        self.head_dim = head_dim
        self.axes = axes
        self._workspace = None

    @property
    def backward_workspace(self):
        """Bytes of scratch of wsattn_qknorm_backward."""
        if self._workspace is None:
            n = _SZ()
            _check(_lib.wsattn_qknorm_backward_workspace(self.handle, ctypes.byref(n)),
                   "wsattn_qknorm_backward_workspace")
            self._workspace = int(n.value)
        return self._workspace

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("rotary plan was destroyed")
        return self._h

    def destroy(self):
        if self._h is not None:
            _lib.wsattn_rotary_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def wsattn_rotary_plan(head_dim, sections=None, base: float = 10000.0, interleaved: bool = True,
                       pair_axis=None, pair_freq=None, axes=None) -> RotaryPlan:
    """Turning rates of a head's pairs.  sections: pairs turned by each axis of
    the positions (time, height, width, ...), in order; pair j of a section of
    n turns by base**(-j / n) radians per unit of its axis, and pairs behind
    the sections are left alone.  Or pair_axis and pair_freq [D / 2] directly,
    with `axes` columns of positions (default: as many as pair_axis names).
    interleaved: pairs are dims (2p, 2p + 1) (as wsattn_produce turns them),
    else (p, p + D / 2)."""
    if (pair_axis is None) != (pair_freq is None) or (sections is None) == (pair_axis is None):
        raise ValueError("give sections, or pair_axis and pair_freq")
    if sections is not None and axes not in (None, len(sections)):
        raise ValueError(f"{len(sections)} sections for {axes} axes")
    half = max(int(head_dim), 0) // 2
    if sections is not None:
        sections = tuple(int(n) for n in sections)
        if not sections or min(sections) < 0 or sum(sections) > half:
            raise ValueError(f"sections {sections} do not fit {half} pairs")
        if not base > 0:
            raise ValueError("base must be positive")
        axes, first = len(sections), 0
        axis, freq = np.zeros(half, dtype=np.int32), np.zeros(half)
        for a, n in enumerate(sections):
            axis[first:first + n] = a
            freq[first:first + n] = float(base) ** (np.arange(n) / -max(n, 1))
            first += n
    else:
        axis = np.ascontiguousarray(pair_axis, dtype=np.int32)
        freq = np.ascontiguousarray(pair_freq, dtype=np.float64)
        if axis.shape != (half,) or freq.shape != (half,):
            raise ValueError(f"pair_axis and pair_freq must have {half} entries")
        axes = axes if axes is not None else int(axis.max()) + 1 if half else 0
    h = _P()
    _check(_lib.wsattn_rotary_plan(int(head_dim), int(axes), axis.ctypes.data, freq.ctypes.data,
                                   int(bool(interleaved)), ctypes.byref(h)), "wsattn_rotary_plan")
    return RotaryPlan(h, int(head_dim), int(axes))


def wsattn_rotary_destroy(rot: RotaryPlan):
    rot.destroy()


def _head_view(t, name, shape, dtype, dev):
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _check_tensor(t, name, dev, dtype)
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    sb, sh, sn, sd = t.stride()
    if sd != 1 and t.numel():
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return _HEADS(t.data_ptr(), shape[1], sb, sh, sn)


def _positions(rot, t, batch, tokens, dev):
    """(pointer, batch stride) of the positions."""
    if t.dtype is not torch.float32 or t.get_device() != dev:
        _check_tensor(t, "positions", dev, torch.float32)
    axes, shape, st = rot.axes, t.shape, t.stride()
    if shape == (tokens, axes):
        stride = 0
    elif shape == (batch, tokens, axes):
        stride = st[0] if batch > 1 else 0
    else:
        raise ValueError(f"positions must be [{tokens}, {axes}] or [{batch}, {tokens}, {axes}], "
                         f"got {list(shape)}")
    if (axes > 1 and st[-1] != 1 or tokens > 1 and st[-2] != axes) and t.numel():
        raise ValueError("positions must be contiguous")
    return t.data_ptr(), stride


_INT_MAX = (1 << 31) - 1  # batch elements and heads are ints of the C ABI


def _heads_shape(t, name, rot):
    shape = t.shape
    if len(shape) != 4 or shape[3] != rot.head_dim:
        raise ValueError(f"{name} must be [B, H, N, {rot.head_dim}], got {list(shape)}")
    if shape[0] > _INT_MAX or shape[1] > _INT_MAX:  # ctypes would drop the upper bits
        raise ValueError(f"{name} has more than {_INT_MAX} batch elements or heads: {list(shape)}")
    return shape


def wsattn_rotary(rot: RotaryPlan, x, positions, inverse: bool = False, out=None, stream=None):
    """x [B, H, N, D] (bf16, fp16 or fp32; any strides, last dimension
    contiguous) turned by positions fp32 [N, axes] or [B, N, axes]; inverse
    turns back (the gradient).  out: default a contiguous tensor; may be x."""
    dev = _device_of(x, "x")
    shape, dt = _heads_shape(x, "x", rot), x.dtype
    code = _dtype_code(x, "x")
    raw = _raw_stream(dev, stream)
    pos, pos_b = _positions(rot, positions, shape[0], shape[2], dev)
    if out is None:
        out = _empty(shape, dt, x, stream)
    _run(dev, "wsattn_rotary", _lib.wsattn_rotary, rot.handle, code, shape[0], shape[2],
         _head_view(x, "x", shape, dt, dev), pos, pos_b, 1 if inverse else 0,
         _head_view(out, "out", shape, dt, dev), raw)
    return out


def _gains(q_weight, k_weight, dim, dtype, code, dev):
    """Pointers of the gain vectors and their dtype code."""
    ptr, kind = [None, None], None
    for i, t in enumerate((q_weight, k_weight)):
        if t is None:
            continue
        name = "qk"[i] + "_weight"
        _check_tensor(t, name, dev)
        if t.shape != (dim,) or t.stride(0) != 1:
            raise ValueError(f"{name} must be contiguous [{dim}], got {list(t.shape)}")
        if t.dtype != dtype and t.dtype != torch.float32:
            raise TypeError(f"{name} must be {dtype} or torch.float32, got {t.dtype}")
        if kind is not None and kind != t.dtype:
            raise TypeError("q_weight and k_weight must have one type")
        kind, ptr[i] = t.dtype, t.data_ptr()
    return ptr[0], ptr[1], FP32 if kind == torch.float32 else code


def _qkv_shapes(rot, q, k, v):
    """Checked shapes of q, k and v (or of their gradients)."""
    sq, sk = _heads_shape(q, "q", rot), _heads_shape(k, "k", rot)
    sv = None if v is None else _heads_shape(v, "v", rot)
    for name, sh in (("k", sk), ("v", sv)):
        if sh is not None and (sh[0] != sq[0] or sh[2] != sq[2]):
            raise ValueError(f"{name} must have q's batch and tokens, got {list(sh)}")
    return sq, sk, sv


def wsattn_qknorm(rot: RotaryPlan, q, k, positions, q_weight=None, k_weight=None,
                  eps: float = 1e-6, v=None, q_out=None, k_out=None, v_out=None, stream=None):
    """Per-head RMS norm (with gains [D]) and rotation of q [B, Hq, N, D] and
    k [B, Hk, N, D], and a copy of v, in one pass; q, k, v may be views of one
    projection's rows.  Returns (q, k) or (q, k, v), by default contiguous, as
    wsattn_prepare and wsattn_forward read them; an output may be its input."""
    dev = _device_of(q, "q")
    sq, sk, sv = _qkv_shapes(rot, q, k, v)
    if v is None and v_out is not None:
        raise ValueError("v_out without v")
    raw = _raw_stream(dev, stream)
    code, dt = _dtype_code(q, "q"), q.dtype
    wq, wk, wcode = _gains(q_weight, k_weight, rot.head_dim, dt, code, dev)
    pos, pos_b = _positions(rot, positions, sq[0], sq[2], dev)
    q_out = _empty(sq, dt, q, stream) if q_out is None else q_out
    k_out = _empty(sk, dt, q, stream) if k_out is None else k_out
    if v is not None and v_out is None:
        v_out = _empty(sv, dt, q, stream)
    _run(dev, "wsattn_qknorm", _lib.wsattn_qknorm, rot.handle, code, sq[0], sq[2],
         _head_view(q, "q", sq, dt, dev), _head_view(k, "k", sk, dt, dev),
         None if v is None else _head_view(v, "v", sv, dt, dev), wq, wk, wcode, eps, pos, pos_b,
         _head_view(q_out, "q_out", sq, dt, dev), _head_view(k_out, "k_out", sk, dt, dev),
         None if v is None else _head_view(v_out, "v_out", sv, dt, dev), raw)
    return (q_out, k_out) if v is None else (q_out, k_out, v_out)


def wsattn_qknorm_backward_workspace(rot: RotaryPlan) -> int:
    """Bytes of scratch wsattn_qknorm_backward takes for the gains' gradients."""
    return rot.backward_workspace


def _scratch_args(workspace, dev):
    if workspace is None:
        return None, 0
    _check_tensor(workspace, "workspace", dev)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def wsattn_qknorm_backward(rot: RotaryPlan, dq_out, dk_out, q, k, positions, q_weight=None,
                           k_weight=None, eps: float = 1e-6, dv_out=None, dq=None, dk=None,
                           dv=None, workspace=None, stream=None):
    """Gradients of wsattn_qknorm: (dq, dk, dv, dq_weight, dk_weight).  dq, dk
    and dv may be views of one packed gradient (default: contiguous); dv is
    None without dv_out, and a gain's gradient (fp32 [D]) None without the gain."""
    dev = _device_of(q, "q")
    sq, sk, sv = _qkv_shapes(rot, q, k, dv_out)
    if dv_out is None and dv is not None:
        raise ValueError("dv without dv_out")
    raw = _raw_stream(dev, stream)
    code, dt, dim = _dtype_code(q, "q"), q.dtype, rot.head_dim
    wq, wk, wcode = _gains(q_weight, k_weight, dim, dt, code, dev)
    pos, pos_b = _positions(rot, positions, sq[0], sq[2], dev)
    dq = _empty(sq, dt, q, stream) if dq is None else dq
    dk = _empty(sk, dt, q, stream) if dk is None else dk
    if dv_out is not None and dv is None:
        dv = _empty(sv, dt, q, stream)
    dwq = None if wq is None else _empty((dim,), torch.float32, q, stream)
    dwk = None if wk is None else _empty((dim,), torch.float32, q, stream)
    if workspace is None and (dwq is not None or dwk is not None):
        workspace = _empty((rot.backward_workspace,), torch.uint8, q, stream)
    ws, ws_bytes = _scratch_args(workspace, dev)
    _run(dev, "wsattn_qknorm_backward", _lib.wsattn_qknorm_backward, rot.handle, code, sq[0],
         sq[2], _head_view(dq_out, "dq_out", sq, dt, dev),
         _head_view(dk_out, "dk_out", sk, dt, dev),
         None if dv is None else _head_view(dv_out, "dv_out", sv, dt, dev),
         _head_view(q, "q", sq, dt, dev), _head_view(k, "k", sk, dt, dev), wq, wk, wcode, eps, pos,
         pos_b, _head_view(dq, "dq", sq, dt, dev), _head_view(dk, "dk", sk, dt, dev),
         None if dv is None else _head_view(dv, "dv", sv, dt, dev),
         None if dwq is None else dwq.data_ptr(), None if dwk is None else dwk.data_ptr(), ws,
         ws_bytes, raw)
    return dq, dk, dv, dwq, dwk


def _rows(t, name, cols, lead, dtype, dev):
    """Row stride of t seen as a matrix of `cols` columns under the leading
    dimensions `lead` (None: any), which must lie one row stride apart."""
    if t.dtype is not dtype or t.get_device() != dev:
        _check_tensor(t, name, dev, dtype)
    shape = t.shape
    if not shape or shape[-1] != cols or (lead is not None and shape[:-1] != lead):
        want = "..." if lead is None else ", ".join(str(x) for x in lead)
        raise ValueError(f"{name} must be [{want}, {cols}], got {list(shape)}")
    if t.is_contiguous():
        return cols
    st = t.stride()
    rows, ld = 1, None
    if t.numel() == 0:
        return cols
    if cols > 1 and st[-1] != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    for n, step in zip(reversed(shape[:-1]), reversed(st[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = step
        elif step != ld * rows:
            raise ValueError(f"{name}'s rows must lie one stride apart")
        rows *= n
    if ld is not None and ld < cols:
        raise ValueError(f"{name}'s rows must not overlap")
    return cols if ld is None else ld


def _activation(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}")
    return code


def _scratch(query, what, args, workspace, dev, like, stream):
    """(pointer, bytes, tensor) of a call's workspace, allocated when needed."""
    if workspace is None:
        n = _SZ()
        _run(dev, what, query, args, ctypes.byref(n))
        if not n.value:
            return None, 0, None
        workspace = _empty((n.value,), torch.uint8, like, stream)
    return *_scratch_args(workspace, dev), workspace


def _linear_args(x, weight, bias, residual, activation, preact, out, out_dtype, stream, query=False):
    """The packed wsattn_linear_args, the output and the device.  query: for
    the workspace's size, which depends on x and weight alone (no output)."""
    dev = _device_of(weight, "weight")
    if weight.dim() != 2:
        raise ValueError(f"weight must be [n, k], got {list(weight.shape)}")
    n, k = weight.shape
    dt, code = weight.dtype, _dtype_code(weight, "weight", (BF16, FP16))
    act = _activation(activation)
    if x.dtype is dt:
        lead, heads, tokens = x.shape[:-1], 0, 0
        ldx = _rows(x, "x", k, None, dt, dev)
    else:
        if x.dtype != torch.float32 or x.dim() != 4:
            raise TypeError(f"x must be {dt} (or wsattn_forward's fp32 output), got {x.dtype}")
        _check_tensor(x, "x", dev)
        B, heads, tokens, D = x.shape
        if heads * D != k or not x.is_contiguous():
            raise ValueError(f"x must be contiguous [B, H, N, D] with H * D = {k}, "
                             f"got {list(x.shape)}")
        lead, ldx = torch.Size((B, tokens)), 0
    m = lead.numel()
    ldw = _rows(weight, "weight", k, None, dt, dev)
    xp, wp = x.data_ptr(), weight.data_ptr()
    bp = rp = pp = ldr = ldp = 0
    if query:
        return _LINEAR(code, code, m, n, k, xp, ldx, heads, tokens, wp, ldw, bp, rp, ldr, 0, n, pp,
                       ldp, act), None, dev, False
    if bias is not None:
        _check_tensor(bias, "bias", dev, dt)
        if bias.shape != (n,) or (n > 1 and bias.stride(0) != 1):
            raise ValueError(f"bias must be contiguous [{n}], got {list(bias.shape)}")
        bp = bias.data_ptr()
    if out is None:
        out = _empty(lead + (n,), dt if out_dtype is None else out_dtype, weight, stream)
    elif out_dtype not in (None, out.dtype):
        raise TypeError(f"out is {out.dtype}, not {out_dtype}")
    odt = out.dtype
    ocode = code if odt is dt else _dtype_code(out, "out", (FP32,))
    ldo = _rows(out, "out", n, lead, odt, dev)
    if residual is not None:
        ldr, rp = _rows(residual, "residual", n, lead, odt, dev), residual.data_ptr()
    if preact is not None:
        ldp, pp = _rows(preact, "preact", n, lead, dt, dev), preact.data_ptr()
    # no workspace: operands whose rows start on 16-byte boundaries, and too
    # little work for a contraction to be split
    plain = not (heads or (xp | wp) & 15 or (ldx | ldw) & 7 or m * n * k >= 1 << 33)
    return _LINEAR(code, ocode, m, n, k, xp, ldx, heads, tokens, wp, ldw, bp, rp, ldr,
                   out.data_ptr(), ldo, pp, ldp, act), out, dev, plain


def wsattn_linear(x, weight, bias=None, residual=None, activation="none", preact=None, out=None,
                  out_dtype=None, workspace=None, stream=None):
    """residual + act(x weight^T + bias): x [..., k] in weight's type (bf16 or
    fp16), or wsattn_forward's fp32 output [B, H, N, D], whose heads are merged
    (the result is then [B, N, n]).  activation: a name in ACTIVATIONS.
    preact: a tensor that receives x weight^T + bias, for
    wsattn_linear_backward.  out (or out_dtype): weight's type or fp32, and
    the residual's; residual may be out."""
    args, out, dev, plain = _linear_args(x, weight, bias, residual, activation, preact, out,
                                         out_dtype, stream)
    raw = _raw_stream(dev, stream)
    ws = nbytes = _hold = None
    if workspace is not None or not plain:
        ws, nbytes, _hold = _scratch(_lib.wsattn_linear_workspace, "wsattn_linear_workspace", args,
                                     workspace, dev, weight, stream)
    _run(dev, "wsattn_linear", _lib.wsattn_linear, args, ws, nbytes or 0, raw)
    return out


def wsattn_linear_workspace(x, weight) -> int:
    """Bytes of scratch wsattn_linear takes for these operands (0 for products
    below 2^33 multiply-adds whose rows start on 16-byte boundaries, unless x
    is the attention's output)."""
    args, _, dev, _ = _linear_args(x, weight, None, None, "none", None, None, None, None, query=True)
    n = _SZ()
    _run(dev, "wsattn_linear_workspace", _lib.wsattn_linear_workspace, args, ctypes.byref(n))
    return int(n.value)


def _linear_grad_args(dout, x, weight, preact, activation, dx, dw, db, need_dx, need_dw, need_db,
                      stream, query=False):
    """The packed wsattn_linear_grad_args, the gradients and the device.  query:
    for the workspace's size, which depends on which gradients are wanted, not
    on where they go (any address stands for them, and nothing is allocated)."""
    dev = _device_of(weight, "weight")
    if weight.dim() != 2:
        raise ValueError(f"weight must be [n, k], got {list(weight.shape)}")
    n, k = weight.shape
    dt, code = weight.dtype, _dtype_code(weight, "weight", (BF16, FP16))
    act = _activation(activation)
    if act and preact is None:
        raise ValueError("an activation's gradient needs preact")
    ldx = _rows(x, "x", k, None, dt, dev)
    lead = x.shape[:-1]
    m = lead.numel()
    ldd = _rows(dout, "dout", n, lead, dt, dev)
    ldw = _rows(weight, "weight", k, None, dt, dev)
    pp = ldp = dxp = lddx = dwp = lddw = dbp = 0
    if preact is not None:
        ldp, pp = _rows(preact, "preact", n, lead, dt, dev), preact.data_ptr()
    if query:
        dxp, dwp, dbp = (256 if need else 0 for need in (need_dx, need_dw, need_db))
        return _LINEAR_GRAD(code, m, n, k, dout.data_ptr(), ldd, x.data_ptr(), ldx,
                            weight.data_ptr(), ldw, pp, ldp, act, dxp, k, dwp, k, dbp), dx, dw, db, dev
    if need_dx or dx is not None:
        dx = _empty(x.shape, dt, weight, stream) if dx is None else dx
        lddx, dxp = _rows(dx, "dx", k, lead, dt, dev), dx.data_ptr()
    if need_dw or dw is not None:
        dw = _empty((n, k), dt, weight, stream) if dw is None else dw
        lddw, dwp = _rows(dw, "dw", k, (n,), dt, dev), dw.data_ptr()
    if need_db or db is not None:
        db = _empty((n,), torch.float32, weight, stream) if db is None else db
        _check_tensor(db, "db", dev, torch.float32)
        if db.shape != (n,) or (n > 1 and db.stride(0) != 1):
            raise ValueError(f"db must be contiguous [{n}], got {list(db.shape)}")
        dbp = db.data_ptr()
    args = _LINEAR_GRAD(code, m, n, k, dout.data_ptr(), ldd, x.data_ptr(), ldx, weight.data_ptr(),
                        ldw, pp, ldp, act, dxp, lddx, dwp, lddw, dbp)
    return args, dx, dw, db, dev


def wsattn_linear_backward(dout, x, weight, preact=None, activation="none", dx=None, dw=None,
                           db=None, need_dx=True, need_dw=True, need_db=True, workspace=None,
                           stream=None):
    """Gradients of wsattn_linear from dout [..., n]: (dx, dw, db), dx and dw in
    weight's type, db fp32; None for what is not needed.  preact: what
    wsattn_linear left there (not needed without an activation).  The
    residual's gradient is dout itself."""
    args, dx, dw, db, dev = _linear_grad_args(dout, x, weight, preact, activation, dx, dw, db,
                                              need_dx, need_dw, need_db, stream)
    raw = _raw_stream(dev, stream)
    ws, nbytes, _hold = _scratch(_lib.wsattn_linear_backward_workspace,
                                 "wsattn_linear_backward_workspace", args, workspace, dev, weight,
                                 stream)
    _run(dev, "wsattn_linear_backward", _lib.wsattn_linear_backward, args, ws, nbytes, raw)
    return dx, dw, db


def wsattn_linear_backward_workspace(dout, x, weight, preact=None, activation="none", need_dx=True,
                                     need_dw=True, need_db=True) -> int:
    """Bytes of scratch wsattn_linear_backward takes for these operands."""
    args, *_, dev = _linear_grad_args(dout, x, weight, preact, activation, None, None, None,
                                      need_dx, need_dw, need_db, None, query=True)
    n = _SZ()
    _run(dev, "wsattn_linear_backward_workspace", _lib.wsattn_linear_backward_workspace, args,
         ctypes.byref(n))
    return int(n.value)


def wsattn_op_status(stream=None) -> int:
    """Status of the operators above on the stream's device (default: the
    current stream).  One word a device, shared by its streams: see wsattn.h.
    Synchronises the stream."""
    dev = _current_device() if stream is None else stream.device.index
    raw = _raw_stream(dev, stream)
    if _current_device() == dev:
        return int(_lib.wsattn_op_status(raw))
    with torch.cuda.device(dev):
        return int(_lib.wsattn_op_status(raw))


def raw_call(name: str):
    """The ctypes function for an exported symbol (for tests of the ABI)."""
    return getattr(_lib, name)
