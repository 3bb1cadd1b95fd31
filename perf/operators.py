"""The operators around the attention and the sizes they are measured at.

Five paths of a block of a video transformer that attends with this library:

  rotary       x [B, H, N, D] turned by positions on several axes (time, height, width), or back
  qknorm       per-head RMS norm of q and k with a gain, the same rotation, v copied, packed for the attention
  qknorm_bwd   its gradients
  linear       residual + act(x W^T + bias)
  linear_bwd   its gradients

Sizes come from the library's own workloads (tiny: 2 heads of 64, 240 tokens; small: 8 heads of 128, 2080 tokens;
sr_long: 54080 tokens; dense: 2 x 21952 tokens, 40 heads of 128) and from odd ones between them.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BASE = 10000.0
_EPS = 1e-6


# ----------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of a stream: every head of one position, far from the start
        dict(name="rotary one token", op="rotary", dtype="bf16", batch=1, heads=8, tokens=1, dim=128, axes=1, interleaved=False,
             inverse=False, rows=1, cols=1, start=70001),
        # fp32 activations of a long clip (the sr_long token count), turned back as a backward pass does
        dict(name="rotary long fp32 back", op="rotary", dtype="fp32", batch=1, heads=16, tokens=54080, dim=128, axes=3, interleaved=True,
             inverse=True, rows=52, cols=40, start=0),
        # the tiny workload: a packed projection split into normed and turned q and k, and v
        dict(name="qknorm tiny fp16", op="qknorm", dtype="fp16", batch=1, heads=2, kv_heads=2, tokens=240, dim=64, axes=3, interleaved=True,
             gain="fp32", rows=6, cols=8, start=0),
        # the dense workload: 28 x 56 latent grid, 14 frames, two clips
        dict(name="qknorm dense bf16", op="qknorm", dtype="bf16", batch=2, heads=40, kv_heads=40, tokens=21952, dim=128, axes=3,
             interleaved=True, gain="same", rows=28, cols=56, start=0),
        # shared key heads, a head width that is no power of two, a ragged token count
        dict(name="qknorm back shared heads", op="qknorm_bwd", dtype="fp16", batch=3, heads=18, kv_heads=6, tokens=1999, dim=96, axes=2,
             interleaved=False, gain="same", rows=25, cols=20, start=300),
        # the dense workload trained
        dict(name="qknorm back dense", op="qknorm_bwd", dtype="bf16", batch=2, heads=40, kv_heads=40, tokens=21952, dim=128, axes=3,
             interleaved=True, gain="fp32", rows=28, cols=56, start=0),
        # the output projection of one token
        dict(name="linear one token", op="linear", dtype="bf16", rows=1, k=5120, n=5120, bias=True, act="none", residual=True, keep=False),
        # a ragged one: nothing is a multiple of a tile or of 16 bytes
        dict(name="linear ragged fp16", op="linear", dtype="fp16", rows=333, k=1001, n=779, bias=True, act="silu", residual=True, keep=True),
        # the small workload's first feed-forward product in training: keeps what the backward pass needs
        dict(name="linear small gelu", op="linear", dtype="bf16", rows=2080, k=1024, n=4096, bias=True, act="gelu_tanh", residual=False, keep=True),
        # the dense workload's output projection: bias and the residual stream
        dict(name="linear dense residual", op="linear", dtype="bf16", rows=43904, k=5120, n=5120, bias=True, act="none", residual=True, keep=False),
        # the small workload's first feed-forward product, backwards
        dict(name="linear back small gelu", op="linear_bwd", dtype="bf16", rows=2080, k=1024, n=4096, act="gelu_tanh"),
        # one clip of the dense workload, backwards
        dict(name="linear back dense", op="linear_bwd", dtype="bf16", rows=21952, k=5120, n=5120, act="gelu"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "qknorm", "qknorm_bwd", "linear", "linear_bwd"])
    if op in ("linear", "linear_bwd"):
        # any width: multiples of 64 as models have them, and odd ones
        k, n = (64 * _log(rng, 1, 80) if rng.random() < 0.6 else _log(rng, 33, 5120) for _ in range(2))
        most = 43904 if op == "linear" else 21952
        case = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), rows=_log(rng, 1, most), k=k, n=n,
                    act=rng.choice(["none", "gelu", "gelu_tanh", "silu"]))
        if op == "linear":
            case.update(bias=rng.random() < 0.7, residual=rng.random() < 0.5, keep=rng.random() < 0.4)
        return case
    dim = rng.choice([32, 64, 80, 96, 128, 128, 256])
    batch, kv = _log(rng, 1, 4), _log(rng, 1, 12)
    heads = kv * rng.choice([1, 1, 2, 4])
    # at most a third of what the dense workload moves
    most = max(1, min(54080, 150_000_000 // (batch * heads * dim)))
    rows, cols = _log(rng, 1, 40), _log(rng, 1, 64)
    case = dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), batch=batch, heads=heads, tokens=_log(rng, 1, most), dim=dim,
                axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5, rows=rows, cols=cols, start=rng.choice([0, 17, 4096, 200000]))
    if op == "rotary":
        case.update(inverse=rng.random() < 0.5)
    else:
        case.update(kv_heads=kv, gain=rng.choice(["same", "fp32", "none"]))
    return case


# ---------------------------------------------------------------------------------------------------------- inputs

def _sections(case):
    """Pairs of a head that each axis turns: rows and columns a third each, time the rest (all, or halves, with fewer axes)."""
    half = case["dim"] // 2
    if case["axes"] == 3:
        return (half - 2 * (half // 3), half // 3, half // 3)
    return (half - half // 2, half // 2) if case["axes"] == 2 else (half,)


def _positions(case):
    """fp32 [N, axes] of a grid walked frame by frame, row by row."""
    n = torch.arange(case["tokens"], dtype=torch.int64)
    if case["axes"] == 1:
        p = n[:, None] + case["start"]
    else:
        area, cols = case["rows"] * case["cols"], case["cols"]
        frame, row, col = n // area + case["start"], n % area // cols, n % cols
        p = torch.stack([frame, row, col] if case["axes"] == 3 else [frame * case["rows"] + row, col], 1)
    return p.to(torch.float32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": dict(case)}
    if case["op"] in ("linear", "linear_bwd"):
        m, k, n = case["rows"], case["k"], case["n"]
        s["x"] = normal(m, k)
        s["w"] = normal(n, k, std=k ** -0.5)
        if case["op"] == "linear":
            s["bias"] = normal(n, std=0.5) if case["bias"] else None
            s["residual"] = normal(m, n) if case["residual"] else None
        else:
            s["dy"] = normal(m, n, std=0.1)
            s["z"] = None if case["act"] == "none" else normal(m, n)  # what the forward pass kept
        return s
    b, h, n, d = case["batch"], case["heads"], case["tokens"], case["dim"]
    s["positions"] = _positions(case)
    if case["op"] == "rotary":
        s["x"] = normal(b, n, h, d).transpose(1, 2)  # heads of a projection, not yet packed
    else:
        kv = case["kv_heads"]
        # one projection's output: q, k and v features of a token next to each other
        rows = normal(b, n, h + 2 * kv, d, std=2.0).transpose(1, 2)
        s["q"], s["k"], s["v"] = rows[:, :h], rows[:, h:h + kv], rows[:, h + kv:]
        gt = torch.float32 if case["gain"] == "fp32" else dt
        s["wq"], s["wk"] = ((1 + normal(d, std=0.2, dtype=torch.float32)).to(gt) if case["gain"] != "none" else None for _ in range(2))
        if case["op"] == "qknorm_bwd":
            s["gq"], s["gk"], s["gv"] = normal(b, h, n, d), normal(b, kv, n, d), normal(b, kv, n, d)
    if own:
        import frame_aligned_window_gb300 as fw
        s["rot"] = fw.wsattn_rotary_plan(d, _sections(case), base=_BASE, interleaved=case["interleaved"])
    return s


# --------------------------------------------------------------------------------------------------------- one pass

def _turns(case, positions):
    """cos, sin [N, D / 2] in fp32, from angles in 64 bits."""
    sec = torch.tensor(_sections(case), device="cuda")
    axis = torch.repeat_interleave(torch.arange(len(sec), device="cuda"), sec)
    j = torch.arange(len(axis), device="cuda") - torch.repeat_interleave(torch.cumsum(sec, 0) - sec, sec)
    angle = positions.double()[:, axis] * torch.exp(-math.log(_BASE) * (j.double() / sec[axis].double()))
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turn(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def _slope(z, act):
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _norm_back(g, x, w, cos, sin, interleaved):
    """Gradients of turn(w x / rms(x)) by x (rounded to its type) and by w (fp32)."""
    g, xf = _turn(g.float(), cos, -sin, interleaved), x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + _EPS)
    xh = xf * r
    gw = g if w is None else g * w.float()
    dx = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), None if w is None else (g * xh).sum((0, 1, 2))


def _plain(s):
    c = s["case"]
    if c["op"] == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(s["x"].dtype), **({"z": z.to(s["x"].dtype)} if c["keep"] else {})}
    if c["op"] == "linear_bwd":
        dz = s["dy"].float()
        if s["z"] is not None:
            dz = dz * _slope(s["z"].float(), c["act"])
        dt = s["x"].dtype
        return {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt), "db": dz.sum(0)}
    cos, sin = _turns(c, s["positions"])
    if c["op"] == "rotary":
        y = _turn(s["x"].float(), cos, -sin if c["inverse"] else sin, c["interleaved"])
        return {"y": y.to(s["x"].dtype)}
    if c["op"] == "qknorm":
        def normed(x, w):
            xf = x.float()
            xf = xf * torch.rsqrt((xf * xf).mean(-1, keepdim=True) + _EPS)
            return _turn(xf if w is None else xf * w.float(), cos, sin, c["interleaved"]).to(x.dtype)
        return {"q": normed(s["q"], s["wq"]), "k": normed(s["k"], s["wk"]), "v": s["v"].contiguous()}
    (dq, dwq), (dk, dwk) = (_norm_back(s["g" + i], s[i], s["w" + i], cos, sin, c["interleaved"]) for i in "qk")
    # the projection's gradient, packed as its output was
    out = {"d": torch.cat((dq, dk, s["gv"]), 1).transpose(1, 2).contiguous()}
    return out if dwq is None else {**out, "dwq": dwq, "dwk": dwk}


def _own(s):
    import frame_aligned_window_gb300 as fw
    c = s["case"]
    if c["op"] == "linear":
        z = torch.empty((c["rows"], c["n"]), dtype=s["x"].dtype, device="cuda") if c["keep"] else None
        y = fw.wsattn_linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"], activation=c["act"], preact=z)
        return {"y": y, **({"z": z} if c["keep"] else {})}
    if c["op"] == "linear_bwd":
        dx, dw, db = fw.wsattn_linear_backward(s["dy"], s["x"], s["w"], preact=s["z"], activation=c["act"])
        return {"dx": dx, "dw": dw, "db": db}
    if c["op"] == "rotary":
        return {"y": fw.wsattn_rotary(s["rot"], s["x"], s["positions"], inverse=c["inverse"])}
    if c["op"] == "qknorm":
        q, k, v = fw.wsattn_qknorm(s["rot"], s["q"], s["k"], s["positions"], q_weight=s["wq"], k_weight=s["wk"], eps=_EPS, v=s["v"])
        return {"q": q, "k": k, "v": v}
    h, kv = c["heads"], c["kv_heads"]
    d = torch.empty((c["batch"], c["tokens"], h + 2 * kv, c["dim"]), dtype=s["q"].dtype, device="cuda")
    t = d.transpose(1, 2)
    _, _, _, dwq, dwk = fw.wsattn_qknorm_backward(s["rot"], s["gq"], s["gk"], s["q"], s["k"], s["positions"], q_weight=s["wq"],
                                                  k_weight=s["wk"], eps=_EPS, dv_out=s["gv"], dq=t[:, :h], dk=t[:, h:h + kv], dv=t[:, h + kv:])
    return {"d": d} if dwq is None else {"d": d, "dwq": dwq, "dwk": dwk}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------------------ floors

def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] in ("linear", "linear_bwd"):
        m, k, n = case["rows"], case["k"], case["n"]
        if case["op"] == "linear":
            b = size * (m * k + n * k + m * n * (1 + case["residual"] + case["keep"]) + n * case["bias"])
            return {"bytes": b, "flops": 2 * m * n * k}
        return {"bytes": size * (2 * m * k + 2 * n * k + m * n * (1 if case["act"] == "none" else 2)) + 4 * n, "flops": 4 * m * n * k}
    b, h, n, d = case["batch"], case["heads"], case["tokens"], case["dim"]
    pos = 4 * n * case["axes"]
    if case["op"] == "rotary":
        return {"bytes": 2 * size * b * h * n * d + pos, "flops": 3 * b * h * n * d}
    qk, v = b * n * d * (h + case["kv_heads"]), b * n * d * case["kv_heads"]
    gain = 0 if case["gain"] == "none" else 2 * d * (4 if case["gain"] == "fp32" else size)
    if case["op"] == "qknorm":
        return {"bytes": 2 * size * (qk + v) + pos + gain, "flops": 7 * qk}
    return {"bytes": size * (3 * qk + 2 * v) + pos + gain + (8 * d if gain else 0), "flops": 16 * qk}


# ---------------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f = lambda t: t.to(torch.float64)  # noqa: E731
    if case["op"] in ("linear", "linear_bwd"):
        act = None if case["act"] == "none" else case["act"]
        cdf = {"gelu": lambda z: 0.5 * torch.special.erfc(-z / math.sqrt(2.0)),
               "gelu_tanh": lambda z: torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)),
               "silu": torch.sigmoid}
        if case["op"] == "linear":
            z = torch.einsum("mk,nk->mn", f(s["x"]), f(s["w"]))
            if case["bias"]:
                z += f(s["bias"])
            y = z * cdf[act](z) if act else z.clone()
            if case["residual"]:
                y += f(s["residual"])
            return {"y": y, "z": z} if case["keep"] else {"y": y}
        dz = f(s["dy"])
        if act:
            # the slope of z * c(z) is c + z c'
            z = f(s["z"])
            c = cdf[act](z)
            if act == "gelu":
                dc = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
            elif act == "gelu_tanh":
                dc = c * (1 - c) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z ** 2)
            else:
                dc = c * (1 - c)
            dz = dz * (c + z * dc)
            del z, c, dc
        return {"dx": torch.einsum("mn,nk->mk", dz, f(s["w"])), "dw": torch.einsum("mn,mk->nk", dz, f(s["x"])), "db": dz.sum(0)}

    # the rotation as a product of complex numbers
    freqs = [[float(_BASE) ** (-j / n) for j in range(n)] for n in _sections(case)]
    pos = f(s["positions"])
    angle = torch.cat([pos[:, i:i + 1] * torch.tensor([w], dtype=torch.float64, device="cuda") for i, w in enumerate(freqs)], 1)
    unit = torch.polar(torch.ones_like(angle), angle)

    def turned(x, by):
        if case["interleaved"]:
            return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * by).flatten(-2)
        half = x.shape[-1] // 2
        y = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * by
        return torch.cat((y.real, y.imag), -1)

    if case["op"] == "rotary":
        return {"y": turned(f(s["x"]), unit.conj() if case["inverse"] else unit)}
    one = torch.ones(case["dim"], dtype=torch.float64, device="cuda")
    gains = {i: one if s["w" + i] is None else f(s["w" + i]) for i in "qk"}
    if case["op"] == "qknorm":
        out = {}
        for i in "qk":
            x = f(s[i])
            out[i] = turned(x / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + _EPS) * gains[i], unit)
        return {**out, "v": f(s["v"])}
    d, dw = [], {}
    for i in "qk":
        x, g = f(s[i]), turned(f(s["g" + i]), unit.conj())
        ms = torch.mean(x ** 2, -1, keepdim=True) + _EPS
        if s["w" + i] is not None:
            dw["dw" + i] = torch.einsum("bhnd,bhnd->d", g, x / torch.sqrt(ms))
        g *= gains[i]
        d.append(g / torch.sqrt(ms) - x * torch.sum(g * x, -1, keepdim=True) / (case["dim"] * ms ** 1.5))
    return {"d": torch.cat((*d, f(s["gv"])), 1).transpose(1, 2), **dw}
