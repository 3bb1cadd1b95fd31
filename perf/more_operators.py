"""The rest of a block: attention to an encoder's states, and the norms around each part. Sizes they are measured at.

Four paths of a block of a video transformer that is conditioned on an encoder's states (a text of some tokens, the
patches of images, a long memory) and on modulation vectors (one set for each clip, frame or token):

  cross       softmax(c q k^T) v of queries [B, H, N, D] over the encoder's M keys, of which each batch element has some
  cross_bwd   its gradients
  norm        hidden = residual_scale * residual + gate * u, u = x or its norm with a gain (the end of one part), and
              out = (norm(hidden) * weight + bias) * (1 + scale) + shift (the start of the next one)
  norm_bwd    its gradients

Sizes come from the library's own workloads (tiny: 2 heads of 64, 240 tokens; small: 10 frames of 208 tokens; sr: 24 heads
of 128, 22880 tokens; sr_long: 54080 tokens; dense: 2 x 21952 tokens in frames of 1568, 40 heads of 128) and from odd ones
between them; encoders' lengths are those of short and long texts, image patches and a clip's own tokens.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_EPS = 1e-6


# ----------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of a stream that reads a long text
        dict(name="cross one token", op="cross", dtype="bf16", batch=1, heads=8, kv_heads=8, tokens=1, keys=512, dim=128, lengths="full"),
        # the tiny workload and a short prompt, padded to 77 tokens
        dict(name="cross tiny fp16", op="cross", dtype="fp16", batch=1, heads=2, kv_heads=2, tokens=240, keys=77, dim=64, lengths="ragged"),
        # a few learned queries that read a whole clip (the sr_long token count), with shared key heads
        dict(name="cross few over long", op="cross", dtype="bf16", batch=1, heads=24, kv_heads=6, tokens=77, keys=54080, dim=128,
             lengths="full"),
        # the sr workload and a text of 226 tokens
        dict(name="cross sr", op="cross", dtype="bf16", batch=1, heads=24, kv_heads=24, tokens=22880, keys=226, dim=128, lengths="full"),
        # the dense workload, two clips with texts of their own lengths in 512 padded tokens
        dict(name="cross dense", op="cross", dtype="bf16", batch=2, heads=40, kv_heads=40, tokens=21952, keys=512, dim=128,
             lengths="ragged"),
        # shared key heads, a head width that is no power of two, ragged counts
        dict(name="cross back shared heads", op="cross_bwd", dtype="fp16", batch=3, heads=18, kv_heads=6, tokens=1999, keys=333, dim=96,
             lengths="ragged"),
        # the dense workload trained
        dict(name="cross back dense", op="cross_bwd", dtype="bf16", batch=2, heads=40, kv_heads=40, tokens=21952, keys=512, dim=128,
             lengths="full"),
        # one token between two parts of a block
        dict(name="norm one token", op="norm", dtype="bf16", residual="same", vectors="same", batch=1, frames=1, per_frame=1, width=5120,
             kind="layer", post="none", modulated="clip", affine=False, residual_scale=1.0),
        # no multiple of a tile or of 16 bytes; norms before and after, with gains and no modulation, beside an fp32 residual stream
        dict(name="norm ragged fp16", op="norm", dtype="fp16", residual="fp32", vectors="fp32", batch=3, frames=1, per_frame=333, width=779,
             kind="rms", post="rms", modulated="none", affine=True, residual_scale=0.5),
        # the dense workload: a clip's gate, scale and shift
        dict(name="norm dense", op="norm", dtype="bf16", residual="same", vectors="same", batch=2, frames=14, per_frame=1568, width=5120,
             kind="layer", post="none", modulated="clip", affine=False, residual_scale=1.0),
        # the small workload trained: every frame has its own modulation
        dict(name="norm back small frames", op="norm_bwd", dtype="bf16", residual="fp32", vectors="fp32", batch=1, frames=10, per_frame=208,
             width=1024, kind="rms", post="rms", modulated="frame", affine=True, residual_scale=1.0),
        # the dense workload trained
        dict(name="norm back dense", op="norm_bwd", dtype="bf16", residual="same", vectors="same", batch=2, frames=14, per_frame=1568,
             width=5120, kind="layer", post="none", modulated="clip", affine=False, residual_scale=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cross", "cross", "cross_bwd", "cross_bwd", "norm", "norm_bwd"])
    if op in ("cross", "cross_bwd"):
        dim = rng.choice([32, 64, 64, 80, 96, 128, 128, 128])
        batch, kv = _log(rng, 1, 4), _log(rng, 1, 16)
        heads = kv * rng.choice([1, 1, 1, 2, 4])
        # texts and images mostly, long memories sometimes
        keys = _log(rng, 1, 1024) if rng.random() < 0.8 else _log(rng, 1024, 54080)
        # at most a quarter of the dense workload's pairs, and its tokens
        most = max(1, min(43904 // batch, 450_000_000 // (batch * heads * keys)))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), batch=batch, heads=heads, kv_heads=kv, tokens=_log(rng, 1, most),
                    keys=keys, dim=dim, lengths=rng.choice(["full", "ragged", "ragged", "one empty"]))
    # widths: multiples of 64 as models have them, and odd ones
    width = 64 * _log(rng, 1, 80) if rng.random() < 0.6 else _log(rng, 1, 5120)
    batch, frames = _log(rng, 1, 3), _log(rng, 1, 16)
    modulated = rng.choice(["clip", "clip", "frame", "token", "none"])
    most = max(1, min(43904, 60_000_000 // width) // (batch * frames))
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    return dict(op=op, dtype=dtype, residual=rng.choice(["same", "same", "fp32", "none"]), vectors=rng.choice(["same", "fp32"]),
                batch=batch, frames=frames, per_frame=_log(rng, 1, most), width=width, kind=rng.choice(["layer", "rms"]),
                post=rng.choice(["none", "none", "rms", "layer"]), modulated=modulated, affine=rng.random() < 0.4,
                residual_scale=rng.choice([1.0, 1.0, 0.70703125]))


# ---------------------------------------------------------------------------------------------------------- inputs

def _grouped(case):
    return case["heads"] // case["kv_heads"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = {"case": dict(case)}
    if case["op"] in ("cross", "cross_bwd"):
        b, h, kv, n, m, d = (case[i] for i in ("batch", "heads", "kv_heads", "tokens", "keys", "dim"))
        s["q"] = normal(b, n, h, d, std=1.5).transpose(1, 2)  # heads of one projection, k and v of another
        rows = normal(b, m, 2 * kv, d).transpose(1, 2)
        s["k"], s["v"] = rows[:, :kv], rows[:, kv:]
        s["len"] = None
        if case["lengths"] != "full":
            s["len"] = torch.randint(1, m + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
            if case["lengths"] == "one empty":
                s["len"][-1] = 0
        if case["op"] == "cross_bwd":
            # what the forward pass left, and the gradient that comes back, as the output projection packs it
            s["out"], s["lse"] = _attend(s)
            s["dout"] = normal(b, n, h, d, std=0.1).transpose(1, 2)
        return s
    rows, c = case["batch"] * case["frames"] * case["per_frame"], case["width"]
    lead = (case["batch"], case["frames"] * case["per_frame"])
    rt = torch.float32 if case["residual"] == "fp32" else dt
    vt = torch.float32 if case["vectors"] == "fp32" else dt
    s["x"] = normal(*lead, c)
    s["residual"] = None if case["residual"] == "none" else normal(*lead, c, std=2.0, mean=0.3, dtype=rt)
    s["gate"] = s["scale"] = s["shift"] = s["weight"] = s["bias"] = s["post_weight"] = None
    if case["modulated"] != "none":
        shape = {"clip": lead[:1], "frame": (case["batch"], case["frames"]), "token": lead}[case["modulated"]]
        # gate, scale and shift lie side by side, as one projection of the conditioning makes them
        s["gate"], s["scale"], s["shift"] = normal(*shape, 3 * c, std=0.5, dtype=vt).split(c, -1)
    if case["affine"]:
        s["weight"] = normal(c, std=0.2, mean=1.0, dtype=vt)
        if case["kind"] == "layer":
            s["bias"] = normal(c, std=0.2, dtype=vt)
    if case["post"] != "none":
        s["post_weight"] = normal(c, std=0.2, mean=1.0, dtype=vt)
    if case["op"] == "norm_bwd":
        s["hidden"] = _hidden(s).to(rt) if _joins(case) else s["x"]
        s["dout"], s["dhidden"] = normal(*lead, c, std=0.1), normal(*lead, c, std=0.1, dtype=rt if _joins(case) else dt)
    return s


def _joins(case):
    """Whether anything happens in front of the second norm."""
    return case["residual"] != "none" or case["modulated"] != "none" or case["post"] != "none"


# --------------------------------------------------------------------------------------------------------- one pass

def _heads_of(t, groups):
    """fp32 keys or values, one head for each query head."""
    return t.float().repeat_interleave(groups, 1) if groups > 1 else t.float()


def _logits(s, k):
    x = torch.matmul(s["q"].float(), k.transpose(2, 3)) * s["q"].shape[-1] ** -0.5
    if s["len"] is not None:
        x = x.masked_fill(torch.arange(k.shape[2], device=x.device) >= s["len"][:, None, None, None], -math.inf)
    return x


def _attend(s):
    """(out, lse): rows that see no key are zero and -inf."""
    r = _grouped(s["case"])
    x = _logits(s, _heads_of(s["k"], r))
    top = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    x = torch.exp(x.sub_(top))
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, _heads_of(s["v"], r)) / total.clamp_min(1.0)  # the largest term is 1
    return o.to(s["q"].dtype), (top + torch.log(total)).squeeze(-1)


def _attend_back(s):
    c, r = s["case"], _grouped(s["case"])
    k, v, do = _heads_of(s["k"], r), _heads_of(s["v"], r), s["dout"].float()
    p = torch.exp(_logits(s, k) - s["lse"].clamp_min(torch.finfo(torch.float32).min)[..., None])
    dv = torch.matmul(p.transpose(2, 3), do)
    d = (do * s["out"].float()).sum(-1, keepdim=True)
    ds = p.mul_(torch.matmul(do, v.transpose(2, 3)).sub_(d)).mul_(c["dim"] ** -0.5)
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(2, 3), s["q"].float())
    if r > 1:
        dk, dv = (t.unflatten(1, (-1, r)).sum(2) for t in (dk, dv))
    return {"dq": dq.to(s["q"].dtype), "dk": dk.to(s["q"].dtype), "dv": dv.to(s["q"].dtype)}


def _spread(t, rows):
    """fp32 vectors of groups of rows, for [..., C] of `rows` rows."""
    t = t.float()
    n = rows // t.shape[:-1].numel()
    return t.flatten(0, -2) if n == 1 else t.flatten(0, -2).repeat_interleave(n, 0)


def _normed(x, kind):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    return x * r, r


def _hidden(s):
    c, x = s["case"], s["x"].float()
    if c["post"] != "none":
        x = _normed(x, c["post"])[0] * s["post_weight"].float()
    if s["gate"] is not None:
        x = x * _spread(s["gate"], x.shape[:-1].numel()).view(x.shape)
    return x if s["residual"] is None else c["residual_scale"] * s["residual"].float() + x


def _norm(s):
    c, h = s["case"], _hidden(s)
    out = _normed(h, c["kind"])[0]
    if s["weight"] is not None:
        out = out * s["weight"].float()
    if s["bias"] is not None:
        out = out + s["bias"].float()
    if s["scale"] is not None:
        rows = h.shape[:-1].numel()
        out = out * (1 + _spread(s["scale"], rows).view(h.shape)) + _spread(s["shift"], rows).view(h.shape)
    r = {"out": out.to(s["x"].dtype)}
    if _joins(c):
        r["hidden"] = h.to(s["x"].dtype if s["residual"] is None else s["residual"].dtype)
    return r


def _back(g, n, r, kind):
    """Gradient of a norm by its input."""
    t = g - n * (g * n).mean(-1, keepdim=True)
    if kind == "layer":
        t = t - g.mean(-1, keepdim=True)
    return t * r


def _norm_back(s):
    c, width = s["case"], s["case"]["width"]
    h, dy, x = (s[i].float().flatten(0, -2) for i in ("hidden", "dout", "x"))
    rows, out = h.shape[0], {}
    n, r = _normed(h, c["kind"])
    w = None if s["weight"] is None else s["weight"].float()

    def group(t, like):  # sums over the rows of a group
        return t.view(like.shape[:-1].numel(), -1, width).sum(1).view(like.shape)

    g = dy
    if s["scale"] is not None:
        a = n if w is None else n * w
        out["dscale"] = group(dy * (a if s["bias"] is None else a + s["bias"].float()), s["scale"])
        out["dshift"] = group(dy, s["shift"])
        g = dy * (1 + _spread(s["scale"], rows))
    if w is not None:
        out["dweight"] = (g * n).sum(0)
        if s["bias"] is not None:
            out["dbias"] = g.sum(0)
        g = g * w
    dh = s["dhidden"].float().flatten(0, -2) + _back(g, n, r, c["kind"])
    if s["residual"] is not None:
        out["dresidual"] = (c["residual_scale"] * dh).to(s["residual"].dtype).view(s["residual"].shape)
    du, u = dh, x
    if c["post"] != "none":
        u, r = _normed(x, c["post"])
    if s["gate"] is not None:
        out["dgate"] = group(dh * (u if c["post"] == "none" else u * s["post_weight"].float()), s["gate"])
        du = dh * _spread(s["gate"], rows)
    if c["post"] != "none":
        out["dpost_weight"] = (du * u).sum(0)
        du = _back(du * s["post_weight"].float(), u, r, c["post"])
    out["dx"] = du.to(s["x"].dtype).view(s["x"].shape)
    return out


def _plain(s):
    op = s["case"]["op"]
    if op == "cross":
        return dict(zip(("out", "lse"), _attend(s)))
    return {"cross_bwd": _attend_back, "norm": _norm, "norm_bwd": _norm_back}[op](s)


def _own(s):
    import frame_aligned_window_gb300 as fw
    c = s["case"]
    if c["op"] == "cross":
        lse = torch.empty(s["q"].shape[:3], dtype=torch.float32, device="cuda")
        return {"out": fw.wsattn_cross(s["q"], s["k"], s["v"], k_lengths=s["len"], lse=lse), "lse": lse}
    if c["op"] == "cross_bwd":
        dq, dk, dv = fw.wsattn_cross_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], k_lengths=s["len"])
        return {"dq": dq, "dk": dk, "dv": dv}
    post = None if c["post"] == "none" else c["post"]
    same = dict(norm=c["kind"], post_norm=post, eps=_EPS, residual_scale=c["residual_scale"],
                **{i: s[i] for i in ("gate", "scale", "weight", "bias", "post_weight")})
    if c["op"] == "norm":
        out, hidden = fw.wsattn_block_norm(s["x"], s["residual"], shift=s["shift"], **same)
        return {"out": out, **({"hidden": hidden} if _joins(c) else {})}
    d = fw.wsattn_block_norm_backward(s["dout"], s["hidden"], s["x"], dhidden=s["dhidden"],
                                      need_dresidual=s["residual"] is not None, **same)
    return {i: t for i, t in d._asdict().items() if t is not None}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------------------ floors

def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] in ("cross", "cross_bwd"):
        b, h, kv, n, m, d = (case[i] for i in ("batch", "heads", "kv_heads", "tokens", "keys", "dim"))
        # the keys that count: all of them, or on average half
        m = m if case["lengths"] == "full" else (m + 1) / 2
        q, k, rows = 2 * b * n * h * d, 2 * b * m * kv * d, 4 * b * h * n
        if case["op"] == "cross":
            return {"bytes": 2 * q + 2 * k + rows, "flops": 4 * b * h * n * m * d}
        return {"bytes": 4 * q + 4 * k + rows, "flops": 10 * b * h * n * m * d}
    rows, c = case["batch"] * case["frames"] * case["per_frame"], case["width"]
    wide, vec = 4 if case["residual"] == "fp32" else size, 4 if case["vectors"] == "fp32" else size
    groups = {"none": 0, "clip": case["batch"], "frame": case["batch"] * case["frames"], "token": rows}[case["modulated"]]
    singles = case["affine"] * (2 if case["kind"] == "layer" else 1) + (case["post"] != "none")
    res = case["residual"] != "none"
    if case["op"] == "norm":
        b = rows * c * (2 * size + wide * (res + _joins(case))) + vec * c * (3 * groups + singles)
        return {"bytes": b, "flops": 12 * rows * c}
    # x counts where the gate's or the first norm's gradient needs it
    b = rows * c * (size * (2 + (groups > 0 or case["post"] != "none")) + wide * (2 + res))
    return {"bytes": b + c * (vec * (2 * groups + singles) + 4 * (3 * groups + singles)), "flops": 30 * rows * c}


# ---------------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f = lambda t: t.to(torch.float64)  # noqa: E731
    if case["op"] in ("cross", "cross_bwd"):
        b, h, kv, n, m, d = (case[i] for i in ("batch", "heads", "kv_heads", "tokens", "keys", "dim"))
        back = case["op"] == "cross_bwd"
        lens = [m] * b if s["len"] is None else s["len"].tolist()
        r = dict(dq=f(torch.zeros_like(s["q"])), dk=f(torch.zeros_like(s["k"])), dv=f(torch.zeros_like(s["v"]))) if back else dict(
            out=f(torch.zeros_like(s["q"])), lse=torch.full((b, h, n), -math.inf, dtype=torch.float64, device="cuda"))
        for i in range(b):
            for j in range(h):
                if lens[i] == 0:
                    continue
                e = j // (h // kv)
                q, k, v = f(s["q"][i, j]), f(s["k"][i, e, :lens[i]]), f(s["v"][i, e, :lens[i]])
                logits = torch.einsum("nd,md->nm", q, k) / math.sqrt(d)
                if not back:
                    r["lse"][i, j] = torch.logsumexp(logits, -1)
                    r["out"][i, j] = torch.einsum("nm,md->nd", torch.softmax(logits, -1), v)
                    continue
                p = torch.softmax(logits, -1)
                do = f(s["dout"][i, j])
                r["dv"][i, e, :lens[i]] += torch.einsum("nm,nd->md", p, do)
                dp = torch.einsum("nd,md->nm", do, v) - torch.einsum("nd,nd->n", do, f(s["out"][i, j]))[:, None]
                p *= dp / math.sqrt(d)
                r["dq"][i, j] = torch.einsum("nm,md->nd", p, k)
                r["dk"][i, e, :lens[i]] += torch.einsum("nm,nd->md", p, q)
        return r

    # the norms' gradients by differentiating the definition, some rows of one group at a time
    c, width = case, case["width"]
    x = f(s["x"]).reshape(-1, width)
    rows = x.shape[0]
    groups = 1 if s["gate"] is None else s["gate"].shape[:-1].numel()
    per = rows // groups
    vec = {i: None if s[i] is None else f(s[i]).reshape(-1, width).clone() for i in ("gate", "scale", "shift", "weight", "bias", "post_weight")}
    res = None if s["residual"] is None else f(s["residual"]).reshape(-1, width)

    def std(t, kind):
        if kind == "rms":
            return t / torch.sqrt(torch.mean(t ** 2, -1, keepdim=True) + _EPS)
        return (t - torch.mean(t, -1, keepdim=True)) / torch.sqrt(torch.var(t, -1, keepdim=True, correction=0) + _EPS)

    def first(t, v):
        if c["post"] != "none":
            t = std(t, c["post"]) * v["post_weight"]
        return t if v["gate"] is None else t * v["gate"]

    def second(t, v):
        t = std(t, c["kind"])
        if v["weight"] is not None:
            t = t * v["weight"]
        if v["bias"] is not None:
            t = t + v["bias"]
        return t if v["scale"] is None else t * (1 + v["scale"]) + v["shift"]

    step, pieces = max(1, 40_000_000 // width), []
    at = lambda v, i: v if v is None or v.shape[0] == 1 else v[i:i + 1]  # noqa: E731
    if groups * -(-per // step) > 300:  # a group of a row or two: all of them side by side
        at = lambda v, i: v  # noqa: E731
        spans = [(None, 0, rows)]
        vec = {i: v if v is None or v.shape[0] != groups else v.repeat_interleave(per, 0) for i, v in vec.items()}
    else:
        spans = [(i, i * per + j, i * per + min(j + step, per)) for i in range(groups) for j in range(0, per, step)]
    if case["op"] == "norm":
        for i, a, e in spans:
            v = {name: at(t, i) for name, t in vec.items()}
            h = first(x[a:e], v)
            h = h if res is None else case["residual_scale"] * res[a:e] + h
            pieces.append((second(h, v), h))
        r = {"out": torch.cat([p[0] for p in pieces]).view(s["x"].shape)}
        if _joins(case):
            r["hidden"] = torch.cat([p[1] for p in pieces]).view(s["x"].shape)
        return r
    h, dy, dh = (f(s[i]).reshape(-1, width) for i in ("hidden", "dout", "dhidden"))
    total = {name: None if t is None else torch.zeros_like(t) for name, t in vec.items()}
    dres, dx = [], []
    for i, a, e in spans:
        v = {name: None if t is None else at(t, i).clone().requires_grad_() for name, t in vec.items()}
        hh, xx = h[a:e].clone().requires_grad_(), x[a:e].clone().requires_grad_()
        y = second(hh, v)
        used = [name for name in ("scale", "shift", "weight", "bias") if v[name] is not None]
        got = torch.autograd.grad(y, [hh] + [v[name] for name in used], dy[a:e])
        gh = got[0] + dh[a:e]
        for name, t in zip(used, got[1:]):
            at(total[name], i).add_(t)
        u = first(xx, v)
        used = [name for name in ("gate", "post_weight") if v[name] is not None]
        got = torch.autograd.grad(u, [xx] + [v[name] for name in used], gh) if u is not xx else [gh]
        for name, t in zip(used, got[1:]):
            at(total[name], i).add_(t)
        dres.append(gh)
        dx.append(got[0])
    r = {}
    for name, t in total.items():
        if t is not None:
            r["d" + name] = t.view(s[name].shape[:-1].numel(), -1, width).sum(1).view(s[name].shape)
    if res is not None:
        r["dresidual"] = case["residual_scale"] * torch.cat(dres).view(s["x"].shape)
    r["dx"] = torch.cat(dx).view(s["x"].shape)
    return r
