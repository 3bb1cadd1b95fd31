"""Plain 64-bit definitions of a block's norms and of cross attention, and how
far the kernels' fp32 arithmetic and their roundings may take them from it."""
import torch

from _ops_ref import half_step, tiny

# A row of up to 12288 columns is summed as 32 in sequence and 10 in pairs, each
# rounded by 2^-24, and a value goes through at most 20 roundings more: below
# 64 * 2^-24 of the sum of magnitudes.
E = 2.0 ** -18


def std(t, kind, eps):
    """(std(t), 1 / deviation)."""
    if kind == "layer":
        t = t - t.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((t * t).mean(-1, keepdim=True) + eps)
    return t * r, r


def spread(t, m):
    """[G, n] vectors (or None) for m rows."""
    return None if t is None else t.double().cpu().reshape(-1, t.shape[-1]).repeat_interleave(m // t.shape[:-1].numel(), 0)


def flat(t):
    return None if t is None else t.double().cpu().reshape(-1, t.shape[-1])


def mul(a, b):
    return a if b is None else a * b


def stats_error(h, s, r, kind, dh):
    """Error of std(h) where h is off by dh: mean, deviation and 1 / deviation."""
    size = h.abs().mean(-1, keepdim=True) if kind == "layer" else 0.0
    rms = torch.sqrt((dh * dh).mean(-1, keepdim=True))
    return 2 * (r * (dh + dh.mean(-1, keepdim=True) + E * size) + s.abs() * (E + r * rms))


def norm_forward(x, residual, gate, scale, shift, weight, bias, norm, eps, post_norm, post_weight, res_scale):
    """(out, its tolerance, hidden, its tolerance), before rounding."""
    xf, m = flat(x), x.shape[:-1].numel()
    u, du = xf, torch.zeros_like(xf)
    if post_norm:
        s, r = std(xf, post_norm, eps)
        w = flat(post_weight)
        u, du = mul(s, w), mul(stats_error(xf, s, r, post_norm, du), None if w is None else w.abs())
    g = spread(gate, m)
    h, dh = mul(u, g), mul(du + E * u.abs(), None if g is None else g.abs())
    if residual is not None:
        h = h + res_scale * flat(residual)
        dh = dh + E * abs(res_scale) * flat(residual).abs()
    s, r = std(h, norm, eps)
    ds = stats_error(h, s, r, norm, dh)
    y, dy, size = s, ds, s.abs()
    if weight is not None:
        y, dy, size = y * flat(weight), dy * flat(weight).abs(), size * flat(weight).abs()
    if bias is not None:
        y, size = y + flat(bias), size + flat(bias).abs()
    sc, sh = spread(scale, m), spread(shift, m)
    if sc is not None:
        y, dy, size = y * (1 + sc), dy * (1 + sc).abs(), size * (1 + sc.abs())
    if sh is not None:
        y, size = y + sh, size + sh.abs()
    return y, dy + E * size, h, dh


def norm_backward(dout, hidden, x, dhidden, gate, scale, shift, weight, bias, norm, eps, post_norm, post_weight, res_scale):
    """{name: (gradient, tolerance)} before rounding."""
    like = dout if dout is not None else dhidden
    m, n = like.shape[:-1].numel(), like.shape[-1]
    out, zero = {}, torch.zeros((m, n), dtype=torch.float64)
    g_, s_, w_, b_, p_ = spread(gate, m), spread(scale, m), flat(weight), flat(bias), flat(post_weight)

    def group(t, like_t, tol):
        """Sums over groups: m terms in sequence at most, each rounded."""
        k = like_t.shape[:-1].numel()
        return (t.view(k, -1, n).sum(1), (tol + (m // k + 64) * 2.0 ** -24 * t.abs()).view(k, -1, n).sum(1))

    dh, tol = zero, zero
    if dout is not None:
        dy, h = flat(dout), flat(hidden)
        s, r = std(h, norm, eps)
        ds = stats_error(h, s, r, norm, zero)
        g = mul(mul(dy, w_), None if s_ is None else 1 + s_)
        a = mul(s, w_)
        if b_ is not None:
            a = a + b_
        if s_ is not None:
            size = mul(ds + E * s.abs(), None if w_ is None else w_.abs()) + E * a.abs()
            out["dscale"] = group(dy * a, scale, dy.abs() * size)
        if s_ is not None or shift is not None:
            out["dshift"] = group(dy, shift if shift is not None else scale, zero)
        f = dy if s_ is None else dy * (1 + s_)
        if w_ is not None:
            t, e = group(f * s, torch.empty(1, n), f.abs() * (ds + E * s.abs()))
            out["dweight"] = t[0], e[0]
        if b_ is not None:
            t, e = group(f, torch.empty(1, n), E * f.abs())
            out["dbias"] = t[0], e[0]
        gs = (g * s).mean(-1, keepdim=True)
        t = g - s * gs
        if norm == "layer":
            t = t - g.mean(-1, keepdim=True)
        dh = r * t
        amp = 1 + (r * h.abs().mean(-1, keepdim=True) if norm == "layer" else 0.0)
        ga = g.abs()
        tol = 4 * E * amp * r * (ga + ga.mean(-1, keepdim=True) + s.abs() * (ga * s.abs()).mean(-1, keepdim=True)) \
            + r * (ds * gs.abs() + s.abs() * (ga * ds).mean(-1, keepdim=True)) \
            + E * amp * dh.abs()
    else:
        for name, t in (("dscale", scale), ("dshift", shift if shift is not None else scale), ("dweight", weight), ("dbias", bias)):
            if t is not None:
                k = flat(t)
                out[name] = (torch.zeros_like(k), torch.zeros_like(k)) if t.dim() > 1 else (torch.zeros(n).double(),) * 2
    if dhidden is not None:
        dh = dh + flat(dhidden)
        tol = tol + E * flat(dhidden).abs()
    out["dresidual"] = res_scale * dh, abs(res_scale) * (tol + E * dh.abs())
    xf = None if x is None else flat(x)
    xh, dxh, rx = xf, zero, None
    if post_norm:
        xh, rx = std(xf, post_norm, eps)
        dxh = stats_error(xf, xh, rx, post_norm, zero)
    if g_ is not None:
        u = mul(xh, p_)
        size = tol * u.abs() + dh.abs() * (mul(dxh, None if p_ is None else p_.abs()) + E * u.abs())
        out["dgate"] = group(dh * u, gate, size)
    du, tol = mul(dh, g_), mul(tol + E * dh.abs(), None if g_ is None else g_.abs())
    if post_norm:
        if p_ is not None:
            t, e = group(du * xh, torch.empty(1, n), tol * xh.abs() + du.abs() * (dxh + E * xh.abs()))
            out["dpost_weight"] = t[0], e[0]
        du, tol = mul(du, p_), mul(tol + E * du.abs(), None if p_ is None else p_.abs())
        m2 = (du * xh).mean(-1, keepdim=True)
        t = du - xh * m2
        if post_norm == "layer":
            t = t - du.mean(-1, keepdim=True)
        amp = 1 + (rx * xf.abs().mean(-1, keepdim=True) if post_norm == "layer" else 0.0)
        da = du.abs()
        tol = rx * (tol + tol.mean(-1, keepdim=True) + xh.abs() * (tol * xh.abs()).mean(-1, keepdim=True)) \
            + 4 * E * amp * rx * (da + da.mean(-1, keepdim=True) + xh.abs() * (da * xh.abs()).mean(-1, keepdim=True)) \
            + rx * (dxh * m2.abs() + xh.abs() * (da * dxh).mean(-1, keepdim=True))
        du = rx * t
    out["dx"] = du, tol
    return out


def rounded(tol, want, dtype):
    """A tolerance with the rounding to a type."""
    return tol + half_step(dtype) * (want.abs() + tol) + tiny(dtype) + 1e-37


# ------------------------------------------------------------ cross attention

# The exponential of the special-function unit counts what is below fp32's normal
# values as zero: a probability is off by less than 2^-126 for that.
LEAST = 2.0 ** -126

def heads_of(t, h):
    return t.double().repeat_interleave(h // t.shape[1], 1)


def lengths_of(lengths, b, m, dev):
    if lengths is None:
        return torch.full((b,), m, device=dev)
    return lengths.long().clamp(0, m)


def cleaned(t, lens):
    """fp64 keys or values with zeros behind each length."""
    keep = torch.arange(t.shape[2], device=t.device) < lens[:, None]
    return torch.where(keep[:, None, :, None], t.double(), 0.0)


def logits(q, k, lens, scale):
    """(scale q k^T with -inf behind the lengths, its error on the tensor cores)."""
    h, d = q.shape[1], q.shape[3]
    qd, kd = q.double(), heads_of(cleaned(k, lens), h)
    s = scale * qd @ kd.transpose(2, 3)
    size = scale * qd.abs() @ kd.abs().transpose(2, 3)
    dead = torch.arange(k.shape[2], device=k.device) >= lens[:, None, None, None]
    # truncations of the product's partial sums, the multiplication by scale log2(e) and the subtraction of the maximum
    # or the sum (fp32, of values up to `size` and 40 more), the exponential's own 2^-22
    err = (d / 16 + 8) * 2.0 ** -22 * size + 2.0 ** -22 * (size.amax(-1, keepdim=True) + 40) if k.shape[2] else size
    return s.masked_fill(dead, float("-inf")), torch.where(dead, 0.0, err)


def cross_forward(q, k, v, lengths, scale):
    """(out, its tolerance, lse, its tolerance)."""
    b, h, n, d = q.shape
    m, dt = k.shape[2], q.dtype
    lens = lengths_of(lengths, b, m, q.device)
    if m == 0:
        zero = torch.zeros((b, h, n, d), dtype=torch.float64, device=q.device)
        return zero, zero, torch.full((b, h, n), float("-inf"), dtype=torch.float64, device=q.device), torch.zeros((b, h, n)).to(q.device)
    s, es = logits(q, k, lens, scale)
    lse = torch.logsumexp(s, -1)
    empty = (lens == 0)[:, None, None]
    p = torch.where(empty[..., None], 0.0, torch.exp(s - lse.masked_fill(empty, 0.0)[..., None]))
    vd = heads_of(cleaned(v, lens), h)
    out = p @ vd
    # p: rounded, and off by its logit's error; below the type's smallest values relative to the largest p (1 / sum >= p)
    step = half_step(dt) + 2 * es + 2.0 ** -20
    small = torch.where(empty[..., None], 0.0, torch.exp(s.amax(-1, keepdim=True) - lse[..., None])) * max(tiny(dt), LEAST)
    tol = (p * step) @ vd.abs() + small * vd.abs().sum(2, keepdim=True)
    # the sum of the probabilities is off by as much as they are, and the product by its truncations
    rel = (p * (2 * es + 2.0 ** -20)).sum(-1, keepdim=True) + 2.0 ** -19
    tol = tol + rel * out.abs() + (m / 16 + 8) * 2.0 ** -22 * (p @ vd.abs())
    return out, tol, lse, torch.where(empty, 0.0, rel.squeeze(-1) + 2.0 ** -22 * (1 + lse.masked_fill(empty, 0.0).abs()))


def cross_backward(dout, q, k, v, out, lse, lengths, scale):
    """{name: (gradient, tolerance)} of the definition with out and lse as given."""
    b, h, n, d = q.shape
    hk, m, dt = k.shape[1], k.shape[2], q.dtype
    r = h // hk
    lens = lengths_of(lengths, b, m, q.device)
    s, es = logits(q, k, lens, scale)
    empty = (lens == 0)[:, None, None]
    p = torch.exp(s - lse.double().masked_fill(empty, 0.0)[..., None])
    do, qd = dout.double(), q.double()
    kd, vd = heads_of(cleaned(k, lens), h), heads_of(cleaned(v, lens), h)
    delta = (do * out.double()).sum(-1, keepdim=True)
    dp = do @ vd.transpose(2, 3)
    ds = p * (dp - delta)
    rel = 2 * es + 2.0 ** -20
    size = do.abs() @ vd.abs().transpose(2, 3)
    e_ds = ds.abs() * (rel + half_step(dt) + 2.0 ** -21) + tiny(dt) * (p > 0) \
        + p * ((d / 16 + 8) * 2.0 ** -22 * size + 2.0 ** -20 * (do * out.double()).abs().sum(-1, keepdim=True)) \
        + LEAST * (dp - delta).abs() * (p > 0)

    def shared(t):
        return t.view(b, hk, r, m, d).sum(2)

    w = {}
    w["dq"] = scale * ds @ kd, scale * (e_ds @ kd.abs() + (m / 16 + 8) * 2.0 ** -22 * (ds.abs() @ kd.abs()))
    many = (n * r / 16 + 8) * 2.0 ** -22
    w["dk"] = scale * shared(ds.transpose(2, 3) @ qd), \
        scale * shared(e_ds.transpose(2, 3) @ qd.abs() + many * (ds.abs().transpose(2, 3) @ qd.abs()))
    e_p = p * (rel + half_step(dt)) + (tiny(dt) + LEAST) * (p > 0)
    w["dv"] = shared(p.transpose(2, 3) @ do), shared(e_p.transpose(2, 3) @ do.abs() + many * (p.transpose(2, 3) @ do.abs()))
    return w
