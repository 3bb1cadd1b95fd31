"""Plain 64-bit definitions of the operators around the attention, and how far
a kernel's rounded result may be from them."""
import math

import torch


def half_step(t):
    """Relative rounding error of a type: half its spacing."""
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the spacing of a type's smallest (subnormal) values."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def sections_for(dim, axes):
    """Uneven sections over all but one of the pairs (the last is left alone)."""
    left, out = dim // 2 - 1, []
    for a in range(axes):
        n = left if a == axes - 1 else max(1, left // 3)
        out.append(n)
        left -= n
    return tuple(out)


def angles(positions, sections, dim, base=10000.0):
    """[..., N, D / 2] angles in 64 bits."""
    p = positions.double().cpu()
    cols = []
    for a, n in enumerate(sections):
        for j in range(n):
            cols.append(p[..., a] * base ** (-j / n))
    while len(cols) < dim // 2:
        cols.append(torch.zeros_like(p[..., 0]))
    return torch.stack(cols, -1)


def turn(x, ang, interleaved, sign=1):
    """x [B, H, N, D] in 64 bits turned by ang [N, D / 2] or [B, N, D / 2]."""
    c, s = torch.cos(ang), sign * torch.sin(ang)
    if ang.dim() == 3:
        c, s = c[:, None], s[:, None]
    y = torch.empty_like(x)
    half = x.shape[-1] // 2
    first = slice(0, None, 2) if interleaved else slice(0, half)
    second = slice(1, None, 2) if interleaved else slice(half, None)
    a, b = x[..., first], x[..., second]
    y[..., first] = a * c - b * s
    y[..., second] = a * s + b * c
    return y


def normed(x, w, eps):
    """(x / rms, g x / rms, 1 / rms) in 64 bits."""
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * r
    return xh, (xh if w is None else xh * w), r


def act(z, name):
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z / (1 + torch.exp(-z)) if name == "silu" else z


def assert_close(got, want, tol, what=""):
    """Elementwise |got - want| <= tol (a tensor or a number), no NaN let through."""
    g = got.detach().double().cpu()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    bad = ~((g - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((g - want).abs().max()),
                           bad.nonzero()[:3].tolist())


# fp32 error of a rotation by a reduced angle, relative to |a| + |b|: the
# fraction of a turn is off by 2^-25 + 2^-26 turns (2.8e-7 rad), sine and cosine
# by 2 ulp (2^-23 each) and the two products and the sum by 2^-24 each: < 2^-20
TURN = 2.0 ** -20
# ... of a norm over D <= 256 in 16 sequential and 4 pairwise sums: 20 * 2^-24 on
# the sum, half of it on the root, 6 more roundings: < 2^-19 relative
NORM = 2.0 ** -19


def product_tol(s, k):
    """fp32 error of a product of 16-bit rows over k values on the tensor cores:
    at most two truncations (2^-23) of a partial sum per 16 values and one
    rounding for each of 8 partial results, of the sum s of magnitudes."""
    return (k / 16 + 8) * 2.0 ** -22 * s
