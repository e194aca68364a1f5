"""Plain 64-bit forms of the head operators, and the bounds that the kernels'
outputs are held to.

The bounds come from the definitions and from the arithmetic alone (u = 2^-24,
the unit roundoff of fp32; K = D / 16 + 24, which no kernel's row sum passes in
additions one after another: a lane's own elements, then levels):

  mean      u (K + 2) mean|x|
  rstd      e_r = u (K / 2 + 10) + (mean's error)^2 / (var + eps), relative: the
            sum, each square, the division, eps, rsqrtf's 2 ulp
  n         e = |gamma| (|xhat| (e_r + 4 u) + rstd (mean's error)) + 4 u |beta|
  cos, sin  4 u: the angle as an fp32 number of half turns (pi 2^-25), two ulp
            of sincospif; and 2^-65 turns times the position
  y         e_a + e_b + (8 u + 2 pi |position| 2^-65) (|n_a| + |n_b|): cos and sin, their products with
            gamma and n, one addition; then half a step of the stored type
  t         (as y, of dy)
  dx        r (e_g + e_c1 + |xhat| e_c2 + 4 u (|g| + |c1| + 2 |xhat c2|)) + 2 u |dx|,
            e_g = |gamma| e_t + u |g|, xhat within 3 u, e_c2 = mean(e_g |xhat| + 3 u |g xhat|) + u (K + 2) mean|g xhat|
  dgamma    sum(e_t |xhat| + 4 u |t xhat|) + u N sum|t xhat| with N = heads / 1024 + 64 (a grid of 304 CTAs of
            8 warps that add their heads one after another, then the warps, then the partial rows; with the grid
            capped, at most 1100 heads over the 32 groups of lanes of a CTA)
"""
import math

import torch

from q8_ref import TYPES, U, held  # noqa: F401


def angles(positions, inv_freq, pair_axis, B, S):
    """[B, S, 1, pairs], and the largest |position| of each token."""
    p = positions.double()
    p = p if pair_axis is not None else p[None]
    p = p.reshape(p.shape[0], -1, S).expand(-1, B, S)
    axis = pair_axis if pair_axis is not None else [0] * inv_freq.numel()
    a = torch.stack([p[axis[j]] * inv_freq[j].double() for j in range(inv_freq.numel())], -1)
    return a[:, :, None], p.abs().amax(0)[:, :, None, None]


def pairs(rot, inter):
    j = torch.arange(rot // 2)
    return (2 * j, 2 * j + 1) if inter else (j, j + rot // 2)


def rotate(v, angle, rot, inter, sign=1.0):
    if rot == 0:
        return v.clone()
    a, b = pairs(rot, inter)
    c, s = torch.cos(angle), torch.sin(angle) * sign
    out = v.clone()
    out[..., a] = v[..., a] * c - v[..., b] * s
    out[..., b] = v[..., b] * c + v[..., a] * s
    return out


def rotate_tol(v, e, far, rot, inter):
    """Bound of a rotated v that is off by e."""
    tol = e.clone()
    if rot:
        a, b = pairs(rot, inter)
        t = e[..., a] + e[..., b] + (8 * U + 2 * math.pi * far * 2.0 ** -65) * (v[..., a].abs() + v[..., b].abs())
        tol[..., a] = t
        tol[..., b] = t
    return tol


def depth(D):
    return D / 16 + 24


def norm(ln, x, gamma, beta, eps):
    """mean, rstd, n with their bounds, of [..., D]."""
    v, D = x.double(), x.shape[-1]
    K = depth(D)
    mean = v.mean(-1, keepdim=True) if ln else torch.zeros_like(v[..., :1])
    em = U * (K + 2) * v.abs().mean(-1, keepdim=True) if ln else torch.zeros_like(mean)
    var = (v - mean).square().mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    er = U * (K / 2 + 10) + em.square() / (var + eps)
    xhat = (v - mean) * rstd
    g = gamma.double() if gamma is not None else torch.ones(D, dtype=torch.float64)
    b = beta.double() if (ln and beta is not None) else torch.zeros(D, dtype=torch.float64)
    n = xhat * g + b
    e = g.abs() * (xhat.abs() * (er + 4 * U) + rstd * em) + 4 * U * b.abs()
    return (mean[..., 0], em[..., 0]), (rstd[..., 0], (er * rstd)[..., 0]), (n, e)


def forward(mode, x, gamma, beta, eps, angle, far, rot, inter, sign=1.0):
    """(mean, bound), (rstd, bound), (y, bound); mode None: the rotation alone."""
    if mode is None:
        n, e, m, r = x.double(), torch.zeros_like(x, dtype=torch.float64), None, None
    else:
        m, r, (n, e) = norm(mode, x, gamma, beta, eps)
    return m, r, (rotate(n, angle, rot, inter, sign), rotate_tol(n, e, far, rot, inter))


def backward(ln, dy, x, gamma, mean, rstd, angle, far, rot, inter):
    """(dx, bound), (dgamma, bound), (dbeta, bound) from the saved statistics [B, S, H]."""
    D = x.shape[-1]
    K, r = depth(D), rstd.double()[..., None]
    t = rotate(dy.double(), angle, rot, inter, -1.0)
    et = rotate_tol(dy.double(), torch.zeros_like(t), far, rot, inter)
    xh = (x.double() - (mean.double()[..., None] if ln else 0.0)) * r
    w = gamma.double() if gamma is not None else torch.ones(D, dtype=torch.float64)
    g = t * w
    eg = w.abs() * et + U * g.abs()
    c2 = (g * xh).mean(-1, keepdim=True)
    e2 = (eg * xh.abs() + 3 * U * (g * xh).abs()).mean(-1, keepdim=True) \
        + U * (K + 2) * (g * xh).abs().mean(-1, keepdim=True)
    c1 = g.mean(-1, keepdim=True) if ln else torch.zeros_like(c2)
    e1 = eg.mean(-1, keepdim=True) + U * (K + 2) * g.abs().mean(-1, keepdim=True) if ln else torch.zeros_like(c2)
    dx = r * (g - c1 - xh * c2)
    tol = r * (eg + e1 + xh.abs() * e2 + 4 * U * (g.abs() + c1.abs() + 2 * (xh * c2).abs())) + 2 * U * dx.abs()
    dims = tuple(range(x.dim() - 1))
    N = U * (x.numel() / D / 1024 + 64)
    dg, db = (t * xh).sum(dims), t.sum(dims)
    tg = (et * xh.abs() + 4 * U * (t * xh).abs()).sum(dims) + N * (t * xh).abs().sum(dims)
    return (dx, tol), (dg, tg), (db, et.sum(dims) + N * t.abs().sum(dims))


def heads(B, S, H, D, dtype, seed, shift=0.0):
    """Heads drawn on the CPU: N(shift, 1), with one of zeros, a constant and a large one where there are enough."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, S, H, D, generator=g) + shift
    flat = x.view(-1, D)
    if flat.shape[0] >= 4:
        flat[1] = 0.0
        flat[2] = 1.5
        flat[3] *= 100.0
    return x.to(dtype)
