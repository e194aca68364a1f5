"""Plain 64-bit forms of the 8-bit operators, and the bounds that the kernels'
outputs are held to.

The bounds come from the definitions and from the arithmetic alone (u = 2^-24,
the unit roundoff of fp32): half a step of the stored type, plus a first-order
bound on fp32 computations of the given length.  Nothing is measured.

  statistics    1e-5 relative (rstd), 1e-5 (|mean| + sigma) (mean)
  y             what these leave: T = |gamma| (4 u |xhat| + 1e-5 (|xhat| + |mean| rstd + 1)) + 4 u |beta|
  8-bit output  |Q scale - max|y|| <= max T + 4 u max|y|;
                |code scale - y| <= half a code's step + T + 4 u |y|, where half a step is 2^-4 |y| (e4m3, at least
                2^-10 scale, half the smallest code) or scale / 2 (int8)
  checkpoint    scale, mid and codes bit for bit (they are defined by fp32 steps)
"""
import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24
TINY = 2.0 ** -100
QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def half_step(t):
    """Relative size of half a rounding step of a storage type."""
    return torch.finfo(t).eps / 2


def rows(M, N, dtype, seed, shift=0.0, special=True):
    """Rows drawn on the CPU: N(shift, 1), one row of zeros, a constant one, one 100 times larger."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N, generator=g) + shift
    if special and M >= 4:
        x[1] = 0.0
        x[2] = 1.5
        x[3] *= 100.0
    return x.to(dtype)


def add(x, r):
    """h: the sum in fp32, rounded once (the fp32 sum of two values of one type rounds as the exact sum does)."""
    return x if r is None else (x.float() + r.float()).to(x.dtype)


def norm(ln, h, gamma, beta, eps):
    v = h.double()
    mean = v.mean(1, keepdim=True) if ln else torch.zeros_like(v[:, :1])
    var = (v - mean).square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    xhat = (v - mean) * rstd
    g = gamma.double() if gamma is not None else torch.ones_like(v[0])
    b = beta.double() if (ln and beta is not None) else torch.zeros_like(g)
    y = xhat * g + b
    tol = g.abs() * (4 * U * xhat.abs() + 1e-5 * (xhat.abs() + mean.abs() * rstd + (1.0 if ln else 0.0))) + 4 * U * b.abs()
    return mean[:, 0], rstd[:, 0], y, tol


def blocks(v, group):
    return torch.split(v, group or v.shape[1], 1)


def spread(s, group, n):
    return s.repeat_interleave(group or n, 1)[:, :n]


def check_q8(ln, h, gamma, q, scale, group, y, tol):
    """The 8-bit output against y and its bound; rows of h * gamma below 2^-100 are not among the inputs, zeros are."""
    Q = QMAX[q.dtype]
    q, scale, n = q.cpu().float().double(), scale.cpu().double(), y.shape[1]
    amax = torch.stack([b.abs().amax(1) for b in blocks(y, group)], 1)
    t = torch.stack([b.amax(1) for b in blocks(tol, group)], 1)
    assert ((Q * scale - amax).abs() <= t + 4 * U * amax).all(), "scale"
    s = spread(scale, group, n)
    half = s / 2 if Q == 127 else torch.maximum(y.abs() * 2.0 ** -4, s * 2.0 ** -10)
    off = (q * s - y).abs() - (half + tol + 4 * U * y.abs())
    assert (off <= 0).all(), f"codes: {off.max().item():.3g} over the bound"
    assert (q.abs() <= Q).all()
    assert (q[scale[:, 0] == 0] == 0).all() if group == 0 else True


def checkpoint(h, group):
    """codes, scales: fp32 steps."""
    codes, scales = [], []
    for b in blocks(h.float(), group):
        top, low = b.amax(1, keepdim=True), b.amin(1, keepdim=True)
        mid = top * 0.5 + low * 0.5
        half = torch.maximum(top - mid, mid - low)
        scale = torch.where(half < TINY, torch.zeros_like(half), half / torch.full_like(half, 127.0))
        inv = torch.where(half < TINY, torch.zeros_like(half), torch.ones_like(half) / scale)
        codes.append(torch.round((b - mid) * inv).to(torch.int8))
        scales.append(torch.cat([scale, mid], 1))
    return torch.cat(codes, 1), torch.stack(scales, 1)


def values(codes, scales, group):
    """What a checkpoint stands for, and |mid| + |scale code| (the sizes its fp32 evaluation rounds at)."""
    n = codes.shape[1]
    s, m = spread(scales[..., 0].double(), group, n), spread(scales[..., 1].double(), group, n)
    return m + s * codes.double(), m.abs() + (s * codes.double()).abs()


def backward(ln, dy, codes, scales, group, gamma, mean, rstd, dres):
    """dx, dgamma, dbeta in 64 bits from the checkpoint and the saved fp32 statistics, each with its bound
    (before dx's own rounding)."""
    v, size = values(codes, scales, group)
    M, N = v.shape
    mu = mean.double()[:, None] if ln else torch.zeros_like(v[:, :1])
    r = rstd.double()[:, None]
    xh = (v - mu) * r
    ex = 4 * U * r * (size + mu.abs())  # of xhat
    d = dy.double()
    g = d * (gamma.double() if gamma is not None else 1.0)
    c2 = (g * xh).mean(1, keepdim=True)
    c1 = g.mean(1, keepdim=True) if ln else torch.zeros_like(c2)
    dx = r * (g - c1 - xh * c2)
    dr = dres.double() if dres is not None else torch.zeros_like(dx)
    s2, s1 = (g * xh).abs().mean(1, keepdim=True), g.abs().mean(1, keepdim=True)
    K = N / 128 + 32  # terms a thread adds one after another, and the levels above it
    tol = U * r * (8 * (g.abs() + c1.abs() + (xh * c2).abs()) + K * (xh.abs() * s2 + s1)) + 2 * U * (dr.abs() + dx.abs())
    tol = tol + r * (ex * c2.abs() + xh.abs() * (g.abs() * ex).mean(1, keepdim=True))
    KM = M / 64 + 64  # rows a partial sum adds one after another, then the partial rows
    dg_tol = (d.abs() * ex).sum(0) + KM * U * (d * xh).abs().sum(0)
    db_tol = KM * U * d.abs().sum(0)
    return (dx + dr, tol), ((d * xh).sum(0), dg_tol), (d.sum(0), db_tol)


def held(name, got, want, tol, dtype=None):
    """|got - want| <= half a step of the stored type + tol (subnormals: half the smallest one)."""
    got = got.cpu().double()
    step = 0.0
    if dtype is not None and dtype != torch.float32:
        step = half_step(dtype) * (want.abs() + tol) + torch.finfo(dtype).smallest_normal * half_step(dtype)
    off = (got - want).abs() - (step + tol)
    assert not torch.isnan(got).any(), f"{name}: NaN"
    assert (off <= 0).all(), f"{name}: {off.max().item():.3g} over the bound"
