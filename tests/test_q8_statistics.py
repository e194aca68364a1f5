"""Statistics of the 8-bit forwards, and what is made of them, at bounds derived from the arithmetic (GPU).

u = 2^-24.  D: roundings along the longest chain of a row sum.  Rows in registers: at most 16 elements one after
another (32 in two lanes of a pair), those joined, 5 levels of a warp, 5 of 32 warps, 3 of 8 CTAs; products with counts
and their reciprocals, two for a thread's mean and three for each level above: 41.  Element by element: N / 256 one
after another, 5 levels, 8 warps in order and 4 for the operations around them.

  rstd, RMSNorm    e_r = u (D / 2 + 7): half of what the sum of squares, the division and eps make of the variance, and
                   the 2 ulp (4 u) that rsqrtf is documented to be off by at most
  rstd, LayerNorm  e_r = u (D / 2 + 8) + 48 u rms(h) sigma / (var + eps) + (u D rms(h))^2 / (var + eps).  The second
                   term, rows in registers only: the threads' means are off by up to 19 u mean|h|, the warps' by 27 u,
                   the CTAs' by 35 u, each meets the part of the spread that lies between the means of its level, and
                   by Cauchy-Schwarz they make (19^2 + 27^2 + 35^2)^(1/2) u rms(h) sigma at most.  The third: their
                   squares, which alone are left where sigma is 0
  mean             e_mu = u (D + 2) mean|h|
  y                |gamma| (rstd e_mu + |xhat| e_r) + 4 u (|xhat gamma| + |beta|)
"""
import pytest
import torch

import q8_ref as ref
from q8_ref import TYPES, U
from test_q8 import E4M3, I8, cuda, lib, params

pytestmark = pytest.mark.gpu


def norm(ln, h, gamma, beta, eps, elem):
    """mean, rstd, y in 64 bits, and the bounds of the three."""
    N = h.shape[1]
    D = N / 256 + 17 if elem else 41
    mean, rstd, y, _ = ref.norm(ln, h, gamma, beta, eps)
    v = h.double()
    rms2, var = v.square().mean(1), 1 / rstd.square()  # var + eps
    e_r = U * (D / 2 + 7) * torch.ones_like(rstd)
    if ln:
        sigma = (var - eps).clamp(min=0).sqrt()
        e_r = e_r + U + (0 if elem else 48 * U) * rms2.sqrt() * sigma / var + (U * D) ** 2 * rms2 / var
    e_mu = U * (D + 2) * v.abs().mean(1) if ln else torch.zeros_like(mean)
    gm = gamma.double().abs()
    xhat = (v - mean[:, None] if ln else v).abs() * rstd[:, None]
    tol = gm * ((rstd * e_mu)[:, None] + xhat * e_r[:, None]) + 4 * U * xhat * gm
    if ln:
        tol = tol + 4 * U * beta.double().abs()
    return mean, rstd, y, e_mu, e_r, tol


def outliers(M, N, dtype, shift, seed):
    """ref.rows with the 40th element of each hundred 50 times larger, in some rows one that starts a chunk of 8."""
    x = ref.rows(M, N, torch.float32, seed, shift)
    x[: M // 2, 39::100] *= 50
    x[M // 2:, ::32] *= 50
    return x.to(dtype)


@pytest.mark.parametrize("N", [96, 1000, 1003, 4096, 5120, 8192, 12288, 16384, 32768, 40001, 140000])
@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("dt,pdt", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_at_derived_bounds(N, ln, dt, pdt):
    g = lib()
    M, eps = 21, 1e-6
    h = outliers(M, N, TYPES[dt], 0.5 if ln else 0.0, N)
    gamma, beta = params(N, ln, TYPES[pdt])
    mean, rstd, y, e_mu, e_r, tol = norm(ln, h, gamma, beta, eps, N > 131072)
    par = (h.cuda(), gamma.cuda(), cuda(beta), eps)
    for group, fmt in ((0, E4M3), (128, I8)):
        q, s, _, m, r = g.norm_fwd_q8(ln, *par, group=group, fmt=fmt)
        assert ((r.cpu().double() - rstd).abs() <= e_r * rstd).all()
        assert not ln or ((m.cpu().double() - mean).abs() <= e_mu).all()
        ref.check_q8(ln, h, gamma, q, s, group, y, tol)
    yy, _, _, m, r = g.norm_fwd_ck8(ln, *par, y_dtype=torch.float32)
    assert ((r.cpu().double() - rstd).abs() <= e_r * rstd).all()
    assert not ln or ((m.cpu().double() - mean).abs() <= e_mu).all()
    ref.held("y", yy, y, tol)


@pytest.mark.parametrize("vec", [True, False])
@pytest.mark.parametrize("big", [3600, 3637, 3859])
def test_variance_of_rows_with_an_outlier_in_every_thread(vec, big):
    """LayerNorm rows of 8192 in which every thread holds the same integers, one large, first, and small ones, with an
    integer mean: the thread's mean, its deviations and their squares' sums (below 2^24) are exact, and the sums of
    equal parts too.  So the variance is, and rstd is off by rsqrtf's 2 ulp, 4 u, alone.  Sums of squares about
    anything but the mean would pass 2^24 and be rounded."""
    g = lib()
    N, n = 8192, 32 if vec else 16
    pat = torch.tensor([big] + [(7 * i * i + 3 * i) % 61 - 30 for i in range(1, n)], dtype=torch.float64)
    pat[-1] -= pat.sum() % n
    j = torch.arange(N)
    at = j % 8 + 8 * (j // 2048) if vec else j % 256 // 32 + 8 * (j // 4096)
    assert (torch.bincount(at) == N // n).all() and (pat - pat.mean()).square().sum() < 2 ** 24
    x = torch.zeros(3, N + 4, device="cuda")[:, :N] if vec else torch.zeros(3, N + 5, device="cuda")[:, 1:N + 1]
    x.copy_(pat[at].float()[None].expand(3, N))
    rstd = 1 / pat.var(unbiased=False).sqrt().item()
    for group in (0, 128):
        _, _, _, m, r = g.norm_fwd_q8(True, x, None, None, 0.0, group=group)
        assert g.q8_last_variant(0) == ("rows256x4c1" if vec else "any512x2c1")
        assert (m.cpu().double() == pat.mean()).all()
        assert ((r.cpu().double() - rstd).abs() <= 4 * U * rstd).all()


@pytest.mark.parametrize("N", [256, 1003, 5128, 40000, 40001, 140000])
def test_squares_beyond_fp32_near_the_end_of_the_range(N):
    """LayerNorm rows whose squares pass fp32 and whose sums of magnitudes do not: rstd 0, zeros, a finite mean."""
    g = lib()
    x = torch.randn(3, N, generator=torch.Generator().manual_seed(1))
    x[1] = torch.where(torch.arange(N) % 2 == 0, 1.0, -1.0) * (2.0 ** 127 / N)
    mean = x[1].double().mean().item()
    for group in (0, 128):
        q, s, _, m, rstd = g.norm_fwd_q8(True, x.cuda(), None, None, 1e-6, group=group)
        assert rstd[1] == 0 and (s[1] == 0).all() and (q[1].float() == 0).all()
        assert abs(m[1].item() - mean) <= U * (N / 256 + 64) * 2.0 ** 127 / N
        assert torch.isfinite(s).all() and (rstd[0] > 0) and (rstd[2] > 0)
