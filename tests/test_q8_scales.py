"""Scales of the 8-bit output: the division that defines them, NaN in rows with groups of zeros, products h * gamma
beyond fp32 (GPU)."""
import pytest
import torch

import q8_ref as ref
from test_q8 import E4M3, I8, lib, params, same_bits

pytestmark = pytest.mark.gpu
# one row group, without vectors, over a cluster, that without vectors, element by element
KERNELS = [(512, "rows"), (1003, "any"), (40000, "rows"), (40001, "any"), (140000, "elem")]


@pytest.mark.parametrize("N,kernel", KERNELS)
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("fmt", [E4M3, I8])
def test_nan_reaches_groups_of_zeros(N, kernel, group, fmt):
    """RMSNorm of a row with a NaN: y is NaN everywhere, so is every scale, where the row or gamma is zero too.  Groups
    of zeros in rows without one keep scale 0, beside an infinity (rstd 0) and in a row of zeros with eps 0 (rstd
    infinite) as well."""
    g = lib()
    x = ref.rows(5, N, torch.bfloat16, 1, special=False)
    gamma = params(N, False, torch.bfloat16)[0]
    x[:, :group] = 0.0
    gamma[2 * group:3 * group] = 0.0
    x[3, N - 1] = float("nan")
    x[4, N - 1] = float("inf")
    q, s, _, _, rstd = g.norm_fwd_q8(False, x.cuda(), gamma.cuda(), None, 1e-6, group=group, fmt=fmt)
    assert kernel in g.q8_last_variant(0)
    assert torch.isnan(rstd[3]) and torch.isnan(s[3]).all()
    assert torch.isnan(g.read_q8(q, s, group)[3]).all()
    for i in (0, 1, 2, 4):
        assert s[i, 0] == 0 and s[i, 2] == 0
        assert (q[i, :group].float() == 0).all() and (q[i, 2 * group:3 * group].float() == 0).all()
    assert torch.isfinite(s[:3]).all() and (s[:3, 1] > 0).all()
    q, s, _, _, rstd = g.norm_fwd_q8(False, torch.zeros_like(x).cuda(), gamma.cuda(), None, 0.0, group=group, fmt=fmt)
    assert torch.isinf(rstd).all() and (s == 0).all() and (q.float() == 0).all()


@pytest.mark.parametrize("N,kernel", KERNELS)
@pytest.mark.parametrize("group", [0, 32, 256])
@pytest.mark.parametrize("fmt", [E4M3, I8])
def test_scales_are_the_division(N, kernel, group, fmt):
    """scale = max|y| / Q in fp32, the same bits from every kernel: RMSNorm's from max|h gamma| and the saved rstd,
    LayerNorm's where y is exact (rows of zeros: y is beta)."""
    g = lib()
    x = ref.rows(7, N, torch.bfloat16, 3)
    gamma, beta = params(N, True, torch.bfloat16)
    _, s, _, _, rstd = g.norm_fwd_q8(False, x.cuda(), gamma.cuda(), None, 1e-6, group=group, fmt=fmt)
    assert kernel in g.q8_last_variant(0)
    t = x.float() * gamma.float()
    amax = torch.stack([b.abs().amax(1) for b in ref.blocks(t, group)], 1)
    Q = torch.full_like(amax, ref.QMAX[fmt])
    assert same_bits(s, (amax * rstd.cpu()[:, None]) / Q)
    _, s, *_ = g.norm_fwd_q8(True, torch.zeros_like(x).cuda(), gamma.cuda(), beta.cuda(), 1e-6, group=group, fmt=fmt)
    amax = torch.stack([b.abs().amax(1) for b in ref.blocks(beta.float()[None].expand(7, N), group)], 1)
    assert same_bits(s, amax / Q)


@pytest.mark.parametrize("N,kernel", KERNELS)
@pytest.mark.parametrize("group", [0, 64])
def test_products_beyond_fp32(N, kernel, group):
    """RMSNorm where h gamma passes fp32 although y does not: a scale that is not finite, not a wrong value."""
    g = lib()
    x = torch.full((2, N), 1e10)
    x[1] = 1.0
    q, s, *_ = g.norm_fwd_q8(False, x.cuda(), torch.full((N,), 1e30).cuda(), None, 1e-6, group=group)
    assert kernel in g.q8_last_variant(0)
    assert not torch.isfinite(s[0]).any()
    assert torch.isfinite(s[1]).all() and (q[1].float() == 448).all()
