"""Head operators at the edges of what their documentation allows: very many tokens, parameters that
are not finite (GPU)."""
import pytest
import torch

import rope_ref as ref
from test_rope import EPS, _no_device_fault, cuda, lib, place, plan, positions, rotation  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ln", [False, True])
def test_workspace_of_more_tokens_than_a_batch_may_have(ln):
    """The size is of batches * tokens; beyond what fills the grid it does not grow."""
    size = lib().qk_norm_rope_bwd_workspace_size
    full = size(ln, 2 ** 31 - 1, 8, 2, 128)
    assert full > 0
    for tokens in (2 ** 31, 2 ** 32, 2 ** 40):
        assert size(ln, tokens, 8, 2, 128) == full
    assert size(ln, 2 ** 40 + 1, 8, 2, 128) == 0 and size(ln, -1, 8, 2, 128) == 0


def test_backward_of_more_than_2_31_tokens():
    """Batches of the same tokens (stride 0) all get the gradient of one batch."""
    g = lib()
    B, S, D = 32769, 65536, 2
    q, dy = (ref.heads(1, S, 1, D, torch.bfloat16, s).cuda() for s in (1, 2))
    r, pos = plan(rotation(D)[0], None, False), positions(1, S, 1)[0].cuda()
    rstd = g.qk_norm_rope_fwd(False, q, None, None, None, EPS, pos, r)[3]
    want = g.qk_norm_rope_bwd(False, dy, None, q, None, None, None, None, rstd, pos, r, need_dgamma=False)[0]
    dx = g.qk_norm_rope_bwd(False, dy.expand(B, S, 1, D), None, q.expand(B, S, 1, D), None, None, None, None,
                            rstd.expand(B, S, 1).contiguous(), pos, r, need_dgamma=False)[0]
    assert B * S > 2 ** 31 and torch.equal(dx, want.expand_as(dx))


@pytest.mark.parametrize("dt,how", [("bf16", "dense"), ("bf16", "two"), ("fp32", "dense"), ("fp16", "odd")])
@pytest.mark.parametrize("D,rot", [(128, 64), (128, 0), (80, 32), (72, 24), (98, 40), (600, 64)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_parameter_that_is_not_finite_reaches_its_own_element(D, rot, inter, bad, dt, how):
    """A NaN or an infinity in gamma or beta reaches its element, that one's partner if the pair is rotated, no other."""
    g = lib()
    if rot == 0 and inter:
        pytest.skip("no pairs")
    dtype = ref.TYPES[dt]
    r, pos = (plan(rotation(rot)[0], None, inter), positions(1, 3, 1).cuda() + 1) if rot else (None, None)
    q = place(torch.randn(1, 3, 5, D, generator=torch.Generator().manual_seed(1)).to(dtype), how)
    a, b = ref.pairs(rot, inter)
    for at in {0, max(rot - 1, 0), rot, (rot + D) // 2, D - 1}:
        hit = torch.zeros(D, dtype=torch.bool)
        hit[at] = True
        if at < rot:
            j = [i for i in range(rot // 2) if at in (a[i], b[i])][0]
            hit[a[j]] = hit[b[j]] = True
        w = torch.ones(D, dtype=dtype)
        w[at] = bad
        none = torch.ones(D, dtype=dtype)
        for ln, gamma, beta in ((False, w, None), (True, w, None), (True, none, w)):
            y = g.qk_norm_rope_fwd(ln, q, None, cuda(gamma), None, EPS, pos, r, beta_q=cuda(beta))[0].cpu()
            assert not torch.isfinite(y[..., hit]).any() and torch.isfinite(y[..., ~hit]).all(), (at, ln, beta is None)
