"""Head operators at the edges of what their documentation allows: very many tokens (GPU)."""
import pytest
import torch

import rope_ref as ref
from test_rope import EPS, _no_device_fault, lib, plan, positions, rotation  # noqa: F401

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
