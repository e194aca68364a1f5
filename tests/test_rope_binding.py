"""What the binding of the head operators refuses before it allocates or launches anything (CPU only)."""
import os

import pytest
import torch

from test_rope_abi import LIB, OnDevice0


@pytest.fixture(scope="module")
def rope():
    if not os.path.exists(LIB):
        from rmsnorm_norm_fwd_gb300 import build
        build.build()
    from rmsnorm_norm_fwd_gb300 import rope
    return rope


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice0)


S, H, D = 4, 2, 64


@pytest.fixture(scope="module")
def where(rope):
    return zeros(S, dtype=torch.int32), rope.Rotary(zeros(D // 2, dtype=torch.float32), False, 1, None)


@pytest.mark.parametrize("given", [False, True])
def test_keys_outputs_and_gradients_without_keys(rope, where, given):
    """yk, dk or dyk without k: nothing would write or read them."""
    q, rstd = zeros(S, H, D), zeros(S, H, dtype=torch.float32)
    out = zeros(S, H, D) if given else None
    for f in (lambda: rope.rope_fwd(q, None, *where, yq=out, yk=zeros(S, H, D)),
              lambda: rope.qk_norm_rope_fwd(False, q, None, None, None, 1e-6, *where, yq=out, yk=zeros(S, H, D)),
              lambda: rope.rope_bwd(q, None, *where, dq=out, dk=zeros(S, H, D)),
              lambda: rope.qk_norm_rope_bwd(False, q, None, q, None, None, None, None, rstd, *where, dq=out,
                                            dk=zeros(S, H, D)),
              lambda: rope.qk_norm_rope_bwd(False, q, zeros(S, H, D), q, None, None, None, None, rstd, *where, dq=out)):
        with pytest.raises(ValueError, match="without k"):
            f()


def test_a_dtype_that_the_given_output_contradicts(rope, where):
    q, y = zeros(S, H, D), zeros(S, H, D, dtype=torch.float16)
    for f in (lambda: rope.rope_fwd(q, None, *where, y_dtype=torch.float32, yq=y),
              lambda: rope.qk_norm_rope_fwd(False, q, None, None, None, 1e-6, *where, y_dtype=torch.bfloat16, yq=y),
              lambda: rope.rope_bwd(q, None, *where, dx_dtype=torch.float32, dq=y)):
        with pytest.raises(ValueError, match="dtype"):
            f()
