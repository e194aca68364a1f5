"""The 8-bit binding's stream argument (CPU: every call here is refused before anything is launched)."""
from types import SimpleNamespace

import pytest
import torch


class OnDevice0(torch.Tensor):
    """A host tensor that says it lies on device 0."""
    is_cuda = True

    def get_device(self):
        return 0


def test_a_stream_of_another_device_is_refused():
    from rmsnorm_norm_fwd_gb300 import Checkpoint8, norm_bwd_ck8, norm_fwd_ck8, norm_fwd_q8, read_ck8, read_q8
    x = torch.zeros(4, 64).as_subclass(OnDevice0)
    ck = Checkpoint8(torch.zeros(4, 64, dtype=torch.int8).as_subclass(OnDevice0), torch.zeros(4, 1, 2), 64)
    s = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    for f in (lambda: norm_fwd_q8(False, x, None, None, 1e-6, stream=s),
              lambda: norm_fwd_q8(False, x=x, gamma=None, beta=None, eps=1e-6, stream=s),
              lambda: norm_fwd_ck8(False, x, None, None, 1e-6, stream=s),
              lambda: norm_bwd_ck8(False, x, ck, None, None, x[:, 0], stream=s),
              lambda: read_q8(ck.codes, x[:, :1], stream=s),
              lambda: read_ck8(ck, stream=s),
              lambda: read_ck8(checkpoint=ck, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            f()
