"""The head operators captured into a graph as the first calls that a process makes of them (GPU)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import sys, torch
import rmsnorm_norm_fwd_gb300 as g
D, ln = int(sys.argv[1]), sys.argv[2] == "ln"
B, S, hq, hk = 1, 130, 6, 3
r = g.rotary(torch.tensor([1e4 ** (-2 * j / D) for j in range(D // 2)], dtype=torch.float32).cuda())
q, k = (torch.zeros(B, S, h, D, device="cuda", dtype=torch.bfloat16) for h in (hq, hk))
pos = torch.zeros(B, S, device="cuda", dtype=torch.int32)
def calls():
    yq, yk, mean, rstd = g.qk_norm_rope_fwd(ln, q, k, None, None, 1e-6, pos, r)
    return (yq, yk, rstd, *g.qk_norm_rope_bwd(ln, yq, yk, q, k, None, None, mean, rstd, pos, r)[:3],
            *g.rope_fwd(q, k, pos, r), *g.rope_bwd(yq, yk, pos, r))
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    out = calls()
for seed in (1, 2):
    gen = torch.Generator().manual_seed(seed)
    for t in (q, k):
        t.copy_(torch.randn(t.shape, generator=gen))
    pos.copy_(torch.randint(0, 5000, (B, S), generator=gen))
    graph.replay()
    for a, b in zip(out, calls()):
        assert torch.equal(a, b) and torch.isfinite(a.float()).all() and a.any()
assert g.read_fault(reset=True) == 0
print("same", g.rope_last_variant(0), g.rope_last_variant(1), g.rope_last_variant(2))
"""


@pytest.mark.parametrize("D,kernel", [(128, "vec8"), (72, "vec4"), (98, "any")])
@pytest.mark.parametrize("norm", ["rms", "ln"])
def test_captured_before_any_call_of_the_process(D, kernel, norm):
    """What a kernel's first call on a device does (its limit of shared memory, what an SM holds of it) happens inside
    the capture; replayed on other inputs and positions."""
    r = subprocess.run([sys.executable, "-c", FIRST, str(D), norm], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split()[0] == "same" and all(n.startswith(kernel) for n in r.stdout.split()[1:])
