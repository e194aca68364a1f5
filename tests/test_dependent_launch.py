"""Kernels that are launched while their predecessor still runs (programmatic dependent launch) read what it writes by
loads that see it: not through the read-only path, which is for memory that nobody writes while the kernel is resident
(`__ldg`, or what the compiler makes of a `const __restrict__` pointer)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rmsnorm_norm_fwd_gb300", "csrc")


def kernels():
    """(name, parameters, body) of every __global__ function that waits for its predecessor."""
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\s*\([^{;]*?\)\s*)?(\w+)\s*\(([^{;]*)\)\s*\{", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            if "pdl_wait_primary()" in text[m.end():i]:
                out.append((m.group(1), m.group(2), text[m.end():i]))
    return out


def test_there_are_such_kernels():
    assert {k[0] for k in kernels()} >= {"colreduce", "rope_columns"}


@pytest.mark.parametrize("name,parameters,body", kernels(), ids=[k[0] for k in kernels()])
def test_reads_what_the_predecessor_writes(name, parameters, body):
    assert "__ldg" not in body and "ld.global.nc" not in body and "__restrict__" not in parameters + body
    after = body[body.index("pdl_wait_primary()"):]
    assert "__ldcg(" in after and "__ldcg(" not in body[:body.index("pdl_wait_primary()")]
