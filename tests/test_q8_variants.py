"""Every compiled kernel of the 8-bit operators that holds rows in registers runs, at the row lengths that select it
(GPU)."""
import pytest
import torch

from test_q8 import I8, lib, run_backward, run_forward

pytestmark = pytest.mark.gpu

# (threads of a row, chunks or blocks of a thread, CTAs of a cluster[, rows at a time]) by capacity
FWD = {
    False: [(32, 1, 1), (32, 2, 1), (32, 4, 1), (64, 4, 1), (128, 4, 1), (256, 3, 1), (256, 4, 1), (512, 3, 1), (512, 4, 1),
            (512, 3, 2), (512, 4, 2), (512, 3, 4), (512, 4, 4), (512, 3, 8), (512, 4, 8)],
    True: [(32, 1, 1), (32, 2, 1), (32, 4, 1), (64, 4, 1), (128, 4, 1), (160, 4, 1), (256, 3, 1), (256, 4, 1), (512, 3, 1),
           (512, 4, 1), (256, 3, 4), (256, 4, 4), (256, 3, 8), (256, 4, 8), (512, 3, 8), (512, 4, 8)],
}
BWD = {
    False: [(32, 1, 1, 2), (32, 2, 1, 2), (32, 4, 1, 1), (64, 4, 1, 1), (128, 4, 1, 1), (160, 4, 1, 1), (256, 3, 1, 1),
            (256, 4, 1, 1), (512, 3, 1, 1), (512, 4, 1, 1), (256, 3, 4, 1), (256, 4, 4, 1), (256, 3, 8, 1), (256, 4, 8, 1),
            (512, 4, 8, 1)],
    True: [(32, 1, 1, 2), (32, 2, 1, 2), (64, 2, 1, 2), (128, 2, 1, 2), (256, 2, 1, 2), (320, 2, 1, 1), (512, 2, 1, 2),
           (256, 2, 4, 2), (256, 2, 8, 2), (512, 2, 8, 2), (512, 4, 8, 1)],
}
ANY = [(32, 1, 1), (32, 2, 1), (64, 2, 1), (128, 2, 1), (256, 2, 1), (512, 2, 1), (512, 2, 2), (512, 2, 4), (512, 2, 8),
       (1024, 2, 8)]


def lengths(table, step):
    """(N, geometry) for each entry: just past what the entry before holds, and all that it holds (without vectors: one
    element less)."""
    before = 0
    for geom in table:
        most = geom[0] * geom[1] * geom[2] * 8
        yield before + step, geom
        yield (most if step == 8 else most - 1), geom
        before = most


def name(prefix, geom):
    return f"{prefix}{geom[0]}x{geom[1]}c{geom[2]}" + (f"r{geom[3]}" if len(geom) > 3 else "")


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("prefix", ["rows", "any"])
def test_every_forward(ln, prefix):
    g = lib()
    for N, geom in lengths(FWD[ln], 8) if prefix == "rows" else lengths(ANY, 1):
        for kw in (dict(dt="bf16", group=32, ck=32), dict(dt="fp16", pdt="fp32", group=0, ck=128, fmt=I8),
                   dict(dt="fp32", group=0, residual=False), dict(dt="bf16", group=256), dict(dt="bf16", out="ck8", ck=64)):
            run_forward(ln, 3, N, **kw)
            assert g.q8_last_variant(0) == name(prefix, geom), (N, kw)


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("prefix", ["rows", "any"])
def test_every_backward(ln, prefix):
    g = lib()
    for N, geom in lengths(BWD[ln], 8) if prefix == "rows" else lengths(ANY, 1):
        for kw in (dict(dt="bf16", group=32), dict(dt="fp16"), dict(dt="fp32", dres=False), dict(dt="bf16", ydt="fp32")):
            run_backward(ln, 3, N, **kw)
            assert g.q8_last_variant(1) == name(prefix, geom), (N, kw)
