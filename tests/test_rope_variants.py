"""Every kernel of the head operators by name, at the head sizes that select it, and the order in which a warp takes
tokens (GPU)."""
import pytest
import torch

import rope_ref as ref
from test_rope import EPS, _no_device_fault, lib, plan, positions, rotation, run_backward, run_forward  # noqa: F401

pytestmark = pytest.mark.gpu


def names():
    g = lib()
    return [g.rope_last_variant(i) for i in range(3)]


# 16-byte vectors: 2 * V * L elements fill L lanes (fp32 has powers of two alone); eight fewer leave a chunk out.
WHOLE = [(dt, v, L) for dt, v in (("bf16", 8), ("fp16", 8), ("fp32", 4)) for L in (4, 5, 6, 8, 10, 16, 32)]


def lanes(dt, L):
    return {5: 8, 6: 8, 10: 16}.get(L, L) if dt == "fp32" else L


@pytest.mark.parametrize("dt,v,L", WHOLE)
@pytest.mark.parametrize("inter", [False, True])
def test_whole_heads(dt, v, L, inter):
    D, forward = 2 * v * L, "" if L == 32 else "n" if inter else "h"
    n = f"vec{v}x{lanes(dt, L)}"
    want = [n + forward, n + ("" if inter else forward), n + forward]  # the backward has none for neighbours
    for hq, hk in ((7, 3), (32 // L, 1)):
        for mode in (False, True):
            run_forward(mode, 2, 5, hq, hk, D, dt=dt, inter=inter)
            run_backward(mode, 2, 5, hq, hk, D, dt=dt, inter=inter)
        run_forward(None, 2, 5, hq, hk, D, dt=dt, inter=inter)
        assert names() == want
    if inter:  # a chunk missing: an odd number of them
        run_forward(True, 1, 5, 7, 3, D - v, dt=dt, inter=True)
        run_backward(True, 1, 5, 7, 3, D - v, dt=dt, inter=True)
        assert names()[:2] == want[:2]


@pytest.mark.parametrize("dt,v,L", WHOLE)
def test_parts_of_heads(dt, v, L):
    D, name = 2 * v * L, f"vec{v}x{lanes(dt, L)}"
    for rot, inter in ((2 * v, False), (0, False), (D - 2 * v, False), (3 * v, True), (D - v, True)):
        for mode in (False, True):
            run_forward(mode, 1, 5, 7, 3, D, rot, dt=dt, inter=inter)
            run_backward(mode, 1, 5, 7, 3, D, rot, dt=dt, inter=inter)
        assert names()[:2] == [name] * 2
        if rot:
            run_forward(None, 1, 5, 7, 3, D, rot, dt=dt, inter=inter)
            assert names()[2] == name


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D,L", [(8, 4), (24, 4), (40, 4), (56, 4), (72, 5), (88, 6), (104, 8), (136, 10), (152, 10),
                                 (200, 16), (256, 16), (424, 32)])
def test_vectors_of_four(dt, D, L):
    how = "packed" if D < 200 else "dense"
    rot = D if D != 256 else 200  # half of 200 is no multiple of eight
    for mode in (False, True):
        run_forward(mode, 1, 9, 7, 3, D, rot, dt=dt, how=how)
        run_backward(mode, 1, 9, 7, 3, D, rot, dt=dt, how=how)
    run_forward(None, 1, 9, 7, 3, D, rot, dt=dt, how=how)
    kind = "h" if rot == D and L != 32 else ""
    assert names() == [f"vec4x{L}{kind}", f"vec4x{L}", f"vec4x{L}{kind}"]


@pytest.mark.parametrize("D,L", [(32, 4), (64, 4), (80, 8), (128, 8), (256, 16), (512, 32)])
@pytest.mark.parametrize("xt,yt", [("fp32", "bf16"), ("bf16", "fp32"), ("fp16", "bf16"), ("fp32", "fp16")])
def test_differing_types(D, L, xt, yt):
    for inter in (False, True):
        for mode in (False, True):
            run_forward(mode, 1, 9, 7, 3, D, dt=xt, ydt=yt, inter=inter, pdt="fp32")
            run_backward(mode, 1, 9, 7, 3, D, dt=xt, ydt=yt, inter=inter, pdt="fp32")
        run_forward(None, 1, 9, 7, 3, D, D // 2, dt=xt, ydt=yt, inter=inter)
        assert names() == [f"vec4x{L}"] * 3


# Halves of an even number of pairs, or neighbours, on boundaries of two elements.
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,rot,inter,L", [(4, 4, False, 4), (2, 2, True, 4), (44, 44, False, 4), (98, 98, True, 8),
                                           (100, 44, False, 8), (130, 130, True, 16), (250, 20, True, 16),
                                           (252, 252, False, 16), (258, 258, True, 32)])
def test_vectors_of_two(dt, D, rot, inter, L):
    if dt == "fp32":
        L = 2 * L if 2 * 2 * L * 2 < D + 8 else L  # eight elements a lane, not sixteen
        if D >= 258:
            return
    for mode in (False, True):
        run_forward(mode, 1, 9, 7, 3, D, rot, dt=dt, inter=inter, how="two")
        run_backward(mode, 1, 9, 7, 3, D, rot, dt=dt, inter=inter, how="two")
    run_forward(None, 1, 9, 7, 3, D, rot, dt=dt, inter=inter, how="two")
    assert all(n.startswith("vec2x") for n in names()), names()
    if dt != "fp32":
        assert names() == [f"vec2x{L}"] * 3


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("D,rot,name", [(1, 0, "any4x8"), (63, 62, "any4x8"), (66, 66, "any8x8"), (127, 20, "any8x8"),
                                        (128, 18, "any8x8"), (255, 254, "any16x8"), (511, 100, "any32x8"),
                                        (1022, 1022, "any32x16"), (1024, 14, "any32x16")])
def test_element_by_element(dt, D, rot, name):
    for inter in (False, True) if rot else (False,):
        if rot % 4 == 0 and inter and D % 4 == 0:
            continue
        for mode in (False, True):
            run_forward(mode, 1, 9, 9, 3, D, rot, dt=dt, inter=inter, how="odd")
            run_backward(mode, 1, 9, 9, 3, D, rot, dt=dt, inter=inter, how="odd")
        assert names()[:2] == [name] * 2
        if rot:
            run_forward(None, 1, 9, 9, 3, D, rot, dt=dt, inter=inter, how="odd")
            assert names()[2] == name


@pytest.mark.parametrize("limit", [1, 2])
@pytest.mark.parametrize("B,S", [(1, 97), (40, 3), (7, 25), (131, 1), (2, 64), (33, 2)])
def test_whole_tokens_then_the_rest(limit, B, S):
    """With few warps each takes every W-th token, over the ends of batches, and a share of what is left."""
    g = lib()
    try:
        g.set_grid_limit(limit)
        for D in (128, 98):
            for hq, hk in ((9, 2), (3, 0), (1, 5)):
                run_forward(True, B, S, hq, hk, D)
                run_forward(None, B, S, hq, hk, D, out="major")
                run_backward(False, B, S, hq, hk, D)
    finally:
        g.set_grid_limit(0)


@pytest.mark.parametrize("D,dt", [(128, "bf16"), (72, "fp16"), (98, "bf16")])
def test_many_tokens(D, dt):
    """More tokens than four times the warps of the device's grid."""
    run_forward(False, 3, 4001, 5, 2, D, dt=dt)
    run_forward(None, 1, 20011, 2, 1, D, dt=dt, axes=3)
    run_backward(True, 3, 4001, 5, 2, D, dt=dt)


@pytest.mark.parametrize("D", [128, 80, 98])
def test_a_tensor_does_not_change_the_other(D):
    """Keys beside the queries change no bit of them, in whatever share of the work: forward and rotation."""
    g = lib()
    S, f = 301, rotation(D)[0]
    q, k = (ref.heads(1, S, h, D, torch.bfloat16, h).cuda() for h in (6, 3))
    r, pos = plan(f, None, False), positions(1, S, 1).cuda()
    a = g.qk_norm_rope_fwd(False, q, k, None, None, EPS, pos, r)
    b, c = (g.qk_norm_rope_fwd(False, t, None, None, None, EPS, pos, r) for t in (q, k))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], c[0]) and torch.equal(a[3], torch.cat([b[3], c[3]], 2))
    x = g.rope_fwd(q, k, pos, r)
    assert torch.equal(x[0], g.rope_fwd(q, None, pos, r)[0]) and torch.equal(x[1], g.rope_fwd(k, None, pos, r)[0])
