"""Argument checks of the head operators' C entry points (CPU only: every call
here is rejected before any device is touched), and their binding's checks of
the stream."""
import ctypes
import os
from types import SimpleNamespace

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "rmsnorm_norm_fwd_gb300", "libgbnorm.so")
BAD, BF16 = 1, 2


@pytest.fixture(scope="module")
def rope():
    if not os.path.exists(LIB):
        from rmsnorm_norm_fwd_gb300 import build
        build.build()
    from rmsnorm_norm_fwd_gb300 import rope
    return rope


def at(k):
    """Fake, never-dereferenced addresses, 16 MiB apart."""
    return 0x1000000 * (k + 1)


B, S, HQ, HK, D = 2, 8, 4, 2, 64
ES = 2
SHAPE = dict(B=B, S=S, hq=HQ, hk=HK, D=D, xdt=BF16, ydt=BF16, pdt=BF16, inter=0, rot=D, axes=1, posdt=0, res=0, pos=at(20),
             pa=0, pb=S, pt=1, freq=at(21), pair=0)


def dense(p, h):
    return [p, S * h * D, h * D, D]


def call(rope, which, shape=None, x=None, y=None, g=None, ln=0, eps=1e-6, gamma=(at(10), at(11)), beta=(0, 0), mean=None,
         rstd=at(14), dgamma=at(15), dbeta=None, ws=at(16), wsb=1 << 24):
    s = {**SHAPE, **(shape or {})}
    if s["axes"] > 1 and s["pair"] == 0 and "pair" not in (shape or {}):
        pairs = (ctypes.c_uint8 * (D // 2))()
        s["pair"] = ctypes.addressof(pairs)
    elif isinstance(s["pair"], list):
        pairs = (ctypes.c_uint8 * (D // 2))(*s["pair"])
        s["pair"] = ctypes.addressof(pairs)
    r = rope._ROPE(*s.values())

    def heads(q, k):
        return rope._HEADS(*q, *k)
    x = heads(*(x or (dense(at(0), HQ), dense(at(1), HK))))
    y = heads(*(y or (dense(at(2), HQ), dense(at(3), HK))))
    g = heads(*(g or (dense(at(4), HQ), dense(at(5), HK))))
    ga, be = rope._TWO(*gamma), rope._TWO(*beta)
    if which == "fwd":
        return rope.lib.qk_norm_rope_fwd(ln, eps, r, x, y, ga, be, mean, rstd, None)
    if which == "bwd":
        return rope.lib.qk_norm_rope_bwd(ln, r, g, x, y, ga, mean, rstd, dgamma, dbeta, ws, wsb, None)
    return getattr(rope.lib, which)(r, x, y, None)


SHAPES = [dict(B=-1), dict(S=-1), dict(hq=0), dict(hk=-1), dict(hq=65537), dict(D=0), dict(D=1025), dict(xdt=3),
          dict(ydt=-1), dict(pdt=5), dict(inter=2), dict(rot=63), dict(rot=66), dict(rot=-2), dict(axes=0), dict(axes=5),
          dict(posdt=2), dict(pos=0), dict(pos=at(20) + 2), dict(posdt=1, pos=at(20) + 4), dict(freq=0),
          dict(freq=at(21) + 2), dict(axes=2, pair=0), dict(axes=2, pair=[0] * 31 + [2]), dict(pair=[0] * 31 + [1]),
          dict(pb=-1), dict(pt=-1), dict(axes=2, pa=-4), dict(pt=1 << 59), dict(B=1 << 41), dict(B=1 << 30, S=1 << 30)]


@pytest.mark.parametrize("which", ["fwd", "bwd", "rope_fwd", "rope_bwd"])
@pytest.mark.parametrize("change", SHAPES)
def test_shapes_refused(rope, which, change):
    assert call(rope, which, change) == BAD


def test_rotation_of_nothing_refused(rope):
    assert call(rope, "rope_fwd", dict(rot=0)) == BAD and call(rope, "rope_bwd", dict(rot=0)) == BAD


# What an output may not be: q's heads and k's heads as changed [pointer, batch, token, head].
PACKED = [[at(0), S * 8 * D, 8 * D, D], [at(0) + 4 * D * ES, S * 8 * D, 8 * D, D]]
OUTPUTS = [
    dict(y=([0] + dense(0, HQ)[1:], dense(at(3), HK))), dict(y=(dense(at(2), HQ), dense(0, HK))),
    dict(y=(dense(at(2) + 1, HQ), dense(at(3), HK))),
    dict(y=(dense(at(2), HQ), dense(at(2), HK))), dict(y=(dense(at(0), HK), dense(at(3), HK))),  # other strides
    dict(y=(dense(at(0) + 2, HQ), dense(at(3), HK))), dict(y=(dense(at(1), HQ), dense(at(3), HK))),
    dict(y=(dense(at(2), HQ), dense(at(1) + 64, HK))), dict(y=(dense(at(2), HQ), dense(at(0), HK))),
    dict(y=([at(2), 0, HQ * D, D], dense(at(3), HK))), dict(y=([at(2), S * HQ * D, 0, D], dense(at(3), HK))),
    dict(y=([at(2), S * HQ * D, HQ * D, 0], dense(at(3), HK))), dict(y=([at(2), S * HQ * D, HQ * D, D - 1], dense(at(3), HK))),
    dict(y=([at(2), S * HQ * D, HQ * D - 2, D], dense(at(3), HK))), dict(y=([at(2), -5, HQ * D, D], dense(at(3), HK))),
    dict(y=([at(2), 1 << 60, HQ * D, D], dense(at(3), HK))), dict(x=([at(0), -1, HQ * D, D], dense(at(1), HK))),
    dict(x=(dense(0, HQ), dense(at(1), HK))), dict(x=(dense(at(0) + 1, HQ), dense(at(1), HK))),
    # packed inputs, the output over the other tensor, or over part of both
    dict(x=PACKED, y=(PACKED[0][:1] + [S * 8 * D, 8 * D, D // 2], dense(at(3), HK))),
    dict(x=PACKED, y=([at(0) + 2 * D * ES, S * 8 * D, 8 * D, D], dense(at(3), HK))),
    dict(x=PACKED, y=(dense(at(2), HQ), [at(0) + 5 * D * ES, S * 8 * D, 8 * D, D])),
    dict(x=PACKED, y=([at(0), S * 4 * D, 4 * D, D], dense(at(3), HK))),
    dict(y=(dense(at(20), HQ), dense(at(3), HK))), dict(y=(dense(at(21), HQ), dense(at(3), HK))),
]


@pytest.mark.parametrize("which", ["fwd", "bwd", "rope_fwd"])
@pytest.mark.parametrize("change", OUTPUTS)
def test_outputs_refused(rope, which, change):
    assert call(rope, which, **change) == BAD


@pytest.mark.parametrize("change", [dict(ln=2), dict(eps=-1.0), dict(eps=float("inf")), dict(eps=float("nan")),
                                    dict(rstd=at(0)), dict(rstd=at(2)), dict(rstd=at(14) + 2), dict(ln=1, mean=at(14)),
                                    dict(ln=1, mean=at(14) + 4), dict(gamma=(at(10) + 1, 0)), dict(gamma=(0, at(2))),
                                    dict(ln=1, beta=(at(3), 0)), dict(ln=1, beta=(0, at(12) + 1)),
                                    dict(shape=dict(xdt=0), y=(dense(at(0), HQ), dense(at(3), HK)))])
def test_forward_refuses(rope, change):
    assert call(rope, "fwd", **change) == BAD


@pytest.mark.parametrize("change", [dict(ln=-1), dict(rstd=None), dict(ln=1, mean=None), dict(rstd=at(2)),
                                    dict(rstd=at(14) + 1), dict(dgamma=at(2)), dict(dgamma=at(14)), dict(dgamma=at(15) + 2),
                                    dict(ln=1, mean=at(13), dbeta=at(15)), dict(ln=1, mean=at(13) + 2),
                                    dict(y=(dense(at(0), HQ), dense(at(3), HK))),  # dx is x
                                    dict(y=(dense(at(5), HQ), dense(at(3), HK))),
                                    dict(g=(dense(0, HQ), dense(at(5), HK))), dict(gamma=(at(2), 0)),
                                    dict(shape=dict(ydt=0), y=(dense(at(4), HQ), dense(at(3), HK)))])
def test_backward_refuses(rope, change):
    assert call(rope, "bwd", **change) == BAD


def test_parts_of_one_tensor_are_not_refused(rope):
    """In place in a packed projection passes every check (what follows them needs a device)."""
    if torch.cuda.is_available():
        pytest.skip("would run on the fake addresses")
    for x in (PACKED, [[at(0), 6 * S * D, D, S * D], [at(0) + 4 * S * D * ES, 6 * S * D, D, S * D]]):
        assert call(rope, "fwd", x=x, y=x) not in (0, BAD)
        assert call(rope, "bwd", g=x, y=x, x=(dense(at(2), HQ), dense(at(3), HK))) not in (0, BAD)
        assert call(rope, "rope_bwd", x=x, y=x) not in (0, BAD)
    # inputs of the same values for all tokens or heads
    assert call(rope, "fwd", x=([at(0), 0, 0, 0], [at(1), 0, 0, 0])) not in (0, BAD)


def test_workspace_size_and_last_variant(rope):
    size = rope.lib.qk_norm_rope_bwd_workspace_size
    for bad in ((2, 8, 4, 2, 64), (0, -1, 4, 2, 64), (0, 8, 0, 2, 64), (0, 8, 4, -1, 64), (0, 8, 4, 2, 0), (0, 8, 4, 2, 1025)):
        assert size(*bad) == 0
    buf = ctypes.create_string_buffer(16)
    last = rope.lib.gbnorm_rope_last_variant
    assert last(3, buf, 16) == BAD and last(-1, buf, 16) == BAD and last(0, None, 16) == BAD and last(0, buf, 0) == BAD
    assert last(0, buf, 16) == 0 and buf.value == b""


def test_struct_layouts(rope):
    """The binding's packed forms have the header's layout."""
    class Heads(ctypes.Structure):
        _fields_ = [("p", ctypes.c_void_p), ("batch", ctypes.c_int64), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]

    class Rope(ctypes.Structure):
        _fields_ = [(n, ctypes.c_int64) for n in ("B", "S", "hq", "hk", "D")] + \
            [(n, ctypes.c_int32) for n in ("xdt", "ydt", "pdt", "inter", "rot", "axes", "posdt", "res")] + \
            [("pos", ctypes.c_void_p)] + [(n, ctypes.c_int64) for n in ("pa", "pb", "pt")] + \
            [("freq", ctypes.c_void_p), ("pair", ctypes.c_void_p)]
    values = {n: 3 * i + 1 for i, (n, _) in enumerate(Rope._fields_)}
    assert bytes(Rope(**values)) == rope._ROPE(*values.values())
    two = (Heads * 2)(Heads(1, 2, 3, 4), Heads(5, 6, 7, 8))
    assert bytes(two) == rope._HEADS(*range(1, 9))


class OnDevice0(torch.Tensor):
    """A host tensor that says it lies on device 0."""
    is_cuda = True

    def get_device(self):
        return 0


def test_a_stream_of_another_device_is_refused(rope):
    q = torch.zeros(4, 2, 64).as_subclass(OnDevice0)
    s = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    for f in (lambda: rope.qk_norm_rope_fwd(False, q, None, None, None, 1e-6, stream=s),
              lambda: rope.qk_norm_rope_bwd(False, q, None, q, None, None, None, None, q, stream=s),
              lambda: rope.rope_fwd(q, None, None, None, stream=s), lambda: rope.rope_bwd(q, None, None, None, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            f()
