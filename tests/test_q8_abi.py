"""Argument checks of the 8-bit operators' C entry points (CPU only: every
call here is rejected before any device is touched)."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "rmsnorm_norm_fwd_gb300", "libgbnorm.so")
BAD, BF16 = 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from rmsnorm_norm_fwd_gb300 import build
        build.build()
    from rmsnorm_norm_fwd_gb300 import q8
    return q8.lib


def at(k):
    """Fake, never-dereferenced addresses, 16 MiB apart."""
    return ctypes.c_void_p(0x1000000 * (k + 1))


M, N = 8, 512
FWD = dict(ln=0, M=M, N=N, eps=1e-6, x=at(0), ldx=N, xdt=BF16, res=at(1), ldr=N, h=at(2), ldh=N, gamma=at(3), beta=None,
           pdt=BF16)
CK = dict(c=at(6), ldc=N, cg=128, cs=at(7), ldcs=8)
Q8 = dict(FWD, q=at(4), ldq=N, fmt=0, qg=128, qs=at(5), qr=4, qgs=1, **CK, mean=None, rstd=at(8), stream=None)
CK8 = dict(FWD, y=at(4), ldy=N, ydt=BF16, **CK, mean=None, rstd=at(8), stream=None)
BWD = dict(ln=0, M=M, N=N, dy=at(0), lddy=N, ydt=BF16, **CK, dres=at(1), lddres=N, gamma=at(3), pdt=BF16, mean=None,
           rstd=at(8), dx=at(2), lddx=N, xdt=BF16, dgamma=at(9), dbeta=None, ws=at(10), wsb=1 << 20, stream=None)
READ = dict(M=M, N=N, q=at(0), ldq=N, fmt=1, qg=128, scale=at(1), mid=None, sr=4, sg=1, mean=at(2), rstd=at(3),
            gamma=at(4), beta=at(5), pdt=BF16, y=at(6), ldy=N, ydt=BF16, stream=None)


def off(p, by):
    return ctypes.c_void_p(p.value + by)


FORWARD = [dict(ln=2), dict(M=-1), dict(N=0), dict(N=(1 << 24) + 1), dict(M=1 << 60), dict(eps=-1.0), dict(eps=float("inf")),
           dict(x=None), dict(ldx=N - 1), dict(xdt=3), dict(pdt=-1), dict(res=None), dict(ldr=N - 1), dict(ldh=0),
           dict(rstd=at(2)), dict(h=off(at(1), 2)), dict(h=at(0), ldh=N + 8), dict(cg=0), dict(cg=96), dict(cs=None),
           dict(cs=off(at(7), 4)), dict(ldcs=6), dict(ldcs=9), dict(c=at(0)), dict(c=at(2)), dict(cs=at(8)),
           dict(x=off(at(0), 1)), dict(gamma=off(at(3), 1)), dict(rstd=off(at(8), 2))]


@pytest.mark.parametrize("change", FORWARD + [dict(q=None), dict(fmt=2), dict(qg=100), dict(qg=512), dict(qs=None),
                                              dict(qr=0), dict(qr=1, qgs=1), dict(qr=3), dict(qr=-4), dict(qgs=0),
                                              dict(qs=off(at(5), 2)), dict(qs=at(7)), dict(q=at(0)), dict(q=at(1)),
                                              dict(ldq=N - 1), dict(qs=at(0)), dict(q=off(at(6), 100))])
def test_norm_fwd_q8_refuses(lib, change):
    assert lib.norm_fwd_q8(*{**Q8, **change}.values()) == BAD


@pytest.mark.parametrize("change", FORWARD + [dict(y=None), dict(c=None), dict(ydt=9), dict(ldy=N - 1), dict(y=at(2)),
                                              dict(y=off(at(0), 16)), dict(y=at(0), ydt=0), dict(y=at(3))])
def test_norm_fwd_ck8_refuses(lib, change):
    assert lib.norm_fwd_ck8(*{**CK8, **change}.values()) == BAD


@pytest.mark.parametrize("change", [dict(ln=3), dict(M=-1), dict(N=0), dict(dy=None), dict(c=None), dict(cs=None),
                                    dict(rstd=None), dict(dx=None), dict(ln=1), dict(lddy=N - 1), dict(ldc=1),
                                    dict(lddres=2), dict(lddx=N - 1), dict(cg=0), dict(cg=16), dict(ldcs=7),
                                    dict(ldcs=6), dict(cs=off(at(7), 4)), dict(xdt=5), dict(ydt=5), dict(pdt=5),
                                    dict(dx=at(6)), dict(dx=off(at(0), 2)), dict(dx=at(0), lddx=N + 8),
                                    dict(dx=at(0), ydt=0), dict(dgamma=at(2)), dict(dgamma=at(8)),
                                    dict(ln=1, mean=at(11), dbeta=at(9)), dict(dy=off(at(0), 1)), dict(dx=off(at(2), 1)),
                                    dict(rstd=off(at(8), 2)), dict(dgamma=off(at(9), 2)), dict(dres=off(at(1), 1))])
def test_norm_bwd_ck8_refuses(lib, change):
    assert lib.norm_bwd_ck8(*{**BWD, **change}.values()) == BAD


@pytest.mark.parametrize("change", [dict(M=-1), dict(N=0), dict(q=None), dict(scale=None), dict(y=None), dict(ldq=N - 1),
                                    dict(ldy=N - 1), dict(fmt=2), dict(qg=1), dict(pdt=4), dict(ydt=4), dict(sr=2),
                                    dict(sg=0), dict(y=at(0)), dict(y=at(1)), dict(y=at(4)), dict(mid=off(at(9), 1)),
                                    dict(y=off(at(0), 64)), dict(y=off(at(6), 1)), dict(rstd=off(at(3), 1))])
def test_q8_read_refuses(lib, change):
    assert lib.q8_read(*{**READ, **change}.values()) == BAD


def test_workspace_size_and_last_variant(lib):
    assert lib.norm_bwd_ck8_workspace_size(2, 8, 512) == 0
    assert lib.norm_bwd_ck8_workspace_size(0, -1, 512) == 0
    assert lib.norm_bwd_ck8_workspace_size(0, 8, 0) == 0
    buf = ctypes.create_string_buffer(16)
    assert lib.gbnorm_q8_last_variant(3, buf, 16) == BAD
    assert lib.gbnorm_q8_last_variant(0, None, 16) == BAD
    assert lib.gbnorm_q8_last_variant(0, buf, 16) == 0 and buf.value == b""


def test_groups_beyond_the_list_are_refused_for_empty_checkpoints():
    from rmsnorm_norm_fwd_gb300 import checkpoint8_empty
    for group in (0, 16, 100, 512):
        with pytest.raises(ValueError):
            checkpoint8_empty(4, 64, group, device="cpu")
