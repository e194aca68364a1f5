"""Binding of the 8-bit operators (norm_fwd_q8, norm_fwd_ck8, norm_bwd_ck8 and
q8_read of include/gbnorm.h).

Argument marshalling only, as in ``binding``: tensors are checked, outputs that
the caller does not pass are allocated with torch's caching allocator, and the
call goes to the C ABI on torch's current stream of the tensors' device, or on
the one given as the keyword ``stream``, which every operator takes.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from .binding import DTYPE_CODE, GbnormError, _check, _f, _i64, _int, _sz, _vp, lib

_FWD = [_int, _i64, _i64, _f, _vp, _i64, _int, _vp, _i64, _vp, _i64, _vp, _vp, _int]
_CK = [_vp, _i64, _int, _vp, _i64]
lib.norm_fwd_q8.argtypes = _FWD + [_vp, _i64, _int, _int, _vp, _i64, _i64] + _CK + [_vp, _vp, _vp]
lib.norm_fwd_ck8.argtypes = _FWD + [_vp, _i64, _int] + _CK + [_vp, _vp, _vp]
lib.norm_bwd_ck8_workspace_size.argtypes = [_int, _i64, _i64]
lib.norm_bwd_ck8_workspace_size.restype = _sz
lib.norm_bwd_ck8.argtypes = [_int, _i64, _i64, _vp, _i64, _int] + _CK + [_vp, _i64, _vp, _int, _vp, _vp, _vp, _i64, _int,
                                                                       _vp, _vp, _vp, _sz, _vp]
lib.q8_read.argtypes = [_i64, _i64, _vp, _i64, _int, _int, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _int, _vp, _i64,
                        _int, _vp]
lib.gbnorm_q8_last_variant.argtypes = [_int, ctypes.c_char_p, _sz]
for _fn in ("norm_fwd_q8", "norm_fwd_ck8", "norm_bwd_ck8", "q8_read", "gbnorm_q8_last_variant"):
    getattr(lib, _fn).restype = _int

Q8_CODE = {torch.float8_e4m3fn: 0, torch.int8: 1}
GROUPS = (32, 64, 128, 256)


class Checkpoint8(NamedTuple):
    """An 8-bit checkpoint of [M, N] rows: int8 codes [M, N], float32 scales
    [M, ceil(N / group), 2] (scale and mid of each group), columns per group."""
    codes: torch.Tensor
    scales: torch.Tensor
    group: int


def _groups(n: int, group: int) -> int:
    return -(-n // group) if group else 1


def checkpoint8_empty(M: int, N: int, group: int = 128, device="cuda") -> Checkpoint8:
    """Buffers for a checkpoint of [M, N] rows."""
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}")
    return Checkpoint8(torch.empty(M, N, device=device, dtype=torch.int8),
                       torch.empty(M, _groups(N, group), 2, device=device, dtype=torch.float32), group)


# The current stream's handle without a Stream object around it (a call of a
# few microseconds would spend a fifth of its time on that), where this torch
# has the function.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


class _Call:
    """Checks of one call's tensors against its first one, and its launch on that one's device."""

    __slots__ = ("dev", "shape", "M", "N")

    def __init__(self, name, t):
        self.dev = t.get_device()
        if self.dev < 0 or not t.is_cuda or t.dim() != 2:
            raise ValueError(f"{name} must be a 2-D CUDA tensor")
        self.shape = t.shape
        self.M, self.N = self.shape

    def rows(self, name, t, dtype=None):
        """(ptr, ld) of [M, N] rows with any row stride."""
        if t is None:
            return None, self.N
        if t.shape != self.shape or t.get_device() != self.dev:
            raise ValueError(f"{name} must be a [{self.M}, {self.N}] CUDA tensor on device {self.dev}")
        ld, col = t.stride()
        if col != 1 and self.N > 1:
            raise ValueError(f"{name} must have unit column stride")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name} must have dtype {dtype}")
        return t.data_ptr(), (ld if ld > self.N or self.M > 1 else self.N)

    def vec(self, name, t, n, dtype):
        if t is None:
            return None
        if t.shape != (n,) or t.get_device() != self.dev or t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 1-D CUDA {dtype} tensor of {n} elements on device {self.dev}")
        return t.data_ptr()

    def params(self, gamma, beta, default):
        """(gamma ptr, beta ptr, dtype code)."""
        pdt = gamma.dtype if gamma is not None else beta.dtype if beta is not None else default
        code = DTYPE_CODE.get(pdt)
        if code is None:
            raise ValueError(f"gamma and beta cannot have dtype {pdt}")
        return self.vec("gamma", gamma, self.N, pdt), self.vec("beta", beta, self.N, pdt), code

    def scales(self, name, t, group):
        """(ptr, row stride, group stride) of [M, G] scales in either order."""
        G = _groups(self.N, group)
        if t.shape != (self.M, G) or t.get_device() != self.dev or t.dtype != torch.float32:
            raise ValueError(f"{name} must be a [{self.M}, {G}] float32 CUDA tensor on device {self.dev}")
        return t.data_ptr(), *t.stride()

    def checkpoint(self, ck):
        """The five checkpoint arguments."""
        if ck is None:
            return None, self.N, 128, None, 2
        codes, scales, group = ck
        if group not in GROUPS:
            raise ValueError(f"checkpoint group must be one of {GROUPS}")
        pc, ldc = self.rows("checkpoint codes", codes, torch.int8)
        G = _groups(self.N, group)
        if scales.shape != (self.M, G, 2) or scales.dtype != torch.float32 or scales.get_device() != self.dev \
                or (self.M > 0 and (scales.stride(2) != 1 or (G > 1 and scales.stride(1) != 2))):
            raise ValueError(f"checkpoint scales must be [{self.M}, {G}, 2] float32 on device {self.dev}, "
                             "each row contiguous")
        return pc, ldc, group, scales.data_ptr(), scales.stride(0) if self.M > 1 else 2 * G

    def stats(self, is_layernorm, mean, rstd, save):
        if save:
            if rstd is None:
                rstd = torch.empty(self.M, device=self.dev, dtype=torch.float32)
            if is_layernorm and mean is None:
                mean = torch.empty(self.M, device=self.dev, dtype=torch.float32)
        return mean, rstd, self.vec("mean", mean, self.M, torch.float32), self.vec("rstd", rstd, self.M, torch.float32)

    def on_device(self, fn, *args):
        """fn(*args) with the tensors' device current."""
        if self.dev == torch.cuda.current_device():
            return fn(*args)
        with torch.cuda.device(self.dev):
            return fn(*args)

    def go(self, name, fn, args):
        """fn(*args, stream) with the tensors' device current, on its current stream."""
        _check(name, self.on_device(fn, *args, _raw_stream(self.dev)))


def _on_stream(f):
    """Adds the argument ``stream``: the call, and with it the allocation of its
    outputs and workspace, under that stream (a workspace of another stream's
    could be handed out again while the kernels still write to it).  A stream of
    another device than the tensors' is refused: the launch would go to that
    device's current stream instead."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        for t in (*args, *kw.values()):
            t = t.codes if isinstance(t, Checkpoint8) else t
            if isinstance(t, torch.Tensor) and t.get_device() != stream.device.index:
                raise ValueError(f"stream is one of {stream.device}, the tensors are on device {t.get_device()}")
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


def _float_code(name, dtype):
    if dtype not in DTYPE_CODE:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, not {dtype}")
    return DTYPE_CODE[dtype]


def _sum_rows(c, x, residual, store_h, h):
    """Pointers and strides of x, residual and h (allocated here where it is to be stored and not given)."""
    px, ldx = c.rows("x", x)
    pr, ldr = c.rows("residual", residual, x.dtype)
    if residual is not None and store_h and h is None:
        h = torch.empty(c.M, c.N, device=x.device, dtype=x.dtype)
    ph, ldh = c.rows("h", h, x.dtype)
    return h, (px, ldx, _float_code("x", x.dtype), pr, ldr, ph, ldh)


@_on_stream
def norm_fwd_q8(is_layernorm: bool, x, gamma, beta, eps: float, residual=None, store_h: bool = True,
                fmt=torch.float8_e4m3fn, group: int = 0, checkpoint: Checkpoint8 | None = None, q=None, scale=None,
                h=None, mean=None, rstd=None, save_stats: bool = True):
    """RMSNorm / LayerNorm of x (+ residual) with the output in 8 bits: codes q
    of dtype ``fmt`` (torch.float8_e4m3fn or torch.int8; q's own if q is given)
    and float32 scales [M, ceil(N / group)], one per ``group`` columns (32, 64,
    128, 256) or per row (0): the output is q * scale.  scale may be given in
    either order of strides.  checkpoint, if given, is filled with the 8-bit
    checkpoint of the normalised rows.  Returns (q, scale, h, mean, rstd); h
    (the stored residual sum) is None without a residual or with store_h
    False, mean None for RMSNorm."""
    c = _Call("x", x)
    if group != 0 and group not in GROUPS:
        raise ValueError(f"group must be 0 (a scale per row) or one of {GROUPS}")
    if q is None:
        q = torch.empty(c.M, c.N, device=x.device, dtype=fmt)
    if q.dtype not in Q8_CODE:
        raise ValueError("8-bit rows must be torch.float8_e4m3fn or torch.int8")
    if scale is None:
        scale = torch.empty(c.M, _groups(c.N, group), device=x.device, dtype=torch.float32)
    h, sums = _sum_rows(c, x, residual, store_h, h)
    par = c.params(gamma, beta, x.dtype)
    mean, rstd, pm, ps = c.stats(is_layernorm, mean, rstd, save_stats)
    c.go("norm_fwd_q8", lib.norm_fwd_q8,
         (int(bool(is_layernorm)), c.M, c.N, eps, *sums, *par, *c.rows("q", q), Q8_CODE[q.dtype], group,
          *c.scales("scale", scale, group), *c.checkpoint(checkpoint), pm, ps))
    return q, scale, h, mean, rstd


@_on_stream
def norm_fwd_ck8(is_layernorm: bool, x, gamma, beta, eps: float, residual=None, store_h: bool = True,
                 group: int = 128, checkpoint: Checkpoint8 | None = None, y_dtype=None, y=None, h=None, mean=None,
                 rstd=None):
    """norm_fwd_ex that also leaves an 8-bit checkpoint of the normalised rows
    for norm_bwd_ck8 (int8 codes about the middle of each group of ``group``
    columns; a checkpoint that is given keeps its own group).  Returns (y, h,
    checkpoint, mean, rstd)."""
    c = _Call("x", x)
    if checkpoint is None:
        checkpoint = checkpoint8_empty(c.M, c.N, group, x.device)
    if y is None:
        y = torch.empty(c.M, c.N, device=x.device, dtype=y_dtype or x.dtype)
    h, sums = _sum_rows(c, x, residual, store_h, h)
    par = c.params(gamma, beta, x.dtype)
    mean, rstd, pm, ps = c.stats(is_layernorm, mean, rstd, True)
    c.go("norm_fwd_ck8", lib.norm_fwd_ck8,
         (int(bool(is_layernorm)), c.M, c.N, eps, *sums, *par, *c.rows("y", y), _float_code("y", y.dtype),
          *c.checkpoint(checkpoint), pm, ps))
    return y, h, checkpoint, mean, rstd


def norm_bwd_ck8_workspace_size(is_layernorm: bool, M: int, N: int) -> int:
    return int(lib.norm_bwd_ck8_workspace_size(int(bool(is_layernorm)), M, N))


@_on_stream
def norm_bwd_ck8(is_layernorm: bool, dy, checkpoint: Checkpoint8, gamma, mean, rstd, dres=None, dx=None, dx_dtype=None,
                 dgamma=None, dbeta=None, workspace=None, need_dgamma: bool = True, need_dbeta: bool = True):
    """Backward of the norm from its 8-bit checkpoint and saved statistics; dres
    (dx's dtype) is added into dx.  Returns (dx, dgamma, dbeta): dx of dx_dtype
    (default dres's, else dy's), dgamma and dbeta in float32 (None where not
    needed; dbeta LayerNorm only)."""
    c = _Call("dy", dy)
    if dx is None:
        dt = dx_dtype or (dres.dtype if dres is not None else dy.dtype)
        dx = torch.empty(c.M, c.N, device=dy.device, dtype=dt)
    pdx, lddx = c.rows("dx", dx)
    pdr, lddr = c.rows("dres", dres, dx.dtype)
    if dgamma is None and need_dgamma:
        dgamma = torch.empty(c.N, device=dy.device, dtype=torch.float32)
    if not is_layernorm:
        dbeta = mean = None
    elif dbeta is None and need_dbeta:
        dbeta = torch.empty(c.N, device=dy.device, dtype=torch.float32)
    if rstd is None or (is_layernorm and mean is None):
        raise ValueError("rstd (and mean for LayerNorm) of the forward are needed")
    pg, _, pdt = c.params(gamma, None, dy.dtype)
    if workspace is None:
        need = c.on_device(lib.norm_bwd_ck8_workspace_size, int(bool(is_layernorm)), c.M, c.N)
        if need == 0:
            raise GbnormError("norm_bwd_ck8_workspace_size", 2)
        workspace = torch.empty(need, device=dy.device, dtype=torch.uint8)
    elif not workspace.is_contiguous() or workspace.get_device() != c.dev:
        raise ValueError(f"workspace must be contiguous on device {c.dev}")
    c.go("norm_bwd_ck8", lib.norm_bwd_ck8,
         (int(bool(is_layernorm)), c.M, c.N, *c.rows("dy", dy), _float_code("dy", dy.dtype),
          *c.checkpoint(checkpoint), pdr, lddr, pg, pdt, c.vec("mean", mean, c.M, torch.float32),
          c.vec("rstd", rstd, c.M, torch.float32), pdx, lddx, _float_code("dx", dx.dtype),
          c.vec("dgamma", dgamma, c.N, torch.float32), c.vec("dbeta", dbeta, c.N, torch.float32),
          workspace.data_ptr(), workspace.numel() * workspace.element_size()))
    return dx, dgamma, dbeta


def _read(c, pq, ldq, code, group, scale, mid, mean, rstd, gamma, beta, y_dtype, y, like):
    if y is None:
        y = torch.empty(c.M, c.N, device=like.device, dtype=y_dtype)
    pg, pb, pdt = c.params(gamma, beta, torch.float32)
    c.go("q8_read", lib.q8_read,
         (c.M, c.N, pq, ldq, code, group, scale[0], mid, scale[1], scale[2], c.vec("mean", mean, c.M, torch.float32),
          c.vec("rstd", rstd, c.M, torch.float32), pg, pb, pdt, *c.rows("y", y), _float_code("y", y.dtype)))
    return y


@_on_stream
def read_q8(q, scale, group: int = 0, mean=None, rstd=None, gamma=None, beta=None, y_dtype=torch.bfloat16, y=None):
    """8-bit rows read back: ((q * scale - mean) * rstd) * gamma + beta in
    y_dtype, with what is None left out."""
    c = _Call("q", q)
    if q.dtype not in Q8_CODE:
        raise ValueError("8-bit rows must be torch.float8_e4m3fn or torch.int8")
    if group != 0 and group not in GROUPS:
        raise ValueError(f"group must be 0 (a scale per row) or one of {GROUPS}")
    return _read(c, *c.rows("q", q), Q8_CODE[q.dtype], group, c.scales("scale", scale, group), None, mean, rstd, gamma,
                 beta, y_dtype, y, q)


@_on_stream
def read_ck8(checkpoint: Checkpoint8, mean=None, rstd=None, gamma=None, beta=None, y_dtype=torch.bfloat16, y=None):
    """A checkpoint read back: the rows it stands for, or, given the saved
    statistics (and gamma, beta), the norm's output computed again from them."""
    c = _Call("checkpoint codes", checkpoint.codes)
    pc, ldc, group, ps, lds = c.checkpoint(checkpoint)
    return _read(c, pc, ldc, Q8_CODE[torch.int8], group, (ps, lds, 2), ps + 4 if ps else None, mean, rstd, gamma, beta,
                 y_dtype, y, checkpoint.codes)


def q8_last_variant(what: int) -> str:
    """The kernel this thread's last 8-bit forward (0), backward (1) or read (2) launched ("" for none)."""
    buf = ctypes.create_string_buffer(64)
    _check("gbnorm_q8_last_variant", lib.gbnorm_q8_last_variant(what, buf, 64))
    return buf.value.decode()
