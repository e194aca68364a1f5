"""Binding of the head operators (qk_norm_rope_fwd, qk_norm_rope_bwd, rope_fwd
and rope_bwd of include/gbnorm.h).

Argument marshalling only, as in ``binding``: tensors are checked, outputs that
the caller does not pass are allocated with torch's caching allocator, and the
call goes to the C ABI on torch's current stream of the tensors' device, or on
the one given as the keyword ``stream``, which every operator takes.

Queries and keys are [tokens, heads, D] or [batches, tokens, heads, D] with any
strides but the last, which is 1: parts of a packed projection, or tensors with
heads outside tokens (transposed).  Positions are int32 or int64, one for each
token ([tokens], or [batches, tokens] or [tokens] with batches); with several
axes these come first ([axes, tokens], [axes, batches, tokens]).
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from .binding import DTYPE_CODE, GbnormError, _check, _f, _int, _i64, _sz, _vp, lib
from .q8 import _on_stream, _raw_stream

lib.qk_norm_rope_fwd.argtypes = [_int, _f, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.qk_norm_rope_bwd_workspace_size.argtypes = [_int, _i64, _i64, _i64, _i64]
lib.qk_norm_rope_bwd_workspace_size.restype = _sz
lib.qk_norm_rope_bwd.argtypes = [_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
lib.rope_fwd.argtypes = lib.rope_bwd.argtypes = [_vp, _vp, _vp, _vp]
lib.gbnorm_rope_last_variant.argtypes = [_int, ctypes.c_char_p, _sz]
for _fn in ("qk_norm_rope_fwd", "qk_norm_rope_bwd", "rope_fwd", "rope_bwd", "gbnorm_rope_last_variant"):
    getattr(lib, _fn).restype = _int

MAX_AXES = 4
_HEADS = struct.Struct("8q").pack    # two gbnorm_heads_t
_ROPE = struct.Struct("5q8i6q").pack  # gbnorm_rope_t
_TWO = struct.Struct("2q").pack
_CONTIGUOUS = torch.contiguous_format
_POS_CODE = {torch.int32: 0, torch.int64: 1}


class Rotary:
    """The rotation of a model's heads, made once (see ``rotary``): float32
    frequencies on the device, the pairing, and the axis of each pair."""

    __slots__ = ("inv_freq", "interleaved", "axes", "rot", "dev", "pair_axis", "_axis_at")

    def __init__(self, inv_freq, interleaved, axes, pair_axis):
        self.inv_freq, self.interleaved, self.axes = inv_freq, bool(interleaved), axes
        self.rot, self.dev = 2 * inv_freq.numel(), inv_freq.get_device()
        self.pair_axis = pair_axis
        self._axis_at = ctypes.addressof(pair_axis) if pair_axis is not None else 0


def rotary(inv_freq, interleaved: bool = False, sections=None, pair_axis=None) -> Rotary:
    """A rotation of 2 len(inv_freq) elements of each head: pair j turns by
    position * inv_freq[j] radians (float32, on the GPU; kept, not copied).
    Pairs are (j, j + len(inv_freq)), or (2 j, 2 j + 1) where interleaved.  With
    several position axes, sections gives the number of consecutive pairs that
    follow each axis, or pair_axis the axis of every pair."""
    if not (isinstance(inv_freq, torch.Tensor) and inv_freq.is_cuda and inv_freq.dim() == 1 and inv_freq.numel() > 0
            and inv_freq.dtype == torch.float32 and inv_freq.is_contiguous()):
        raise ValueError("inv_freq must be a contiguous 1-D float32 CUDA tensor with at least one element")
    n = inv_freq.numel()
    if sections is not None and pair_axis is not None:
        raise ValueError("give sections or pair_axis, not both")
    if sections is not None:
        sections = [int(w) for w in sections]
        if not sections or min(sections) < 0 or sum(sections) != n:
            raise ValueError(f"sections must be numbers of pairs that sum to {n}")
        pair_axis, axes = [a for a, w in enumerate(sections) for _ in range(w)], len(sections)
    elif pair_axis is not None:
        pair_axis = [int(a) for a in pair_axis]
        if len(pair_axis) != n or min(pair_axis) < 0:
            raise ValueError(f"pair_axis must be an axis for each of the {n} pairs")
        axes = max(pair_axis) + 1
    else:
        axes = 1
    if axes > MAX_AXES:
        raise ValueError(f"at most {MAX_AXES} axes")
    return Rotary(inv_freq, interleaved, axes, (ctypes.c_uint8 * n)(*pair_axis) if axes > 1 else None)


class _Call:
    """Checks of one call's tensors against its first one (the queries), and its launch on that one's device."""

    __slots__ = ("dev", "q", "k", "B", "S", "D", "hq", "hk")

    def __init__(self, name, q, k):
        self.q = shape = q.shape
        n = len(shape)
        self.dev = q.get_device()
        if n == 3:
            self.B = 1
            self.S, self.hq, self.D = shape
        elif n == 4:
            self.B, self.S, self.hq, self.D = shape
        if not q.is_cuda or self.dev < 0 or n not in (3, 4):
            raise ValueError(f"{name}q must be a CUDA tensor [tokens, heads, D] or [batches, tokens, heads, D]")
        self.k, self.hk = None, 0
        if k is not None:
            self.k = kshape = k.shape
            if len(kshape) != n or kshape[-1] != self.D or kshape[:-2] != shape[:-2]:
                raise ValueError(f"{name}k must have the batches, tokens and head size of {name}q")
            self.hk = kshape[-2]
            if self.hk == 0:
                raise ValueError("keys without heads are given as None")

    def heads(self, name, q, k, dtype):
        """Two gbnorm_heads_t."""
        if self.k is None:
            if k is not None:
                raise ValueError(f"{name}k is given without k")
            return _HEADS(*self._one(name + "q", q, self.q, dtype), 0, 0, 0, 0)
        return _HEADS(*self._one(name + "q", q, self.q, dtype), *self._one(name + "k", k, self.k, dtype))

    def _one(self, name, t, shape, dtype):
        if t is None or t.shape != shape or t.get_device() != self.dev:
            raise ValueError(f"{name} must be a {list(shape)} CUDA tensor on device {self.dev}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must have dtype {dtype}")
        st = t.stride()
        if len(st) == 3:
            token, head, one = st
            batch = 0
        else:
            batch, token, head, one = st
        if one != 1 and self.D > 1:
            raise ValueError(f"{name} must have unit stride in its last dimension")
        return t.data_ptr(), batch, token, head

    def out(self, name, yq, yk, q, k, dtype):
        """The two outputs, allocated where they are not given, and their gbnorm_heads_t."""
        if k is None and yk is not None:
            raise ValueError(f"{name}k is given without k")
        if yq is not None or yk is not None:
            if yq is None:
                yq = torch.empty_like(q, dtype=dtype, memory_format=_CONTIGUOUS)
            if yk is None and k is not None:
                yk = torch.empty_like(k, dtype=dtype, memory_format=_CONTIGUOUS)
            return yq, yk, self.heads(name, yq, yk, dtype)
        D, tq, tk = self.D, self.hq * self.D, self.hk * self.D
        yq = torch.empty_like(q, dtype=dtype, memory_format=_CONTIGUOUS)
        if k is None:
            return yq, None, _HEADS(yq.data_ptr(), self.S * tq, tq, D, 0, 0, 0, 0)
        yk = torch.empty_like(k, dtype=dtype, memory_format=_CONTIGUOUS)
        return yq, yk, _HEADS(yq.data_ptr(), self.S * tq, tq, D, yk.data_ptr(), self.S * tk, tk, D)

    def sums(self, name, t, shape, needed):
        """A float32 output, allocated where it is needed and not given, and its pointer."""
        if t is not None:
            return t, self.flat(name, t, shape)
        if not needed:
            return None, None
        t = torch.empty(shape, dtype=torch.float32, device=self.dev)
        return t, t.data_ptr()

    def pair(self, name, q, k, dtype):
        """Two pointers to [D] parameters."""
        if q is None and k is None:
            return None
        for w, t in (("q", q), ("k", k)):
            if t is not None and (t.shape != (self.D,) or t.get_device() != self.dev or t.dtype != dtype
                                  or not t.is_contiguous()):
                raise ValueError(f"{name}_{w} must be a contiguous 1-D CUDA {dtype} tensor of {self.D} elements on "
                                 f"device {self.dev}")
        return _TWO(0 if q is None else q.data_ptr(), 0 if k is None else k.data_ptr())

    def flat(self, name, t, shape):
        if t is None:
            return None
        if t.shape != shape or t.get_device() != self.dev or t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {list(shape)} float32 CUDA tensor on device {self.dev}")
        return t.data_ptr()

    def stats_shape(self):
        return (*self.q[:-2], self.hq + self.hk)

    def rope(self, positions, rotary, xdt, ydt, pdt):
        """gbnorm_rope_t."""
        try:
            xdt, ydt, pdt = DTYPE_CODE[xdt], DTYPE_CODE[ydt], DTYPE_CODE[pdt]
        except KeyError:
            raise ValueError(f"tensors must be float32, float16 or bfloat16, not {xdt}, {ydt}, {pdt}") from None
        if rotary is None:
            if positions is not None:
                raise ValueError("positions without a rotation")
            return _ROPE(self.B, self.S, self.hq, self.hk, self.D, xdt, ydt, pdt, 0, 0, 1, 0, 0, 0, 0, 0, 0, 0, 0)
        if rotary.rot > self.D:
            raise ValueError(f"{rotary.rot} rotated elements in heads of {self.D}")
        if positions is None or positions.get_device() != self.dev or rotary.dev != self.dev:
            raise ValueError(f"positions and frequencies must be on device {self.dev}")
        code = _POS_CODE.get(positions.dtype)
        if code is None:
            raise ValueError("positions must be int32 or int64")
        shape, st, axis = positions.shape, positions.stride(), 0
        if rotary.axes > 1:
            if not shape or shape[0] != rotary.axes:
                raise ValueError(f"positions must have {rotary.axes} axes first")
            shape, axis, st = shape[1:], st[0], st[1:]
        if len(shape) == 1 and shape[0] == self.S:
            batch, token = 0, st[0]
        elif len(self.q) == 4 and len(shape) == 2 and shape[0] == self.B and shape[1] == self.S:
            batch, token = st
        else:
            raise ValueError(f"positions must have one value for each of the tokens {list(self.q[:-2])}")
        return _ROPE(self.B, self.S, self.hq, self.hk, self.D, xdt, ydt, pdt, rotary.interleaved, rotary.rot,
                     rotary.axes, code, 0, positions.data_ptr(), axis, batch, token, rotary.inv_freq.data_ptr(),
                     rotary._axis_at)

    def go(self, name, fn, *args):
        """fn(*args, stream) with the tensors' device current, on its current stream."""
        if self.dev == torch.cuda.current_device():
            status = fn(*args, _raw_stream(self.dev))
        else:
            with torch.cuda.device(self.dev):
                status = fn(*args, _raw_stream(self.dev))
        if status:
            _check(name, status)


def _out_dtype(name, out, dtype, default):
    """The type of an output: its own where it is given, which the argument may not contradict."""
    if out is None:
        return dtype or default
    if dtype is not None and out.dtype != dtype:
        raise ValueError(f"{name} has dtype {out.dtype}, not the {dtype} asked for")
    return out.dtype


def _param_dtype(default, *params):
    for t in params:
        if t is not None:
            return t.dtype
    return default


def qk_norm_rope_fwd(is_layernorm: bool, q, k, gamma_q, gamma_k, eps: float, positions=None,
                     rotary: Rotary | None = None, beta_q=None, beta_k=None, y_dtype=None, yq=None, yk=None, mean=None,
                     rstd=None, save_stats: bool = True, stream=None):
    """Each head of the queries q and keys k (None: queries alone) normalised
    by itself (gamma, beta of D elements, None: 1, 0; all of one dtype), then
    rotated by its token's position (rotary None: the norm alone).  Returns
    (yq, yk, mean, rstd): outputs of y_dtype (default q's) with q's and k's
    shapes; mean and rstd float32 [..., heads of q and of k], mean None for
    RMSNorm, both None without save_stats unless given.  yq may be q itself
    and yk k itself.  Without k, gamma_k and beta_k (a layer's) are not read, yk is refused."""
    if stream is not None:
        return _on_stream(qk_norm_rope_fwd)(is_layernorm, q, k, gamma_q, gamma_k, eps, positions, rotary, beta_q,
                                            beta_k, y_dtype, yq, yk, mean, rstd, save_stats, stream=stream)
    c = _Call("", q, k)
    dt = _out_dtype("yq", yq, y_dtype, q.dtype)
    if not is_layernorm:
        mean = beta_q = beta_k = None
    pdt = _param_dtype(q.dtype, gamma_q, gamma_k, beta_q, beta_k)
    r, x = c.rope(positions, rotary, q.dtype, dt, pdt), c.heads("", q, k, q.dtype)
    yq, yk, y = c.out("y", yq, yk, q, k, dt)
    stats = c.stats_shape()
    rstd, ps = c.sums("rstd", rstd, stats, save_stats)
    mean, pm = c.sums("mean", mean, stats, save_stats and is_layernorm)
    c.go("qk_norm_rope_fwd", lib.qk_norm_rope_fwd, int(bool(is_layernorm)), eps, r, x, y,
         c.pair("gamma", gamma_q, gamma_k, pdt), c.pair("beta", beta_q, beta_k, pdt), pm, ps)
    return yq, yk, mean, rstd


def qk_norm_rope_bwd_workspace_size(is_layernorm: bool, tokens: int, heads_q: int, heads_k: int, dim: int) -> int:
    return int(lib.qk_norm_rope_bwd_workspace_size(int(bool(is_layernorm)), tokens, heads_q, heads_k, dim))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(ln, tokens, heads_q, heads_k, dim, dev):
    """A function of the shape and the device alone."""
    with torch.cuda.device(dev):
        need = lib.qk_norm_rope_bwd_workspace_size(ln, tokens, heads_q, heads_k, dim)
    if need == 0:
        raise GbnormError("qk_norm_rope_bwd_workspace_size", 2)
    return need


def qk_norm_rope_bwd(is_layernorm: bool, dyq, dyk, q, k, gamma_q, gamma_k, mean, rstd, positions=None,
                     rotary: Rotary | None = None, dq=None, dk=None, dgamma=None, dbeta=None, workspace=None,
                     need_dgamma: bool = True, need_dbeta: bool = True, stream=None):
    """Backward of qk_norm_rope_fwd from its inputs q and k and its saved
    statistics.  Returns (dq, dk, dgamma, dbeta): dq and dk of q's dtype, dgamma
    and dbeta float32 [2, D] (queries, keys; [1, D] without keys), None where not
    needed, dbeta LayerNorm only.  dq may be dyq itself and dk dyk itself.
    Without k, gamma_k is not read, dyk and dk are refused."""
    if stream is not None:
        return _on_stream(qk_norm_rope_bwd)(is_layernorm, dyq, dyk, q, k, gamma_q, gamma_k, mean, rstd, positions,
                                            rotary, dq, dk, dgamma, dbeta, workspace, need_dgamma, need_dbeta,
                                            stream=stream)
    c = _Call("", q, k)
    dt = q.dtype
    if not is_layernorm:
        dbeta, mean, need_dbeta = None, None, False
    if rstd is None or (is_layernorm and mean is None):
        raise ValueError("rstd (and mean for LayerNorm) of the forward are needed")
    pdt = _param_dtype(dt, gamma_q, gamma_k)
    r, dy, x = c.rope(positions, rotary, dt, dyq.dtype, pdt), c.heads("dy", dyq, dyk, dyq.dtype), c.heads("", q, k, dt)
    dq, dk, dx = c.out("d", dq, dk, q, k, dt)
    sums, stats = (2 if c.hk else 1, c.D), c.stats_shape()
    dgamma, pg = c.sums("dgamma", dgamma, sums, need_dgamma)
    dbeta, pb = c.sums("dbeta", dbeta, sums, need_dbeta)
    if workspace is None:
        workspace = torch.empty(_workspace_bytes(int(bool(is_layernorm)), c.B * c.S, c.hq, c.hk, c.D, c.dev),
                                dtype=torch.uint8, device=c.dev)
    elif not workspace.is_contiguous() or workspace.get_device() != c.dev:
        raise ValueError(f"workspace must be contiguous on device {c.dev}")
    c.go("qk_norm_rope_bwd", lib.qk_norm_rope_bwd, int(bool(is_layernorm)), r, dy, x, dx,
         c.pair("gamma", gamma_q, gamma_k, pdt), c.flat("mean", mean, stats), c.flat("rstd", rstd, stats), pg, pb,
         workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return dq, dk, dgamma, dbeta


def rope_fwd(q, k, positions, rotary: Rotary, y_dtype=None, yq=None, yk=None, stream=None):
    """The heads of q and k (None: of q alone) rotated by their tokens'
    positions.  Returns (yq, yk) of y_dtype (default q's); yq may be q itself
    and yk k itself."""
    if stream is not None:
        return _on_stream(rope_fwd)(q, k, positions, rotary, y_dtype, yq, yk, stream=stream)
    c = _Call("", q, k)
    dt = _out_dtype("yq", yq, y_dtype, q.dtype)
    if rotary is None:
        raise ValueError("rotary is needed")
    r, x = c.rope(positions, rotary, q.dtype, dt, q.dtype), c.heads("", q, k, q.dtype)
    yq, yk, y = c.out("y", yq, yk, q, k, dt)
    c.go("rope_fwd", lib.rope_fwd, r, x, y)
    return yq, yk


def rope_bwd(dyq, dyk, positions, rotary: Rotary, dx_dtype=None, dq=None, dk=None, stream=None):
    """Backward of rope_fwd: gradients turned back.  Returns (dq, dk) of
    dx_dtype (default dyq's); dq may be dyq itself and dk dyk itself."""
    if stream is not None:
        return _on_stream(rope_bwd)(dyq, dyk, positions, rotary, dx_dtype, dq, dk, stream=stream)
    c = _Call("dy", dyq, dyk)
    dt = _out_dtype("dq", dq, dx_dtype, dyq.dtype)
    if rotary is None:
        raise ValueError("rotary is needed")
    r, dy = c.rope(positions, rotary, dt, dyq.dtype, dyq.dtype), c.heads("dy", dyq, dyk, dyq.dtype)
    dq, dk, dx = c.out("d", dq, dk, dyq, dyk, dt)
    c.go("rope_bwd", lib.rope_bwd, r, dy, dx)
    return dq, dk


def rope_last_variant(what: int) -> str:
    """The kernel this thread's last qk_norm_rope_fwd (0), qk_norm_rope_bwd (1) or rotation (2) launched ("" for none)."""
    buf = ctypes.create_string_buffer(64)
    _check("gbnorm_rope_last_variant", lib.gbnorm_rope_last_variant(what, buf, 64))
    return buf.value.decode()
