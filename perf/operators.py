"""Cases of the 8-bit operators: a norm whose output is written in 8 bits with
scales, a norm that leaves an 8-bit checkpoint of its input behind, the
backward pass from that checkpoint, and the reading back of 8-bit rows.

Each operator has its plain form in elementary torch operations (32 bits,
rounded once at the end), the call a user makes of the library (where `own` is
true), and its definition in 64 bits (`exact`).

What is stored in 8 bits:

  output rows   one scale for `group` consecutive columns (group 0: the row),
                scale = max|y| / 448 (e4m3) or / 127 (int8), code = y / scale
                rounded to nearest even.  A group whose values all lie below
                2^-100 has scale 0 and codes 0.
  checkpoint    int8 about the middle of each group's range: mid = max / 2 +
                min / 2, half = max(max - mid, mid - min), scale = half / 127,
                code = rint((h - mid) * (1 / scale)), every step in fp32, so
                that the codes are a function of the stored rows alone.
                half < 2^-100: scale 0, codes 0.
"""
import math

import torch

own = False

EPS = 1e-6
TINY = 2.0 ** -100
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
QMAX = {"e4m3": 448.0, "int8": 127.0}


def _lib():
    import rmsnorm_norm_fwd_gb300
    return rmsnorm_norm_fwd_gb300


# ------------------------------------------------------------------ cases
def _case(name, kind, m, n, ln=False, dtype="bf16", param=None, residual=False, fmt="e4m3", group=0):
    return {"name": name, "kind": kind, "m": m, "n": n, "ln": ln, "dtype": dtype, "param": param or dtype,
            "residual": residual, "fmt": fmt, "group": group}


def listed():
    return [
        # One token of a decoder: latency alone.
        _case("q8 token 1x4096", "q8", 1, 4096, residual=True),
        # A decoding batch, one scale per 128 columns for a block-scaled product.
        _case("q8 batch 48x8192 g128", "q8", 48, 8192, residual=True, group=128),
        # A prefill: residual stream in and out, rows in 8 bits for the next product.
        _case("q8 prefill 16384x8192", "q8", 16384, 8192, residual=True),
        # LayerNorm in fp16 with a row count that divides nothing.
        _case("q8 ln 4111x5120 g128", "q8", 4111, 5120, ln=True, dtype="fp16", group=128),
        # int8 rows written and read back to bf16 for a consumer without 8-bit products.
        _case("q8 int8 there and back 16384x4096", "q8", 16384, 4096, fmt="int8"),
        # Odd rows, no 16-byte vectors anywhere, fp32.
        _case("q8 odd 8191x1003", "q8", 8191, 1003, ln=True, dtype="fp32"),
        # Rows wider than one SM keeps in registers.
        _case("q8 wide 1024x65536 g128", "q8", 1024, 65536, group=128),
        # The forward of a training step: output for the next product, checkpoint
        # for the backward, read back here as what it stands for.
        _case("ck8 forward 16384x4096", "ck8_fwd", 16384, 4096, residual=True, group=128),
        # The backward from a checkpoint, with the residual stream's gradient.
        _case("ck8 backward 16384x8192", "ck8_bwd", 16384, 8192, residual=True, group=128),
        # The same for LayerNorm, both parameter gradients, fp32 parameters.
        _case("ck8 backward ln 16384x4096", "ck8_bwd", 16384, 4096, ln=True, param="fp32", group=128),
        # Forward and backward of a small batch: launches count.
        _case("ck8 step 512x2048", "ck8_step", 512, 2048, ln=True, residual=True, group=64),
        # The norm's output computed again from the checkpoint, for the gradient of
        # the weights that read it.
        _case("read norm 65536x2048", "read", 65536, 2048, group=128),
    ]


def draw(rng):
    kind = rng.choice(["q8", "q8", "ck8_fwd", "ck8_bwd", "ck8_step", "read"])
    n = int(round(math.exp(rng.uniform(math.log(96), math.log(70000)))))
    n = rng.choice([n, n // 8 * 8, -(-n // 128) * 128, -(-n // 128) * 128])
    m = int(round(math.exp(rng.uniform(0.0, math.log(70000)))))
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    c = {"kind": kind, "m": m, "n": n, "ln": rng.random() < 0.5, "dtype": dtype,
         "param": rng.choice([dtype, dtype, "fp32"]), "residual": rng.random() < 0.5,
         "fmt": rng.choice(["e4m3", "e4m3", "int8"]),
         "group": rng.choice([32, 64, 128, 128, 256] + ([0, 0, 0] if kind == "q8" else []))}
    most = max(work(x)["bytes"] for x in listed())
    c["m"] = max(1, min(m, int(m * 0.9 * most / work(c)["bytes"])))
    return c


def _groups(c):
    return -(-c["n"] // c["group"]) if c["group"] else 1


def work(c):
    """Each input read once, each output written once."""
    m, n, b, k = c["m"], c["n"], SIZE[c["dtype"]], c["kind"]
    mn, r, g = m * n, 1 if c["residual"] else 0, _groups(c)
    par = n * SIZE[c["param"]] * (2 if c["ln"] else 1)
    stat = 4 * m * (2 if c["ln"] else 1)
    fwd_in = mn * b * (1 + 2 * r) + par + stat  # x, the residual, h
    back = mn * b * (2 + r) + mn + 8 * m * g + n * SIZE[c["param"]] + stat + 4 * n * (2 if c["ln"] else 1)
    if k == "q8":
        total = fwd_in + mn + 4 * m * g + (mn * 3 + 4 * m * g if c["fmt"] == "int8" else 0)
        return {"bytes": total, "flops": 12 * mn}
    if k == "ck8_fwd":  # y, the codes, and their values in 16 bits
        return {"bytes": fwd_in + mn * b + mn + 8 * m * g + mn * 3 + 8 * m * g, "flops": 16 * mn}
    if k == "ck8_bwd":
        return {"bytes": back, "flops": 16 * mn}
    if k == "ck8_step":
        return {"bytes": fwd_in + mn * b + mn + 8 * m * g + back, "flops": 30 * mn}
    return {"bytes": mn + 8 * m * g + mn * b + par + stat, "flops": 6 * mn}


# ------------------------------------------------------------------ inputs
def _rows(gen, m, n, dt, shift):
    """Activations: unit rows about `shift`, a hundredth of them 100 times larger, some single
    large values, and a padded row of zeros among each few hundred."""
    x = torch.randn(m, n, device="cuda", generator=gen).add_(shift)
    far = torch.rand(m, 1, device="cuda", generator=gen)
    x = torch.where(far < 0.01, x * 100, x)
    at = torch.randint(0, m * n, (max(1, m * n // 1000),), device="cuda", generator=gen)
    x.view(-1)[at] = 60.0
    x = torch.where(far > 0.996, torch.zeros_like(x), x)
    return x.to(dt)


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    m, n, dt, pt, k = c["m"], c["n"], DTYPE[c["dtype"]], DTYPE[c["param"]], c["kind"]
    s = {"case": c, "group": c["group"]}
    x = _rows(gen, m, n, dt, 0.5 if c["ln"] else 0.0)
    s["gamma"] = (1 + 0.1 * torch.randn(n, device="cuda", generator=gen)).to(pt)
    s["beta"] = (0.1 * torch.randn(n, device="cuda", generator=gen)).to(pt) if c["ln"] else None
    if k in ("q8", "ck8_fwd", "ck8_step"):
        s["x"] = x
        s["residual"] = torch.randn(m, n, device="cuda", generator=gen).to(dt) if c["residual"] else None
    if k in ("ck8_bwd", "read"):  # what the forward left
        h = x.float()
        s["mean"] = h.mean(1) if c["ln"] else None
        d = h - s["mean"][:, None] if c["ln"] else h
        s["rstd"] = torch.rsqrt(d.square().mean(1) + EPS)
        s["codes"], s["scales"] = _checkpoint(h, c["group"])
    if k in ("ck8_bwd", "ck8_step"):
        s["dy"] = torch.randn(m, n, device="cuda", generator=gen).to(dt)
        s["dres"] = torch.randn(m, n, device="cuda", generator=gen).to(dt) if c["residual"] else None
    if k == "q8":  # a server keeps its buffers
        f32 = {"device": "cuda", "dtype": torch.float32}
        s["q"] = torch.empty(m, n, device="cuda", dtype=torch.int8 if c["fmt"] == "int8" else torch.float8_e4m3fn)
        s["scale"] = torch.empty(m, _groups(c), **f32)
        s["h"] = torch.empty_like(x) if c["residual"] else None
        s["m"] = torch.empty(m, **f32) if c["ln"] else None
        s["r"] = torch.empty(m, **f32)
    return s


# ------------------------------------------------------------------ plain forms
def _grouped(v, group, fill):
    """[M, N] as [M, G, group], the last group filled up."""
    m, n = v.shape
    group = group or n
    g = -(-n // group)
    if g * group != n:
        v = torch.cat([v, fill.expand(m, g * group - n)], 1)
    return v.reshape(m, g, group)


def _spread(s, group, n):
    """[M, G] to [M, N]."""
    return s.repeat_interleave(group or n, 1)[:, :n]


def _checkpoint(h, group):
    n = h.shape[1]
    v = _grouped(h, group, h[:, -1:])
    top, low = v.amax(2), v.amin(2)
    mid = top * 0.5 + low * 0.5
    half = torch.maximum(top - mid, mid - low)
    scale = torch.where(half < TINY, torch.zeros_like(half), half / torch.full_like(half, 127.0))
    inv = torch.where(half < TINY, torch.zeros_like(half), torch.ones_like(scale) / scale)
    codes = torch.round((h - _spread(mid, group, n)) * _spread(inv, group, n))
    return codes.to(torch.int8), torch.stack([scale, mid], 2)


def _values(codes, scales, group):
    n = codes.shape[1]
    return _spread(scales[..., 1], group, n) + _spread(scales[..., 0], group, n) * codes.float()


def _norm(s, ln, x, residual):
    """h in its type, mean, rstd and y in 32 bits."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    v = h.float()
    mean = v.mean(1, keepdim=True) if ln else None
    d = v - mean if ln else v
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    y = d * rstd * s["gamma"].float()
    if ln:
        y = y + s["beta"].float()
    return h, mean, rstd, y


def _plain_q8(s):
    c = s["case"]
    h, mean, rstd, y = _norm(s, c["ln"], s["x"], s["residual"])
    amax = _grouped(y.abs(), c["group"], y.new_zeros(1, 1)).amax(2)
    small = amax < TINY
    scale = torch.where(small, torch.zeros_like(amax), amax / QMAX[c["fmt"]])
    u = y * _spread(torch.where(small, torch.zeros_like(amax), QMAX[c["fmt"]] / amax), c["group"], c["n"])
    out = {"scale": scale, "rstd": rstd[:, 0]}
    if c["fmt"] == "int8":
        out["values"] = (torch.round(u) * _spread(scale, c["group"], c["n"])).to(torch.bfloat16)
    else:
        out["codes"] = u.to(torch.float8_e4m3fn)
    if c["ln"]:
        out["mean"] = mean[:, 0]
    if c["residual"]:
        out["h"] = h
    return out


def _plain_forward(s):
    """y, h, the checkpoint and the statistics of a training forward."""
    c = s["case"]
    h, mean, rstd, y = _norm(s, c["ln"], s["x"], s["residual"])
    codes, scales = _checkpoint(h.float(), c["group"])
    return y.to(h.dtype), h, codes, scales, mean[:, 0] if c["ln"] else None, rstd[:, 0]


def _plain_backward(s, codes, scales, mean, rstd):
    c = s["case"]
    v = _values(codes, scales, c["group"])
    if c["ln"]:
        v = v - mean[:, None]
    xhat = v * rstd[:, None]
    dy = s["dy"].float()
    g = dy * s["gamma"].float()
    dx = g - xhat * (g * xhat).mean(1, keepdim=True)
    if c["ln"]:
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * rstd[:, None]
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    out = {"dx": dx.to(s["dy"].dtype), "dgamma": (dy * xhat).sum(0)}
    if c["ln"]:
        out["dbeta"] = dy.sum(0)
    return out


def _named(y, h, mean, rstd, c):
    out = {"y": y, "rstd": rstd}
    if c["ln"]:
        out["mean"] = mean
    if c["residual"]:
        out["h"] = h
    return out


def _plain(s):
    c = s["case"]
    if c["kind"] == "q8":
        return _plain_q8(s)
    if c["kind"] == "ck8_fwd":
        y, h, codes, scales, mean, rstd = _plain_forward(s)
        return {**_named(y, h, mean, rstd, c), "scales": scales,
                "values": _values(codes, scales, c["group"]).to(torch.bfloat16)}
    if c["kind"] == "ck8_bwd":
        return _plain_backward(s, s["codes"], s["scales"], s["mean"], s["rstd"])
    if c["kind"] == "ck8_step":
        y, h, codes, scales, mean, rstd = _plain_forward(s)
        return {**_named(y, h, mean, rstd, c), **_plain_backward(s, codes, scales, mean, rstd)}
    v = _values(s["codes"], s["scales"], c["group"])
    if c["ln"]:
        v = v - s["mean"][:, None]
    y = v * s["rstd"][:, None] * s["gamma"].float()
    if c["ln"]:
        y = y + s["beta"].float()
    return {"y": y.to(DTYPE[c["dtype"]])}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    g, c = _lib(), s["case"]
    k, ln = c["kind"], c["ln"]
    if k == "q8":
        q, scale, h, mean, rstd = g.norm_fwd_q8(ln, s["x"], s["gamma"], s["beta"], EPS, residual=s["residual"],
                                                group=c["group"], q=s["q"], scale=s["scale"], h=s["h"],
                                                mean=s["m"], rstd=s["r"])
        out = {"scale": scale, "rstd": rstd}
        if c["fmt"] == "int8":
            out["values"] = g.read_q8(q, scale, group=c["group"], y_dtype=torch.bfloat16)
        else:
            out["codes"] = q
        if ln:
            out["mean"] = mean
        if c["residual"]:
            out["h"] = h
        return out
    if k in ("ck8_fwd", "ck8_step"):
        y, h, ck, mean, rstd = g.norm_fwd_ck8(ln, s["x"], s["gamma"], s["beta"], EPS, residual=s["residual"],
                                              group=c["group"])
        out = _named(y, h, mean, rstd, c)
        if k == "ck8_fwd":
            return {**out, "scales": ck.scales, "values": g.read_ck8(ck, y_dtype=torch.bfloat16)}
        dx, dgamma, dbeta = g.norm_bwd_ck8(ln, s["dy"], ck, s["gamma"], mean, rstd, dres=s["dres"])
    else:
        ck = g.Checkpoint8(s["codes"], s["scales"], c["group"])
        if k == "read":
            return {"y": g.read_ck8(ck, mean=s["mean"], rstd=s["rstd"], gamma=s["gamma"], beta=s["beta"],
                                    y_dtype=DTYPE[c["dtype"]])}
        out = {}
        dx, dgamma, dbeta = g.norm_bwd_ck8(ln, s["dy"], ck, s["gamma"], s["mean"], s["rstd"], dres=s["dres"])
    out.update(dx=dx, dgamma=dgamma)
    if ln:
        out["dbeta"] = dbeta
    return out


def run(s):
    return _own(s) if own else _plain(s)


# ------------------------------------------------------------------ in 64 bits
def _e4m3(v):
    """To the nearest e4m3 value, ties to even; |v| <= 448."""
    e = torch.frexp(v)[1].clamp(min=-5).to(torch.float64) - 4
    return torch.round(v * torch.exp2(-e)) * torch.exp2(e)


def _by_group(v, group, step):
    """`step` for each block of columns, put side by side."""
    return [step(b) for b in torch.split(v, group or v.shape[1], 1)]


def _exact_norm(s, c):
    x = s["x"].double()
    if s["residual"] is not None:  # the sum of two values of a type, rounded once to that type
        x = (s["x"].float() + s["residual"].float()).to(s["x"].dtype).double()
    mean = x.sum(1, keepdim=True) / c["n"] if c["ln"] else torch.zeros_like(x[:, :1])
    var = ((x - mean) ** 2).sum(1, keepdim=True) / c["n"]
    rstd = 1 / torch.sqrt(var + EPS)
    y = (x - mean) * rstd * s["gamma"].double()
    if c["ln"]:
        y += s["beta"].double()
    return x, mean[:, 0], rstd[:, 0], y


def _exact_checkpoint(x, group):
    """The codes are defined by fp32 steps on the stored rows, so they are taken in these; what they stand for, in 64 bits."""
    def block(b):
        b = b.float()
        hi, lo = b.max(1, keepdim=True).values, b.min(1, keepdim=True).values
        mid = (hi / 2) + (lo / 2)
        half = torch.max(hi - mid, mid - lo)
        some = half >= TINY
        scale = half.div(half.new_tensor(127.0)) * some
        inv = torch.where(some, scale.reciprocal(), scale)
        value = mid.double() + scale.double() * ((b - mid) * inv).round().double()
        return value, scale, mid
    v, s, m = zip(*_by_group(x, group, block))
    return torch.cat(v, 1), torch.stack([torch.cat(s, 1), torch.cat(m, 1)], 2)


def _exact_backward(s, c, v, mean, rstd):
    r = rstd.double()[:, None]
    xh = (v - (mean.double()[:, None] if c["ln"] else 0.0)) * r
    dy = s["dy"].double()
    t = dy * s["gamma"].double()
    dx = r * (t - (t.sum(1, keepdim=True) / c["n"] if c["ln"] else 0.0) - xh * ((t * xh).sum(1, keepdim=True) / c["n"]))
    if s["dres"] is not None:
        dx += s["dres"].double()
    return {"dx": dx, "dgamma": (dy * xh).sum(0), **({"dbeta": dy.sum(0)} if c["ln"] else {})}


def exact(c, seed):
    s = prepare(c, seed)
    k = c["kind"]
    if k in ("ck8_bwd", "read"):
        parts = []
        for i, b in enumerate(torch.split(s["codes"], c["group"], 1)):
            parts.append(s["scales"][:, i, 1:].double() + s["scales"][:, i, :1].double() * b.double())
        v = torch.cat(parts, 1)
        if k == "ck8_bwd":
            return _exact_backward(s, c, v, s["mean"], s["rstd"])
        y = (v - (s["mean"].double()[:, None] if c["ln"] else 0.0)) * s["rstd"].double()[:, None] * s["gamma"].double()
        return {"y": y + s["beta"].double() if c["ln"] else y}
    x, mean, rstd, y = _exact_norm(s, c)
    out = {"rstd": rstd, **({"mean": mean} if c["ln"] else {}), **({"h": x} if c["residual"] else {})}
    if k == "q8":
        def block(b):
            top = b.abs().max(1, keepdim=True).values
            scale = torch.where(top < TINY, torch.zeros_like(top), top / QMAX[c["fmt"]])
            u = torch.where(scale > 0, b / scale, torch.zeros_like(b))
            return scale, (torch.round(u) * scale if c["fmt"] == "int8" else _e4m3(u))
        scale, codes = zip(*_by_group(y, c["group"], block))
        return {**out, "scale": torch.cat(scale, 1), "values" if c["fmt"] == "int8" else "codes": torch.cat(codes, 1)}
    v, scales = _exact_checkpoint(x, c["group"])
    out["y"] = y
    if k == "ck8_fwd":
        return {**out, "scales": scales, "values": v}
    return {**out, **_exact_backward(s, c, v, mean, rstd)}
