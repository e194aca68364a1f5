"""Cases of the operators on attention heads: the norm of queries and keys for
each head with the position rotation in the same pass, its backward pass, and
the rotation alone, over one position axis or several (time, height, width).

Each operator has its plain form in elementary torch operations (32 bits,
angles in 64, rounded once at the end), the call a user makes of the library
(where `own` is true), and its definition in 64 bits (`exact`).

For every token and head, with D elements x:

  norm      RMSNorm n = x r gamma, r = 1 / sqrt(mean x^2 + eps), or LayerNorm
            n = (x - mean) r gamma + beta; gamma (beta) of D elements, one for
            the heads of q and one for those of k.
  angle     of pair j: position on the pair's axis times inv_freq[j].
  rotation  pair j is (j, j + rot / 2), or (2 j, 2 j + 1) where interleaved:
            y_a = n_a cos - n_b sin, y_b = n_b cos + n_a sin; elements from
            rot on keep n.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def _lib():
    import rmsnorm_norm_fwd_gb300
    return rmsnorm_norm_fwd_gb300


# ------------------------------------------------------------------ cases
def _case(name, kind, b, s, hq, hk, d, rot=None, ln=False, dtype="bf16", param=None, inter=False, axes=1,
          single=False, pos64=False, major=False, stats=False):
    """kind: forward, backward or step (both) of the norm with the rotation; rope, rope backward: the rotation alone.
    b batches of s tokens; rot rotated elements of d; single: tokens of different sequences, else prompts (one axis) or
    a grid (several); major: gradients come with heads outside tokens."""
    return {"name": name, "kind": kind, "b": b, "s": s, "hq": hq, "hk": hk, "d": d, "rot": d if rot is None else rot,
            "ln": ln, "dtype": dtype, "param": param or dtype, "inter": inter, "axes": axes, "single": single,
            "pos64": pos64, "major": major, "stats": stats}


def listed():
    return [
        # One token of a decoder, q and k inside the packed projection: latency alone.
        _case("qk token 1x(32+8)x128", "forward", 1, 1, 32, 8, 128, single=True, pos64=True),
        # A decoding batch, each token at its own far position, fp32 parameters.
        _case("qk batch 96x(64+8)x128", "forward", 1, 96, 64, 8, 128, param="fp32", single=True),
        # A prefill: prompts one behind another in one packed tensor.
        _case("qk prefill 16384x(32+8)x128", "forward", 1, 16384, 32, 8, 128),
        # Encoder heads: LayerNorm with a bias, a part of the head rotated, pairs interleaved, a ragged token count.
        _case("qk ln 4099x(16+16)x80 rot 32", "forward", 1, 4099, 16, 16, 80, rot=32, ln=True, dtype="fp16", inter=True,
              stats=True),
        # Heads of a size without 16-byte vectors, fp32.
        _case("qk odd 1003x(10+2)x98", "forward", 1, 1003, 10, 2, 98, dtype="fp32", stats=True),
        # The backward of a training step; attention's gradients arrive with heads outside tokens.
        _case("qk backward 4x4096x(32+8)x128", "backward", 4, 4096, 32, 8, 128, param="fp32", major=True),
        # The same for LayerNorm: wide heads, a quarter of each rotated.
        _case("qk backward ln 8191x(16+2)x256 rot 64", "backward", 1, 8191, 16, 2, 256, rot=64, ln=True, dtype="fp16"),
        # Forward and backward of a small batch: launches count.
        _case("qk step 2x256x(20+20)x64", "step", 2, 256, 20, 20, 64, param="fp32", stats=True),
        # Tokens of a video, three axes, q and k of as many heads, pairs interleaved.
        _case("rope video 26520x(40+40)x128", "rope", 1, 26520, 40, 40, 128, inter=True, axes=3),
        # An image encoder: two axes, heads of 80, ragged token count.
        _case("rope image 1369x(16+16)x80", "rope", 1, 1369, 16, 16, 80, dtype="fp16", axes=2),
        # The rotation's backward for text among images, three axes.
        _case("rope backward 2x4096x(28+4)x128", "rope backward", 2, 4096, 28, 4, 128, axes=3, pos64=True, major=True),
        # A decoding batch of the same, three axes, single tokens.
        _case("rope batch 32x(28+4)x128", "rope", 1, 32, 28, 4, 128, axes=3, single=True, pos64=True),
    ]


def draw(rng):
    kind = rng.choice(["forward", "forward", "backward", "backward", "step", "rope", "rope", "rope backward"])
    d = int(round(math.exp(rng.uniform(math.log(24), math.log(300)))))
    d = rng.choice([d, d // 8 * 8, -(-d // 16) * 16, 64, 128, 128])
    rot = rng.choice([d, d, d, d // 2, d // 4]) // 2 * 2
    axes = rng.choice([1, 1, 1, 2, 3]) if "rope" not in kind else rng.choice([1, 2, 3, 3])
    hk = rng.choice([1, 2, 4, 8, 8, 16, rng.randint(1, 20)])
    hq = hk * rng.choice([1, 1, 2, 4, 5, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    tokens = int(round(math.exp(rng.uniform(0.0, math.log(50000)))))
    b = rng.choice([1, 1, 2, 3, 4]) if tokens >= 16 else 1
    c = _case(None, kind, b, max(1, tokens // b), hq, hk, d, rot=max(2, rot), ln=rng.random() < 0.4, dtype=dtype,
              param=rng.choice([dtype, "fp32"]), inter=rng.random() < 0.4, axes=min(axes, max(1, rot // 2)),
              single=tokens < 300 and rng.random() < 0.5, pos64=rng.random() < 0.5, major=rng.random() < 0.4,
              stats=kind == "step" or rng.random() < 0.3)
    del c["name"]
    if kind in ("rope", "rope backward"):
        c["ln"] = c["stats"] = False
    most = max(work(x)["bytes"] for x in listed())
    c["s"] = max(1, min(c["s"], int(c["s"] * 0.9 * most / work(c)["bytes"])))
    return c


def work(c):
    """Each input read once, each output written once."""
    t, h, d, k = c["b"] * c["s"], c["hq"] + c["hk"], c["d"], c["kind"]
    n, e, two = t * h * d, SIZE[c["dtype"]], 2 if c["ln"] else 1
    angles = t * c["axes"] * (8 if c["pos64"] else 4) + 2 * c["rot"]
    if k in ("rope", "rope backward"):
        return {"bytes": 2 * n * e + angles, "flops": 3 * n}
    par, stat, sums = 2 * d * SIZE[c["param"]], 4 * t * h * two, 2 * d * 4 * two
    fwd = 2 * n * e + par * two + (stat if c["stats"] else 0) + angles
    bwd = 3 * n * e + par + stat + sums + angles
    if k == "forward":
        return {"bytes": fwd, "flops": 8 * n}
    if k == "backward":
        return {"bytes": bwd, "flops": 16 * n}
    return {"bytes": fwd + bwd, "flops": 24 * n}


# ------------------------------------------------------------------ inputs
def _sections(c):
    """Rotated pairs of each axis, near equal."""
    n, a = c["rot"] // 2, c["axes"]
    return [n - (a - 1) * (n // a)] + [n // a] * (a - 1)


def _positions(c, gen):
    """[b, s], or [axes, b, s]: far positions of single tokens, prompts one behind another, or the cells of a grid."""
    b, s, a = c["b"], c["s"], c["axes"]
    at = {"device": "cuda", "generator": gen}
    if c["single"]:
        p = torch.randint(0, 131072, (a, b, s), **at)
    elif a == 1:
        starts = (torch.rand(b, s, **at) < 4.0 / s).long()
        starts[:, 0] = 1
        i = torch.arange(s, device="cuda").expand(b, s)
        p = (i - torch.cummax(i * starts, 1).values)[None]
    else:
        side = max(1, round(s ** (1.0 / a)))
        i = torch.arange(s, device="cuda")
        p = torch.stack([i // side ** (a - 1 - k) % (side if k else s) for k in range(a)])
        p = p[:, None] + torch.randint(0, 64, (a, b, 1), **at)
    p = p.to(torch.int64 if c["pos64"] else torch.int32)
    return (p[0] if a == 1 else p).contiguous()


def _heads(gen, c, h, tail=0):
    """Projections: unit heads, one in a hundred larger, some heads of zeros (a padded token among a few hundred)."""
    x = torch.randn(c["b"], c["s"], h + tail, c["d"], device="cuda", generator=gen)
    u = torch.rand(c["b"], c["s"], h + tail, 1, device="cuda", generator=gen)
    x = torch.where(u < 0.01, x * 30, x)
    pad = torch.rand(c["b"], c["s"], 1, 1, device="cuda", generator=gen) > 0.997
    return torch.where(pad & (c["b"] * c["s"] > 1), torch.zeros_like(x), x).to(DTYPE[c["dtype"]])


def _gradient(gen, c, h):
    shape = (c["b"], h, c["s"], c["d"]) if c["major"] else (c["b"], c["s"], h, c["d"])
    g = torch.randn(shape, device="cuda", generator=gen).to(DTYPE[c["dtype"]])
    return g.transpose(1, 2) if c["major"] else g


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    hq, hk, d, k, pt = c["hq"], c["hk"], c["d"], c["kind"], DTYPE[c["param"]]
    s = {"case": c, "positions": _positions(c, gen)}
    n = c["rot"] // 2
    theta = 1e6 if c["single"] or c["axes"] == 1 else 1e4
    s["inv_freq"] = torch.tensor([theta ** (-j / n) for j in range(n)], dtype=torch.float64).to(torch.float32).cuda()
    s["sections"] = _sections(c)
    for name in ("q", "k"):
        s["gamma_" + name] = (1 + 0.1 * torch.randn(d, device="cuda", generator=gen)).to(pt)
        s["beta_" + name] = (0.1 * torch.randn(d, device="cuda", generator=gen)).to(pt) if c["ln"] else None
    if k != "rope backward":
        # the projection's output: q, k and (behind them, not read here) v heads of a token side by side
        s["qkv"] = _heads(gen, c, hq + hk, tail=hk if k in ("forward", "step") else 0)
        s["q"], s["k"] = s["qkv"][:, :, :hq], s["qkv"][:, :, hq:hq + hk]
    if k not in ("forward", "rope"):
        s["dq"], s["dk"] = _gradient(gen, c, hq), _gradient(gen, c, hk)
    if k == "backward":  # what the forward left
        x = s["qkv"].float()
        s["mean"] = x.mean(3) if c["ln"] else None
        v = x - s["mean"][..., None] if c["ln"] else x
        s["rstd"] = torch.rsqrt(v.square().mean(3) + EPS)
    if c["single"]:  # a server keeps its buffers
        s["yq"], s["yk"] = (torch.empty(c["b"], c["s"], h, d, device="cuda", dtype=DTYPE[c["dtype"]]) for h in (hq, hk))
    if own:
        s["rotary"] = _lib().rotary(s["inv_freq"], interleaved=c["inter"], sections=s["sections"])
    return s


# ------------------------------------------------------------------ plain forms
def _angles(s):
    """cos, sin [b, s, 1, rot / 2]: the product in 64 bits, since a far position has more than 24."""
    c, p = s["case"], s["positions"]
    p = p[None] if c["axes"] == 1 else p
    pos = torch.cat([p[a][..., None].expand(*p.shape[1:], n) for a, n in enumerate(s["sections"])], -1)
    a = pos.double() * s["inv_freq"].double()
    return torch.cos(a).float()[:, :, None], torch.sin(a).float()[:, :, None]


def _rotate(v, cos, sin, c):
    r = c["rot"]
    if c["inter"]:
        a, b = v[..., 0:r:2], v[..., 1:r:2]
        out = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = v[..., :r // 2], v[..., r // 2:r]
        out = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([out, v[..., r:]], -1) if r < c["d"] else out


def _plain_forward(s):
    c, (cos, sin) = s["case"], _angles(s)
    out, means, rstds = {}, [], []
    for name in ("q", "k"):
        x = s[name].float()
        if c["ln"]:
            means.append(x.mean(3))
            x = x - means[-1][..., None]
        rstds.append(torch.rsqrt(x.square().mean(3) + EPS))
        n = x * rstds[-1][..., None] * s["gamma_" + name].float()
        if c["ln"]:
            n = n + s["beta_" + name].float()
        out["y" + name] = _rotate(n, cos, sin, c).to(DTYPE[c["dtype"]])
    if c["stats"]:
        out["rstd"] = torch.cat(rstds, 2)
        if c["ln"]:
            out["mean"] = torch.cat(means, 2)
    return out


def _plain_backward(s, mean, rstd):
    c, (cos, sin) = s["case"], _angles(s)
    out, dgamma, dbeta, at = {}, [], [], 0
    for name in ("q", "k"):
        h = s[name].shape[2]
        r = rstd[:, :, at:at + h, None]
        xhat = s[name].float()
        if c["ln"]:
            xhat = xhat - mean[:, :, at:at + h, None]
        xhat = xhat * r
        t = _rotate(s["d" + name].float(), cos, -sin, c)
        g = t * s["gamma_" + name].float()
        dx = g - xhat * (g * xhat).mean(3, keepdim=True)
        if c["ln"]:
            dx = dx - g.mean(3, keepdim=True)
        out["d" + name] = (dx * r).to(DTYPE[c["dtype"]])
        dgamma.append((t * xhat).sum((0, 1, 2)))
        dbeta.append(t.sum((0, 1, 2)))
        at += h
    out["dgamma"] = torch.stack(dgamma)
    if c["ln"]:
        out["dbeta"] = torch.stack(dbeta)
    return out


def _plain(s):
    c = s["case"]
    k = c["kind"]
    if k == "forward":
        return _plain_forward(s)
    if k == "backward":
        return _plain_backward(s, s["mean"], s["rstd"])
    if k == "step":
        out = _plain_forward(s)
        return {**out, **_plain_backward(s, out.get("mean"), out["rstd"])}
    cos, sin = _angles(s)
    if k == "rope":
        return {"y" + n: _rotate(s[n].float(), cos, sin, c).to(DTYPE[c["dtype"]]) for n in ("q", "k")}
    return {"d" + n: _rotate(s["d" + n].float(), cos, -sin, c).to(DTYPE[c["dtype"]]) for n in ("q", "k")}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    g, c = _lib(), s["case"]
    k, ln, where = c["kind"], c["ln"], (s["positions"], s["rotary"])
    if k == "rope":
        yq, yk = g.rope_fwd(s["q"], s["k"], *where, yq=s.get("yq"), yk=s.get("yk"))
        return {"yq": yq, "yk": yk}
    if k == "rope backward":
        dq, dk = g.rope_bwd(s["dq"], s["dk"], *where)
        return {"dq": dq, "dk": dk}
    out, mean, rstd = {}, s.get("mean"), s.get("rstd")
    if k in ("forward", "step"):
        yq, yk, mean, rstd = g.qk_norm_rope_fwd(ln, s["q"], s["k"], s["gamma_q"], s["gamma_k"], EPS, *where,
                                                beta_q=s["beta_q"], beta_k=s["beta_k"], yq=s.get("yq"),
                                                yk=s.get("yk"), save_stats=c["stats"])
        out.update(yq=yq, yk=yk)
        if c["stats"]:
            out["rstd"] = rstd
            if ln:
                out["mean"] = mean
    if k in ("backward", "step"):
        dq, dk, dgamma, dbeta = g.qk_norm_rope_bwd(ln, s["dq"], s["dk"], s["q"], s["k"], s["gamma_q"], s["gamma_k"],
                                                   mean, rstd, *where)
        out.update(dq=dq, dk=dk, dgamma=dgamma)
        if ln:
            out["dbeta"] = dbeta
    return out


def run(s):
    return _own(s) if own else _plain(s)


# ------------------------------------------------------------------ in 64 bits
def _order(c):
    """Elements of a head in the order (first of each pair, second of each pair, rest)."""
    r = c["rot"]
    i = torch.arange(r, device="cuda").view((-1, 2) if c["inter"] else (2, -1))
    i = i.T if c["inter"] else i
    return i.reshape(-1).tolist() + list(range(r, c["d"]))


def _turned(v, s, c, sign):
    """Every pair as a complex number, times e^(sign i angle)."""
    n, order = c["rot"] // 2, _order(c)
    p = s["positions"].double().view(c["axes"], c["b"], c["s"])
    axis = [a for a, w in enumerate(s["sections"]) for _ in range(w)]
    angle = p[axis].permute(1, 2, 0) * s["inv_freq"].double() * sign
    w = v[..., order]
    z = torch.complex(w[..., :n], w[..., n:2 * n]) * torch.polar(torch.ones_like(angle), angle).unsqueeze(2)
    out = torch.empty_like(w)
    out[..., order] = torch.cat([z.real, z.imag, w[..., 2 * n:]], -1)
    return out


def _statistics(s, c, name):
    x = s[name].double()
    m = x.sum(-1, keepdim=True) / c["d"] if c["ln"] else torch.zeros_like(x[..., :1])
    return x, m, 1 / torch.sqrt(((x - m) ** 2).sum(-1, keepdim=True) / c["d"] + EPS)


def exact(c, seed):
    s, k = prepare(c, seed), c["kind"]
    if k in ("rope", "rope backward"):
        sign, i, o = (1, "", "y") if k == "rope" else (-1, "d", "d")
        return {o + n: _turned(s[i + n].double(), s, c, sign) for n in ("q", "k")}
    out, means, rstds, dgamma, dbeta, first = {}, [], [], [], [], 0
    for name in ("q", "k"):
        h = c["h" + name]
        x, m, r = _statistics(s, c, name)
        means.append(m[..., 0])
        rstds.append(r[..., 0])
        w = s["gamma_" + name].double()
        if k in ("forward", "step"):
            n = (x - m) * r * w
            out["y" + name] = _turned(n + s["beta_" + name].double() if c["ln"] else n, s, c, 1)
        if k == "backward":  # from the statistics that the backward is given
            r = s["rstd"][:, :, first:first + h, None].double()
            m = s["mean"][:, :, first:first + h, None].double() if c["ln"] else m
        if k in ("backward", "step"):
            t = _turned(s["d" + name].double(), s, c, -1)
            xh, u = (x - m) * r, t * w
            dot = (u * xh).sum(-1, keepdim=True) / c["d"]
            off = u.sum(-1, keepdim=True) / c["d"] if c["ln"] else 0.0
            out["d" + name] = r * (u - off - xh * dot)
            dgamma.append((t * xh).sum((0, 1, 2)))
            dbeta.append(t.sum((0, 1, 2)))
        first += h
    if c["stats"] and k in ("forward", "step"):
        out["rstd"] = torch.cat(rstds, 2)
        if c["ln"]:
            out["mean"] = torch.cat(means, 2)
    if dgamma:
        out["dgamma"] = torch.stack(dgamma)
        if c["ln"]:
            out["dbeta"] = torch.stack(dbeta)
    return out
