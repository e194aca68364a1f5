"""The head operators (norms of queries and keys with the position rotation,
their backward, the rotation alone) against plain 64-bit forms (GPU)."""
import pytest
import torch

import rope_ref as ref
from rope_ref import TYPES

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(autouse=True)
def _no_device_fault():
    import rmsnorm_norm_fwd_gb300 as g
    g.read_fault(reset=True)
    yield
    assert g.read_fault(reset=True) == 0


def lib():
    import rmsnorm_norm_fwd_gb300 as g
    return g


def params(D, dtype, seed=5):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.1 * torch.randn(D, generator=g)).to(dtype), (0.1 * torch.randn(D, generator=g)).to(dtype)


def cuda(t):
    return None if t is None else t.cuda()


def place(t, how, fill=float("nan")):
    """t on the GPU as: "dense", "packed" (behind other heads of its token), "major" (heads outside tokens), "odd" (one
    element off every boundary), "two" (two off), the rest of the memory holding `fill`."""
    if t is None:
        return None
    B, S, H, D = t.shape
    if how == "dense":
        return t.cuda()
    if how == "major":
        return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    if how == "packed":
        buf = torch.full((B, S, H + 3, D), fill, device="cuda").to(t.dtype)
        out = buf[:, :, 2:2 + H]
    else:
        first = 1 if how == "odd" else 2
        buf = torch.full((B, S, H, D + 2 + first), fill, device="cuda").to(t.dtype)
        out = buf[..., first:first + D]
    out.copy_(t)
    return out


def untouched(t, how, fill):
    """What lies around a tensor that `place` laid out still holds `fill`."""
    if how not in ("packed", "odd", "two"):
        return True
    whole = t._base
    inner = torch.zeros(whole.shape, dtype=torch.bool, device="cuda")
    (inner[:, :, 2:2 + t.shape[2]] if how == "packed" else inner[..., (1 if how == "odd" else 2):][..., :t.shape[3]]).fill_(True)
    return bool((whole[~inner] == fill).all())


def rotation(rot, axes=1, seed=7, theta=1e4, mixed=False):
    """inv_freq and the axis of each pair (None with one axis)."""
    n = rot // 2
    f = torch.tensor([theta ** (-j / n) for j in range(n)], dtype=torch.float64).float()
    if axes == 1:
        return f, None
    if mixed:
        return f, [j % axes for j in range(n)]
    return f, [min(j * axes // n, axes - 1) for j in range(n)]


def plan(f, pair_axis, inter):
    return lib().rotary(f.cuda(), interleaved=inter, pair_axis=pair_axis)


def positions(B, S, axes, dtype=torch.int32, seed=9, most=5000):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, most, (axes, B, S), generator=g).to(dtype)
    return p if axes > 1 else p[0]


def run_forward(mode, B, S, hq, hk, D, rot=None, dt="bf16", pdt=None, ydt=None, inter=False, axes=1, how="dense",
                out="dense", pos=None, gamma=(True, True), beta=(True, True), eps=EPS, stats=True, mixed=False, xs=None,
                f=None):
    """One forward through the public call, held to its bounds; mode False RMSNorm, True LayerNorm, None the rotation
    alone.  Returns yq, yk."""
    g = lib()
    rot = D // 2 * 2 if rot is None else rot
    dtype, yt = TYPES[dt], TYPES[ydt or dt]
    q = ref.heads(B, S, hq, D, dtype, 1, 0.5 if mode else 0.0) if xs is None else xs[0]
    k = ref.heads(B, S, hk, D, dtype, 2) if hk and xs is None else xs[1] if xs else None
    if rot:
        f, pa = rotation(rot, axes, mixed=mixed) if f is None else f
        pos = positions(B, S, axes) if pos is None else pos
        angle, far = ref.angles(pos, f, pa, B, S)
        where = (cuda(pos), plan(f, pa, inter))
    else:
        angle = far = None
        where = (None, None)
    par = [params(D, TYPES[pdt or dt], s) for s in (5, 6)]
    gam = [par[i][0] if gamma[i] else None for i in (0, 1)]
    bet = [par[i][1] if mode and beta[i] else None for i in (0, 1)]
    qd, kd = place(q, how), place(k, how)
    yq = place(torch.full((B, S, hq, D), 7.0, dtype=yt), out, 7.0) if out != "dense" else None
    yk = place(torch.full((B, S, hk, D), 7.0, dtype=yt), out, 7.0) if hk and out != "dense" else None
    if mode is None:
        yq, yk = g.rope_fwd(qd, kd, *where, y_dtype=yt, yq=yq, yk=yk)
        mean = rstd = None
    else:
        yq, yk, mean, rstd = g.qk_norm_rope_fwd(mode, qd, kd, cuda(gam[0]), cuda(gam[1]), eps, *where,
                                                beta_q=cuda(bet[0]), beta_k=cuda(bet[1]), y_dtype=yt, yq=yq, yk=yk,
                                                save_stats=stats)
    assert hk or yk is None
    at = 0
    for x, y, i in ((q, yq, 0), (k, yk, 1)):
        if x is None:
            continue
        m, r, (want, tol) = ref.forward(mode, x, gam[i], bet[i], eps, angle, far, rot, inter)
        assert y.dtype == yt and y.shape == x.shape
        ref.held("yqyk"[2 * i:2 * i + 2], y, want, tol, yt)
        assert untouched(y, out, 7.0)
        if stats and mode is not None:
            ref.held("rstd", rstd[:, :, at:at + x.shape[2]], *r)
            if mode:
                ref.held("mean", mean[:, :, at:at + x.shape[2]], *m)
        at += x.shape[2]
    if mode is not None and stats:
        assert rstd.shape == (B, S, hq + hk) and (mean is None) == (not mode)
    return yq, yk


def run_backward(mode, B, S, hq, hk, D, rot=None, dt="bf16", pdt=None, ydt=None, inter=False, axes=1, how="dense",
                 out="dense", gamma=(True, True), in_place=False, pos=None, sums=True):
    g = lib()
    rot = D // 2 * 2 if rot is None else rot
    dtype, yt = TYPES[dt], TYPES[ydt or dt]
    f, pa = rotation(rot, axes) if rot else (None, None)
    pos = positions(B, S, axes) if pos is None and rot else pos
    angle, far = ref.angles(pos, f, pa, B, S) if rot else (None, None)
    where = (cuda(pos), plan(f, pa, inter)) if rot else (None, None)
    gam = [params(D, TYPES[pdt or dt], s)[0] if gamma[s - 5] else None for s in (5, 6)]
    x = [ref.heads(B, S, hq, D, dtype, 1, 0.5 if mode else 0.0), ref.heads(B, S, hk, D, dtype, 2) if hk else None]
    dy = [ref.heads(B, S, hq, D, yt, 3), ref.heads(B, S, hk, D, yt, 4) if hk else None]
    means, rstds = [], []
    for t in x:
        if t is not None:
            (m, _), (r, _), _ = ref.norm(mode, t, None, None, EPS)
            means.append(m.float())
            rstds.append(r.float())
    mean, rstd = torch.cat(means, 2).contiguous(), torch.cat(rstds, 2).contiguous()
    xd, dyd = [place(t, how) for t in x], [place(t, how) for t in dy]
    dxs = [None, None]
    if in_place:
        dxs = dyd
    elif out != "dense":
        dxs = [place(torch.full(t.shape, 7.0, dtype=dtype), out, 7.0) if t is not None else None for t in x]
    dq, dk, dgamma, dbeta = g.qk_norm_rope_bwd(mode, *dyd, *xd, cuda(gam[0]), cuda(gam[1]), cuda(mean) if mode else None,
                                               cuda(rstd), *where, dq=dxs[0], dk=dxs[1], need_dgamma=sums,
                                               need_dbeta=sums)
    if in_place:
        assert dq is dyd[0] and dk is dyd[1]
    assert (dbeta is None) == (not (mode and sums)) and (dgamma is None) == (not sums)
    at = 0
    for i, got in enumerate((dq, dk)):
        if x[i] is None:
            assert got is None
            continue
        h = x[i].shape[2]
        (wx, tx), (wg, tg), (wb, tb) = ref.backward(mode, dy[i], x[i], gam[i], mean[..., at:at + h], rstd[..., at:at + h],
                                                    angle, far, rot, inter)
        ref.held("d" + "qk"[i], got, wx, tx, dtype)
        assert untouched(got, out, 7.0) or in_place
        if sums:
            ref.held("dgamma", dgamma[i], wg, tg)
            if mode:
                ref.held("dbeta", dbeta[i], wb, tb)
        at += h
    return dq, dk, dgamma, dbeta


SIZES = [(128, 128), (64, 64), (256, 64), (80, 80), (96, 96), (72, 72), (32, 32), (16, 8), (128, 48), (192, 128), (98, 98),
         (7, 6), (2, 2), (1, 0), (200, 200), (320, 64), (512, 512), (576, 64), (1023, 510), (1024, 1024), (128, 0),
         (40, 24), (24, 4), (260, 260)]
DT = ["bf16", "fp16", "fp32"]


@pytest.mark.parametrize("D,rot", SIZES)
@pytest.mark.parametrize("mode", [False, True, None])
def test_forward_sizes(mode, D, rot):
    if mode is None and rot == 0:
        pytest.skip("nothing to rotate")
    for i, dt in enumerate(DT):
        run_forward(mode, 2, 9, 5, 2, D, rot, dt, inter=i == 1)
        run_forward(mode, 1, 3, 2, 1, D, rot, dt, inter=i != 1, axes=2 if rot >= 4 else 1)


@pytest.mark.parametrize("D,rot", SIZES)
@pytest.mark.parametrize("mode", [False, True])
def test_backward_sizes(mode, D, rot):
    for i, dt in enumerate(DT):
        run_backward(mode, 2, 9, 5, 2, D, rot, dt, inter=i == 1)
        run_backward(mode, 1, 3, 2, 1, D, rot, dt, inter=i != 1, axes=2 if rot >= 4 else 1)


@pytest.mark.parametrize("how", ["packed", "major", "odd"])
@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "fp32"), (72, "fp16"), (98, "bf16")])
def test_layouts(how, D, dt):
    for mode in (False, True, None):
        run_forward(mode, 2, 17, 6, 3, D, dt=dt, how=how, out="dense")
        run_forward(mode, 2, 17, 6, 3, D, dt=dt, how="dense", out=how, inter=True)
    for mode in (False, True):
        run_backward(mode, 2, 17, 6, 3, D, dt=dt, how=how, out="dense")
        run_backward(mode, 2, 17, 6, 3, D, dt=dt, how="dense", out=how, inter=True)


@pytest.mark.parametrize("B,S,hq,hk", [(1, 1, 1, 0), (1, 1, 32, 8), (1, 1, 1, 1), (3, 1, 33, 0), (1, 2, 7, 3), (1, 301, 8, 1),
                                       (2, 257, 3, 5), (64, 1, 16, 2), (1, 4099, 4, 4), (1, 40, 130, 70)])
def test_token_and_head_counts(B, S, hq, hk):
    for mode in (False, True, None):
        run_forward(mode, B, S, hq, hk, 64)
    for mode in (False, True):
        run_backward(mode, B, S, hq, hk, 64, 32)


@pytest.mark.parametrize("xt", DT)
@pytest.mark.parametrize("yt", DT)
def test_mixed_types(xt, yt):
    for pt in DT:
        run_forward(False, 1, 21, 4, 2, 128, dt=xt, ydt=yt, pdt=pt)
        run_forward(True, 1, 21, 4, 2, 80, dt=xt, ydt=yt, pdt=pt, inter=True)
        run_backward(False, 1, 21, 4, 2, 128, dt=xt, ydt=yt, pdt=pt)
        run_backward(True, 1, 21, 4, 2, 80, dt=xt, ydt=yt, pdt=pt, inter=True)
    run_forward(None, 1, 21, 4, 2, 128, dt=xt, ydt=yt)


@pytest.mark.parametrize("D", [128, 98])
def test_parameters_left_out(D):
    for on in ((False, False), (True, False), (False, True)):
        run_forward(False, 1, 9, 4, 2, D, gamma=on)
        run_forward(True, 1, 9, 4, 2, D, gamma=on, beta=on[::-1])
        run_forward(True, 1, 9, 4, 2, D, gamma=(True, True), beta=on, inter=True)
        run_backward(False, 1, 9, 4, 2, D, gamma=on)
        run_backward(True, 1, 9, 4, 2, D, gamma=on)
    run_forward(False, 1, 9, 4, 2, D, stats=False)
    run_backward(True, 1, 9, 4, 2, D, sums=False)


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("inter", [False, True])
def test_axes(axes, inter):
    for mixed in (False, True):
        for D in (128, 42):
            run_forward(None, 2, 33, 4, 2, D, axes=axes, inter=inter, mixed=mixed)
            run_forward(False, 2, 33, 4, 2, D, axes=axes, inter=inter, mixed=mixed)
    run_backward(False, 2, 33, 4, 2, 128, axes=axes, inter=inter)


def test_position_types_and_strides():
    g = lib()
    S, D = 37, 128
    for D in (128, 98):
        for dtype in (torch.int32, torch.int64):
            run_forward(False, 3, S, 4, 2, D, pos=positions(3, S, 1, dtype))
            shared = positions(1, S, 2, dtype)[:, 0]  # [axes, tokens], the same for all batches
            run_forward(False, 3, S, 4, 2, D, axes=2, pos=shared)
            run_forward(None, 3, S, 4, 2, D, axes=2, pos=shared)
    # every other position of a longer row, and one position for all tokens
    f, _ = rotation(D)
    q = ref.heads(2, S, 4, D, torch.bfloat16, 1).cuda()
    long = positions(2, 2 * S, 1, torch.int64).cuda()
    r = plan(f, None, False)
    assert torch.equal(g.rope_fwd(q, None, long[:, ::2], r)[0], g.rope_fwd(q, None, long[:, ::2].contiguous(), r)[0])
    one = long[:, :1].expand(2, S)
    assert torch.equal(g.rope_fwd(q, None, one, r)[0], g.rope_fwd(q, None, one.contiguous(), r)[0])
    # three dimensions: tokens without batches
    assert torch.equal(g.rope_fwd(q[1], None, long[1, :S], r)[0], g.rope_fwd(q[1:], None, long[1:, :S], r)[0][0])


@pytest.mark.parametrize("D", [128, 98])
def test_far_positions(D):
    """Angles of far positions are exact: the angle itself in exact integers here (positions up to 2^40, frequencies as
    stored), since 64 bits would round the product."""
    from fractions import Fraction
    g = lib()
    pi = Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)
    n = D // 2
    f = torch.tensor([10000.0 ** (-j / n) for j in range(n)], dtype=torch.float64).float()
    pos = torch.tensor([0, 1, -1, 4097, 1000003, 16777217, 2 ** 31 - 1, -2 ** 31, 2 ** 40 + 12345, -(2 ** 37) - 1])
    turns = [[float((int(p) * Fraction(float(w)) / (2 * pi)) % 1) for w in f] for p in pos]
    angle = 2 * torch.pi * torch.tensor(turns, dtype=torch.float64)[None, :, None]
    far = pos.double().abs()[None, :, None, None]
    q = ref.heads(1, len(pos), 3, D, torch.float32, 1)
    for inter in (False, True):
        want, tol = ref.forward(None, q, None, None, 0, angle, far, D, inter)[2]
        ref.held("yq", g.rope_fwd(q.cuda(), None, pos[None].cuda(), plan(f, None, inter))[0], want, tol + 1e-14)


def test_far_positions_int32():
    pos = torch.tensor([[0, 131071, 1048575, 2 ** 31 - 1, -5]], dtype=torch.int32)
    # 64 bits hold these products to 2^-53 of at most 2^31 radians
    for dt in DT:
        g, D = lib(), 128
        f, _ = rotation(D)
        q = ref.heads(1, 5, 3, D, TYPES[dt], 1)
        angle, far = ref.angles(pos, f, None, 1, 5)
        want, tol = ref.forward(None, q, None, None, 0, angle, far, D, False)[2]
        got = g.rope_fwd(q.cuda(), None, pos.cuda(), plan(f, None, False))[0]
        ref.held("yq", got, want, tol + 2.0 ** -22 * (1 + q.double().abs().amax()), TYPES[dt])


def test_frequencies_of_any_size():
    """0, subnormal, negative and large frequencies; not finite ones make their pairs NaN and no others."""
    g, D = lib(), 32
    f = torch.tensor([0.0, 1e-42, -0.75, 3.0, 1e6, 2.0 ** 60, 1.0, 2.0, 0.1, 1e-7, 0.5, 2.0 ** -100, 7.0, 1.5, -1e-3, 6.25])
    from fractions import Fraction
    pi = Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)
    pos = torch.tensor([[0, 1, 3, 1000]])
    turns = [[float((int(p) * Fraction(float(w)) / (2 * pi)) % 1) for w in f] for p in pos[0]]
    angle = 2 * torch.pi * torch.tensor(turns, dtype=torch.float64)[None, :, None]
    far = pos.double().abs()[..., None, None]
    q = ref.heads(1, 4, 3, D, torch.float32, 1)
    for inter in (False, True):
        want, tol = ref.forward(None, q, None, None, 0, angle, far, D, inter)[2]
        ref.held("yq", g.rope_fwd(q.cuda(), None, pos.cuda(), plan(f, None, inter))[0], want, tol + 1e-12)
        for bad in (float("nan"), float("inf"), -float("inf"), 3e38):
            h = f.clone()
            h[5] = bad
            y = g.rope_fwd(q.cuda(), None, pos.cuda(), plan(h, None, inter))[0].cpu()
            a, b = ref.pairs(D, inter)
            hit = torch.zeros(D, dtype=torch.bool)
            hit[a[5]] = hit[b[5]] = True
            assert torch.isnan(y[..., hit]).all() and not torch.isnan(y[..., ~hit]).any()


@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (80, 32), (98, 40)])
def test_nan_and_infinity_stay_in_their_place(D, rot):
    """A NaN or an infinity reaches its own head (with the norm), its own pair (rotation alone), and nothing else."""
    g = lib()
    S, H = 5, 12
    for inter in (False, True):
        f, _ = rotation(rot)
        r, pos = plan(f, None, inter), positions(1, S, 1).cuda()
        for bad in (float("nan"), float("inf")):
            for at in (0, rot - 1, D - 1):
                q = ref.heads(1, S, H, D, torch.bfloat16, 1)
                q[0, 2, 6, at] = bad
                y = g.rope_fwd(q.cuda(), None, pos, r)[0].cpu()
                hit = torch.zeros(q.shape, dtype=torch.bool)
                hit[0, 2, 6, at] = True
                if at < rot:
                    a, b = ref.pairs(rot, inter)
                    j = [i for i in range(rot // 2) if at in (a[i], b[i])][0]
                    hit[0, 2, 6, a[j]] = hit[0, 2, 6, b[j]] = True
                assert not torch.isfinite(y[hit]).any() and torch.isfinite(y[~hit]).all()
                for ln in (False, True):
                    y = g.qk_norm_rope_fwd(ln, q.cuda(), None, None, None, EPS, pos, r)[0].cpu()
                    hit = torch.zeros(q.shape, dtype=torch.bool)
                    hit[0, 2, 6] = True
                    assert torch.isnan(y[hit]).any() and torch.isfinite(y[~hit]).all()
                    rstd = torch.ones(1, S, H).cuda()
                    dx, _, dg, _ = g.qk_norm_rope_bwd(ln, q.cuda(), None, torch.ones_like(q).cuda(), None, None, None,
                                                      torch.zeros_like(rstd) if ln else None, rstd, pos, r)
                    assert torch.isfinite(dx.cpu()[~hit]).all() and not torch.isfinite(dx.cpu()[hit]).all()


def test_no_tokens():
    g = lib()
    r, D = plan(rotation(64)[0], None, False), 64
    for shape in ((0, 4, D), (2, 0, 4, D), (0, 3, 4, D)):
        q = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
        pos = torch.empty(shape[:-2], device="cuda", dtype=torch.int32)
        yq, yk, mean, rstd = g.qk_norm_rope_fwd(True, q, q, None, None, EPS, pos, r)
        assert yq.shape == shape and rstd.numel() == 0
        dg, db = torch.full((2, D), 5.0, device="cuda"), torch.full((2, D), 5.0, device="cuda")
        g.qk_norm_rope_bwd(True, q, q, q, q, None, None, mean, rstd, pos, r, dgamma=dg, dbeta=db)
        assert not dg.any() and not db.any()
        assert g.rope_fwd(q, None, pos, r)[1] is None and g.rope_last_variant(2) == ""


@pytest.mark.parametrize("D", [128, 98])
def test_in_place_in_a_packed_projection(D):
    """q and k normalised and turned where they lie, v between the tokens untouched."""
    g = lib()
    B, S, hq, hk = 2, 65, 8, 2
    qkv = ref.heads(B, S, hq + 2 * hk, D, torch.bfloat16, 1).cuda()
    r, pos = plan(rotation(D // 2 * 2)[0], None, False), positions(B, S, 1).cuda()
    gq, gk = (params(D, torch.bfloat16, s)[0].cuda() for s in (5, 6))
    q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:]
    keep = v.clone()
    want = g.qk_norm_rope_fwd(False, q, k, gq, gk, EPS, pos, r)
    yq, yk, _, rstd = g.qk_norm_rope_fwd(False, q, k, gq, gk, EPS, pos, r, yq=q, yk=k)
    assert yq is q and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(rstd, want[3])
    assert torch.equal(v, keep)
    back = g.rope_bwd(q, k, pos, r)
    g.rope_bwd(q, k, pos, r, dq=q, dk=k)
    assert torch.equal(q, back[0]) and torch.equal(k, back[1]) and torch.equal(v, keep)
    run_backward(True, 2, 33, 5, 2, D, in_place=True, how="packed")


def test_broadcast_inputs():
    """Inputs with stride 0: one token's heads for all tokens, one head's gradient for all heads."""
    g = lib()
    D, S = 128, 19
    for D in (128, 98):
        r, pos = plan(rotation(D)[0], None, True), positions(1, S, 1)[0].cuda()
        q = ref.heads(1, 1, 8, D, torch.bfloat16, 1)[0].cuda().expand(S, 8, D)
        dy = ref.heads(1, S, 1, D, torch.bfloat16, 2)[0].cuda().expand(S, 8, D)
        full = g.qk_norm_rope_fwd(False, q.contiguous(), None, None, None, EPS, pos, r)
        got = g.qk_norm_rope_fwd(False, q, None, None, None, EPS, pos, r)
        assert torch.equal(got[0], full[0]) and torch.equal(got[3], full[3])
        a = g.qk_norm_rope_bwd(False, dy, None, q, None, None, None, None, got[3], pos, r)
        b = g.qk_norm_rope_bwd(False, dy.contiguous(), None, q.contiguous(), None, None, None, None, got[3], pos, r)
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("D", [128, 98])
def test_rotation_back_and_forth(D):
    """rope_bwd is the inverse: twice half a step of the stored type away, and the rotations' own errors."""
    g = lib()
    r, pos = plan(rotation(D, 3)[0], rotation(D, 3)[1], False), positions(1, 50, 3).cuda()
    q = ref.heads(1, 50, 3, D, torch.float32, 1).cuda()
    back = g.rope_bwd(g.rope_fwd(q, None, pos, r)[0], None, pos, r)[0]
    size = torch.cat([q[..., D // 2:], q[..., :D // 2]], -1).abs() + q.abs()
    assert ((back - q).abs() <= 2 * (8 + 2) * ref.U * 1.5 * size).all()


@pytest.mark.parametrize("limit", [1, 3, 0])
def test_grid_limits(limit):
    g = lib()
    try:
        g.set_grid_limit(limit)
        for D in (128, 98):
            run_forward(False, 1, 77, 6, 2, D)
            run_forward(None, 1, 77, 5, 0, D)
            run_backward(True, 1, 77, 6, 2, D)
            run_backward(False, 1, 77, 1, 1, D)
            run_backward(False, 1, 77, 5, 0, D)
    finally:
        g.set_grid_limit(0)


@pytest.mark.parametrize("D", [128, 98])
def test_same_bits_every_run(D):
    g = lib()
    B, S, hq, hk = 1, 1111, 8, 4
    q, k = (ref.heads(B, S, h, D, torch.bfloat16, h).cuda() for h in (hq, hk))
    dq, dk = (ref.heads(B, S, h, D, torch.bfloat16, h + 1).cuda() for h in (hq, hk))
    r, pos = plan(rotation(D)[0], None, False), positions(B, S, 1).cuda()
    first = None
    for _ in range(3):
        out = g.qk_norm_rope_fwd(True, q, k, None, None, EPS, pos, r)
        out = out + g.qk_norm_rope_bwd(True, dq, dk, q, k, None, None, out[2], out[3], pos, r)
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_offsets_past_32_bits():
    """Tokens 2^30 elements apart."""
    g = lib()
    S, D, H = 4, 128, 2
    step = 2 ** 30
    buf = torch.empty(3 * step + H * D, device="cuda", dtype=torch.bfloat16)
    x = ref.heads(1, S, H, D, torch.bfloat16, 1)[0]
    r, pos = plan(rotation(D)[0], None, False), positions(1, S, 1)[0].cuda()
    for off, d in ((0, D), (0, D - 2)):
        q = buf.as_strided((S, H, d), (step, D, 1))
        q.copy_(x[..., :d])
        rr = plan(rotation(d)[0], None, False) if d != D else r
        dense = q.contiguous()
        a, b = g.qk_norm_rope_fwd(False, q, None, None, None, EPS, pos, rr), g.qk_norm_rope_fwd(
            False, dense, None, None, None, EPS, pos, rr)
        assert torch.equal(a[0], b[0]) and torch.equal(a[3], b[3])
        da = g.qk_norm_rope_bwd(False, q, None, q, None, None, None, None, a[3], pos, rr)
        db = g.qk_norm_rope_bwd(False, dense, None, dense, None, None, None, None, a[3], pos, rr)
        assert torch.equal(da[0], db[0]) and torch.equal(da[2], db[2])
        g.rope_fwd(dense, None, pos, rr, yq=q)
        assert torch.equal(q, g.rope_fwd(dense, None, pos, rr)[0])


def test_capture_before_any_call_and_replay():
    """Captured as the first call of these shapes, replayed on other inputs and positions."""
    g = lib()
    B, S, hq, hk, D = 1, 130, 6, 3, 128
    f, _ = rotation(D)
    for D in (128, 98):
        f, _ = rotation(D)
        r = plan(f, None, False)
        q, k = (torch.zeros(B, S, h, D, device="cuda", dtype=torch.bfloat16) for h in (hq, hk))
        pos = torch.zeros(B, S, device="cuda", dtype=torch.int32)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            yq, yk, mean, rstd = g.qk_norm_rope_fwd(True, q, k, None, None, EPS, pos, r)
            dq, dk, dg, db = g.qk_norm_rope_bwd(True, yq, yk, q, k, None, None, mean, rstd, pos, r)
            zq, zk = g.rope_bwd(yq, yk, pos, r)
        for seed in (1, 2):
            q.copy_(ref.heads(B, S, hq, D, torch.bfloat16, seed))
            k.copy_(ref.heads(B, S, hk, D, torch.bfloat16, seed + 10))
            pos.copy_(positions(B, S, 1, seed=seed))
            graph.replay()
            e = g.qk_norm_rope_fwd(True, q, k, None, None, EPS, pos, r)
            eb = g.qk_norm_rope_bwd(True, e[0], e[1], q, k, None, None, e[2], e[3], pos, r)
            ez = g.rope_bwd(e[0], e[1], pos, r)
            for a, b in zip((yq, yk, mean, rstd, dq, dk, dg, db, zq, zk), (*e, *eb, *ez)):
                assert torch.equal(a, b)


def test_streams_and_host_threads():
    import threading
    g = lib()
    D, S, H = 128, 999, 8
    q = ref.heads(1, S, H, D, torch.bfloat16, 1).cuda()
    r, pos = plan(rotation(D)[0], None, False), positions(1, S, 1).cuda()
    want = g.qk_norm_rope_fwd(False, q, None, None, None, EPS, pos, r)
    wb = g.qk_norm_rope_bwd(False, q, None, q, None, None, None, None, want[3], pos, r)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(20):
            y = g.qk_norm_rope_fwd(False, q, None, None, None, EPS, pos, r, stream=s)
            b = g.qk_norm_rope_bwd(False, q, None, q, None, None, None, None, y[3], pos, r, stream=s)
            s.synchronize()
            if not (torch.equal(y[0], want[0]) and torch.equal(b[0], wb[0]) and torch.equal(b[2], wb[2])):
                bad.append(1)
    ts = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_refused_on_the_gpu():
    g = lib()
    D, S = 64, 6
    q = torch.zeros(S, 4, D, device="cuda", dtype=torch.bfloat16)
    r, pos = plan(rotation(D)[0], None, False), torch.zeros(S, device="cuda", dtype=torch.int32)
    for f in (lambda: g.rope_fwd(q, q, pos, r, yq=q, yk=q),                    # both outputs in one place
              lambda: g.rope_fwd(q, None, pos, r, yq=q[:1].expand(S, 4, D)),   # tokens of the output in one place
              lambda: g.rope_fwd(q[:, :2], None, pos, r, yq=q[:, 1:3])):       # the output over other inputs
        with pytest.raises(g.GbnormError) as e:
            f()
        assert e.value.status == 1
    for f in (lambda: g.rope_fwd(q, None, pos[:3], r), lambda: g.rope_fwd(q, None, pos.float(), r),
              lambda: g.rope_fwd(q, None, pos.cpu(), r), lambda: g.rope_fwd(q, q[:3], pos, r),
              lambda: g.rope_fwd(q, q.half(), pos, r), lambda: g.rope_fwd(q[..., ::2], None, pos, r),
              lambda: g.rope_fwd(q[:, :, :32], None, pos, r), lambda: g.rope_fwd(q, None, pos, None),
              lambda: g.rope_fwd(q, q[:, :0], pos, r), lambda: g.rope_fwd(q.double(), None, pos, r),
              lambda: g.qk_norm_rope_fwd(False, q, None, q[0, 0, :32], None, EPS, pos, r),
              lambda: g.qk_norm_rope_fwd(False, q, q, q[0, 0], q[0, 0].float(), EPS, pos, r),
              lambda: g.qk_norm_rope_fwd(False, q, None, None, None, EPS, pos, None),
              lambda: g.qk_norm_rope_fwd(False, q, None, None, None, EPS, pos, r, rstd=torch.zeros(S, 3, device="cuda")),
              lambda: g.qk_norm_rope_bwd(False, q, None, q, None, None, None, None, None, pos, r),
              lambda: g.qk_norm_rope_bwd(False, q[:3], None, q, None, None, None, None, pos, pos, r),
              lambda: g.rotary(r.inv_freq.half()), lambda: g.rotary(r.inv_freq.cpu()), lambda: g.rotary(r.inv_freq[:0]),
              lambda: g.rotary(r.inv_freq, sections=(16, 15)), lambda: g.rotary(r.inv_freq, pair_axis=[0] * 31),
              lambda: g.rotary(r.inv_freq, sections=(8, 8, 8, 4, 4)),
              lambda: g.rotary(r.inv_freq, sections=(32,), pair_axis=[0] * 32)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(g.GbnormError):
        g.qk_norm_rope_bwd(False, q, None, q, None, None, None, None, torch.ones(S, 4, device="cuda"), pos, r,
                           workspace=torch.empty(16, device="cuda", dtype=torch.uint8))


def test_attention_step():
    """The operators as a training step uses them: hidden rows normalised (with the residual), projected, heads
    normalised and turned, attention, and back through all of it; against 64-bit autograd."""
    g = lib()
    T, C, hq, hk, D = 96, 256, 4, 2, 64
    gen = torch.Generator().manual_seed(3)
    def draw(*s, k=1.0):
        return (torch.randn(*s, generator=gen) * k)
    x, res, w, dout = draw(T, C), draw(T, C), draw(C, (hq + 2 * hk) * D, k=C ** -0.5), draw(T, hq, D)
    gam, gq, gk = 1 + 0.1 * draw(C), 1 + 0.1 * draw(D), 1 + 0.1 * draw(D)
    f, _ = rotation(D)
    pos = torch.arange(T, dtype=torch.int32)

    def attend(q, k, v):
        k, v = (t.repeat_interleave(hq // hk, 1) for t in (k, v))
        s = torch.einsum("thd,shd->hts", q, k) * D ** -0.5
        s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device=q.device).triu(1), float("-inf"))
        return torch.einsum("hts,shd->thd", torch.softmax(s, -1), v)
    # 64 bits
    leaves = [t.double().requires_grad_() for t in (x, res, w, gam, gq, gk)]
    X, R, W, G, GQ, GK = leaves
    h = X + R
    rms = lambda t, gg: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * gg
    qkv = (rms(h, G) @ W).view(T, hq + 2 * hk, D)
    angle, _ = ref.angles(pos, f, None, 1, T)
    turn = lambda t: ref.rotate(t, angle[0], D, False)
    q, k, v = turn(rms(qkv[:, :hq], GQ)), turn(rms(qkv[:, hq:hq + hk], GK)), qkv[:, hq + hk:]
    (attend(q, k, v) * dout.double()).sum().backward()
    # fp32, the library's operators around torch's products
    c = [t.cuda() for t in (x, res, w, gam, gq, gk, dout, pos)]
    r = plan(f, None, False)
    y, hh, _, rs = g.norm_fwd_ex(False, c[0], c[3], None, EPS, residual=c[1])
    p = (y @ c[2]).view(T, hq + 2 * hk, D)
    qf, kf, vf = p[:, :hq], p[:, hq:hq + hk], p[:, hq + hk:]
    yq, yk, _, rstd = g.qk_norm_rope_fwd(False, qf, kf, c[4], c[5], EPS, c[7], r)
    t = [u.detach().clone().requires_grad_() for u in (yq, yk, vf)]
    (attend(*t) * c[6]).sum().backward()
    dp = torch.empty_like(p)
    dp[:, hq + hk:] = t[2].grad
    _, _, dgam, _ = g.qk_norm_rope_bwd(False, t[0].grad, t[1].grad, qf, kf, c[4], c[5], None, rstd, c[7], r,
                                       dq=dp[:, :hq], dk=dp[:, hq:hq + hk])
    dp2 = dp.view(T, -1)
    dw, dy = y.t() @ dp2, dp2 @ c[2].t()
    dx, dg, _ = g.norm_bwd_ex(False, dy, hh, c[3], None, rs)
    # relative L2: some twenty fp32 steps deep, each of a few hundred u at the most (products of length 256)
    for name, got, want in (("dx", dx, X.grad), ("dres", dx, R.grad), ("dw", dw, W.grad), ("dgamma", dg, G.grad),
                            ("dgamma_q", dgam[0], GQ.grad), ("dgamma_k", dgam[1], GK.grad)):
        e = (got.cpu().double() - want).norm() / want.norm()
        assert e <= 20 * 256 * ref.U, (name, e)


@pytest.mark.parametrize("ln", [False, True])
def test_gradient_against_differences(ln):
    """Central differences of L = sum(dy y) through the fp32 forward, step 2^-5: the truncation is at most step^2 / 6
    times the third derivative, the rounding 2 u sum|dy y| / step."""
    g = lib()
    S, H, D = 2, 2, 16
    gen = torch.Generator().manual_seed(1)
    q = torch.randn(S, H, D, generator=gen).cuda()
    dy = torch.randn(S, H, D, generator=gen).cuda()
    gam, bet = (1 + 0.1 * torch.randn(D, generator=gen)).cuda(), torch.zeros(D).cuda() if ln else None
    r, pos = plan(rotation(D)[0], None, False), torch.tensor([3, 70], dtype=torch.int32).cuda()

    def loss(x, w):
        return (g.qk_norm_rope_fwd(ln, x, None, w, None, 1e-2, pos, r, beta_q=bet)[0].double() * dy.double()).sum().item()
    _, _, mean, rstd = g.qk_norm_rope_fwd(ln, q, None, gam, None, 1e-2, pos, r, beta_q=bet)
    dx, _, dg, _ = g.qk_norm_rope_bwd(ln, dy, None, q, None, gam, None, mean, rstd, pos, r)
    e = 2.0 ** -5
    size = 2 * ref.U * 8 * dy.abs().sum().item() * 4 / e
    # third derivatives of x / |x| along one element: below 15 / rms^3 times |dy|, rms above 1/2 here
    third = e * e / 6 * 15 * 8 * dy.abs().max().item()
    assert (rstd < 2).all()
    for at in ((0, 0, 0), (0, 1, 9), (1, 0, 15), (1, 1, 4)):
        hi, lo = q.clone(), q.clone()
        hi[at] += e
        lo[at] -= e
        num = (loss(hi, gam) - loss(lo, gam)) / (2 * e)
        assert abs(num - dx[at].item()) <= size + third, at
    for j in (0, 7, 15):
        hi, lo = gam.clone(), gam.clone()
        hi[j] += e
        lo[j] -= e
        assert abs((loss(q, hi) - loss(q, lo)) / (2 * e) - dg[0, j].item()) <= size, j
