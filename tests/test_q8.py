"""The 8-bit operators: 8-bit norm output, 8-bit checkpoint, the backward from
it and the reading back, against plain 64-bit forms (GPU)."""
import pytest
import torch

import q8_ref as ref
from q8_ref import TYPES, U

pytestmark = pytest.mark.gpu
E4M3, I8 = torch.float8_e4m3fn, torch.int8


@pytest.fixture(autouse=True)
def _no_device_fault():
    import rmsnorm_norm_fwd_gb300 as g
    g.read_fault(reset=True)
    yield
    assert g.read_fault(reset=True) == 0


def lib():
    import rmsnorm_norm_fwd_gb300 as g
    return g


def params(N, ln, dtype, seed=5):
    g = torch.Generator().manual_seed(seed)
    gamma = (1 + 0.1 * torch.randn(N, generator=g)).to(dtype)
    return gamma, (0.1 * torch.randn(N, generator=g)).to(dtype) if ln else None


def cuda(t):
    return None if t is None else t.cuda()


def padded(t, pad, fill=None):
    """t on the GPU with row stride N + pad, the padding holding NaN (or fill)."""
    if t is None:
        return None
    M, N = t.shape
    buf = torch.full((M, N + pad), float("nan") if fill is None else fill, device="cuda").to(t.dtype)
    buf[:, :N].copy_(t)
    return buf[:, :N]


def stats_ok(ln, h, mean, rstd, m, r):
    assert ((rstd.cpu().double() - r).abs() <= 1e-5 * r).all()
    if ln:
        assert ((mean.cpu().double() - m).abs() <= 1e-5 * (m.abs() + 1 / r)).all()


def same_bits(a, b):
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    view = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.shape == b.shape and torch.equal(a.view(view), b.view(view))


def raw(q):
    """8-bit rows as bytes on the CPU."""
    return q.cpu().view(torch.uint8)


def run_forward(ln, M, N, dt, pdt=None, residual=True, fmt=E4M3, group=0, ck=None, pad=0, out="q8", ydt=None, seed=1,
                x=None):
    """One forward through the public call, held to its bounds; what it returned."""
    g = lib()
    dtype, shift = TYPES[dt], 0.5 if ln else 0.0
    x = ref.rows(M, N, dtype, seed, shift) if x is None else x
    r = ref.rows(M, N, dtype, seed + 1, special=False) if residual else None
    if residual and M >= 2:
        r[1] = 0.0
    gamma, beta = params(N, ln, TYPES[pdt or dt])
    eps = 1e-6
    h = ref.add(x, r)
    mean, rstd, y, tol = ref.norm(ln, h, gamma, beta, eps)
    xd, rd = (padded(x, pad), padded(r, pad)) if pad else (cuda(x), cuda(r))
    keep = (xd.clone(), rd.clone() if residual else None)
    if out == "q8":
        c8 = g.checkpoint8_empty(M, N, ck) if ck else None
        q, scale, hh, mm, rr = g.norm_fwd_q8(ln, xd, cuda(gamma), cuda(beta), eps, residual=rd, fmt=fmt, group=group,
                                             checkpoint=c8)
        ref.check_q8(ln, h, gamma, q, scale, group, y, tol)
        got = (q, scale)
    else:
        yy, hh, c8, mm, rr = g.norm_fwd_ck8(ln, xd, cuda(gamma), cuda(beta), eps, residual=rd, group=ck,
                                            y_dtype=TYPES[ydt or dt])
        ref.held("y", yy, y, tol, yy.dtype)
        got = (yy,)
    if residual:
        assert same_bits(hh, h)
    assert same_bits(xd, keep[0]) and (not residual or same_bits(rd, keep[1]))
    stats_ok(ln, h, mm, rr, mean, rstd)
    if ck:
        codes, scales = ref.checkpoint(h, ck)
        assert same_bits(c8.scales, scales), "checkpoint scales"
        assert same_bits(c8.codes, codes), "checkpoint codes"
    return got + (hh, c8, mm, rr)


def run_backward(ln, M, N, dt, pdt=None, ydt=None, group=128, dres=True, pad=0, seed=3, gamma=True, in_place=None):
    g = lib()
    dtype, dyt = TYPES[dt], TYPES[ydt or dt]
    h = ref.rows(M, N, dtype, seed, 0.5 if ln else 0.0)
    gam = params(N, ln, TYPES[pdt or dt])[0] if gamma else None
    mean, rstd, _, _ = ref.norm(ln, h, gam, None, 1e-6)
    mean, rstd = mean.float(), rstd.float()
    codes, scales = ref.checkpoint(h, group)
    dy = ref.rows(M, N, dyt, seed + 1, special=False)
    dr = ref.rows(M, N, dtype, seed + 2, special=False) if dres else None
    (dx, tx), (dg, tg), (db, tb) = ref.backward(ln, dy, codes, scales, group, gam, mean, rstd, dr)
    dyd, drd = (padded(dy, pad), padded(dr, pad)) if pad else (cuda(dy), cuda(dr))
    cod = padded(codes, pad, 0) if pad else cuda(codes)
    out = {"dy": dyd, "dres": drd, None: None}[in_place]
    ck = g.Checkpoint8(cod, cuda(scales), group)
    gx, gg, gb = g.norm_bwd_ck8(ln, dyd, ck, cuda(gam), cuda(mean) if ln else None, cuda(rstd), dres=drd,
                                dx_dtype=dtype, dx=out)
    if in_place:
        assert gx.data_ptr() == out.data_ptr()
    ref.held("dx", gx, dx, tx, dtype)
    ref.held("dgamma", gg, dg, tg)
    if ln:
        ref.held("dbeta", gb, db, tb)
    else:
        assert gb is None
    return gx, gg, gb


# ------------------------------------------------------------------ 8-bit output
LENGTHS = [1, 3, 8, 31, 64, 130, 256, 1000, 1003, 2048, 4096, 5120, 8192, 16384]


@pytest.mark.parametrize("N", LENGTHS)
@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_q8_lengths(N, ln, group):
    for M in (1, 37):
        run_forward(ln, M, N, "bf16", group=group)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pdt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("fmt", [E4M3, I8])
def test_q8_types(dt, pdt, ln, fmt):
    for N, group in ((384, 64), (2056, 0), (777, 256)):
        run_forward(ln, 19, N, dt, pdt=pdt, fmt=fmt, group=group, residual=N != 2056)


@pytest.mark.parametrize("N", [16392, 32768, 40000, 65537, 131072])
@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("group", [0, 256])
def test_q8_wide(N, ln, group):
    run_forward(ln, 6, N, "bf16", group=group, ck=128)


@pytest.mark.parametrize("pad", [8, 16, 3])
@pytest.mark.parametrize("ln", [False, True])
def test_q8_strided(pad, ln):
    for N in (512, 4096):
        run_forward(ln, 45, N, "bf16", group=64, pad=pad, ck=64)
        run_forward(ln, 45, N, "fp32", group=0, pad=pad)


@pytest.mark.parametrize("M", [2, 1000, 4099])
@pytest.mark.parametrize("ln", [False, True])
def test_q8_many_rows(M, ln):
    """More rows than CTAs hold at once, and the checkpoint along with the 8-bit output."""
    run_forward(ln, M, 1024, "bf16", group=128, ck=32)
    run_forward(ln, M, 264, "fp16", group=0, ck=256, fmt=I8)


def test_q8_scale_layouts():
    """Scales in the caller's buffer, rows first or groups first, and 8-bit rows inside wider ones: the same bits, and
    nothing written beside them."""
    g = lib()
    M, N, group = 53, 1000, 128
    x, (gamma, _) = ref.rows(M, N, torch.bfloat16, 1).cuda(), params(N, False, torch.bfloat16)
    gamma, G = gamma.cuda(), 8
    q0, s0, _, _, _ = g.norm_fwd_q8(False, x, gamma, None, 1e-6, group=group)
    for buf in (torch.full((G, M + 3), -1.0, device="cuda"), torch.full((M, G + 5), -1.0, device="cuda")):
        scale = buf[:, :M].t() if buf.shape[0] == G else buf[:, :G]
        qb = torch.full((M, N + 24), 7, device="cuda", dtype=torch.int8).view(E4M3)
        g.norm_fwd_q8(False, x, gamma, None, 1e-6, group=group, q=qb[:, :N], scale=scale)
        assert same_bits(scale, s0) and same_bits(qb[:, :N], q0)
        assert (qb[:, N:].view(torch.int8) == 7).all()
        assert (buf == -1.0).sum() == buf.numel() - M * G
        assert same_bits(g.read_q8(qb[:, :N], scale, group), g.read_q8(q0, s0, group))


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("over", ["x", "residual"])
def test_h_in_place(ln, over):
    """h over x or over the residual: the bits of the call with separate buffers."""
    g = lib()
    for M, N in ((33, 2048), (5, 1003), (3, 40000)):
        x, r = ref.rows(M, N, torch.bfloat16, 1).cuda(), ref.rows(M, N, torch.bfloat16, 2).cuda()
        gamma, beta = (cuda(t) for t in params(N, ln, torch.bfloat16))
        a = g.norm_fwd_q8(ln, x, gamma, beta, 1e-6, residual=r, group=128, checkpoint=g.checkpoint8_empty(M, N))
        x2, r2 = x.clone(), r.clone()
        b = g.norm_fwd_q8(ln, x2, gamma, beta, 1e-6, residual=r2, group=128, h=x2 if over == "x" else r2)
        for p, q in zip(a, b):
            assert (p is None and q is None) or same_bits(p, q)
        a = g.norm_fwd_ck8(ln, x, gamma, beta, 1e-6, residual=r)
        x3, r3 = x.clone(), r.clone()
        b = g.norm_fwd_ck8(ln, x3, gamma, beta, 1e-6, residual=r3, h=x3 if over == "x" else r3,
                           y=r3 if over == "x" else x3)
        for p, q in zip((a[0], a[1], *a[2][:2], *a[3:]), (b[0], b[1], *b[2][:2], *b[3:])):
            assert (p is None and q is None) or same_bits(p, q)


@pytest.mark.parametrize("N", [256, 1003, 8192, 40000])
@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("fmt", [E4M3, I8])
def test_rms_codes_do_not_depend_on_rstd(N, group, fmt):
    """RMSNorm's codes are those of h * gamma: the same bits at any eps, and exact where that product is exact."""
    g = lib()
    x = ref.rows(9, N, torch.bfloat16, 8)
    gamma = params(N, False, torch.bfloat16)[0]
    q, s, *_ = g.norm_fwd_q8(False, x.cuda(), gamma.cuda(), None, 1e-6, group=group, fmt=fmt)
    q2, s2, *_ = g.norm_fwd_q8(False, x.cuda(), gamma.cuda(), None, 3.0, group=group, fmt=fmt)
    assert same_bits(q, q2)
    t = x.float() * gamma.float()
    amax = torch.stack([b.abs().amax(1) for b in ref.blocks(t, group)], 1)
    inv = torch.where(amax < ref.TINY, torch.zeros_like(amax), torch.full_like(amax, ref.QMAX[fmt]) / amax)
    u = t * ref.spread(inv, group, N)
    want = torch.round(u).to(I8) if fmt == I8 else u.clamp(-448, 448).to(E4M3)
    assert torch.equal(q.cpu().float(), want.float())


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("N,group", [(512, 0), (512, 64), (1003, 128), (40000, 0), (40000, 256)])
def test_not_finite(ln, N, group):
    """A NaN makes every scale of its row NaN and its checkpoint group's pair NaN; other rows keep their bits."""
    g = lib()
    x = ref.rows(6, N, torch.bfloat16, 1)
    gamma, beta = (cuda(t) for t in params(N, ln, torch.bfloat16))
    ck0, ck1 = g.checkpoint8_empty(6, N), g.checkpoint8_empty(6, N)
    q0, s0, *_ = g.norm_fwd_q8(ln, x.cuda(), gamma, beta, 1e-6, group=group, checkpoint=ck0)
    x[4, N // 2] = float("nan")
    q, s, _, _, r = g.norm_fwd_q8(ln, x.cuda(), gamma, beta, 1e-6, group=group, checkpoint=ck1)
    assert torch.isnan(s[4]).all() and torch.isnan(r[4])
    assert torch.isnan(ck1.scales[4, (N // 2) // 128]).all()
    keep = torch.arange(6) != 4
    assert same_bits(raw(q)[keep], raw(q0)[keep]) and same_bits(s.cpu()[keep], s0.cpu()[keep])
    assert same_bits(ck1.codes.cpu()[keep], ck0.codes.cpu()[keep])
    x[4, N // 2] = float("inf")
    q, s, *_ = g.norm_fwd_q8(ln, x.cuda(), gamma, beta, 1e-6, group=group, checkpoint=ck1)
    at = (N // 2) // group if group else 0
    assert torch.isnan(s[4, at]) and torch.isnan(ck1.scales[4, (N // 2) // 128, 0])
    assert same_bits(raw(q)[keep], raw(q0)[keep])


def test_extreme_values():
    """fp32 rows near the ends of the range: very small groups become zeros with scale 0, neighbouring values of a huge
    size keep codes inside [-127, 127]."""
    g = lib()
    for N in (256, 1003, 40000):
        x = torch.randn(5, N, generator=torch.Generator().manual_seed(2))
        x[0] = 1e-32 * x[0]
        x[1] = 1e30
        x[1, ::2] = torch.nextafter(torch.tensor(1e30), torch.tensor(2e30))
        x[2] = x[2] * 1e16
        x[3] = 1e-15 * x[3]
        ck = g.checkpoint8_empty(5, N, 64)
        q, s, _, _, _ = g.norm_fwd_q8(False, x.cuda(), None, None, 0.0, group=64, checkpoint=ck)
        codes, scales = ref.checkpoint(x, 64)
        assert same_bits(ck.codes, codes) and same_bits(ck.scales, scales)
        assert (q[0].float() == 0).all() and (s[0] == 0).all()
        _, _, y, tol = ref.norm(False, x[2:], None, None, 0.0)
        ref.check_q8(False, x[2:], None, q[2:], s[2:], 64, y, tol)


ODD = [(300, 32), (500, 64), (1003, 128), (1999, 256), (3001, 128), (6001, 64), (12001, 32), (30001, 128), (60001, 256),
       (100001, 128)]


@pytest.mark.parametrize("N,group", ODD)
@pytest.mark.parametrize("ln", [False, True])
def test_odd_lengths(N, group, ln):
    """Rows without 16-byte vectors, from one warp to a cluster."""
    M = 33 if N < 10000 else 5
    run_forward(ln, M, N, "bf16", group=group, ck=group)
    run_forward(ln, M, N, "fp16", pdt="fp32", group=0, ck=group, residual=False, fmt=I8)
    run_forward(ln, M, N, "fp32", group=group)
    run_forward(ln, M, N, "fp32", group=0)
    run_forward(ln, M, N, "bf16", out="ck8", ck=group)
    run_backward(ln, M, N, "bf16", group=group)
    run_backward(ln, M, N, "fp32", ydt="bf16", group=group, dres=False)


@pytest.mark.parametrize("N", [131080, 200001])
@pytest.mark.parametrize("ln", [False, True])
def test_longer_than_a_cluster_holds(N, ln):
    g = lib()
    run_forward(ln, 3, N, "bf16", group=128, ck=128)
    assert g.q8_last_variant(0) == "elem"
    run_forward(ln, 3, N, "bf16", group=0)
    run_forward(ln, 3, N, "bf16", out="ck8", ck=64)
    run_backward(ln, 3, N, "bf16")
    assert g.q8_last_variant(1) == "elem"


def test_every_kernel_is_reached():
    """One call for each row capacity, aligned and not: the kernel named for it runs."""
    g = lib()
    names = [set(), set(), set()]
    for ln in (False, True):
        for N in (8, 256, 512, 1024, 2048, 4096, 5120, 6144, 8192, 12288, 16384, 32768, 65536, 131072, 131080, 7, 301, 1001,
                  2001, 4001, 8001, 16001, 32001, 65001, 131071):
            run_forward(ln, 2, N, "bf16", group=32, ck=32)
            names[0].add((ln, g.q8_last_variant(0)))
            run_backward(ln, 2, N, "bf16")
            names[1].add((ln, g.q8_last_variant(1)))
    for what, want in ((0, ("rows32x1c1", "rows256x4c1", "any32x1c1", "any512x2c8", "any1024x2c8", "elem")),
                       (1, ("rows32x1c1r2", "rows512x4c8r1", "any32x1c1", "any512x2c4", "any1024x2c8", "elem"))):
        for ln in (False, True):
            have = {v for l, v in names[what] if l == ln}
            assert have >= set(want) - ({"rows256x4c1"} if ln and what else set()), (what, ln, have)


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("N", [256, 1003, 5128, 40000, 140000])
def test_squares_beyond_fp32(N, ln):
    """Finite rows whose squares are not: rstd is 0 and the rows are zeros (scale 0), as the general form's are; the
    rows beside them keep their values."""
    g = lib()
    x = torch.randn(3, N, generator=torch.Generator().manual_seed(1))
    x[1] *= 1e25
    gamma, _ = params(N, ln, torch.float32)
    for group in (0, 128):
        q, s, _, _, rstd = g.norm_fwd_q8(ln, x.cuda(), gamma.cuda(), None, 1e-6, group=group)
        assert rstd[1] == 0 and (s[1] == 0).all()
        _, _, y, tol = ref.norm(ln, x, gamma, None, 1e-6)
        for i in (0, 2):
            ref.check_q8(ln, x[i:i + 1], gamma, q[i:i + 1], s[i:i + 1], group, y[i:i + 1], tol[i:i + 1])
    y, _, _, _, rstd = g.norm_fwd_ck8(ln, x.cuda(), gamma.cuda(), None, 1e-6)
    want, _, _, r = g.norm_fwd_ex(ln, x.cuda(), gamma.cuda(), None, 1e-6)
    assert rstd[1] == 0 and r[1] == 0 and (y[1] == 0).all() and (want[1] == 0).all()


# ------------------------------------------------------------------ checkpointed forward
@pytest.mark.parametrize("N", LENGTHS + [16392, 40000])
@pytest.mark.parametrize("ln", [False, True])
def test_ck8_forward_lengths(N, ln):
    for M, group in ((1, 32), (37, 128)):
        run_forward(ln, M, N, "bf16", out="ck8", ck=group)


@pytest.mark.parametrize("dt,pdt,ydt", [("bf16", "fp32", "bf16"), ("fp16", "fp16", "fp32"), ("fp32", "fp32", "bf16"),
                                        ("fp32", "bf16", "fp32"), ("bf16", "fp16", "fp16")])
@pytest.mark.parametrize("ln", [False, True])
def test_ck8_forward_types(dt, pdt, ydt, ln):
    for N in (512, 1003, 8200, 24576):
        run_forward(ln, 11, N, dt, pdt=pdt, ydt=ydt, out="ck8", ck=256, residual=N != 512)


# ------------------------------------------------------------------ backward
@pytest.mark.parametrize("N", LENGTHS + [16392, 32768, 65537])
@pytest.mark.parametrize("ln", [False, True])
def test_ck8_backward_lengths(N, ln):
    for M, group in ((1, 32), (37, 128)):
        run_backward(ln, M, N, "bf16", group=group)


@pytest.mark.parametrize("dt,pdt,ydt", [("bf16", "fp32", "bf16"), ("fp16", "fp16", "fp16"), ("fp32", "fp32", "fp32"),
                                        ("fp32", "fp32", "bf16"), ("bf16", "bf16", "fp32"), ("fp16", "bf16", "bf16")])
@pytest.mark.parametrize("ln", [False, True])
def test_ck8_backward_types(dt, pdt, ydt, ln):
    for N, group in ((512, 32), (1003, 64), (5120, 128), (16384, 256), (24576, 128)):
        run_backward(ln, 23, N, dt, pdt=pdt, ydt=ydt, group=group, dres=N != 512)


@pytest.mark.parametrize("M", [2, 3, 151, 153, 1000, 4099])
@pytest.mark.parametrize("ln", [False, True])
def test_ck8_backward_many_rows(M, ln):
    run_backward(ln, M, 1024, "bf16")
    run_backward(ln, M, 264, "fp16", dres=False)


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("pad", [8, 16, 3])
def test_ck8_backward_strided(ln, pad):
    for N in (512, 4096, 20480):
        run_backward(ln, 45, N, "bf16", pad=pad)


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("in_place", ["dy", "dres"])
def test_ck8_backward_in_place(ln, in_place):
    for M, N in ((77, 4096), (5, 1003), (9, 32768)):
        run_backward(ln, M, N, "bf16", in_place=in_place)


@pytest.mark.parametrize("ln", [False, True])
def test_ck8_backward_options(ln):
    """No gamma; sums that are not asked for leave the others as they are; the same call twice gives the same bits."""
    g = lib()
    run_backward(ln, 31, 1024, "bf16", gamma=False)
    for N in (1024, 1003, 32768):
        h, dy = ref.rows(300, N, torch.bfloat16, 1).cuda(), ref.rows(300, N, torch.bfloat16, 2).cuda()
        gamma, beta = (cuda(t) for t in params(N, ln, torch.bfloat16))
        _, _, ck, mean, rstd = g.norm_fwd_ck8(ln, h, gamma, beta, 1e-6)
        a = g.norm_bwd_ck8(ln, dy, ck, gamma, mean, rstd)
        b = g.norm_bwd_ck8(ln, dy, ck, gamma, mean, rstd)
        c = g.norm_bwd_ck8(ln, dy, ck, gamma, mean, rstd, need_dgamma=False, need_dbeta=False)
        assert same_bits(a[0], b[0]) and same_bits(a[1], b[1]) and (not ln or same_bits(a[2], b[2]))
        assert same_bits(a[0], c[0]) and c[1] is None and c[2] is None


@pytest.mark.parametrize("ln", [False, True])
def test_gradient_against_differences(ln):
    """dx and dgamma against central differences in 64 bits of L = sum dy * norm(v) about the rows v that the
    checkpoint stands for, with v's own statistics.

    Richardson's combination (4 D(e) - D(2e)) / 3 at e = 1e-4 is off by O(e^4) of derivatives of order one and by
    rounding 2^-53 |L| / e, both below 1e-8; the kernel's fp32 outputs by the bound of ref.backward."""
    g = lib()
    M, N, group, eps = 3, 40, 32, 1e-3
    h = ref.rows(M, N, torch.float32, 4, 0.3, special=False)
    codes, scales = ref.checkpoint(h, group)
    v, _ = ref.values(codes, scales, group)
    gamma, _ = params(N, ln, torch.float32)
    dy = ref.rows(M, N, torch.float32, 6, special=False)

    def loss(v, gam):
        mean = v.mean(1, keepdim=True) if ln else 0.0
        return (dy.double() * ((v - mean) / torch.sqrt((v - mean).square().mean(1, keepdim=True) + eps) * gam)).sum()

    def diff(f, t):
        out = torch.zeros_like(t)
        for i in range(t.numel()):
            d = torch.zeros_like(t)
            d.view(-1)[i] = 1.0
            D = [(f(t + e * d) - f(t - e * d)) / (2 * e) for e in (1e-4, 2e-4)]
            out.view(-1)[i] = (4 * D[0] - D[1]) / 3
        return out
    mean = v.mean(1) if ln else torch.zeros(M, dtype=torch.float64)
    rstd = 1 / torch.sqrt((v - mean[:, None]).square().mean(1) + eps)
    dx, dg, _ = g.norm_bwd_ck8(ln, dy.cuda(), g.Checkpoint8(codes.cuda(), scales.cuda(), group), gamma.cuda(),
                               mean.float().cuda() if ln else None, rstd.float().cuda())
    (_, tx), (_, tg), _ = ref.backward(ln, dy, codes, scales, group, gamma, mean.float(), rstd.float(), None)
    # the statistics rounded to fp32 move every xhat by at most 2 u (|xhat| + |mean| rstd)
    more = 16 * U * rstd.max() * dy.abs().max() * (1 + v.abs().max() * rstd.max()) ** 2 + 1e-8
    ref.held("dx", dx, diff(lambda t: loss(t, gamma.double()), v), tx + more)
    ref.held("dgamma", dg, diff(lambda t: loss(v, t), gamma.double()), tg + M * more)


# ------------------------------------------------------------------ reading back
@pytest.mark.parametrize("N", LENGTHS + [16392, 65536])
@pytest.mark.parametrize("ydt", ["bf16", "fp16", "fp32"])
def test_read(N, ydt):
    """Both formats, with and without the norm on top."""
    g = lib()
    M, yt = 29, TYPES[ydt]
    gen = torch.Generator().manual_seed(N)
    gamma, beta = params(N, True, TYPES[ydt if N % 2 else "fp32"])
    mean, rstd = torch.randn(M, generator=gen), torch.rand(M, generator=gen) + 0.5
    for group in (32, 128, 256):
        codes, scales = ref.checkpoint(ref.rows(M, N, torch.float32, N), group)
        v, size = ref.values(codes, scales, group)
        ck = g.Checkpoint8(codes.cuda(), scales.cuda(), group)
        ref.held("values", g.read_ck8(ck, y_dtype=yt), v, 2 * U * size, yt)
        y = g.read_ck8(ck, mean=mean.cuda(), rstd=rstd.cuda(), gamma=gamma.cuda(), beta=beta.cuda(), y_dtype=yt)
        m, r = mean.double()[:, None], rstd.double()[:, None]
        t = 6 * U * (size + m.abs()) * r * gamma.double().abs() + 2 * U * beta.double().abs()
        ref.held("norm", y, (v - m) * r * gamma.double() + beta.double(), t, yt)
    for group in (0, 64):
        G = -(-N // group) if group else 1
        q = (torch.randn(M, N, generator=gen) * 100).clamp(-448, 448).to(E4M3)
        s = torch.rand(M, G, generator=gen) + 0.1
        want = q.float().double() * ref.spread(s.double(), group, N)
        ref.held("e4m3", g.read_q8(q.cuda(), s.cuda(), group, y_dtype=yt), want, 2 * U * want.abs(), yt)


def test_read_every_code():
    """Every e4m3 and int8 code as itself."""
    g = lib()
    for N in (256, 255):
        b = torch.arange(N, dtype=torch.int16).to(torch.uint8)[None].repeat(3, 1)
        for dt in (E4M3, I8):
            q = b.view(dt)
            y = g.read_q8(q.cuda(), torch.ones(3, 1, device="cuda"), y_dtype=torch.float32).cpu()
            want = q.float()
            assert torch.equal(torch.isnan(y), torch.isnan(want))
            ok = ~torch.isnan(want)
            assert torch.equal(y[ok], want[ok])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("N", [1024, 1003])
def test_training_step(ln, N):
    """A layer's forward and backward as a program runs them: residual sum, 8-bit output for the product and
    checkpoint in one call; the weight gradient from the output computed again; dx of the norm with the residual
    stream's gradient.  The product itself is torch's."""
    g = lib()
    M, K, group = 200, 96, 128
    x, r = ref.rows(M, N, torch.bfloat16, 1), ref.rows(M, N, torch.bfloat16, 2, special=False)
    gamma, beta = params(N, ln, torch.float32)
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(9)) / N ** 0.5
    dout = ref.rows(M, K, torch.bfloat16, 7, special=False)
    dres = ref.rows(M, N, torch.bfloat16, 8, special=False)
    ck = g.checkpoint8_empty(M, N, group)
    q, scale, h, mean, rstd = g.norm_fwd_q8(ln, x.cuda(), gamma.cuda(), cuda(beta), 1e-6, residual=r.cuda(),
                                            checkpoint=ck)
    y8 = g.read_q8(q, scale, y_dtype=torch.float32)
    dy = (dout.cuda().float() @ w.cuda().t()).to(torch.bfloat16)
    y2 = g.read_ck8(ck, mean=mean, rstd=rstd, gamma=gamma.cuda(), beta=cuda(beta), y_dtype=torch.float32)
    dx, dg, db = g.norm_bwd_ck8(ln, dy, ck, gamma.cuda(), mean, rstd, dres=dres.cuda())
    # the forward's values against the norm in 64 bits: half a code's step, half a checkpoint step
    hh = ref.add(x, r)
    _, _, y, tol = ref.norm(ln, hh, gamma, beta, 1e-6)
    ref.check_q8(ln, hh, gamma, q, scale, 0, y, tol)
    assert torch.equal(y8.cpu(), q.cpu().float() * scale.cpu())
    codes, scales = ref.checkpoint(hh, group)
    step = ref.spread(scales[..., 0].double(), group, N) * 0.5 * rstd.cpu().double()[:, None] * gamma.double().abs()
    size = (hh.double().abs() + ref.spread(scales[..., 1].double().abs(), group, N)) * rstd.cpu().double()[:, None]
    ref.held("y again", y2, y, step * (1 + 1e-5) + tol + 16 * U * size * gamma.double().abs())
    (wx, tx), (wg, tg), (wb, tb) = ref.backward(ln, dy.cpu(), codes, scales, group, gamma, mean.cpu() if ln else None,
                                                rstd.cpu(), dres)
    ref.held("dx", dx, wx, tx, torch.bfloat16)
    ref.held("dgamma", dg, wg, tg)
    if ln:
        ref.held("dbeta", db, wb, tb)


def test_streams_and_graph():
    """On a stream of its own, and captured and replayed on new inputs: the bits of the eager calls."""
    g = lib()
    M, N = 64, 4096
    x, r, dy = (ref.rows(M, N, torch.bfloat16, k).cuda() for k in (1, 2, 3))
    gamma = params(N, False, torch.bfloat16)[0].cuda()

    def step(x, r, dy):
        ck = g.checkpoint8_empty(M, N)
        q, s, h, _, rstd = g.norm_fwd_q8(False, x, gamma, None, 1e-6, residual=r, group=128, checkpoint=ck)
        dx, dg, _ = g.norm_bwd_ck8(False, dy, ck, gamma, None, rstd, dres=h)
        return [q, s, h, rstd, dx, dg, g.read_ck8(ck)]
    want = step(x, r, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(x, r, dy)
    torch.cuda.current_stream().wait_stream(side)
    assert all(same_bits(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(torch.cuda.Stream()):  # the argument counts, not the current stream
        y, h, ck, _, rstd = g.norm_fwd_ck8(False, x, gamma, None, 1e-6, residual=r, stream=side)
        dx, dg, _ = g.norm_bwd_ck8(False, dy, ck, gamma, None, rstd, dres=h, stream=side)
        v = g.read_ck8(ck, stream=side)
        q, s, *_ = g.norm_fwd_q8(False, x, gamma, None, 1e-6, residual=r, group=128, stream=side)
        u = g.read_q8(q, s, 128, stream=side)
    side.synchronize()
    assert all(same_bits(a, b) for a, b in zip((q, s, h, rstd, dx, dg, v), want)) and same_bits(u, g.read_q8(q, s, 128))
    xs, rs, ds = (torch.empty_like(t) for t in (x, r, dy))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(xs, rs, ds)
    for k in (0, 10):
        new = [ref.rows(M, N, torch.bfloat16, k + j).cuda() for j in (1, 2, 3)]
        for a, b in zip((xs, rs, ds), new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(out, step(*new)))


def test_captured_before_any_eager_call():
    """A shape and types that nothing ran before, captured at once and replayed; two graphs side by side."""
    g = lib()
    M, N = 21, 2824
    x, dy = ref.rows(M, N, torch.float16, 1).cuda(), ref.rows(M, N, torch.float16, 2).cuda()
    gamma, beta = (cuda(t) for t in params(N, True, torch.float32))

    def step(x):
        y, _, ck, mean, rstd = g.norm_fwd_ck8(True, x, gamma, beta, 1e-5, group=32)
        return [y, *ck[:2], *g.norm_bwd_ck8(True, dy, ck, gamma, mean, rstd), g.read_ck8(ck, y_dtype=torch.float16)]
    x2 = (x * 0.5).contiguous()
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph, t in zip(graphs, (x, x2)):
        with torch.cuda.graph(graph):
            outs.append(step(t))
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for t, out in zip((x, x2), outs):
        assert all(same_bits(a, b) for a, b in zip(out, step(t)))


def test_host_threads():
    """Calls from several host threads, each on its stream, give the bits of the calls one after another."""
    import threading
    g = lib()
    xs = [ref.rows(65, N, torch.bfloat16, k).cuda() for k, N in enumerate((1024, 4096, 1003, 32768))]
    gammas = [params(x.shape[1], False, torch.bfloat16)[0].cuda() for x in xs]

    def step(k):
        q, s, *_ , rstd = g.norm_fwd_q8(False, xs[k], gammas[k], None, 1e-6, group=64)
        y, _, ck, _, r2 = g.norm_fwd_ck8(False, xs[k], gammas[k], None, 1e-6)
        return [q, s, rstd, y, *ck[:2], *g.norm_bwd_ck8(False, xs[k], ck, gammas[k], None, r2)[:2]]
    want = [step(k) for k in range(4)]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(5):
                got[k] = step(k)
        stream.synchronize()
    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(same_bits(a, b) for w, o in zip(want, got) for a, b in zip(w, o))


@pytest.mark.parametrize("N", [256, 1000, 8192, 40000])
@pytest.mark.parametrize("fmt", [E4M3, I8])
def test_unaligned_rows_give_the_same_codes(N, fmt):
    """Rows one element off a 16-byte boundary: the codes and checkpoint bits of the aligned call (they are defined by
    the rows alone), read back to the same values."""
    g = lib()
    M = 19
    x, r = ref.rows(M, N, torch.bfloat16, 1).cuda(), ref.rows(M, N, torch.bfloat16, 2).cuda()
    gamma = params(N, False, torch.bfloat16)[0].cuda()

    def off(t, dtype=None):
        buf = torch.zeros(M, N + 9, device="cuda", dtype=dtype or t.dtype)
        if t is not None:
            buf[:, 1:N + 1].copy_(t)
        return buf[:, 1:N + 1]
    for group in (0, 32, 256):
        a = g.checkpoint8_empty(M, N, 64)
        q, s, h, _, _ = g.norm_fwd_q8(False, x, gamma, None, 1e-6, residual=r, group=group, fmt=fmt, checkpoint=a)
        b = g.Checkpoint8(off(None, torch.int8), torch.empty_like(a.scales), 64)
        q2, s2, h2, _, _ = g.norm_fwd_q8(False, off(x), gamma, None, 1e-6, residual=off(r), group=group, checkpoint=b,
                                         q=off(None, torch.uint8).view(fmt), h=off(None, x.dtype))
        assert "any" in g.q8_last_variant(0) and same_bits(q, q2) and same_bits(h, h2)
        assert same_bits(a.codes, b.codes) and same_bits(a.scales, b.scales)
        assert ((s - s2).abs() <= 1e-5 * s).all()
        assert same_bits(g.read_q8(q, s, group, y=off(None, torch.bfloat16)), g.read_q8(q, s, group))
        assert g.q8_last_variant(2) == "vec"
        assert same_bits(g.read_ck8(b), g.read_ck8(a))


def test_workspace_follows_the_partial_rows():
    """One partial row per row group that runs at once: tens of MB for wide rows, and a workspace one byte short refused."""
    g = lib()
    for N in (1003, 4096, 16384, 131072, 200000):
        for ln in (False, True):
            row = 4 * N * (2 if ln else 1)  # one partial row
            # at most four row groups an SM; a CTA or a cluster an SM for wide rows
            most = (4 if N <= 16384 else 1) * torch.cuda.get_device_properties(0).multi_processor_count
            assert row <= g.norm_bwd_ck8_workspace_size(ln, 1 << 20, N) <= most * row + 255
            assert row <= g.norm_bwd_ck8_workspace_size(ln, 1, N) <= row + 255
    x = ref.rows(64, 4096, torch.bfloat16, 1).cuda()
    _, _, ck, _, rstd = g.norm_fwd_ck8(False, x, None, None, 1e-6)
    need = g.norm_bwd_ck8_workspace_size(False, 64, 4096)
    ws = torch.empty(need, device="cuda", dtype=torch.uint8)
    a = g.norm_bwd_ck8(False, x, ck, None, None, rstd, workspace=ws)
    b = g.norm_bwd_ck8(False, x, ck, None, None, rstd)
    assert same_bits(a[0], b[0]) and same_bits(a[1], b[1])
    with pytest.raises(g.GbnormError):
        g.norm_bwd_ck8(False, x, ck, None, None, rstd, workspace=ws[:need - 1])


def test_offsets_beyond_32_bits():
    """Rows whose strides put the last one past 2^31 elements: the bits of contiguous rows."""
    g = lib()
    M, ld = 3, (1 << 30) + 8
    for N in (4096, 1003):
        x, r, dy = (ref.rows(M, N, torch.bfloat16, k, special=False).cuda() for k in (1, 2, 3))
        gamma = params(N, False, torch.bfloat16)[0].cuda()

        def far(t, dtype=torch.bfloat16):
            buf = torch.empty((M - 1) * ld + N, device="cuda", dtype=torch.uint8 if dtype == E4M3 else dtype)
            v = (buf.view(E4M3) if dtype == E4M3 else buf).as_strided((M, N), (ld, 1))
            if t is not None:
                v.copy_(t)
            return v
        xf, rf, hf = far(x), far(r), far(None)
        want = g.norm_fwd_q8(False, x, gamma, None, 1e-6, residual=r, group=64)
        got = g.norm_fwd_q8(False, xf, gamma, None, 1e-6, residual=rf, group=64, q=far(None, E4M3), h=hf)
        assert all(same_bits(a, b) for a, b in zip(got[:3], want[:3]))
        assert same_bits(g.read_q8(got[0], got[1], 64, y=rf), g.read_q8(want[0], want[1], 64))
        ck = g.Checkpoint8(far(None, torch.int8), torch.empty(M, -(-N // 64), 2, device="cuda"), 64)
        y, _, _, _, rstd = g.norm_fwd_ck8(False, xf, gamma, None, 1e-6, checkpoint=ck, y=hf)
        y2, _, ck2, _, rstd2 = g.norm_fwd_ck8(False, x, gamma, None, 1e-6, group=64)
        assert same_bits(y, y2) and same_bits(ck.codes, ck2.codes) and same_bits(ck.scales, ck2.scales)
        a = g.norm_bwd_ck8(False, far(dy), ck, gamma, None, rstd, dx=xf)
        b = g.norm_bwd_ck8(False, dy, ck2, gamma, None, rstd2)
        assert same_bits(a[0], b[0]) and same_bits(a[1], b[1])


def test_no_rows():
    g = lib()
    x = torch.empty(0, 512, device="cuda", dtype=torch.bfloat16)
    gamma = torch.ones(512, device="cuda", dtype=torch.bfloat16)
    q, s, h, m, r = g.norm_fwd_q8(True, x, gamma, None, 1e-6, residual=x, group=128)
    assert q.shape == (0, 512) and s.shape == (0, 4) and h.shape == (0, 512)
    y, h, ck, m, r = g.norm_fwd_ck8(True, x, gamma, None, 1e-6)
    dx, dg, db = g.norm_bwd_ck8(True, x, ck, gamma, m, r)
    assert dx.shape == (0, 512) and (dg == 0).all() and (db == 0).all()
    assert g.read_ck8(ck).shape == (0, 512)


def test_grid_limit_keeps_the_bits():
    """Fewer CTAs, more rows each: outputs per row are the same bits."""
    g = lib()
    for N in (1024, 1003, 32768):
        x, dy = ref.rows(70, N, torch.bfloat16, 1).cuda(), ref.rows(70, N, torch.bfloat16, 2).cuda()
        gamma, beta = (cuda(t) for t in params(N, True, torch.bfloat16))

        def step():
            ck = g.checkpoint8_empty(70, N)
            q, s, _, mean, rstd = g.norm_fwd_q8(True, x, gamma, beta, 1e-6, checkpoint=ck)
            dx, dg, db = g.norm_bwd_ck8(True, dy, ck, gamma, mean, rstd)
            return (q, s, mean, rstd, *ck[:2], dx), (dg, db)
        a, sa = step()
        g.set_grid_limit(3)
        try:
            b, sb = step()
        finally:
            g.set_grid_limit(0)
        assert all(same_bits(p, q) for p, q in zip(a, b))
        for p, q in zip(sa, sb):  # another order of the same 70 terms: at most 140 roundings of |terms| apart
            assert ((p - q).abs() <= 140 * U * 70 * 60).all()


def test_binding_refuses():
    g = lib()
    x = torch.randn(4, 256, device="cuda", dtype=torch.bfloat16)
    gamma = torch.ones(256, device="cuda", dtype=torch.bfloat16)
    ck = g.checkpoint8_empty(4, 256)
    rstd = torch.ones(4, device="cuda")
    bad = [
        lambda: g.norm_fwd_q8(False, x.cpu(), gamma, None, 1e-6),
        lambda: g.norm_fwd_q8(False, x, gamma.cpu(), None, 1e-6),
        lambda: g.norm_fwd_q8(False, x.t(), gamma, None, 1e-6),
        lambda: g.norm_fwd_q8(False, x, gamma[:128], None, 1e-6),
        lambda: g.norm_fwd_q8(False, x, gamma, None, 1e-6, group=48),
        lambda: g.norm_fwd_q8(False, x, gamma, None, 1e-6, fmt=torch.uint8),
        lambda: g.norm_fwd_q8(False, x, gamma, None, 1e-6, residual=x.float()),
        lambda: g.norm_fwd_q8(False, x, gamma, None, 1e-6, scale=torch.empty(4, device="cuda")),
        lambda: g.norm_fwd_q8(False, x.to(torch.float64), gamma, None, 1e-6),
        lambda: g.norm_fwd_ck8(False, x, gamma, None, 1e-6, group=0),
        lambda: g.norm_fwd_ck8(False, x, gamma, None, 1e-6, checkpoint=g.Checkpoint8(ck.codes, ck.scales, 64)),
        lambda: g.norm_fwd_ck8(False, x, gamma, None, 1e-6, checkpoint=g.checkpoint8_empty(3, 256)),
        lambda: g.norm_fwd_ck8(False, x, gamma, None, 1e-6, y_dtype=torch.int8),
        lambda: g.norm_bwd_ck8(True, x, ck, gamma, None, rstd),
        lambda: g.norm_bwd_ck8(False, x, ck, gamma, None, None),
        lambda: g.norm_bwd_ck8(False, x, ck, gamma, None, rstd[:3]),
        lambda: g.norm_bwd_ck8(False, x, ck, gamma, None, rstd, dres=x.float(), dx=torch.empty_like(x)),
        lambda: g.read_q8(x, rstd[:, None]),
        lambda: g.read_q8(ck.codes, rstd[:, None], group=128),
        lambda: g.read_ck8(ck, y_dtype=torch.int32),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {k} was taken")
    refused = [
        lambda: g.norm_fwd_q8(False, x, gamma, None, float("nan")),
        lambda: g.norm_fwd_q8(False, x, gamma, None, 1e-6, h=torch.empty_like(x)),  # no residual
        lambda: g.norm_fwd_q8(False, x, gamma, None, 1e-6, residual=x, h=gamma.expand(4, 256)),  # stride 0
        lambda: g.norm_fwd_q8(False, x, gamma, None, 1e-6, scale=rstd[:1, None].expand(4, 1)),
        lambda: g.norm_fwd_q8(False, x, gamma, None, 1e-6, q=x.view(torch.int8)[:, :256]),
        lambda: g.norm_bwd_ck8(False, x, ck, gamma, None, rstd, workspace=torch.empty(8, device="cuda")),
    ]
    for k, f in enumerate(refused):
        with pytest.raises(g.GbnormError):
            f()
            pytest.fail(f"call {k} was taken")
