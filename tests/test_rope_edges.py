"""Head operators at the edges of what their documentation allows: very many tokens, parameters that are not finite, large
frequencies; cosines and sines to their last bits, column sums to their additions (GPU)."""
import pytest
import torch

import rope_ref as ref
from test_rope import EPS, _no_device_fault, cuda, lib, place, plan, positions, rotation  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ln", [False, True])
def test_workspace_of_more_tokens_than_a_batch_may_have(ln):
    """The size is of batches * tokens; beyond what fills the grid it does not grow."""
    size = lib().qk_norm_rope_bwd_workspace_size
    full = size(ln, 2 ** 31 - 1, 8, 2, 128)
    assert full > 0
    for tokens in (2 ** 31, 2 ** 32, 2 ** 40):
        assert size(ln, tokens, 8, 2, 128) == full
    assert size(ln, 2 ** 40 + 1, 8, 2, 128) == 0 and size(ln, -1, 8, 2, 128) == 0


def test_backward_of_more_than_2_31_tokens():
    """Batches of the same tokens (stride 0) all get the gradient of one batch."""
    g = lib()
    B, S, D = 32769, 65536, 2
    q, dy = (ref.heads(1, S, 1, D, torch.bfloat16, s).cuda() for s in (1, 2))
    r, pos = plan(rotation(D)[0], None, False), positions(1, S, 1)[0].cuda()
    rstd = g.qk_norm_rope_fwd(False, q, None, None, None, EPS, pos, r)[3]
    want = g.qk_norm_rope_bwd(False, dy, None, q, None, None, None, None, rstd, pos, r, need_dgamma=False)[0]
    dx = g.qk_norm_rope_bwd(False, dy.expand(B, S, 1, D), None, q.expand(B, S, 1, D), None, None, None, None,
                            rstd.expand(B, S, 1).contiguous(), pos, r, need_dgamma=False)[0]
    assert B * S > 2 ** 31 and torch.equal(dx, want.expand_as(dx))


@pytest.mark.parametrize("dt,how", [("bf16", "dense"), ("bf16", "two"), ("fp32", "dense"), ("fp16", "odd")])
@pytest.mark.parametrize("D,rot", [(128, 64), (128, 0), (80, 32), (72, 24), (98, 40), (600, 64)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_parameter_that_is_not_finite_reaches_its_own_element(D, rot, inter, bad, dt, how):
    """A NaN or an infinity in gamma or beta reaches its element, that one's partner if the pair is rotated, no other."""
    g = lib()
    if rot == 0 and inter:
        pytest.skip("no pairs")
    dtype = ref.TYPES[dt]
    r, pos = (plan(rotation(rot)[0], None, inter), positions(1, 3, 1).cuda() + 1) if rot else (None, None)
    q = place(torch.randn(1, 3, 5, D, generator=torch.Generator().manual_seed(1)).to(dtype), how)
    a, b = ref.pairs(rot, inter)
    for at in {0, max(rot - 1, 0), rot, (rot + D) // 2, D - 1}:
        hit = torch.zeros(D, dtype=torch.bool)
        hit[at] = True
        if at < rot:
            j = [i for i in range(rot // 2) if at in (a[i], b[i])][0]
            hit[a[j]] = hit[b[j]] = True
        w = torch.ones(D, dtype=dtype)
        w[at] = bad
        none = torch.ones(D, dtype=dtype)
        for ln, gamma, beta in ((False, w, None), (True, w, None), (True, none, w)):
            y = g.qk_norm_rope_fwd(ln, q, None, cuda(gamma), None, EPS, pos, r, beta_q=cuda(beta))[0].cpu()
            assert not torch.isfinite(y[..., hit]).any() and torch.isfinite(y[..., ~hit]).all(), (at, ln, beta is None)


def test_large_frequencies_at_far_positions():
    """Frequencies up to 2^87 with all bits of their mantissas set, at positions where half a unit of 2^-64 turns in
    the frequency is 2^-25 turns of the angle; against exact turns."""
    from fractions import Fraction
    g = lib()
    pi = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679,
                  10 ** 100)
    big = [2.0 ** e * (2 - 2.0 ** -23) for e in (0, 40, 60, 62, 63, 64, 67, 70, 73, 75, 77, 80, 82, 84, 85, 86)]
    f = torch.tensor([(-1) ** i * v for i, v in enumerate(big)], dtype=torch.float64).float()
    D = 2 * len(big)
    pos = torch.tensor([[1, 2 ** 20 + 1, 2 ** 33 - 7, -2 ** 36 + 5, 2 ** 40, 2 ** 40 - 1]])
    turns = [[float((int(p) * Fraction(float(w)) / (2 * pi)) % 1) for w in f] for p in pos[0]]
    angle = 2 * torch.pi * torch.tensor(turns, dtype=torch.float64)[None, :, None]
    far = pos.double().abs()[..., None, None]
    q = ref.heads(1, pos.shape[1], 3, D, torch.float32, 1)
    for inter in (False, True):
        want, tol = ref.forward(None, q, None, None, 0, angle, far, D, inter)[2]
        ref.held("yq", g.rope_fwd(q.cuda(), None, pos.cuda(), plan(f, None, inter))[0], want, tol + 1e-14)


@pytest.mark.parametrize("D,inter,how", [(128, False, "dense"), (128, True, "dense"), (98, True, "two"), (98, False, "odd")])
def test_cosines_and_sines_to_an_fp32_unit(D, inter, how):
    """Pairs (1, 0) turned are the cosine and the sine themselves: 1 ulp of sinpi and cospi below 1 (2^-24), and the
    angle's rounding to fp32 when at most an eighth of a turn is left of it (pi 2^-27).  The angles here are below 2^12
    radians, the reference's own product within 2^-41."""
    g = lib()
    S, gen = 4096, torch.Generator().manual_seed(3)
    f = torch.rand(D // 2, generator=gen)
    a, b = ref.pairs(D, inter)
    q = torch.zeros(1, S, 1, D)
    q[..., a] = 1.0
    angle, _ = ref.angles(torch.arange(S)[None], f, None, 1, S)
    y = g.rope_fwd(place(q, how), None, torch.arange(S)[None].cuda(), plan(f, None, inter))[0].cpu().double()
    tol = 2.0 ** -24 + torch.pi * 2.0 ** -27 + 2.0 ** -40
    assert (y[..., a] - torch.cos(angle)).abs().max() <= tol and (y[..., b] - torch.sin(angle)).abs().max() <= tol


@pytest.mark.parametrize("D,rot,dt,how", [(128, 128, "bf16", "dense"), (128, 64, "fp16", "dense"), (80, 32, "bf16", "dense"),
                                          (64, 64, "fp32", "two"), (98, 40, "bf16", "odd")])
@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_in_the_backwards_input(D, rot, dt, how, ln, inter, bad):
    """With the statistics given, a NaN or an infinity in x reaches its head of dx and its column of its tensor's dgamma,
    an infinity as an infinity; every other output keeps its bits.  The heads do not fill their passes."""
    g = lib()
    S, heads, dtype = 5, (11, 3), ref.TYPES[dt]
    r, pos = plan(rotation(rot)[0], None, inter), positions(1, S, 1).cuda()
    x = [ref.heads(1, S, h, D, dtype, h) for h in heads]
    dy = [place(torch.randn(1, S, h, D, generator=torch.Generator().manual_seed(h)).to(dtype), how) for h in heads]
    rstd, mean = torch.ones(1, S, sum(heads)).cuda(), torch.zeros(1, S, sum(heads)).cuda() if ln else None

    def run():
        return g.qk_norm_rope_bwd(ln, *dy, *[place(t, how) for t in x], None, None, mean, rstd, pos, r)
    clean = run()
    for i in (0, 1):
        for head in (heads[i] - 1, heads[i] // 2):
            for at in (0, rot - 1, D - 1):
                x[i][0, 2, head, at], keep = bad, x[i][0, 2, head, at].clone()
                got = run()
                x[i][0, 2, head, at] = keep
                assert not torch.isfinite(got[i][0, 2, head]).all()
                got[i][0, 2, head] = clean[i][0, 2, head]
                value = got[2][i, at].item()
                assert abs(value) == bad if bad == float("inf") else value != value
                got[2][i, at] = clean[2][i, at]
                assert all(torch.equal(a, b) for a, b in zip(got[:3], clean[:3]))
                assert (got[3] is None) if not ln else torch.equal(got[3], clean[3])


@pytest.mark.parametrize("limit", [1, 2])
@pytest.mark.parametrize("B,S,hq,hk", [(7, 25, 9, 2), (131, 1, 9, 2), (1, 97, 3, 1), (40, 3, 5, 0)])
@pytest.mark.parametrize("D", [128, 80, 98])
@pytest.mark.parametrize("ln", [False, True])
def test_column_sums_of_few_warps(limit, B, S, hq, hk, D, ln):
    """dgamma and dbeta on a grid of one or two CTAs, held to the additions that its longest chain makes: a lane adds a
    value a pass of its warp (whole tokens, then a share of the other passes), then come the groups of lanes of a warp,
    the 8 warps of a CTA, and the partial rows, one after another."""
    import re
    g = lib()
    try:
        g.set_grid_limit(limit)
        f, _ = rotation(D)
        pos = positions(B, S, 1)
        angle, far = ref.angles(pos, f, None, B, S)
        r = plan(f, None, False)
        H = [h for h in (hq, hk) if h]
        x = [ref.heads(B, S, h, D, torch.bfloat16, h, 0.5 if ln else 0.0) for h in H]
        dy = [ref.heads(B, S, h, D, torch.bfloat16, h + 20) for h in H]
        stats = [ref.norm(ln, t, None, None, EPS) for t in x]
        mean, rstd = (torch.cat([s[i][0].float() for s in stats], 2).contiguous() for i in (0, 1))
        more = [None] * (2 - len(H))
        _, _, dgamma, dbeta = g.qk_norm_rope_bwd(ln, *[cuda(t) for t in dy + more + x + more], None, None,
                                                 cuda(mean) if ln else None, cuda(rstd), cuda(pos), r)
        groups = 32 // int(re.match(r"(?:vec\d+x|any)(\d+)", g.rope_last_variant(1)).group(1))
    finally:
        g.set_grid_limit(0)
    passes = [-(-h // groups) for h in H]
    tokens, units = B * S, B * S * sum(passes)
    warps = min(8 * limit, units)
    rounds = tokens // warps  # whole tokens of a warp, where there are four or more
    rest = -(-(tokens - rounds * warps) * sum(passes) // warps)
    at = 0
    for i, h in enumerate(H):
        chain = (rounds * passes[i] + rest if rounds >= 4 else -(-units // warps)) + groups + 8 + limit
        t = ref.rotate(dy[i].double(), angle, D, False, -1.0)
        et = ref.rotate_tol(dy[i].double(), torch.zeros_like(t), far, D, False)
        xh = x[i].double() - (mean[..., at:at + h, None].double() if ln else 0.0)
        xh = xh * rstd[..., at:at + h, None].double()
        p, dims = (t * xh).abs(), (0, 1, 2)
        tol = (et * xh.abs() + 4 * ref.U * p).sum(dims) + chain * ref.U * p.sum(dims)
        ref.held("dgamma", dgamma[i], (t * xh).sum(dims), tol)
        if ln:
            ref.held("dbeta", dbeta[i], t.sum(dims), et.sum(dims) + chain * ref.U * t.abs().sum(dims))
        at += h
