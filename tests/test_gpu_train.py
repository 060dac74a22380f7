"""The training operators (8-bit checkpoints, the norm's passes, the weight gradient)
against the float64 oracle.

Bounds.  u = 2^-24 is fp32's unit roundoff.  A sum of k fp32 terms in any order differs
from the exact one by at most (k - 1) u sum |terms|; the kernels add in trees and over
slices, so a chain has far fewer links than there are terms: CHAIN bounds it (terms per
thread, plus the levels of the tree, plus the slices' partial sums).  Results are then
rounded once to their type: half a unit in the last place."""

import numpy as np
import pytest
import torch

from oracle import train64 as t64
from tests.helpers import library, require_gpu, to64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CHAIN = 512
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
FMTS = ["int8", "e4m3"]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, seed, dtype=torch.float32, std=1.0):
    return (std * torch.randn(shape, generator=gen(seed), device="cuda")).to(dtype)


def strided(t, ld, offset=0):
    """A copy of t whose rows lie ld elements apart, `offset` elements into a buffer; the
    gaps hold NaN."""
    rows, cols = t.shape
    buf = torch.full((rows * ld + offset + 8,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf.as_strided((rows, cols), (ld, 1), offset)
    v.copy_(t)
    return v


def gaps_untouched(v):
    """Whether everything of v's buffer outside v is still NaN."""
    buf = v._base if v._base is not None else v
    keep = torch.ones(buf.numel(), dtype=torch.bool, device=v.device)
    keep.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(False)
    return bool(torch.isnan(buf.flatten()[keep].float()).all())


def rounded(x64, bound, dtype):
    """Elementwise bound on a result of dtype within `bound` of x64 before its rounding."""
    return bound + HALF_ULP[dtype] * (np.abs(x64) + bound) + TINY[dtype]


def same_norm(a, b, dtype):
    """Two results of the same norm whose sums may have run in another order: statistics
    and outputs to rounding, codes at most one step apart."""
    assert torch.allclose(a.rstd, b.rstd, rtol=1e-5, atol=0)
    assert torch.allclose(a.y.float(), b.y.float(), rtol=2 * HALF_ULP[dtype], atol=1e-5)
    if a.q is not None:
        cols = a.q.shape[1]
        va, vb = (t64.restore(f.q.cpu().numpy(), f.scale.cpu().numpy(), cols, "int8")
                  for f in (a, b))
        step = np.ldexp(1.0, np.maximum(a.scale.cpu().numpy(), b.scale.cpu().numpy())
                        .astype(int) - 127)
        assert (np.abs(va - vb) <= np.repeat(step, 32, axis=1)).all()


def check(got, want, bound, what):
    d = np.abs(to64(got) - want)
    assert got.shape == want.shape and (d <= bound).all(), (what, float((d / bound).max()))


# ---------------------------------------------------------------- checkpoints

SHAPES = [(1, 1), (1, 2048), (3, 31), (5, 32), (4, 33), (7, 257), (33, 1000), (2, 16385),
          (129, 64)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_compress_and_restore_match_oracle_bit_for_bit(shape, dtype, fmt):
    require_gpu()
    dr = library()
    rows, cols = shape
    x = randn(shape, 1)
    # Groups of very different size, exact ties and exact powers of two, zeros.
    x = (x * torch.exp2(torch.randint(-12, 12, shape, generator=gen(2), device="cuda").float()))
    x.view(-1)[::7] = 0.0
    x.view(-1)[::11] = torch.round(x.view(-1)[::11] * 2) / 2
    x = x.to(dtype)
    q, s = dr.act_compress(x, fmt)
    q64, s64 = t64.compress(to64(x), fmt)
    assert (s.cpu().numpy() == s64).all()
    v64 = t64.restore(q64, s64, cols, fmt)
    assert (t64.restore(q.cpu().numpy(), s.cpu().numpy(), cols, fmt) == v64).all()
    pad = t64.restore(q.cpu().numpy(), s.cpu().numpy(), q.shape[1], fmt)[:, cols:]
    assert (pad == 0).all()
    for out in DTYPES:
        got = dr.act_restore(q, s, cols, fmt, out)
        assert (got.cpu() == torch.from_numpy(v64).to(out)).all()


@pytest.mark.parametrize("fmt,top", [("int8", 127.0), ("e4m3", 448.0)])
def test_compress_at_the_scale_boundaries(fmt, top):
    require_gpu()
    dr = library()
    # amax just below, at and above the values that round past the largest code, over the
    # whole exponent range; subnormals and the largest floats.
    m = {"int8": 127.5 / 64, "e4m3": 464.0 / 256}[fmt]
    rows = []
    for e in list(range(-140, 128, 9)) + [-149, -133, -127, -126, -125, -124, 126, 127]:
        for f in (1.0, np.nextafter(np.float32(m), np.float32(0)), m,
                  np.nextafter(np.float32(m), np.float32(9)), 1.9999999):
            with np.errstate(over="ignore"):
                v = np.float32(f) * np.float32(2.0) ** np.float32(e)
            rows.append(np.float32(v) if np.isfinite(v) else np.float32(3.4e38))
    a = np.array(rows, dtype=np.float32)
    x = np.zeros((len(a), 32), dtype=np.float32)
    x[:, 3] = -a
    x[:, 5:32] = a[:, None] * np.linspace(-1, 1, 27, dtype=np.float32)
    q, s = dr.act_compress(torch.from_numpy(x).cuda(), fmt)
    q64, s64 = t64.compress(x, fmt)
    assert (s.cpu().numpy() == s64).all()
    assert (t64.restore(q.cpu().numpy(), s.cpu().numpy(), 32, fmt)
            == t64.restore(q64, s64, 32, fmt)).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_non_finite_values_stay_in_their_group(fmt):
    require_gpu()
    dr = library()
    x = randn((4, 100), 3)
    clean = dr.act_restore(*dr.act_compress(x, fmt), 100, fmt, torch.float32)
    y = x.clone()
    y[1, 40], y[2, 99], y[3, 0] = float("nan"), float("inf"), float("-inf")
    q, s = dr.act_compress(y, fmt)
    got = dr.act_restore(q, s, 100, fmt, torch.float32)
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[1, 32:64], bad[2, 96:], bad[3, :32] = True, True, True
    assert torch.isnan(got[bad]).all() and (got[~bad] == clean[~bad]).all()
    assert (s == 255).sum() == 3


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols,ld,off", [(96, 104, 0), (96, 104, 8), (96, 101, 3), (100, 128, 1),
                                         (2048, 2056, 4)])
def test_checkpoints_of_strided_views(cols, ld, off, dtype):
    require_gpu()
    dr = library()
    x = randn((9, cols), 4, dtype)
    xs = strided(x, ld, off)
    q, s = dr.act_compress(xs, "int8")
    q0, s0 = dr.act_compress(x, "int8")
    assert (q == q0).all() and (s == s0).all()
    out = strided(torch.zeros_like(x), ld, off)
    dr.act_restore(q, s, cols, "int8", out=out)
    assert (out == dr.act_restore(q, s, cols, "int8", dtype)).all() and gaps_untouched(out)


# ---------------------------------------------------------------- norm, forward

NORM_SHAPES = [(1, 1), (1, 2048), (2, 2), (3, 31), (5, 33), (7, 264), (19, 777), (6, 1024),
               (5, 2040), (4, 5632), (3, 8200), (2, 16383), (3, 16384)]


def forward_bounds(r64, gamma64, beta64, eps, center):
    """(y, n, mean, rstd) in 64 bits and bounds on their fp32 errors."""
    y, n, mean, rstd = t64.norm_forward(r64, gamma64, beta64, eps, center)
    cols = r64.shape[1]
    # mean: a chain of additions.  d = r - mean inherits it; the sum of squares of d
    # (relative chain error, and d's own error, which enters the variance at most as
    # 2 |d| e_d + e_d^2 averaged); rstd and n follow.
    e_mean = CHAIN * U * np.abs(r64).sum(axis=1) / cols if center else np.zeros(len(r64))
    d = np.abs(r64 - mean[:, None])
    e_d = e_mean[:, None] + U * d
    var = 1.0 / rstd ** 2
    e_var = CHAIN * U * var + (2 * d * e_d + e_d ** 2).sum(axis=1) / cols
    rel = e_var / var / 2 + 4 * U
    e_rstd = rstd * rel
    e_n = e_d * rstd[:, None] + np.abs(n) * (rel[:, None] + 2 * U)
    g = 1.0 if gamma64 is None else np.abs(gamma64)
    e_y = e_n * g + 2 * U * np.abs(n) * g
    if beta64 is not None:
        e_y = e_y + U * np.abs(y) + U * np.abs(beta64)
    return (y, n, mean, rstd), (e_y, e_n, e_mean + U * np.abs(mean), e_rstd)


def check_codes(dr, q, s, n, e_n, cols, fmt):
    """The checkpoint's values are roundings of a number within e_n of n."""
    v = t64.restore(q.cpu().numpy(), s.cpu().numpy(), cols, fmt)
    rows = n.shape[0]
    ng = s.shape[1]
    e = s.cpu().numpy().astype(int) - 127
    step = np.repeat(np.ldexp(1.0, e), 32, axis=1)[:, :cols]
    if fmt == "int8":
        half = step / 2
    else:
        # Half the spacing of 4-bit significands at the value (or at the next binade).
        half = np.maximum((np.abs(n) + e_n) / 16, step * 2.0 ** -10)
    assert (np.abs(v - n) <= half + e_n).all()
    # The scale is that of an amax within e_n of the exact one.
    p = np.zeros((rows, ng * 32))
    p[:, :cols] = np.abs(n)
    w = np.zeros((rows, ng * 32))
    w[:, :cols] = e_n
    lo = np.maximum(p - w, 0).reshape(rows, ng, 32).max(axis=2)
    hi = (p + w).reshape(rows, ng, 32).max(axis=2)
    for i in np.ndindex(lo.shape):
        assert t64.scale_exponent(lo[i], fmt) <= e[i] <= t64.scale_exponent(hi[i], fmt)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_forward_matches_oracle(shape, dtype, center):
    require_gpu()
    dr = library()
    rows, cols = shape
    fmt = FMTS[(rows + center) % 2]
    wdt = dtype if rows % 2 else torch.float32
    x = randn(shape, 5, dtype, 3.0) + 1.0
    gamma = (1 + 0.3 * randn((cols,), 6)).to(wdt)
    beta = randn((cols,), 7).to(wdt) if center else None
    f = dr.layer_norm_forward(x, gamma, beta, 1e-5, center=center, ckpt=fmt)
    (y, n, mean, rstd), (ey, en, em, er) = forward_bounds(
        to64(x), to64(gamma), None if beta is None else to64(beta), 1e-5, center)
    check(f.y, y, rounded(y, ey, dtype), "y")
    check(f.rstd, rstd, er, "rstd")
    if center:
        check(f.mean, mean, em + 1e-30, "mean")
    else:
        assert f.mean is None
    assert f.r is None
    check_codes(dr, f.q, f.scale, n, en, cols, fmt)
    # The bare form gives the same y.
    g = dr.layer_norm_forward(x, gamma, beta, 1e-5, center=center, stats=False)
    assert (g.y == f.y).all() and g.rstd is None and g.q is None


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 2048), (9, 1030), (40, 96), (3, 9000)])
def test_forward_residual_and_in_place(shape, dtype):
    require_gpu()
    dr = library()
    x, res = randn(shape, 8, dtype), randn(shape, 9, dtype, 4.0)
    r = x + res  # rounded once to dtype
    f = dr.layer_norm_forward(x, residual=res, ckpt="int8")
    g = dr.layer_norm_forward(r, ckpt="int8")
    assert (f.r == r).all()
    same_norm(f, g, dtype)
    keep = res.clone()
    h = dr.layer_norm_forward(x, residual=keep, r=keep)
    assert (keep == r).all() and (h.y == f.y).all()
    keep = x.clone()
    h = dr.layer_norm_forward(keep, residual=res, r=keep)
    assert (keep == r).all() and (h.y == f.y).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols,ld,off", [(96, 104, 0), (96, 101, 3), (2048, 2056, 8),
                                         (2048, 2050, 0), (1000, 1000, 1)])
def test_norm_of_strided_views(cols, ld, off, dtype):
    require_gpu()
    dr = library()
    x, res, dy = (randn((6, cols), 10 + i, dtype) for i in range(3))
    gamma, beta = randn((cols,), 13, dtype), randn((cols,), 14, dtype)
    f = dr.layer_norm_forward(x, gamma, beta, residual=res, ckpt="int8")
    xs, rs, ys, ds, us = (strided(t, ld, off) for t in (x, res, torch.zeros_like(x), dy,
                                                        torch.zeros_like(x)))
    # Vectors that no wide access fits either.
    gs, bs = (strided(t[None], cols + 1, 1)[0] for t in (gamma, beta))
    h = dr.layer_norm_forward(xs, gs, bs, residual=rs, ckpt="int8", y=ys, r=rs)
    assert h.y is ys and (rs == f.r).all()
    assert gaps_untouched(ys) and gaps_untouched(rs)
    same_norm(f, h, dtype)
    for kw0, kw1 in (({"x": f.r, "mean": f.mean}, {"x": rs, "mean": f.mean}),
                     ({"q": f.q, "scale": f.scale},) * 2):
        a = dr.layer_norm_backward(dy, f.rstd, gamma, dres=x, **kw0)
        b = dr.layer_norm_backward(ds, f.rstd, gs, dres=xs, dx=us, **kw1)
        assert b[0] is us and gaps_untouched(us)
        for p, q in zip(a, b):
            assert torch.allclose(p.float(), q.float(), rtol=2 * HALF_ULP[dtype],
                                  atol=2e-5 * float(p.float().abs().max()))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("off", range(8))
@pytest.mark.parametrize("cols,ld", [(5, 7), (250, 259), (513, 513), (1603, 1606), (4101, 4104),
                                     (12293, 12300)])
def test_any_alignment(cols, ld, off, dtype):
    """Rows that start anywhere, of several warps: the same bits as aligned ones from the
    checkpoint kernels, the same results to rounding from the norm's."""
    require_gpu()
    dr = library()
    rows = 11
    x, res, dy = (randn((rows, cols), 60 + i, dtype) for i in range(3))
    wide = -(-cols // 8) * 8
    ax, ares, ady = (strided(t, wide) for t in (x, res, dy))  # aligned rows
    ux, ures, udy, out = (strided(t, ld, off) for t in (x, res, dy, torch.zeros_like(x)))
    q, s = dr.act_compress(ax, "int8")
    uq, us = dr.act_compress(ux, "int8")
    assert (q == uq).all() and (s == us).all()
    dr.act_restore(q, s, cols, "int8", out=out)
    assert (out == dr.act_restore(q, s, cols, "int8", dtype)).all() and gaps_untouched(out)
    r = ures  # in place
    f = dr.layer_norm_forward(ux, residual=ures, r=r, y=out)
    assert (r == x + res).all() and gaps_untouched(r) and gaps_untouched(out)
    want = torch.nn.functional.layer_norm((x + res).double(), (cols,), None, None, 1e-5)
    d = (out.double() - want).abs()
    assert (d <= HALF_ULP[dtype] * want.abs() + 1e-5).all()
    dr.layer_norm_backward(udy, f.rstd, q=q, scale=s, fmt="int8", dx=udy)  # in place
    n = dr.act_restore(q, s, cols, "int8", torch.float32).double()
    g = dy.double()
    m1, m2 = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
    want = f.rstd.double()[:, None] * (g - m1 - n * m2)
    d = (udy.double() - want).abs()
    assert (d <= HALF_ULP[dtype] * want.abs() + 2e-5 * want.abs().max()).all()
    assert gaps_untouched(udy)


def test_constant_and_non_finite_rows():
    require_gpu()
    dr = library()
    x = randn((5, 300), 15)
    x[1] = 7.25           # no variance: n = 0, rstd = eps^(-1/2)
    x[2, 17] = float("nan")
    x[3, 5] = float("inf")
    f = dr.layer_norm_forward(x, eps=1e-4, ckpt="int8")
    assert (f.y[1] == 0).all() and abs(float(f.rstd[1]) - 100.0) < 1e-4
    assert (dr.act_restore(f.q, f.scale, 300)[1] == 0).all()
    for bad in (2, 3):
        assert torch.isnan(f.y[bad]).all()
    for good in (0, 4):
        alone = dr.layer_norm_forward(x[good:good + 1], eps=1e-4).y
        assert torch.allclose(f.y[good], alone[0], rtol=1e-5, atol=1e-5)
    # A non-finite row leaves the other rows' dx alone and spoils the column sums.
    dy = randn((5, 300), 16)
    dx, _, dbeta = dr.layer_norm_backward(dy, f.rstd, q=f.q, scale=f.scale, fmt="int8")
    assert torch.isfinite(dx[[0, 1, 4]]).all() and torch.isnan(dx[2]).all()
    assert torch.isfinite(dbeta).all()


# ---------------------------------------------------------------- norm, backward


def backward_bounds(dy, n, e_n, rstd, gamma, center, dres):
    dx, dg, db = t64.norm_backward(dy, n, rstd, gamma, center, dres)
    cols = dy.shape[1]
    g = np.abs(dy if gamma is None else dy * gamma)
    n1 = np.abs(n)
    e_c1 = (CHAIN + 2) * U * g.sum(axis=1) / cols if center else np.zeros(len(dy))
    e_c2 = ((CHAIN + 2) * U * g * n1 + g * e_n).sum(axis=1) / cols
    c1 = g.sum(axis=1) / cols if center else np.zeros(len(dy))
    c2 = (g * n1).sum(axis=1) / cols
    inner = g + c1[:, None] + n1 * c2[:, None]
    e = 6 * U * inner + e_c1[:, None] + n1 * e_c2[:, None] + e_n * c2[:, None]
    e = e * np.abs(rstd)[:, None]
    if dres is not None:
        e = e + 2 * U * (np.abs(dres) + np.abs(dx))
    e_dg = (np.abs(dy) * ((CHAIN + 2) * U * n1 + e_n)).sum(axis=0)
    e_db = CHAIN * U * np.abs(dy).sum(axis=0)
    return (dx, dg, db), (e, e_dg + 1e-30, e_db + 1e-30)


BWD_SHAPES = NORM_SHAPES + [(400, 160), (1025, 72), (300, 1111), (500, 2048)]


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", BWD_SHAPES)
def test_backward_from_checkpoint_matches_oracle(shape, dtype, center):
    require_gpu()
    dr = library()
    rows, cols = shape
    fmt = FMTS[(rows + cols + center) % 2]
    q, s = dr.act_compress(randn(shape, 17), fmt)
    n = t64.restore(q.cpu().numpy(), s.cpu().numpy(), cols, fmt)
    dy = randn(shape, 18, dtype, 0.1)
    rstd = randn((rows,), 19).abs() + 0.1
    gamma = randn((cols,), 20, dtype) if cols % 3 else None
    dres = randn(shape, 21, dtype, 0.1) if rows % 2 else None
    dx, dg, db = dr.layer_norm_backward(dy, rstd, gamma, q=q, scale=s, fmt=fmt, center=center,
                                        dres=dres)
    (dx0, dg0, db0), (ex, eg, eb) = backward_bounds(
        to64(dy), n, 0 * n, to64(rstd), None if gamma is None else to64(gamma), center,
        None if dres is None else to64(dres))
    check(dx, dx0, rounded(dx0, ex, dtype), "dx")
    check(db, db0, eb, "dbeta")
    if gamma is None:
        assert dg is None
    else:
        check(dg, dg0, eg, "dgamma")


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", BWD_SHAPES)
def test_backward_from_input_matches_oracle(shape, dtype, center):
    require_gpu()
    dr = library()
    rows, cols = shape
    x = randn(shape, 22, dtype, 2.0)
    dy = randn(shape, 23, dtype, 0.1)
    gamma = randn((cols,), 24)
    mean = randn((rows,), 25, std=0.1) if center else None
    rstd = randn((rows,), 26).abs() + 0.1
    dx, dg, db = dr.layer_norm_backward(dy, rstd, gamma, x=x, mean=mean, center=center,
                                        beta=center)
    m = to64(mean)[:, None] if center else 0.0
    n = (to64(x) - m) * to64(rstd)[:, None]
    e_n = 3 * U * (np.abs(to64(x)) + np.abs(m)) * to64(rstd)[:, None]
    (dx0, dg0, db0), (ex, eg, eb) = backward_bounds(to64(dy), n, e_n, to64(rstd), to64(gamma),
                                                    center, None)
    check(dx, dx0, rounded(dx0, ex, dtype), "dx")
    check(dg, dg0, eg, "dgamma")
    if center:
        check(db, db0, eb, "dbeta")
    else:
        assert db is None


def test_backward_in_place_and_without_rows():
    require_gpu()
    dr = library()
    for shape in ((9, 700), (3, 12000)):
        dy, dres = randn(shape, 27, torch.bfloat16), randn(shape, 28, torch.bfloat16)
        gamma = randn((shape[1],), 29)
        q, s = dr.act_compress(randn(shape, 30))
        rstd = randn((shape[0],), 31).abs()
        want = dr.layer_norm_backward(dy, rstd, gamma, q=q, scale=s, dres=dres)
        for i in range(2):
            a, b = dy.clone(), dres.clone()
            got = dr.layer_norm_backward(a, rstd, gamma, q=q, scale=s, dres=b, dx=(a, b)[i])
            assert got[0] is (a, b)[i]
            assert all((p == w).all() for p, w in zip(got, want))
    z = torch.zeros((0, 64), device="cuda")
    q, s = dr.act_compress(z)
    dx, dg, db = dr.layer_norm_backward(z, z[:, 0].contiguous(), gamma[:64].contiguous(), q=q,
                                        scale=s)
    assert dx.shape == (0, 64) and (dg == 0).all() and (db == 0).all()
    f = dr.layer_norm_forward(z, ckpt="int8")
    assert f.y.shape == (0, 64) and f.q.shape == (0, 64)


@pytest.mark.parametrize("center", [True, False])
def test_norm_gradients_match_differences(center):
    """The kernels' gradients against central differences of the float64 forward pass,
    along random directions."""
    require_gpu()
    dr = library()
    rows, cols, h = 24, 200, 1e-5
    x, dy = randn((rows, cols), 32, std=2.0), randn((rows, cols), 33)
    gamma, beta = 1 + 0.2 * randn((cols,), 34), randn((cols,), 35)
    f = dr.layer_norm_forward(x, gamma, beta, center=center)
    dx, dg, db = dr.layer_norm_backward(dy, f.rstd, gamma, x=x, mean=f.mean, center=center)
    args = [to64(x), to64(gamma), to64(beta)]
    for k, grad in enumerate((dx, dg, db)):
        for seed in range(3):
            v = np.random.default_rng(seed).standard_normal(args[k].shape)

            def loss(t):
                a = [w + t * v if i == k else w for i, w in enumerate(args)]
                return (to64(dy) * t64.norm_forward(*a, center=center)[0]).sum()

            slope = (loss(h) - loss(-h)) / (2 * h)
            # fp32 sums of the products' magnitudes; h^2 truncation is far below.
            bound = 64 * U * (np.abs(to64(grad)) * np.abs(v)).sum() + 1e-6
            assert abs(slope - (to64(grad) * v).sum()) <= bound


# ---------------------------------------------------------------- weight gradient

WG_SHAPES = [(1, 1, 1), (1, 64, 64), (3, 40, 33), (17, 130, 129), (64, 128, 256), (65, 257, 100),
             (200, 96, 500), (515, 300, 520), (1031, 264, 136), (4096, 128, 320)]


def wg_bound(dz, n, gamma, beta, parts):
    """Every tensor-core instruction adds a slice of 16 tokens to the running sum with an
    error of at most two units in the last place of the larger of both; split sums and the
    scaling add a few more."""
    dw, db = t64.weight_grad(dz, n, gamma, beta)
    steps = parts * (dz.shape[0] // 16 + 4) + 16
    y = np.abs(n) if gamma is None else np.abs(n) * np.abs(gamma)
    e_db = CHAIN * U * np.abs(dz).sum(axis=0)
    e = 4 * U * steps * (np.abs(dz).T @ y)
    if beta is not None:
        e = e + np.outer(e_db, np.abs(beta)) + 4 * U * np.abs(np.outer(db, beta))
    return dw, db, e + 1e-30, e_db + 1e-30


PARTS = {torch.float32: 3, torch.bfloat16: 1, torch.float16: 2}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", WG_SHAPES)
def test_weight_grad_matches_oracle(shape, dtype):
    require_gpu()
    dr = library()
    rows, outs, cols = shape
    i = WG_SHAPES.index(shape)
    fmt = FMTS[(i + (dtype == torch.float32)) % 2]
    odt = [torch.float32, dtype][i % 2]
    q, s = dr.act_compress(randn((rows, cols), 36), fmt)
    n = t64.restore(q.cpu().numpy(), s.cpu().numpy(), cols, fmt)
    dz = randn((rows, outs), 37, dtype)
    gamma = randn((cols,), 38, dtype) if i % 3 else None
    beta = randn((cols,), 39, dtype) if i % 4 else None
    dw0, db0, e, e_db = wg_bound(to64(dz), n, None if gamma is None else to64(gamma),
                                 None if beta is None else to64(beta), PARTS[dtype])
    dw, db = dr.weight_grad(dz, q, s, cols, fmt, gamma, beta, dtype=odt, bias=True)
    assert dw.dtype == odt
    check(dw, dw0, rounded(dw0, e, odt), "dW")
    check(db, db0, e_db, "db")
    # Without db the same dW, and as blocks what pack_blocks makes of it.
    again, none = dr.weight_grad(dz, q, s, cols, fmt, gamma, beta, dtype=odt)
    assert none is None and (again == dw).all()
    for B in (128, 256, 384):
        blocks, _ = dr.weight_grad(dz, q, s, cols, fmt, gamma, beta, B=B, dtype=odt)
        want, _, _ = dr.pack_blocks(dw, B)
        assert torch.allclose(blocks.float(), want.float(), rtol=2 * HALF_ULP[odt],
                              atol=float(e.max()))
        assert ((blocks == 0) | (want != 0)).all()
    assert dr.device_status() == 0


# Tiles for more than one round of the CTA pairs and a token-split tail, one and several
# parts, both accumulations.
WG_LARGE = [(2048, 2304, 2304, torch.bfloat16, torch.bfloat16, "int8"),
            (2048, 2304, 2304, torch.bfloat16, torch.bfloat16, "e4m3"),
            (4100, 2200, 1090, torch.bfloat16, torch.float32, "int8"),
            (2048, 2304, 2304, torch.float16, torch.float16, "int8"),
            (2048, 2304, 1152, torch.float32, torch.float32, "e4m3"),
            (8192, 5632, 2048, torch.bfloat16, torch.bfloat16, "int8")]


@pytest.mark.parametrize("rows,outs,cols,dtype,odt,fmt", WG_LARGE)
def test_weight_grad_over_many_tiles_every_run(rows, outs, cols, dtype, odt, fmt):
    """Many tiles per CTA pair, run again and again: every run gives the same bits, within
    a bound that one wrong token in one tile would break.

    The bound.  An instruction adds 16 tokens of one part to the running sum S and loses at
    most two units in the last place of the larger of |S| and the slice's sum of
    magnitudes; |S| is followed in float64, slot by slot.  One token's product is near 1,
    the bound below 0.25 before the rounding to dW's type."""
    require_gpu()
    dr = library()
    q, s = dr.act_compress(randn((rows, cols), 60), fmt)
    dz = randn((rows, outs), 61, dtype)
    n64, dz64 = dr.act_restore(q, s, cols, fmt, torch.float32).double(), dz.double()
    want = torch.zeros((outs, cols), dtype=torch.float64, device="cuda")
    top = torch.zeros_like(want)
    for t in range(0, rows, 64):
        a, b = dz64[t:t + 64].t(), n64[t:t + 64]
        want += a @ b
        top = torch.maximum(top, want.abs() + a.abs() @ b.abs())
    steps = PARTS[dtype] * (-(-rows // 16)) + 16
    bound = 4 * U * steps * top
    assert float(bound.max()) < 0.25
    bound = bound + HALF_ULP[odt] * (want.abs() + bound) + TINY[odt]
    first, _ = dr.weight_grad(dz, q, s, cols, fmt, dtype=odt)
    assert ((first.double() - want).abs() <= bound).all()
    ws = torch.empty(dr.weight_grad_workspace_size(rows, outs, cols, dtype, out_dtype=odt),
                     dtype=torch.uint8, device="cuda")
    for _ in range(24):
        again, _ = dr.weight_grad(dz, q, s, cols, fmt, dtype=odt, ws=ws)
        assert (again == first).all()
    assert dr.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("exp", [-126, -118, -90, 90, 118, 126])
def test_weight_grad_at_the_ends_of_the_scale(exp, fmt):
    """Checkpoints whose values lie at either end of fp32's range (below, some are bf16
    subnormals), with dz at the other end, so that the sums are ordinary numbers."""
    require_gpu()
    dr = library()
    rows, outs, cols = 200, 130, 300
    x = torch.ldexp(randn((rows, cols), 62).clamp(-1.9, 1.9),
                    torch.tensor(float(exp), device="cuda"))
    q, s = dr.act_compress(x, fmt)
    n = t64.restore(q.cpu().numpy(), s.cpu().numpy(), cols, fmt)
    dz = torch.ldexp(randn((rows, outs), 63, torch.bfloat16).clamp(-1.9, 1.9),
                     torch.tensor(float(-exp), device="cuda", dtype=torch.bfloat16))
    for odt in (torch.float32, torch.bfloat16):
        dw0, _, e, _ = wg_bound(to64(dz), n, None, None, 1)
        dw, _ = dr.weight_grad(dz, q, s, cols, fmt, dtype=odt)
        check(dw, dw0, rounded(dw0, e, odt), "dW")
    assert dr.device_status() == 0


@pytest.mark.parametrize("odt", DTYPES)
@pytest.mark.parametrize("off", range(8))
@pytest.mark.parametrize("cols,ld", [(1, 3), (15, 15), (17, 23), (255, 257), (530, 531)])
def test_weight_grad_stores_any_alignment(cols, ld, off, odt):
    """dW rows that begin and end anywhere: the same bits as aligned ones, and nothing
    outside them."""
    require_gpu()
    dr = library()
    rows, outs = 70, 300
    dtype = torch.float32 if off % 2 else torch.bfloat16
    q, s = dr.act_compress(randn((rows, cols), 64))
    dz = randn((rows, outs), 65, dtype)
    gamma, beta = randn((cols,), 66), randn((cols,), 67)
    wide = strided(torch.zeros((outs, cols), dtype=odt, device="cuda"), -(-cols // 8) * 8)
    dr.weight_grad(dz, q, s, cols, gamma=gamma, beta=beta, out=wide)
    out = strided(torch.zeros((outs, cols), dtype=odt, device="cuda"), ld, off)
    dr.weight_grad(dz, q, s, cols, gamma=gamma, beta=beta, out=out)
    assert (out == wide).all() and gaps_untouched(out) and gaps_untouched(wide)
    assert dr.device_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_weight_grad_of_strided_views(dtype):
    require_gpu()
    dr = library()
    rows, outs, cols = 150, 200, 300
    q, s = dr.act_compress(randn((rows, cols), 40))
    dz = randn((rows, outs), 41, dtype)
    dw, _ = dr.weight_grad(dz, q, s, cols)
    for ld, off in ((208, 0), (201, 1), (216, 8)):
        out = strided(torch.zeros_like(dw), cols + 5, 3)
        got, _ = dr.weight_grad(strided(dz, ld, off), q, s, cols, out=out)
        assert got is out and (out == dw).all() and gaps_untouched(out)


def test_weight_grad_without_tokens_and_non_finite():
    require_gpu()
    dr = library()
    z = torch.zeros((0, 40), device="cuda", dtype=torch.bfloat16)
    q, s = dr.act_compress(torch.zeros((0, 70), device="cuda"))
    out = torch.full((40, 70), 5.0, device="cuda", dtype=torch.bfloat16)
    dw, db = dr.weight_grad(z, q, s, 70, beta=torch.ones(70, device="cuda"), bias=True, out=out)
    assert (dw == 0).all() and (db == 0).all()
    # A NaN group of the checkpoint spoils its 32 columns, a NaN token output its row.
    for dtype in DTYPES:
        x, dz = randn((100, 200), 42), randn((100, 150), 43, dtype)
        x[7, 40] = float("nan")
        dz[9, 3], dz[11, 5] = float("nan"), float("inf")
        q, s = dr.act_compress(x)
        dw, _ = dr.weight_grad(dz, q, s, 200, dtype=torch.float32)
        bad = torch.zeros((150, 200), dtype=torch.bool, device="cuda")
        bad[:, 32:64], bad[3], bad[5] = True, True, True
        assert not torch.isfinite(dw[bad]).any() and torch.isfinite(dw[~bad]).all()


def test_weight_grad_matches_differences():
    """dW and db against central differences of the float64 layer."""
    require_gpu()
    dr = library()
    rows, outs, cols = 48, 40, 72
    x, dz = randn((rows, cols), 44), randn((rows, outs), 45)
    gamma, beta = 1 + 0.2 * randn((cols,), 46), randn((cols,), 47)
    f = dr.layer_norm_forward(x, gamma, beta, ckpt="e4m3")
    dw, db = dr.weight_grad(dz, f.q, f.scale, cols, "e4m3", gamma, beta, bias=True)
    n = t64.restore(f.q.cpu().numpy(), f.scale.cpu().numpy(), cols, "e4m3")
    y = n * to64(gamma) + to64(beta)
    for seed in range(3):
        rng = np.random.default_rng(seed)
        V, v = rng.standard_normal((outs, cols)), rng.standard_normal(outs)

        def loss(t):
            return (to64(dz) * (y @ (t * V).T + t * v)).sum()

        slope = (loss(1.0) - loss(-1.0)) / 2
        bound = 1e-5 * ((np.abs(to64(dz)).T @ np.abs(y)) * np.abs(V)).sum()
        assert abs(slope - (to64(dw) * V).sum() - (to64(db) * v).sum()) <= bound


# ---------------------------------------------------------------- use


def test_runs_are_reproducible_and_capture_in_a_graph():
    require_gpu()
    dr = library()
    rows, cols, outs = 700, 1000, 300
    x, dz = randn((rows, cols), 48, torch.bfloat16), randn((rows, outs), 49, torch.bfloat16)
    gamma = randn((cols,), 50)
    wsb = torch.empty(dr.layer_norm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    wsw = torch.empty(dr.weight_grad_workspace_size(rows, outs, cols), dtype=torch.uint8,
                      device="cuda")

    def step():
        f = dr.layer_norm_forward(x, gamma, ckpt="int8")
        dw, db = dr.weight_grad(dz, f.q, f.scale, cols, gamma=gamma, bias=True, ws=wsw)
        return (f.y, f.q, dw, db) + dr.layer_norm_backward(x, f.rstd, gamma, q=f.q, scale=f.scale,
                                                           ws=wsb)

    first = step()
    for _ in range(3):
        assert all((a == b).all() for a, b in zip(first, step()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = step()
    torch.cuda.current_stream().wait_stream(s)
    assert all((a == b).all() for a, b in zip(first, side))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all((a == b).all() for a, b in zip(first, out))


def test_offsets_past_32_bits():
    require_gpu()
    dr = library()
    rows, cols = 135000, 16000  # 2.16e9 elements
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen(51))
    f = dr.layer_norm_forward(x, ckpt="int8")
    tail = dr.layer_norm_forward(x[-3:].clone(), ckpt="int8")
    same_norm(dr.NormForward(*(None if t is None else t[-3:] for t in f)), tail, x.dtype)
    q, s = dr.act_compress(x)
    q1, s1 = dr.act_compress(x[-3:].clone())
    assert (q[-3:] == q1).all() and (s[-3:] == s1).all()
    back = dr.act_restore(q, s, cols)
    assert (back[-3:] == dr.act_restore(q1, s1, cols)).all()
    del back, q, s
    # Only the last rows carry a gradient: the column sums are those of these rows.
    dy = torch.zeros_like(x)
    dy[-3:] = 1.0
    dx, dg, db = dr.layer_norm_backward(dy, f.rstd, torch.ones(cols, device="cuda"), q=f.q,
                                        scale=f.scale)
    dx1, dg1, db1 = dr.layer_norm_backward(dy[-3:].clone(), f.rstd[-3:].clone(),
                                           torch.ones(cols, device="cuda"),
                                           q=f.q[-3:].clone(), scale=f.scale[-3:].clone())
    assert torch.allclose(dx[-3:].float(), dx1.float(), rtol=2 * HALF_ULP[x.dtype], atol=1e-5)
    assert (dx[:-3] == 0).all()
    assert torch.allclose(dg, dg1, rtol=1e-6, atol=1e-6) and (db == 3).all()
    del dx
    # The weight gradient over as many tokens of a wide dz.
    dw, _ = dr.weight_grad(dy, f.q[:, :64].contiguous(), f.scale[:, :2].contiguous(), 64,
                           dtype=torch.float32)
    want = dr.act_restore(f.q[-3:, :64].contiguous(), f.scale[-3:, :2].contiguous(), 64,
                          dtype=torch.float32).sum(dim=0)
    assert torch.allclose(dw, want.expand_as(dw), rtol=1e-5, atol=1e-5)


def test_python_refusals():
    require_gpu()
    dr = library()
    x = randn((4, 64), 52)
    q, s = dr.act_compress(x)
    rstd = torch.ones(4, device="cuda")
    gamma = torch.ones(64, device="cuda")
    bad = [
        (ValueError, lambda: dr.act_compress(x, "int4")),
        (TypeError, lambda: dr.act_compress(x.cpu())),
        (TypeError, lambda: dr.act_compress(x[0])),
        (ValueError, lambda: dr.act_compress(x.t())),
        (dr.DashError, lambda: dr.act_compress(x.double())),
        (ValueError, lambda: dr.act_restore(q, s, 100)),
        (ValueError, lambda: dr.act_restore(q[:2], s, 64)),
        (TypeError, lambda: dr.act_restore(q.float(), s, 64)),
        (ValueError, lambda: dr.layer_norm_forward(x, gamma[:3].contiguous())),
        (TypeError, lambda: dr.layer_norm_forward(x, gamma, gamma.half())),
        (TypeError, lambda: dr.layer_norm_forward(x, residual=x.half())),
        (dr.DashError, lambda: dr.layer_norm_forward(x, eps=-1.0)),
        (dr.DashError, lambda: dr.layer_norm_forward(x, eps=float("nan"))),
        (dr.DashError, lambda: dr.layer_norm_forward(torch.ones((2, 16385), device="cuda"))),
        (ValueError, lambda: dr.layer_norm_forward(x[:1].expand(4, 64), y=x[:1].expand(4, 64))),
        (ValueError, lambda: dr.layer_norm_backward(x, rstd, gamma)),
        (ValueError, lambda: dr.layer_norm_backward(x, rstd, gamma, x=x, q=q, scale=s)),
        (ValueError, lambda: dr.layer_norm_backward(x, rstd, gamma, x=x)),
        (ValueError, lambda: dr.layer_norm_backward(x, rstd[:2], gamma, q=q, scale=s)),
        (dr.DashError, lambda: dr.layer_norm_backward(x, rstd, gamma, q=q, scale=s,
                                                      ws=torch.empty(8, device="cuda"))),
        (ValueError, lambda: dr.weight_grad(x, q, s, 65)),
        (dr.DashError, lambda: dr.weight_grad(x, q, s, 64, B=100)),
        (ValueError, lambda: dr.weight_grad(x, q, s, 64, out=torch.empty((64, 63), device="cuda"))),
        (dr.DashError, lambda: dr.weight_grad(x, q, s, 64, ws=torch.empty(8, device="cuda"))),
    ]
    for err, call in bad:
        with pytest.raises(err):
            call()
    torch.cuda.synchronize()
    assert dr.device_status() == 0


@pytest.mark.parametrize("rows,outs,cols,B", [(2, 448, 192, 1024), (3, 153, 1200, 1024),
                                              (40, 300, 70, 512), (5, 129, 129, 384)])
@pytest.mark.parametrize("odt", [torch.float32, torch.bfloat16])
def test_weight_grad_blocks_of_mostly_padding(rows, outs, cols, B, odt):
    """Few small tiles in large blocks: the same values as the matrix, zeros everywhere
    else, from a buffer of NaN."""
    require_gpu()
    dr = library()
    q, s = dr.act_compress(randn((rows, cols), 70))
    dz = randn((rows, outs), 71, torch.bfloat16)
    dw, _ = dr.weight_grad(dz, q, s, cols, dtype=odt)
    nb = -(-outs // B) * -(-cols // B)
    out = torch.full((nb, B, B), float("nan"), dtype=odt, device="cuda")
    dr.weight_grad(dz, q, s, cols, B=B, out=out)
    want, _, _ = dr.pack_blocks(dw, B)
    assert (out == want).all()
    assert dr.device_status() == 0
