"""Float64 oracle: 8-bit activation checkpoints, the norm and the weight gradient.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain NumPy in float64.  The pages
have no counterpart of these operators; the formulas are those of include/dashroot.h.

* Checkpoint.  Groups of 32 columns share a scale 2^e.  The codes of a format are listed
  in a table of non-negative values (index = code); a value goes to the nearest entry,
  ties to the even code.
* Norm.  r = x + residual, n = (r - mean) rstd, y = n gamma + beta; center False takes
  mean = 0.
* Weight gradient.  dW = dz^T (n gamma + beta), db the column sums of dz.
"""

import numpy as np

GROUP = 32
# Non-negative code values, by code.
INT8_TABLE = np.arange(128, dtype=np.float64)
E4M3_TABLE = np.array([(m * 2.0 ** -9) if ex == 0 else (8 + m) * 2.0 ** (ex - 10)
                       for ex in range(16) for m in range(8)][:127])
TABLES = {"int8": INT8_TABLE, "e4m3": E4M3_TABLE}
E_MIN = -124
E_MAX = {"int8": 121, "e4m3": 119}
NAN_BYTE = 255


def nearest_code(v, fmt):
    """Index of the table entry nearest to v >= 0, ties to even, saturating."""
    t = TABLES[fmt]
    hi = np.clip(np.searchsorted(t, v), 0, len(t) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = v - t[lo], t[hi] - v
    take_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    return np.where(v >= t[-1], len(t) - 1, np.where(take_lo, lo, hi))


def scale_exponent(amax, fmt):
    """The smallest e in range at which amax 2^-e does not round past the largest code."""
    t = TABLES[fmt]
    # Where the next code above the largest would start: half its step above it.
    limit = 127.5 if fmt == "int8" else 464.0
    if amax == 0:
        return E_MIN
    e = int(np.floor(np.log2(amax))) - int(np.floor(np.log2(t[-1]))) - 2
    while amax * 2.0 ** -e > limit or (fmt == "int8" and amax * 2.0 ** -e == limit):
        e += 1
    return min(max(e, E_MIN), E_MAX[fmt])


def compress(x, fmt):
    """(q (rows, 32 G) uint8, scale (rows, G) uint8) of a matrix."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    ng = -(-cols // GROUP)
    p = np.zeros((rows, ng * GROUP))
    p[:, :cols] = x
    p = p.reshape(rows * ng, GROUP)
    q = np.zeros(p.shape, dtype=np.uint8)
    scale = np.zeros(rows * ng, dtype=np.uint8)
    for i, g in enumerate(p):
        if not np.isfinite(g).all():
            scale[i] = NAN_BYTE
            continue
        e = scale_exponent(np.abs(g).max(), fmt)
        c = nearest_code(np.abs(g) * 2.0 ** -e, fmt).astype(np.int64)
        if fmt == "int8":
            q[i] = (np.where(g < 0, -c, c) & 0xFF).astype(np.uint8)
        else:
            q[i] = np.where(np.signbit(g), c | 0x80, c).astype(np.uint8)
        scale[i] = e + 127
    return q.reshape(rows, ng * GROUP), scale.reshape(rows, ng)


def restore(q, scale, cols, fmt):
    """The values of a checkpoint."""
    q = np.asarray(q).astype(np.int64)
    if fmt == "int8":
        v = np.where(q > 127, q - 256, q).astype(np.float64)
    else:
        mag = E4M3_TABLE[np.minimum(q & 0x7F, 126)]
        v = np.where(q & 0x80, -mag, mag)
    s = np.asarray(scale).astype(np.int64)
    f = np.where(s == NAN_BYTE, np.nan, np.ldexp(1.0, s - 127))
    return (v * np.repeat(f, GROUP, axis=1))[:, :cols]


def norm_forward(r, gamma=None, beta=None, eps=1e-5, center=True):
    """(y, n, mean, rstd) of the rows of r (the sum that the stream carries)."""
    r = np.asarray(r, dtype=np.float64)
    cols = r.shape[1]
    mean = r.sum(axis=1) / cols if center else np.zeros(r.shape[0])
    d = r - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).sum(axis=1) / cols + eps)
    n = d * rstd[:, None]
    y = n if gamma is None else n * np.asarray(gamma, dtype=np.float64)
    if beta is not None:
        y = y + np.asarray(beta, dtype=np.float64)
    return y, n, mean, rstd


def norm_backward(dy, n, rstd, gamma=None, center=True, dres=None):
    """(dx, dgamma, dbeta) from the normalised rows n."""
    dy = np.asarray(dy, dtype=np.float64)
    n = np.asarray(n, dtype=np.float64)
    cols = dy.shape[1]
    g = dy if gamma is None else dy * np.asarray(gamma, dtype=np.float64)
    c1 = g.sum(axis=1) / cols if center else np.zeros(dy.shape[0])
    c2 = (g * n).sum(axis=1) / cols
    dx = np.asarray(rstd, dtype=np.float64)[:, None] * (g - c1[:, None] - n * c2[:, None])
    if dres is not None:
        dx = dx + np.asarray(dres, dtype=np.float64)
    return dx, (dy * n).sum(axis=0), dy.sum(axis=0)


def weight_grad(dz, n, gamma=None, beta=None):
    """(dW (outs, cols), db (outs,))."""
    dz = np.asarray(dz, dtype=np.float64)
    y = np.asarray(n, dtype=np.float64)
    if gamma is not None:
        y = y * np.asarray(gamma, dtype=np.float64)
    if beta is not None:
        y = y + np.asarray(beta, dtype=np.float64)
    return dz.T @ y, dz.sum(axis=0)
