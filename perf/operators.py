"""Operators of a training step around the preconditioner, as measured cases.

The framework's preconditioner consumes the weight gradients of a transformer's linear
layers.  The operators here stand in front of it: the norm that feeds a linear layer
(forward and backward), the 8-bit checkpoint of an activation that is kept between the
two passes, and the weight gradient computed from that checkpoint.

The checkpoint format: a row is cut into groups of 32 columns (the last one padded with
zeros); a group has one scale 2^e, stored as the byte e + 127, and 32 values q of 8 bits,
int8 or e4m3 (bit patterns in a uint8 tensor), with value q 2^e.  e is the smallest
exponent at which the group's largest magnitude does not round past 127 (int8) or 448
(e4m3).

Four kinds of case:
  checkpoint     x -> 8 bits -> x again: what a checkpoint costs on its own.
  norm_forward   y = gamma n + beta with n = (r - mean) rstd, r = x + residual; for
                 training with the statistics and the checkpoint of n, for serving y (and
                 r) alone.  center = False leaves the mean out (root-mean-square norm).
  norm_backward  dx, dgamma, dbeta from dy and either the checkpoint of n or r itself.
  weight_grad    dW = dz^T (gamma n + beta) from the checkpoint of n, as a matrix or cut
                 into the B x B blocks the preconditioner takes, and db = sum of dz.
"""

import math

import torch

own = False

GROUP = 32
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
# Most elements of a norm or checkpoint case, and most products of a weight gradient.
MAX_ELEMS = 16384 * 8192
MAX_PRODUCTS = 16384 * 8192 * 8192


def _norm(name, direction, rows, cols, dtype, wdtype, **kw):
    case = {"name": name, "kind": "norm_" + direction, "rows": rows, "cols": cols,
            "dtype": dtype, "wdtype": wdtype, "center": True, "beta": True,
            "residual": False, "ckpt": ""}
    case.update(kw)
    return case


def listed():
    return [
        # One token of a served model: the call is all latency.
        _norm("forward_one_token", "forward", 1, 2048, "bf16", "bf16", center=False, beta=False,
              residual=True),
        # A batch of served tokens, an odd number of them, with the widest rows.
        _norm("forward_decode_batch", "forward", 77, 16384, "fp16", "fp32"),
        # The training forward of a d = 2048 layer: residual sum, statistics, checkpoint.
        _norm("forward_train", "forward", 8192, 2048, "bf16", "bf16", center=False, beta=False,
              residual=True, ckpt="int8"),
        # Rows that no vector access fits (odd width), in 32 bits.
        _norm("forward_odd", "forward", 1021, 1537, "fp32", "fp32", ckpt="e4m3"),
        # The training backward of the same layer, from the checkpoint.
        _norm("backward_train", "backward", 8192, 2048, "bf16", "bf16", center=False, beta=False,
              residual=True, ckpt="int8"),
        # The same from the saved input, ragged.
        _norm("backward_odd", "backward", 1021, 1537, "fp32", "fp32"),
        # A large model's norm over a long batch, with all gradients.
        _norm("backward_large", "backward", 16384, 8192, "bf16", "fp32", ckpt="e4m3"),
        # A few tokens' activations, and the hidden activations of a 5632-wide MLP.
        {"name": "checkpoint_small", "kind": "checkpoint", "rows": 33, "cols": 2048,
         "dtype": "fp16", "ckpt": "e4m3"},
        {"name": "checkpoint_mlp", "kind": "checkpoint", "rows": 8192, "cols": 5632,
         "dtype": "bf16", "ckpt": "int8"},
        # A small ragged projection, matrix output with its bias gradient, in 32 bits.
        {"name": "weight_grad_ragged", "kind": "weight_grad", "rows": 515, "cols": 777,
         "outs": 1000, "dtype": "fp32", "wdtype": "fp32", "out": "fp32", "block": 0,
         "gamma": True, "beta": True, "bias": True, "ckpt": "e4m3"},
        # The d = 2048 layer's MLP weight, its gradient cut into 1024 x 1024 blocks.
        {"name": "weight_grad_mlp_blocks", "kind": "weight_grad", "rows": 8192, "cols": 2048,
         "outs": 5632, "dtype": "bf16", "wdtype": "bf16", "out": "bf16", "block": 1024,
         "gamma": True, "beta": False, "bias": False, "ckpt": "int8"},
        # A large model's projection over a long batch.
        {"name": "weight_grad_large", "kind": "weight_grad", "rows": 16384, "cols": 8192,
         "outs": 8192, "dtype": "bf16", "wdtype": "bf16", "out": "bf16", "block": 0,
         "gamma": True, "beta": True, "bias": True, "ckpt": "int8"},
    ]


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]; half of them multiples of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 128 and rng.random() < 0.5:
        v = (v + 32) // 64 * 64
    v = min(max(v, lo), hi)
    return v - 1 if v == 3072 else v


def draw(rng):
    kind = rng.choice(["checkpoint", "norm_forward", "norm_backward", "weight_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    fmt = rng.choice(["int8", "e4m3"])
    if kind == "weight_grad":
        while True:
            rows, cols, outs = (_log_int(rng, 1, 16384), _log_int(rng, 64, 8192),
                                _log_int(rng, 64, 8192))
            # A 16-bit pass costs the largest listed case's work at most; a 32-bit one
            # takes three products for each of the formula's.
            if rows * cols * outs * (3 if dtype == "fp32" else 1) <= MAX_PRODUCTS // 2:
                break
        return {"kind": kind, "rows": rows, "cols": cols, "outs": outs, "dtype": dtype,
                "wdtype": rng.choice([dtype, "fp32"]), "out": rng.choice([dtype, "fp32"]),
                "block": rng.choice([0, 0, 256, 1024]), "gamma": rng.random() < 0.75,
                "beta": rng.random() < 0.5, "bias": rng.random() < 0.5, "ckpt": fmt}
    while True:
        rows, cols = _log_int(rng, 1, 32768), _log_int(rng, 64, 16384)
        if rows * cols * (2 if dtype == "fp32" else 1) <= MAX_ELEMS // 2:
            break
    if kind == "checkpoint":
        return {"kind": kind, "rows": rows, "cols": cols, "dtype": dtype, "ckpt": fmt}
    center = rng.random() < 0.6
    return {"kind": kind, "rows": rows, "cols": cols, "dtype": dtype,
            "wdtype": rng.choice([dtype, "fp32"]), "center": center,
            "beta": center and rng.random() < 0.8, "residual": rng.random() < 0.5,
            "ckpt": rng.choice(["", fmt])}


# ---------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _stream(g, rows, cols):
    """Rows of a residual stream: columns of unlike scale, a few far above the rest."""
    scale = torch.exp(0.5 * _randn(g, cols))
    scale[torch.randint(0, cols, (1 + cols // 512,), generator=g, device="cuda")] *= 12.0
    return _randn(g, rows, cols) * scale + 0.1 * _randn(g, cols)


def _grads(g, rows, cols):
    """Gradients of activations: tokens of unlike weight."""
    return 0.1 * _randn(g, rows, cols) * torch.exp(0.5 * _randn(g, rows, 1))


def _pow2(e):
    """2^e in 32 bits, e in [-126, 127], from its bit pattern."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _encode(x, fmt):
    """The checkpoint of a matrix in 32 bits: (q (rows, 32 G), scale (rows, G)), uint8."""
    rows, cols = x.shape
    ng = -(-cols // GROUP)
    p = torch.zeros((rows, ng * GROUP), device=x.device, dtype=torch.float32)
    p[:, :cols] = x
    p = p.view(rows, ng, GROUP)
    amax = p.abs().amax(dim=2)
    # The exponent of amax, one higher where amax rounds past the largest value: the
    # mantissa bits from which it does are 0x7f0000 (127.5 / 64) and 0x680001 (464 / 256).
    bits = amax.view(torch.int32)
    if fmt == "int8":
        e = ((bits + 0x10000) >> 23) - 127 - 6
        top = 121
    else:
        e = ((bits + 0x17FFFF) >> 23) - 127 - 8
        top = 119
    e = e.clamp(-124, top)
    s = p * _pow2(-e)[:, :, None]
    if fmt == "int8":
        q = s.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    else:
        q = s.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(rows, ng * GROUP), (e + 127).to(torch.uint8)


def _decode(q, scale, cols, fmt):
    """The values of a checkpoint, in 32 bits."""
    v = q.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()
    s = _pow2(scale.to(torch.int32) - 127)
    rows, ng = scale.shape
    return (v.view(rows, ng, GROUP) * s[:, :, None]).view(rows, ng * GROUP)[:, :cols]


def _weights(g, case, n):
    gamma = (1.0 + 0.2 * _randn(g, n)).to(DTYPES[case["wdtype"]])
    beta = (0.2 * _randn(g, n)).to(DTYPES[case["wdtype"]])
    return gamma, beta


def prepare(case, seed):
    g = _gen(seed)
    kind, rows, cols = case["kind"], case["rows"], case["cols"]
    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    if kind == "checkpoint":
        st["x"] = _stream(g, rows, cols).to(dt)
        return st
    gamma, beta = _weights(g, case, cols)
    if kind == "weight_grad":
        st["gamma"] = gamma if case["gamma"] else None
        st["beta"] = beta if case["beta"] else None
        st["dz"] = _grads(g, rows, case["outs"]).to(dt)
        st["q"], st["scale"] = _encode(_randn(g, rows, cols), case["ckpt"])
        return st
    st["gamma"] = gamma
    st["beta"] = beta if case["beta"] else None
    x = _stream(g, rows, cols).to(dt)
    if kind == "norm_forward":
        st["x"] = x
        st["residual"] = _stream(g, rows, cols).to(dt) if case["residual"] else None
        return st
    st["dy"] = _grads(g, rows, cols).to(dt)
    st["dres"] = _grads(g, rows, cols).to(dt) if case["residual"] else None
    xf = x.float()
    mean = xf.mean(dim=1) if case["center"] else torch.zeros(rows, device="cuda")
    xc = xf - mean[:, None]
    rstd = torch.rsqrt((xc * xc).mean(dim=1) + EPS)
    st["mean"] = mean if case["center"] else None
    st["rstd"] = rstd
    if case["ckpt"]:
        st["q"], st["scale"] = _encode(xc * rstd[:, None], case["ckpt"])
    else:
        st["x"] = x
    return st


# ---------------------------------------------------------------- one pass


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import matrix_inverse_roots_gb300 as dr

    case = st["case"]
    kind, cols, fmt = case["kind"], case["cols"], case["ckpt"]
    if kind == "checkpoint":
        q, scale = dr.act_compress(st["x"], fmt)
        return dr.act_restore(q, scale, cols, fmt, st["x"].dtype)
    if kind == "norm_forward":
        f = dr.layer_norm_forward(st["x"], st["gamma"], st["beta"], EPS, center=case["center"],
                                  residual=st["residual"], ckpt=fmt or None, stats=bool(fmt))
        out = {"y": f.y}
        if case["residual"]:
            out["r"] = f.r
        if fmt:
            out["rstd"] = f.rstd
            if case["center"]:
                out["mean"] = f.mean
            out["n"] = dr.act_restore(f.q, f.scale, cols, fmt, st["x"].dtype)
        return out
    if kind == "norm_backward":
        if fmt:
            src = {"q": st["q"], "scale": st["scale"], "fmt": fmt}
        else:
            src = {"x": st["x"], "mean": st["mean"]}
        dx, dgamma, dbeta = dr.layer_norm_backward(st["dy"], st["rstd"], st["gamma"],
                                                   center=case["center"], dres=st["dres"],
                                                   beta=case["beta"], **src)
        out = {"dx": dx, "dgamma": dgamma}
        if case["beta"]:
            out["dbeta"] = dbeta
        return out
    dw, db = dr.weight_grad(st["dz"], st["q"], st["scale"], cols, fmt, st["gamma"], st["beta"],
                            B=case["block"] or None, dtype=DTYPES[case["out"]],
                            bias=case["bias"])
    return {"dw": dw, "db": db} if case["bias"] else {"dw": dw}


def _run_plain(st):
    case = st["case"]
    kind, cols, fmt = case["kind"], case["cols"], case["ckpt"]
    dt = DTYPES[case["dtype"]]
    if kind == "checkpoint":
        return _decode(*_encode(st["x"].float(), fmt), cols, fmt).to(dt)
    if kind == "norm_forward":
        r = st["x"].float()
        out = {}
        if case["residual"]:
            # The stream is carried in the model's type; the norm sees what is carried.
            out["r"] = (r + st["residual"].float()).to(dt)
            r = out["r"].float()
        if case["center"]:
            mean = r.mean(dim=1)
            r = r - mean[:, None]
        rstd = torch.rsqrt((r * r).mean(dim=1) + EPS)
        n = r * rstd[:, None]
        y = n * st["gamma"].float()
        if st["beta"] is not None:
            y = y + st["beta"].float()
        out["y"] = y.to(dt)
        if fmt:
            out["rstd"] = rstd
            if case["center"]:
                out["mean"] = mean
            out["n"] = _decode(*_encode(n, fmt), cols, fmt).to(dt)
        return out
    if kind == "norm_backward":
        if fmt:
            n = _decode(st["q"], st["scale"], cols, fmt)
        else:
            n = st["x"].float()
            if case["center"]:
                n = n - st["mean"][:, None]
            n = n * st["rstd"][:, None]
        dy = st["dy"].float()
        g = dy * st["gamma"].float()
        dx = g - n * (g * n).mean(dim=1, keepdim=True)
        if case["center"]:
            dx = dx - g.mean(dim=1, keepdim=True)
        dx = dx * st["rstd"][:, None]
        if st["dres"] is not None:
            dx = dx + st["dres"].float()
        out = {"dx": dx.to(dt), "dgamma": (dy * n).sum(dim=0)}
        if case["beta"]:
            out["dbeta"] = dy.sum(dim=0)
        return out
    n = _decode(st["q"], st["scale"], cols, fmt)
    if st["gamma"] is not None:
        n = n * st["gamma"].float()
    if st["beta"] is not None:
        n = n + st["beta"].float()
    dz = st["dz"].float()
    dw = (dz.t() @ n).to(DTYPES[case["out"]])
    out = {"dw": _blocks(dw, case["block"]) if case["block"] else dw}
    if case["bias"]:
        out["db"] = dz.sum(dim=0)
    return out


def _blocks(m, b):
    """The zero-padded row-block-major (., b, b) blocks of a matrix."""
    nr, nc = -(-m.shape[0] // b), -(-m.shape[1] // b)
    p = torch.zeros((nr * b, nc * b), device=m.device, dtype=m.dtype)
    p[:m.shape[0], :m.shape[1]] = m
    return p.view(nr, b, nc, b).transpose(1, 2).reshape(nr * nc, b, b)


# ---------------------------------------------------------------- 64 bits


def _two64(e):
    """2^e in 64 bits from its bit pattern."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _code64(v, fmt):
    """The values nearest to v (64 bits) that a checkpoint in this format can hold."""
    rows, cols = v.shape
    out = torch.empty_like(v)
    for c in range(0, cols, 8192):
        w = v[:, c:c + 8192]
        width = w.shape[1]
        w = torch.nn.functional.pad(w, (0, -width % GROUP)).reshape(rows, -1, GROUP)
        top = w.abs().amax(dim=2, keepdim=True)
        mant, ex = torch.frexp(top)
        if fmt == "int8":
            # top = mant 2^ex with mant in [1/2, 1): seven bits, unless it rounds to 128.
            e = (ex - 7) + (mant * 128 >= 127.5).to(ex.dtype)
            e = torch.where(top > 0, e, torch.full_like(e, -124)).clamp(-124, 121)
            step = _two64(e)
            w = torch.round(w / step).clamp(-127, 127) * step
        else:
            e = (ex - 9) + (mant * 512 > 464).to(ex.dtype)
            e = torch.where(top > 0, e, torch.full_like(e, -124)).clamp(-124, 119)
            unit = _two64(e)
            w = w / unit
            # Four significant bits down to 2^-6, then steps of 2^-9.
            _, we = torch.frexp(w)
            step = _two64((we - 4).clamp(min=-9))
            w = (torch.round(w / step) * step).clamp(-448, 448) * unit
        out[:, c:c + 8192] = w.reshape(rows, -1)[:, :width]
    return out


def _values64(st, cols, fmt):
    """The values that a given checkpoint holds, read bit by bit."""
    b = st["q"].to(torch.int32)
    if fmt == "int8":
        v = torch.where(b > 127, b - 256, b).double()
    else:
        ex, m = (b >> 3) & 15, (b & 7).double()
        mag = torch.where(ex > 0, (8 + m) * _two64(ex - 10), m * 2.0 ** -9)
        v = torch.where(b > 127, -mag, mag)
    s = _two64(st["scale"].to(torch.int64) - 127)
    return (v * s.repeat_interleave(GROUP, dim=1))[:, :cols]


def exact(case, seed):
    st = prepare(case, seed)
    kind, rows, cols, fmt = case["kind"], case["rows"], case["cols"], case["ckpt"]
    if kind == "checkpoint":
        return _code64(st["x"].double(), fmt)
    if kind == "norm_forward":
        r = st["x"].double()
        out = {}
        if case["residual"]:
            total = r + st["residual"].double()
            out["r"] = total
            # What the stream carries is the sum in the model's type, rounded once.
            r = total.to(DTYPES[case["dtype"]]).double()
        mu = r.sum(dim=1) / cols if case["center"] else torch.zeros_like(r[:, 0])
        var = ((r - mu[:, None]) ** 2).sum(dim=1) / cols
        scale = 1.0 / torch.sqrt(var + EPS)
        n = (r - mu[:, None]) * scale[:, None]
        shift = 0.0 if st["beta"] is None else st["beta"].double()
        out["y"] = torch.addcmul(torch.zeros_like(n) + shift, n, st["gamma"].double())
        if fmt:
            out["rstd"] = scale
            if case["center"]:
                out["mean"] = mu
            out["n"] = _code64(n, fmt)
        return out
    if kind == "norm_backward":
        if fmt:
            n = _values64(st, cols, fmt)
        else:
            mu = st["mean"].double() if case["center"] else torch.zeros(rows, device="cuda").double()
            n = (st["x"].double() - mu[:, None]) * st["rstd"].double()[:, None]
        dy = st["dy"].double()
        g = dy * st["gamma"].double()
        c2 = torch.einsum("rc,rc->r", g, n) / cols
        c1 = g.sum(dim=1) / cols if case["center"] else torch.zeros_like(c2)
        dx = st["rstd"].double()[:, None] * (g - c1[:, None] - n * c2[:, None])
        if case["residual"]:
            dx = dx + st["dres"].double()
        out = {"dx": dx, "dgamma": torch.einsum("rc,rc->c", dy, n)}
        if case["beta"]:
            out["dbeta"] = torch.ones(rows, dtype=torch.float64, device="cuda") @ dy
        return out
    if rows * cols * case["outs"] > MAX_PRODUCTS:
        return None
    dz = st["dz"].double()
    db = torch.ones(rows, dtype=torch.float64, device="cuda") @ dz
    dw = dz.t() @ _values64(st, cols, fmt)
    if case["gamma"]:
        dw = dw * st["gamma"].double()
    if case["beta"]:
        dw = dw + torch.outer(db, st["beta"].double())
    b = case["block"]
    if b:
        nr, nc = -(-case["outs"] // b), -(-cols // b)
        cut = torch.zeros((nr * nc, b, b), dtype=torch.float64, device="cuda")
        for i in range(nr):
            for j in range(nc):
                part = dw[i * b:(i + 1) * b, j * b:(j + 1) * b]
                cut[i * nc + j, :part.shape[0], :part.shape[1]] = part
        dw = cut
    return {"dw": dw, "db": db} if case["bias"] else {"dw": dw}


# ---------------------------------------------------------------- work


def work(case):
    kind, rows, cols = case["kind"], case["rows"], case["cols"]
    e = BYTES[case["dtype"]]
    n = rows * cols
    code = n + rows * -(-cols // GROUP)
    if kind == "checkpoint":
        # Read, encoded, read as a code, written again.
        return {"bytes": 2 * n * e + 2 * code, "flops": 6 * n}
    w = BYTES[case["wdtype"]]
    if kind == "norm_forward":
        streams = 2 + (2 if case["residual"] else 0)
        b = streams * n * e + cols * w * (2 if case["beta"] else 1)
        if case["ckpt"]:
            # Statistics, the checkpoint, and its values as the pass returns them.
            b += rows * 4 * (2 if case["center"] else 1) + 2 * code + n * e
        return {"bytes": b, "flops": 8 * n}
    if kind == "norm_backward":
        b = (2 + (1 if case["residual"] else 0)) * n * e + (code if case["ckpt"] else n * e)
        b += rows * 4 * (2 if case["center"] and not case["ckpt"] else 1)
        b += cols * w + cols * 4 * (2 if case["beta"] else 1)
        return {"bytes": b, "flops": 12 * n}
    outs, blk = case["outs"], case["block"]
    cells = outs * cols
    if blk:
        cells = -(-outs // blk) * blk * -(-cols // blk) * blk
    b = rows * outs * e + code + cells * BYTES[case["out"]]
    b += cols * w * (int(case["gamma"]) + int(case["beta"])) + (outs * 4 if case["bias"] else 0)
    return {"bytes": b, "flops": 2 * rows * cols * outs}
