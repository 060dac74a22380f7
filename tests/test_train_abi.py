"""Host-side refusals of the training operators' C entry points: every bad argument is
rejected before anything is launched, so no GPU is needed."""

import ctypes

from tests.helpers import library

INVALID, UNSUPPORTED, TOO_SMALL = 1, 2, 4
P = 4096          # an aligned address that is never dereferenced
ODD = 4097


def f(x):
    return ctypes.c_float(x)


def compress(lib, x=P, dt=1, rows=4, cols=64, ld=64, fmt=0, q=P, scale=P):
    return lib.act_compress(x, dt, rows, cols, ld, fmt, q, scale, None)


def restore(lib, q=P, scale=P, fmt=0, rows=4, cols=64, x=P, dt=1, ld=64):
    return lib.act_restore(q, scale, fmt, rows, cols, x, dt, ld, None)


def forward(lib, x=P, ldx=64, res=None, ldres=64, dt=1, rows=4, cols=64, gamma=None, beta=None,
            wdt=0, eps=1e-5, r=None, ldr=64, y=P, ldy=64, mean=None, rstd=None, fmt=0, q=None,
            scale=None):
    return lib.layer_norm_forward(x, ldx, res, ldres, dt, rows, cols, gamma, beta, wdt, eps, 1, r,
                                  ldr, y, ldy, mean, rstd, fmt, q, scale, None)


def backward(lib, dy=P, lddy=64, dt=1, rows=4, cols=64, x=None, ldx=64, mean=None, q=P, scale=P,
             fmt=0, rstd=P, gamma=None, wdt=0, center=1, dres=None, lddres=64, dx=P, lddx=64,
             dg=None, db=None, ws=None, wsb=0):
    return lib.layer_norm_backward(dy, lddy, dt, rows, cols, x, ldx, mean, q, scale, fmt, rstd,
                                   gamma, wdt, center, dres, lddres, dx, lddx, dg, db, ws, wsb,
                                   None)


def wgrad(lib, dz=P, dt=1, lddz=32, rows=4, outs=32, q=P, scale=P, fmt=0, cols=64, gamma=None,
          beta=None, wdt=0, dw=P, odt=1, ldw=64, B=0, db=None, ws=P, wsb=1 << 30):
    return lib.weight_grad(dz, dt, lddz, rows, outs, q, scale, fmt, cols, gamma, beta, wdt, dw,
                           odt, ldw, B, db, ws, wsb, None)


def test_checkpoint_refusals():
    lib = library().load_library()
    for call in (compress, restore):
        for kw in ({"dt": 3}, {"fmt": 2}, {"fmt": -1}, {"rows": -1}, {"cols": -1}, {"ld": 63},
                   {"x": None}, {"x": ODD}, {"q": None}, {"q": P + 8}, {"scale": None},
                   {"rows": 1 << 31}):
            assert call(lib, **kw) == INVALID, kw
        assert call(lib, rows=0, x=None, q=None, scale=None) == 0
        assert call(lib, cols=0, x=None) == 0


def test_norm_refusals():
    lib = library().load_library()
    for kw in ({"dt": 3}, {"wdt": 4}, {"fmt": 2}, {"rows": -1}, {"cols": -5}, {"ldx": 63},
               {"ldy": 10}, {"x": None}, {"y": None}, {"x": ODD}, {"y": ODD}, {"res": ODD},
               {"res": P, "ldres": 1}, {"r": P, "ldr": 63}, {"gamma": P + 2}, {"beta": P + 1},
               {"mean": P + 2}, {"rstd": P + 1}, {"q": P}, {"scale": P},
               {"q": P + 4, "scale": P}, {"eps": f(-1e-5)}, {"eps": f(float("inf"))},
               {"eps": f(float("nan"))}):
        assert forward(lib, **kw) == INVALID, kw
    assert forward(lib, cols=16385, ldx=20000, ldy=20000) == UNSUPPORTED
    assert forward(lib, rows=0, x=None, y=None) == 0
    for kw in ({"dt": 3}, {"wdt": 4}, {"fmt": 2}, {"rows": -1}, {"lddy": 63}, {"lddx": 63},
               {"dy": None}, {"dx": None}, {"rstd": None}, {"rstd": P + 2}, {"q": None},
               {"x": P}, {"q": None, "x": P}, {"q": None, "x": P, "mean": P + 2},
               {"q": None, "x": P, "mean": P, "ldx": 60}, {"scale": None}, {"q": P + 8},
               {"dres": P, "lddres": 5}, {"dres": ODD}, {"gamma": P + 2}, {"dg": P + 2},
               {"db": P, "wsb": 1 << 20}, {"db": P, "ws": P + 16, "wsb": 1 << 20}):
        assert backward(lib, **kw) == INVALID, kw
    assert backward(lib, dg=P, ws=P, wsb=8) == TOO_SMALL
    assert backward(lib, cols=16385, lddy=20000, lddx=20000) == UNSUPPORTED
    n = ctypes.c_size_t(0)
    assert lib.dash_layer_norm_workspace_size(-1, 4, ctypes.byref(n)) == INVALID
    assert lib.dash_layer_norm_workspace_size(4, 4, None) == INVALID
    assert lib.dash_layer_norm_workspace_size(4, 20000, ctypes.byref(n)) == UNSUPPORTED


def test_weight_grad_refusals():
    lib = library().load_library()
    for kw in ({"dt": 3}, {"odt": 3}, {"wdt": 9}, {"fmt": 5}, {"rows": -1}, {"outs": -1},
               {"cols": -1}, {"lddz": 31}, {"ldw": 63}, {"B": 100}, {"B": 64}, {"B": 4096},
               {"dz": None}, {"dz": ODD}, {"dw": None}, {"dw": ODD}, {"q": None}, {"q": P + 8},
               {"scale": None}, {"gamma": P + 2}, {"beta": P + 1}, {"db": P + 2}, {"ws": None},
               {"ws": P + 128}):
        assert wgrad(lib, **kw) == INVALID, kw
    assert wgrad(lib, wsb=0) == TOO_SMALL
    assert wgrad(lib, outs=0) == 0 and wgrad(lib, cols=0) == 0
    assert wgrad(lib, dw=P + 2, B=128) == INVALID
    assert wgrad(lib, outs=1 << 23, lddz=1 << 23, cols=1 << 23, ldw=1 << 23) == INVALID
    n = ctypes.c_size_t(0)
    size = lib.dash_weight_grad_workspace_size
    assert size(4, 4, -1, 1, 1, 0, 0, ctypes.byref(n)) == INVALID
    assert size(4, 4, 4, 7, 1, 0, 0, ctypes.byref(n)) == INVALID
    assert size(4, 4, 4, 1, 9, 0, 0, ctypes.byref(n)) == INVALID
    assert size(4, 4, 4, 1, 1, 0, 100, ctypes.byref(n)) == INVALID
    assert size(4, 4, 4, 1, 1, 0, 0, None) == INVALID


def test_format_names():
    dr = library()
    assert dr.Q8_FORMATS == {"int8": 0, "e4m3": 1}
    assert len(dr.TRACE_KINDS) == 10
