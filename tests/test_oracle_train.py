"""Pins of the float64 oracle of the training operators: the checkpoint format against
brute force over its codes, the norm's gradients and the weight gradient against
differences of the forward pass."""

import numpy as np
import pytest

from oracle import train64 as t64


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_codes_are_nearest_by_brute_force(fmt):
    rng = np.random.default_rng(1)
    table = t64.TABLES[fmt]
    v = np.concatenate([rng.uniform(0, table[-1], 300), table, (table[1:] + table[:-1]) / 2])
    got = t64.nearest_code(v, fmt)
    for x, c in zip(v, got):
        d = np.abs(table - x)
        best = np.flatnonzero(d == d.min())
        assert c in best
        if len(best) == 2:
            assert c % 2 == 0


def test_e4m3_table_matches_torch():
    torch = pytest.importorskip("torch")
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    assert (codes.double().numpy() == t64.E4M3_TABLE).all()


@pytest.mark.parametrize("fmt,limit", [("int8", 127.5), ("e4m3", 464.0)])
def test_scale_is_the_smallest_that_does_not_overflow(fmt, limit):
    rng = np.random.default_rng(2)
    for _ in range(200):
        amax = float(2.0 ** rng.uniform(-60, 60))
        e = t64.scale_exponent(amax, fmt)
        assert amax * 2.0 ** -e <= limit < amax * 2.0 ** -(e - 1) * (1 + 1e-12)
    # The boundary itself: 127.5 would round to 128, 464 rounds to 448.
    assert t64.scale_exponent(127.5, "int8") == 1 and t64.scale_exponent(464.0, "e4m3") == 0
    assert t64.scale_exponent(0.0, fmt) == -124


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_every_value_is_a_bf16_number(fmt):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((40, 70)) * 2.0 ** rng.uniform(-130, 126, (40, 1))
    v = t64.restore(*t64.compress(x, fmt), 70, fmt).astype(np.float32)
    assert (v.view(np.uint32) & 0xFFFF == 0).all() and np.isfinite(v).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rounding_error_and_idempotence(fmt):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((9, 100))
    q, s = t64.compress(x, fmt)
    v = t64.restore(q, s, 100, fmt)
    step = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)[:, :100]
    # int8: half a step; e4m3: 1/16 relative, or half the smallest step.
    bound = step / 2 if fmt == "int8" else np.maximum(np.abs(x) / 16, step * 2.0 ** -10)
    assert (np.abs(v - x) <= bound).all()
    assert (t64.restore(*t64.compress(v, fmt), 100, fmt) == v).all()


@pytest.mark.parametrize("center", [True, False])
def test_norm_gradients_match_differences(center):
    rng = np.random.default_rng(5)
    rows, cols, h = 3, 7, 1e-6
    x, dy = rng.standard_normal((2, rows, cols))
    gamma, beta = rng.standard_normal((2, cols))

    def loss(x, gamma, beta):
        return (dy * t64.norm_forward(x, gamma, beta, center=center)[0]).sum()

    _, n, _, rstd = t64.norm_forward(x, gamma, beta, center=center)
    dx, dg, db = t64.norm_backward(dy, n, rstd, gamma, center)
    for arg, grad in ((0, dx), (1, dg), (2, db)):
        args = [x, gamma, beta]
        for idx in np.ndindex(args[arg].shape):
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[arg][idx] += h
            lo[arg][idx] -= h
            assert abs((loss(*hi) - loss(*lo)) / (2 * h) - grad[idx]) < 1e-7


def test_weight_gradient_matches_differences():
    rng = np.random.default_rng(6)
    n, dz = rng.standard_normal((5, 4)), rng.standard_normal((5, 3))
    gamma, beta = rng.standard_normal((2, 4))
    W, b = rng.standard_normal((3, 4)), rng.standard_normal(3)

    def loss(W, b):
        return (dz * ((n * gamma + beta) @ W.T + b)).sum()

    dW, db = t64.weight_grad(dz, n, gamma, beta)
    for i in range(3):
        e = np.zeros(3)
        e[i] = 1.0
        assert abs(loss(W, b + e) - loss(W, b) - db[i]) < 1e-9
        for j in range(4):
            E = np.zeros((3, 4))
            E[i, j] = 1.0
            assert abs(loss(W + E, b) - loss(W, b) - dW[i, j]) < 1e-9
