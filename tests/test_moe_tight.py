"""The bounds of tests/moe_tight.py by themselves: the arithmetic that they follow, computed here in whole numbers, keeps them,
and each of its digits left out, swapped or cut breaks them."""
from __future__ import annotations

import numpy as np
import pytest

import moe_tight as tight

FORMS = [(tight.I8, 0), (tight.I8, 64), (tight.I4, 0), (tight.I4, 64), (tight.I2, 0), (tight.I2, 64)]


def products(x, codes, scales, gs, mistake=None):
    """Codes times activations in units of 2^-29 (rows whose largest magnitude is 1), four signed base-256 digits at a time."""
    n = np.rint(x.astype(np.float64) * 2.0 ** 29).astype(np.int64)
    digits = []
    for _ in range(4):
        d = (n + 128) % 256 - 128
        digits.append(d)
        n = (n - d) // 256
    weights = [1, 256, 65536, 16777216]
    if mistake in range(4):
        digits[mistake] = digits[mistake] * 0
    elif mistake == "swapped":
        weights[0], weights[1] = weights[1], weights[0]
    elif mistake == "unsigned":
        digits[0] = digits[0] % 256
    y = np.zeros((x.shape[0], codes.shape[0]))
    for g in range(scales.shape[1] if gs else 1):
        c = slice(g * gs, (g + 1) * gs) if gs else slice(None)
        v = sum(w * (d[:, c] @ codes[:, c].T) for w, d in zip(weights, digits))
        y += v * 2.0 ** -29 * (scales[:, g] if gs else scales)
    return y.astype(np.float32)


@pytest.mark.parametrize("fmt,gs", FORMS)
def test_bounds_tell_digits_apart(fmt, gs):
    rng = np.random.default_rng(61)
    x = tight.cancelling_rows(rng, 12)
    codes = tight.cancelling_codes(rng, 50, fmt)
    scales = 2.0 ** rng.integers(-3, 4, (50, 2) if gs else 50).astype(np.float32)
    m = tight.Matrix(tight.pack(codes, fmt), scales, tight.COLS, fmt, gs)
    assert np.array_equal(m.w, codes * (np.repeat(scales, 64, 1)[:, :tight.COLS] if gs else scales[:, None]))
    want, bound = m.product(x.astype(np.float64), np.zeros(x.shape))
    off = lambda mistake: (np.abs(products(x, codes, scales, gs, mistake) - want) / bound).max(1)  # noqa: E731
    assert (off(None) <= 1).all()
    t = np.arange(12)
    assert (off(0)[t % 4 == 0] > 1).all() and (off(1)[t % 4 == 1] > 1).all() and (off(2)[t % 4 == 2] > 1).all() and (off(1)[t % 4 == 3] > 1).all()
    assert (off("swapped")[t % 4 == 1] > 1).all() and (off("unsigned")[t % 4 == 0] > 1).all()


def test_bounds_of_far_values():
    """The largest digit, and ordinary data: fp32 sums over the steps of a long row stay within."""
    rng = np.random.default_rng(62)
    codes = rng.integers(-128, 128, (20, 900))
    m = tight.Matrix(tight.pack(codes, tight.I8), np.ones(20, np.float32), 900, tight.I8, 0)
    x = rng.uniform(-1, 1, (5, 900)).astype(np.float32)
    x[:, 0] = 1
    want, bound = m.product(x.astype(np.float64), np.zeros(x.shape))
    got = np.zeros((5, 20), np.float32)
    for s in range(0, 900, 128):
        got += products(x[:, s:s + 128], codes[:, s:s + 128], np.ones(20, np.float32), 0)
    assert (np.abs(got - want) <= bound).all() and (bound < 1e-5 * (np.abs(x) @ np.abs(codes).T)).all()
    wrong = got - products(x[:, :128], codes[:, :128], np.ones(20, np.float32), 0) + products(x[:, :128], codes[:, :128], np.ones(20, np.float32), 0, 3)
    assert (np.abs(wrong - want) > bound).any()
