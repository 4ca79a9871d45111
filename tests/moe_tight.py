"""The expert layer in 64 bits with error bounds that follow its arithmetic: activations as integers in units of a power of two
that a step shares, exact sums within a step, fp32 sums over steps. Nothing here shares code with the kernels."""
from __future__ import annotations

import numpy as np

from moe_ref import BITS, I2, I4, I8, open_matrix, silu  # noqa: F401

U = 2.0 ** -24  # half a step of fp32, relative to the value
WAVES = 4  # at most as many partial sums of a row are added


class Matrix:
    """One matrix of codes uint8 [rows, row bytes] and scales [rows] or [rows, groups], as float64, with its terms: the runs of
    columns whose sums are exact. They are the 128 bytes of a step, with group scales its halves or (groups that do not cover
    whole halves) its runs of 64 columns. Rows without group scales keep whole KiB in another order: there `shared` is the KiB's
    columns, among which a step's largest activation is, and a term is one column (the sum of magnitudes bounds a step's sum)."""

    def __init__(self, codes, scales, cols, fmt, gs):
        self.codes, self.scales, self.cols, self.fmt, self.gs = codes, scales, cols, fmt, gs
        self.w = open_matrix(codes, scales, cols, fmt, gs)
        per = 8 // BITS[fmt]
        step, at = 128 * per, np.arange(cols)
        self.steps = -(-cols // step)
        if gs:
            run = 64 * per if gs % (64 * per) == 0 else 64
            self.shared, self.term, self.each = at // step, at // run, step // run
        else:
            whole = codes.shape[1] // 1024 * 1024 * per  # columns in whole KiB
            self.shared = np.where(at < whole, at // (8 * step), 10 ** 6 + (at - whole) // step)
            self.term = np.where(at < whole, at, 10 ** 9 + (at - whole) // step)
            self.each = 1

    def product(self, x, Ex):
        """(x @ w.T, bound) of x float64 [S, cols] that is itself within Ex.

        An activation is within 2^-30 of its step's largest magnitude (largest below 2^-96: within 2^-126). Four digits' sums make
        a term in three roundings relative to it (and less than 2^-37 of the largest times the codes where the digits cancel),
        its scale is one rounding, each term's addition one of the sum so far, and the sum over waves and a row's scale follow. Sums
        are kept in units of 2^16: with group scales a term and an addition each lose at most 2^-134 below the smallest number."""
        S = x.shape[0]
        aw = np.abs(self.w).T
        near = np.abs(x) + Ex
        unit = np.empty_like(x)
        for s in np.unique(self.shared):
            unit[:, self.shared == s] = near[:, self.shared == s].max(1, keepdims=True)
        off = (Ex + np.maximum(1.01 * 2.0 ** -30 * unit, 1.01 * 2.0 ** -126) * (x.shape[1] > 0)) @ aw
        y, total = x @ self.w.T, np.zeros((S, self.w.shape[0]))
        if len(np.unique(self.term)) > 64:
            total = near @ aw
        else:
            for t in np.unique(self.term):
                c = self.term == t
                total += np.abs(x[:, c] @ self.w[:, c].T)
            total += off
        roundings = 3 + 1 + self.steps * self.each + WAVES + 1
        return y, 1.01 * off + 1.01 * U * roundings * total + 2 * self.steps * self.each * 2.0 ** -134


def rows_of(x, gate, up, down):
    """(y, bound) of an expert's feed-forward of x float64 [S, D]. silu's slope is at most 1.1; in fp32 its exponential is within
    4 roundings, with sum, quotient and the product with up 8 in all; below -88 the exponential overflows and silu, at most
    3e-37 there, is 0."""
    g, Eg = gate.product(x, np.zeros_like(x))
    u, Eu = up.product(x, np.zeros_like(x))
    h = silu(g) * u
    Eh = 1.1 * Eg * (np.abs(u) + Eu) + (np.abs(silu(g)) + 3e-37) * Eu + 3e-37 * np.abs(u)
    Eh += 8 * U * (np.abs(h) + Eh) + 2.0 ** -140
    return down.product(h, Eh)


def moe(x, ids, w, experts, add=None):
    """(y, bound before y's own rounding); experts: (gate, up, down) of every id."""
    T, k = ids.shape
    rows = experts[0][2].w.shape[0]
    v, b = np.zeros((T, k, rows)), np.zeros((T, k, rows))
    sets = {}
    for t, j in np.ndindex(T, k):
        if 0 <= ids[t, j] < len(experts):
            sets.setdefault(tuple(map(id, experts[ids[t, j]])), (experts[ids[t, j]], []))[1].append((t, j))
    for mats, at in sets.values():
        t, j = np.array(at).T
        v[t, j], b[t, j] = rows_of(x[t], *mats)
    wj = w.astype(np.float64)[..., None]
    y = (v * wj).sum(1) + (0 if add is None else add)
    terms = np.abs(v * wj).sum(1) + (0 if add is None else np.abs(add))
    bound = (b * np.abs(wj)).sum(1)
    return y, bound + (k + 1) * U * (terms + bound)


def pack(codes, fmt):
    """uint8 [rows, row bytes] of whole codes [rows, cols]."""
    per = 8 // BITS[fmt]
    q = (codes + (0 if fmt == I8 else 2 ** (BITS[fmt] - 1))).astype(np.int64) & (2 ** BITS[fmt] - 1)
    q = np.pad(q, ((0, 0), (0, -q.shape[1] % per)))
    return sum(q[:, i::per] << (BITS[fmt] * i) for i in range(per)).astype(np.uint8)


COLS = 120  # of the rows below: one step of any format, in two groups of 64
PAIRS = [(g + 2 * i + 1, g + 2 * i + 2) for g in (0, 64) for i in range(10)]  # columns that cancel, in one group
SMALL = [c for c in range(1, COLS) if c not in sum(PAIRS, ())]


def cancelling_rows(rng, T):
    """float32 [T, COLS]: 1 in column 0, ones of both signs in PAIRS and in SMALL numbers of one base-256 digit in units of 2^-29,
    the lowest in token 0, the next in token 1, the third in token 2, two of them in token 3, and so on."""
    x = np.zeros((T, COLS))
    x[:, 0] = 1
    for t in range(T):
        for i, j in PAIRS:
            x[t, i] = rng.choice([-1, 1])
            x[t, j] = -x[t, i]
        m = rng.integers(1, 128, len(SMALL)) * rng.choice([-1, 1], len(SMALL)) * 256.0 ** (t % 4 % 3)
        if t % 4 == 3:
            m += rng.integers(-128, 128, len(SMALL)) * 256.0
        x[t, SMALL] = m * 2.0 ** -29
    return x.astype(np.float32)


def cancelling_codes(rng, rows, fmt):
    """Codes [rows, COLS]: none in column 0, equal ones in a pair's columns, any in SMALL."""
    top = 2 ** (BITS[fmt] - 1)
    q = rng.integers(-top, top, (rows, COLS))
    q[:, 0] = 0
    for i, j in PAIRS:
        q[:, i] = q[:, j]
    return q
