"""Plain forms in 64 bits of the mixture-of-experts operators and of the norms around a block, on the CPU, with the error
bounds that their tests use. Nothing here shares code with the kernels."""
from __future__ import annotations

import numpy as np

I8, I4, I2 = 1, 2, 3
BITS = {I8: 8, I4: 4, I2: 2}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step, relative to the value
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}  # the smallest step


def route(scores, k, bias=None, gating="softmax", groups=1, top_groups=1, normalise=True, scale=1.0):
    """(ids, weights) of scores float64 [T, E], one token at a time."""
    T, E = scores.shape
    n = E // groups
    ids, weights = np.empty((T, k), dtype=np.int64), np.empty((T, k))
    for t in range(T):
        x = np.where(np.isnan(scores[t]), -np.inf, np.minimum(scores[t], float(np.finfo(np.float32).max)))
        with np.errstate(over="ignore"):
            if gating == "softmax":
                top = x.max()
                e = np.zeros(E) if top == -np.inf else np.exp(x - top)
                p = e / (e.sum() if e.sum() > 0 else 1.0)
            else:
                p = 1 / (1 + np.exp(-x))
        c = p if bias is None else p + bias.astype(np.float64)
        c = np.where(np.isnan(c), -np.inf, c)
        value = []
        for g in range(groups):
            best = sorted(c[g * n:(g + 1) * n])[::-1][:2]
            value.append(sum(best))
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
        allowed = [e for e in range(E) if e // n in kept]
        ids[t] = sorted(allowed, key=lambda e: (-c[e], e))[:k]
        w = p[ids[t]]
        if normalise:
            w = w / w.sum() if w.sum() > 0 else w * 0
        weights[t] = w * scale
    return ids, weights


def open_matrix(codes, scales, cols, fmt, gs):
    """float64 [rows, cols] of packed codes uint8 [rows, row bytes]."""
    per = 8 // BITS[fmt]
    if fmt == I8:
        q = codes.view(np.int8).astype(np.float64)
    else:
        q = np.empty((codes.shape[0], codes.shape[1] * per))
        for i in range(per):
            q[:, i::per] = ((codes >> (BITS[fmt] * i)) & (2 ** BITS[fmt] - 1)).astype(np.float64) - 2 ** (BITS[fmt] - 1)
    s = scales.astype(np.float64)
    return q[:, :cols] * (np.repeat(s, gs, 1)[:, :cols] if gs else s[:, None])


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1 + np.exp(-z))


def product(x, Ex, w):
    """(x @ w.T, bound) of x float64 [S, I] that is itself within Ex: sums within 1e-5 of the sum of the terms' magnitudes (the
    matmuls' contract), and activations as integers of 31 bits: within 2^-31 of the largest that shares their unit, here of all."""
    a, near = np.abs(w).T, np.abs(x) + Ex
    return x @ w.T, 1e-5 * (near @ a) + Ex @ a + 2.0 ** -31 * near.max(1, keepdims=True) * a.sum(0) + 1e-30


def expert_rows(x, gate, up, down):
    """(y, bound) of one expert's feed-forward of x float64 [S, D]: products as above, silu's slope at most 1.1, fp32's silu and
    product within 2e-6."""
    none = np.zeros_like(x)
    (g, Eg), (u, Eu) = product(x, none, gate), product(x, none, up)
    h = silu(g) * u
    Eh = 1.1 * Eg * (np.abs(u) + Eu) + np.abs(silu(g)) * Eu
    Eh += 2e-6 * (np.abs(h) + Eh) + 1e-30
    return product(h, Eh, down)


def moe(x, ids, weights, mats, add=None):
    """(y, bound before y's own rounding); mats: a list of (gate, up, down) float64."""
    T, k = ids.shape
    O = mats[0][2].shape[0]
    y = np.zeros((T, O)) if add is None else add.astype(np.float64).copy()
    terms, bound = np.abs(y), np.zeros((T, O))
    for e, (gate, up, down) in enumerate(mats):
        for t, j in zip(*np.nonzero(ids == e)):
            v, b = expert_rows(x[t:t + 1], gate, up, down)
            w = float(weights[t, j])
            y[t] += w * v[0]
            bound[t] += abs(w) * b[0]
            terms[t] += np.abs(w * v[0])
    return y, bound + (k + 1) * 2.0 ** -24 * (terms + bound)


def block_norm(x, res, w_post, gate, alpha, w_pre, eps):
    """(r, bound of r, y, bound of y before y's own rounding) of float64 rows. A sum of squares is within 64 roundings (at most 32
    elements a thread and 16 partial sums more), its root within half of that and two more; three products follow."""
    u = 2.0 ** -24
    z = x.astype(np.float64)
    Ez = np.zeros_like(z)
    if w_post is not None:
        z = z / np.sqrt((z ** 2).mean(1, keepdims=True) + eps) * w_post
        Ez = 40 * u * np.abs(z)
    s = alpha * z * (1 if gate is None else gate)
    Es = Ez * np.abs(alpha * (1 if gate is None else gate)) + 2 * u * np.abs(s)
    r = res + s
    Er = Es + u * (np.abs(r) + Es)
    ms = (r ** 2).mean(1, keepdims=True) + eps
    if w_pre is None:
        return r, Er, None, None
    y = r / np.sqrt(ms) * w_pre
    shift = np.sqrt((Er ** 2).mean(1, keepdims=True) / ms)
    return r, Er, y, 1.01 * (Er / np.sqrt(ms) * np.abs(w_pre) + np.abs(y) * (shift + 40 * u))
