"""Plain forms in 64 bits of the operators between a decoder layer's products, on the CPU, and builders of their
inputs. Nothing here shares code with the kernels: rows are opened element by element with numpy."""
from __future__ import annotations

import numpy as np

F16, I8, I4 = 0, 1, 2
TINY = 2.0 ** -100


def row_bytes(kind, D):
    return (2 * D, D, D // 2)[kind]


def open_rows(rows, kind):
    """Codes (float64) of uint8 rows [..., row bytes]."""
    rows = np.ascontiguousarray(rows)
    if kind == F16:
        return rows.view(np.float16).astype(np.float64)
    if kind == I8:
        return rows.view(np.int8).astype(np.float64)
    out = np.empty(rows.shape[:-1] + (2 * rows.shape[-1],))
    out[..., 0::2] = (rows & 15).astype(np.float64) - 8
    out[..., 1::2] = (rows >> 4).astype(np.float64) - 8
    return out


def quantise(x, kind):
    """(rows uint8, scales float32) of x float32 [..., D], by the definition of the cache's formats."""
    x = np.asarray(x, dtype=np.float32)
    bad = ~np.isfinite(x).all(-1)
    x64 = np.where(bad[..., None], 0.0, x.astype(np.float64))
    top = np.abs(x64).max(-1)
    zero = (top < TINY) | bad
    safe = np.where(zero, 1.0, top)
    if kind == F16:
        scale = 2.0 ** (np.floor(np.log2(safe)) - 14)
        codes = (np.where(zero[..., None], 0, x64) / scale[..., None]).astype(np.float32).astype(np.float16)
        rows = codes.view(np.uint8)
    else:
        scale = (safe / (127 if kind == I8 else 7)).astype(np.float32).astype(np.float64)
        codes = np.rint(np.where(zero[..., None], 0, x64) / scale[..., None]).astype(np.int64)
        if kind == I8:
            rows = codes.astype(np.int8).view(np.uint8)
        else:
            u = (codes + 8).astype(np.uint8)
            rows = u[..., 0::2] | (u[..., 1::2] << 4)
    scale = np.where(bad, np.nan, np.where(zero, 0.0, scale)).astype(np.float32)
    return rows, scale


def place(kv_len, q_start, table, pages, page, b, tok):
    """(page, slot) of a new token, or None."""
    p = int(kv_len[b]) - int(q_start[b + 1]) + tok
    return place_at(table, pages, page, b, p)


def place_at(table, pages, page, b, t):
    if t < 0 or t // page >= table.shape[1]:
        return None
    pg = int(table[b, t // page])
    return (pg, t % page) if 0 <= pg < pages else None


def attention(q, kind, k, v, ks, vs, q_start, kv_len, table, scale, causal, window):
    """q float64 [T, H, D]; pools as numpy [pages, heads, page, ...]. Returns o, lse, and for the error bounds
    A = sum_t w_t |v_t| and S = max_t |scale| sum_d |q_d k_td| of every row."""
    T, H, D = q.shape
    pages, heads, page = ks.shape
    G = H // heads
    o, A = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, S = np.full((T, H), -np.inf), np.zeros((T, H))
    for b in range(len(kv_len)):
        n, kv = int(q_start[b + 1]) - int(q_start[b]), int(kv_len[b])
        at = [place_at(table, pages, page, b, t) for t in range(kv)]
        there = np.array([a is not None for a in at], dtype=bool)
        pg = np.array([a[0] if a else 0 for a in at], dtype=int)
        sl = np.array([a[1] if a else 0 for a in at], dtype=int)
        pos = np.arange(kv)
        if n == 0 or kv == 0:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            for h in range(heads):
                K = open_rows(k[pg, h, sl], kind) * ks[pg, h, sl].astype(np.float64)[:, None]
                V = open_rows(v[pg, h, sl], kind) * vs[pg, h, sl].astype(np.float64)[:, None]
                for i in range(n):
                    p = kv - n + i
                    seen = there.copy()
                    if causal:
                        seen &= pos <= p
                    if window:
                        seen &= pos > p - window
                    if not seen.any():
                        continue
                    for g in range(G):
                        x = q[q_start[b] + i, h * G + g]
                        s = scale * (K[seen] @ x)
                        m = s.max()
                        w = np.exp(s - m)
                        l = w.sum()
                        o[q_start[b] + i, h * G + g] = (w / l) @ V[seen]
                        A[q_start[b] + i, h * G + g] = (w / l) @ np.abs(V[seen])
                        lse[q_start[b] + i, h * G + g] = m + np.log(l)
                        S[q_start[b] + i, h * G + g] = abs(scale) * (np.abs(K[seen]) @ np.abs(x)).max()
    return o, lse, A, S


def rope(x, pos, rot, pairing, theta, sections):
    """x float64 [T, H, D], pos int [axes, T]."""
    y, first = x.copy(), 0
    for axis, n in enumerate(sections):
        for i in range(first, first + n):
            phi = pos[axis].astype(np.longdouble) * np.exp(np.longdouble(-2 * i) / rot * np.log(np.longdouble(theta)))
            c, s = np.cos(phi).astype(np.float64)[:, None], np.sin(phi).astype(np.float64)[:, None]
            a, b = (i, i + rot // 2) if pairing == 0 else (2 * i, 2 * i + 1)
            y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        first += n
    return y


def paging(rng, kv_len, page, spare=2, width=None):
    """(pages, table int32): the sequences' pages in no order, -1 past their ends."""
    need = [-(-int(n) // page) for n in kv_len]
    pages = sum(need) + spare
    order = rng.permutation(pages)[: sum(need)]
    width = max(max(need), 1) if width is None else width
    table = np.full((len(kv_len), width), -1, dtype=np.int32)
    first = 0
    for b, n in enumerate(need):
        table[b, :n] = order[first:first + n]
        first += n
    return pages, table
