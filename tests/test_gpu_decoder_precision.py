"""What attention keeps of its probabilities and of codes that are not finite, tighter than in test_gpu_decoder.py.

Probabilities times their values' scales enter the matrix units in two f16 parts for f16 queries (22 bits: r = 2^-21 of
sum_t w_t |v_t|), as for f32; in one part (2^-11) they would be as coarse as an f16 output, which shows wherever an
output is smaller than what it sums. The other terms of the bound are test_gpu_decoder.py's: a score within
e = (D + 8) u S, sums over kv positions within (kv + 72) u, half a step of the output."""
from __future__ import annotations

import numpy as np
import pytest

import decoder_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("no GPU", allow_module_level=True)

import gpu_util as gu  # noqa: E402
from test_gpu_decoder import Case, HALF, SMALL, U, attend, f64, queries  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    gu.reinit_with_env(WQ_FORCE_PATH=None, WQ_FAULT=None, WQ_MEM_LIMIT_BYTES=None)
    yield


@pytest.mark.parametrize("kind", [ref.F16, ref.I8, ref.I4])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len,kv_len,G", [([1, 2], [900, 333], 4), ([150, 1], [700, 90], 2)])
def test_f16_probabilities(kind, D, q_len, kv_len, G):
    gu.banner("f16 probabilities kind=%d D=%d q=%s" % (kind, D, q_len))
    c = Case(D + kind + 1, kind, D, 1, 16, q_len, kv_len)
    q = queries(c, G, "f16", 1.0)
    o, _ = attend(c, q, "f16")
    want, _, A, S = ref.attention(f64(q), kind, *c.host(), c.q_start, c.kv_len, c.table, D ** -0.5, True, 0)
    tol = A * (2 * (D + 8) * U * S + (max(kv_len) + 72) * U + 2.0 ** -21)[..., None] + 1.01 * HALF["f16"] * np.abs(want) + SMALL["f16"]
    err = np.abs(f64(o) - want)
    assert (err <= tol).all(), "%d of %d off, worst %.3g of the bound" % ((err > tol).sum(), err.size, (err / tol).max())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len", [[3], [70], [300]])
def test_f16_codes_that_are_not_finite(dtype, D, q_len):
    """An infinite or NaN code of a value makes its own element of the tokens that see it not finite, and touches nothing else."""
    n, kv, window = q_len[0], 700, 150
    gu.banner("infinite codes %s D=%d q=%d" % (dtype, D, n))
    c = Case(D + n, ref.F16, D, 2, 16, q_len, [kv])
    q = queries(c, 4, dtype, 1.0)
    o, l = attend(c, q, dtype, window=window)
    # bad codes in the last pages: before, among and after the new tokens' positions
    codes = c.dev[1].view(torch.float16)
    put = [(kv - n - 20, 5, float("inf")), (kv - n // 2 - 1, D - 1, -float("inf")), (kv - 2, 17, float("nan")), (kv - 1, 18, float("inf"))]
    for t, d, x in put:
        pg, slot = ref.place_at(c.table, c.pages, 16, 0, t)
        codes[pg, 1, slot, d] = x
    o2, l2 = attend(c, q, dtype, window=window)
    assert torch.equal(l, l2) and torch.equal(o[:, :2], o2[:, :2])  # the other key/value head
    bad = torch.zeros_like(o[:, 2:], dtype=torch.bool)
    p = torch.arange(kv - n, kv, device="cuda")
    for t, d, _ in put:
        bad[(p >= t) & (p < t + window), :, d] = True
    assert torch.equal(~o2[:, 2:].isfinite(), bad)  # an infinity or, where parts of a probability differ in sign, a NaN
    assert torch.equal(o2[:, 2:][~bad], o[:, 2:][~bad])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", [ref.F16, ref.I8])
@pytest.mark.parametrize("first", [0.0, 2.0 ** -60, 2.0 ** 60])
@pytest.mark.parametrize("q_len,kv_len,border", [([1], 300, 150), ([1], 6000, 3000), ([90], 700, 350), ([200], 3000, 1500)])
def test_value_scales_that_differ_widely(dtype, kind, first, q_len, kv_len, border):
    """Rows of zeros, or of values 2^120 apart, in one context: every position keeps its weight in the softmax, within a
    step, between the waves of a block and between splits."""
    gu.banner("value scales %s kind=%d first=%g q=%s kv=%d" % (dtype, kind, first, q_len, kv_len))
    c = Case(kv_len + kind, kind, 64, 1, 16, q_len, [kv_len])
    vs = c.dev[3].cpu()
    for t in range(kv_len):
        pg, slot = ref.place_at(c.table, c.pages, 16, 0, t)
        vs[pg, 0, slot] *= first if t < border else (2.0 ** -60 if first > 1 else 2.0 ** 60)
    c.dev[3].copy_(vs)
    q = queries(c, 4, dtype, 0.3)
    o, l = attend(c, q, dtype)
    want, lse, A, S = ref.attention(f64(q), kind, *c.host(), c.q_start, c.kv_len, c.table, 64 ** -0.5, True, 0)
    e = (64 + 8) * U * S
    r = 2.0 ** -21 if dtype == "f32" or q_len[0] == 1 else 2 * 2.0 ** -11
    tol = A * (2 * e + (kv_len + 72) * U + r)[..., None] + 1.01 * HALF[dtype] * np.abs(want) + SMALL[dtype]
    err = np.abs(f64(o) - want)
    assert (err <= tol).all(), "%d of %d off, worst %.3g of the bound" % ((err > tol).sum(), err.size, np.nanmax(err / tol))
    assert (np.abs(f64(l) - lse) <= e + (kv_len + 72) * U + U * np.abs(lse) + U).all()
