"""The expert layer over the ranges of activations and scales, within bounds that follow its arithmetic."""
from __future__ import annotations

import numpy as np
import pytest

import moe_ref as ref
import moe_tight as tight

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("no GPU", allow_module_level=True)

import gpu_util as gu  # noqa: E402
import weight_only_quantized_matmul_amd as wq  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True)
def _init():
    gu.reinit_with_env(WQ_FAULT=None, WQ_MEM_LIMIT_BYTES=None)
    yield
    torch.cuda.synchronize()


class Layer:
    """Experts of (gate, up, down) matrices; an expert's number is modulo their number where more are asked for."""

    def __init__(self, mats, E=None):
        self.mats = mats
        up = lambda m: (wq.wq_tensor_upload_gs(None, 0, m.fmt, m.w.shape[0], m.cols, m.gs, m.codes, m.scales) if m.gs  # noqa: E731
                        else wq.wq_tensor_upload(None, 0, m.fmt, m.w.shape[0], m.cols, m.codes, m.scales))
        self.handles = [[up(m) for m in ms] for ms in mats]
        E = len(mats) if E is None else E
        self.experts = [mats[e % len(mats)] for e in range(E)]
        self.moe = wq.wq_moe_create(*([self.handles[e % len(mats)][n] for e in range(E)] for n in range(3)))

    def check(self, x, ids, w, what="", dtype="f32", apart=False):
        """x float32 [T, D] numpy, taken in dtype (apart: in rows of odd stride), ids, w numpy: the result, which is within its bound."""
        gu.banner("moe %s T=%d k=%d E=%d D=%d F=%d %s" % (what, x.shape[0], ids.shape[1], len(self.experts), self.moe.D, self.moe.F, dtype))
        x = torch.from_numpy(x).cuda().to(DT[dtype])
        if apart:
            x = torch.cat([x, x[:, :1 + x.shape[1] % 2]], 1)[:, :x.shape[1]]
        y = torch.full((x.shape[0], self.moe.D_out), 7.0, dtype=x.dtype, device="cuda")
        wq.wq_moe_ffn_dev(self.moe, x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), y)
        torch.cuda.synchronize()
        want, bound = tight.moe(x.double().cpu().numpy(), ids, w, self.experts)
        bound = bound + ref.HALF[dtype] * (np.abs(want) + bound) + ref.TINY[dtype]
        worst = (np.abs(y.double().cpu().numpy() - want) / bound).max()
        assert worst <= 1, "%s: worst err/bound %.3g" % (what, worst)
        return y

    def free(self):
        torch.cuda.synchronize()
        wq.wq_moe_free(self.moe)
        for t in sum(self.handles, []):
            wq.wq_tensor_free(t)


def matrix(rng, fmt, rows, cols, gs, scale):
    codes = rng.integers(0, 256, (rows, -(-cols * ref.BITS[fmt] // 8)), dtype=np.uint8)
    shape = (rows, -(-cols // gs)) if gs else (rows,)
    return tight.Matrix(codes, (rng.uniform(0.5, 1.5, shape) * scale).astype(np.float32), cols, fmt, gs)


def choose(rng, T, E, k):
    return np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32), rng.uniform(0.1, 1.0, (T, k)).astype(np.float32)


@pytest.mark.parametrize("x,gate,up,down", [
    (2.0 ** -96, 2.0 ** 94, 2.0 ** -10, 2.0 ** 96),  # the smallest activations that keep their bits
    (1.0, 0.05, 1e-33, 1e30), (1.0, 0.05, 2.0 ** -95, 2.0 ** -25),  # small scales, small intermediates
    (2.0 ** 118, 2.0 ** -121, 2.0 ** -8, 2.0 ** -120),  # products with the codes alone would overflow
    (2.0 ** -60, 2.0 ** 56, 2.0 ** 60, 2.0 ** -70), (2.0 ** 60, 2.0 ** -64, 2.0 ** -60, 2.0 ** 70)])
@pytest.mark.parametrize("fmt,gs", [(ref.I8, 0), (ref.I8, 64), (ref.I4, 0), (ref.I4, 64), (ref.I4, 128), (ref.I2, 0), (ref.I2, 64), (ref.I2, 256)])
def test_moe_small_and_large_scales(fmt, gs, x, gate, up, down):
    """Results that are normal numbers keep their accuracy whatever the activations' unit and the scales are by themselves."""
    rng = np.random.default_rng(31)
    spread = {ref.I8: 74.0, ref.I4: 4.6, ref.I2: 1.2}[fmt] / 4.6
    D, F = 517, 300
    layer = Layer([[matrix(rng, fmt, F, D, gs, gate / spread), matrix(rng, fmt, F, D, gs, up / spread), matrix(rng, fmt, 40, F, gs, down / spread)] for _ in range(3)])
    for T, k in ((1, 2), (7, 2), (40, 1)):  # one, two and four operands
        ids, w = choose(rng, T, 3, k)
        layer.check((rng.normal(0, 1, (T, D)) * x).astype(np.float32), ids, w, "fmt %d gs %d x %g scales %g %g %g" % (fmt, gs, x, gate, up, down))
    layer.free()


@pytest.mark.parametrize("T", [2, 9, 40])
@pytest.mark.parametrize("fmt,gs", [(ref.I8, 0), (ref.I8, 128), (ref.I4, 0), (ref.I4, 64), (ref.I4, 128), (ref.I2, 0), (ref.I2, 64), (ref.I2, 256)])
def test_moe_rows_that_are_not_finite(fmt, gs, T):
    """A token with an infinity or a NaN anywhere is NaN or infinite throughout, whatever the form; the others keep their bits."""
    rng = np.random.default_rng(32)
    D, F = 700, 300
    spread = {ref.I8: 74.0, ref.I4: 4.6, ref.I2: 1.2}[fmt]
    layer = Layer([[matrix(rng, fmt, r, c, gs, 1 / (spread * np.sqrt(c))) for r, c in ((F, D), (F, D), (40, F))] for _ in range(3)])
    x, (ids, w) = rng.normal(0, 1, (T, D)).astype(np.float32), choose(rng, T, 3, 2)
    clean = layer.check(x, ids, w, "fmt %d gs %d" % (fmt, gs))
    bad = x.copy()
    bad[0, D - 1], bad[T - 1, 3] = np.nan, np.inf
    y = torch.empty_like(clean)
    wq.wq_moe_ffn_dev(layer.moe, torch.from_numpy(bad).cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), y)
    torch.cuda.synchronize()
    assert not torch.isfinite(y[[0, T - 1]]).any() and torch.equal(y[1:T - 1], clean[1:T - 1])
    layer.free()


@pytest.mark.parametrize("fmt,gs", [(ref.I8, 0), (ref.I8, 64), (ref.I4, 0), (ref.I4, 64), (ref.I2, 0), (ref.I2, 64)])
@pytest.mark.parametrize("T", [3, 8, 14, 40])  # one, two, four and eight operands
def test_moe_every_digit_counts(fmt, gs, T):
    """Large activations cancel and the result is that of small ones, of one base-256 digit each. Gate's only code makes z = 64,
    whose silu is 64 exactly. First the product with up is such a one, then, with up the identity (h = 64 x exactly), down's."""
    rng = np.random.default_rng(33)
    n = tight.COLS
    one = lambda codes, scale: tight.Matrix(tight.pack(codes, fmt), np.full((n, 2) if gs else n, scale, np.float32), n, fmt, gs)  # noqa: E731
    first, eye = np.zeros((n, n), np.int64), np.eye(n, dtype=np.int64)
    first[:, 0] = 1
    scales = (2.0 ** rng.integers(-3, 4, (n, 2) if gs else n)).astype(np.float32)
    codes = [tight.cancelling_codes(rng, n, fmt) for _ in range(2)]
    mixed = [tight.Matrix(tight.pack(q, fmt), scales, n, fmt, gs) for q in codes]
    x = tight.cancelling_rows(rng, T)
    ids, w = (np.arange(T, dtype=np.int32) % 2)[:, None], np.ones((T, 1), np.float32)
    for up, down in (([m for m in mixed], [one(eye, 1)] * 2), ([one(eye, 1)] * 2, mixed)):
        layer = Layer([[one(first, 64), u, d] for u, d in zip(up, down)])
        gu.banner("digits fmt %d gs %d T=%d" % (fmt, gs, T))
        y = torch.empty((T, n), device="cuda")
        wq.wq_moe_ffn_dev(layer.moe, torch.from_numpy(x).cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), y)
        torch.cuda.synchronize()
        for t in range(T):
            x64 = x[t:t + 1].astype(np.float64)
            u, Eu = up[t % 2].product(x64, np.zeros((1, n))) if down is not mixed else (x64, np.zeros((1, n)))
            # 64 u is exact in fp32; y passes one sum over its only expert, without rounding, and its own type, fp32
            want, bound = down[t % 2].product(64 * u, 64 * Eu)
            bound = bound + tight.U * (np.abs(want) + bound)
            err = np.abs(y[t].double().cpu().numpy() - want[0])
            assert (err <= bound[0]).all(), "token %d: worst err/bound %.3g" % (t, (err / bound[0]).max())
        layer.free()
