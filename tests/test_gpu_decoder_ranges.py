"""Inputs far from one: the operators between a decoder layer's products keep their results over fp32's whole range.

Bounds as in test_gpu_decoder.py (u = 2^-24, h(t) half a step of the output type): a norm's output is within
(36 u + h(t)) |y|, its int8 scale within 38 u of max|y| / 127; codes are exact."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("no GPU", allow_module_level=True)

import decoder_ref as ref  # noqa: E402
import gpu_util as gu  # noqa: E402
import weight_only_quantized_matmul_amd as wq  # noqa: E402

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SMALL = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}  # half a step next to zero


@pytest.fixture(scope="module", autouse=True)
def device():
    gu.reinit_with_env(WQ_FORCE_PATH=None, WQ_FAULT=None, WQ_MEM_LIMIT_BYTES=None)
    yield


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def norm_and_check(x, w, eps, out, residual=None):
    rows, n = x.shape
    y = torch.empty((rows, n), dtype=torch.int8 if out == "i8" else DT[out], device="cuda")
    sc = torch.full((rows,), 5.0, device="cuda") if out == "i8" else None
    wq.wq_rmsnorm_dev(x, w, eps, y, residual=residual, y_scale=sc)
    torch.cuda.synchronize()
    t, w64 = f64(x if residual is None else x.float() + residual.float()), f64(w)
    with np.errstate(invalid="ignore"):  # a row of zeros without eps is 0 / 0
        want = t / np.sqrt((t * t).mean(1, keepdims=True) + float(np.float32(eps))) * w64
    if out != "i8":
        none = np.isnan(want)
        assert np.array_equal(np.isnan(f64(y)), none)
        assert (np.abs(f64(y) - want) <= (36 * U + 1.01 * HALF[out]) * np.abs(want) + SMALL[out])[~none].all()
        return
    tw = t * w64
    top = np.abs(tw).max(1, keepdims=True)
    assert np.array_equal(y.cpu().numpy(), np.rint(tw * 127 / np.where(top == 0, 1, top)))
    scale = np.where(top[:, 0] == 0, 0, np.abs(want).max(1) / 127)
    assert (np.abs(f64(sc) - scale) <= 38 * U * scale + 2.0 ** -149).all()


@pytest.mark.parametrize("rows,n", [(3, 300), (3, 9001), (2051, 1000)])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_rows_of_zeros(rows, n, eps):
    """Codes and scale of a row of zeros are 0, its neighbours' what they are; NaN rows keep their NaN scale."""
    x = torch.randn((rows, n), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    x[1] = 0
    x[rows - 1] = 0
    norm_and_check(x, torch.ones(n, device="cuda"), eps, "i8")
    x[1, n - 1] = float("nan")
    y, sc = torch.full((rows, n), 9, dtype=torch.int8, device="cuda"), torch.zeros(rows, device="cuda")
    wq.wq_rmsnorm_dev(x, torch.ones(n, device="cuda"), eps, y, y_scale=sc)
    assert sc[1].isnan() and not y[1].any() and sc[0] > 0 and sc[rows - 1] == 0


EXPONENTS = (-146, -126, -100, -70, -64, -60, -50, 0, 50, 60, 63, 64, 70, 100, 124)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16", "i8"])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
@pytest.mark.parametrize("rows,n", [(len(EXPONENTS), 300), (len(EXPONENTS), 40), (len(EXPONENTS), 20001), (3003, 1000)])
def test_norm_rows_of_any_size(dtype, out, eps, rows, n):
    """Rows of every size beside each other, in one call: each decides by itself how its squares are summed."""
    gu.banner("norm sizes %s -> %s eps=%g %d x %d" % (dtype, out, eps, rows, n))
    rng = np.random.default_rng(rows + n)
    e = np.resize(EXPONENTS, rows)[:, None]
    x = torch.from_numpy(np.ldexp(rng.uniform(0.5, 1.5, (rows, n)) * rng.choice([-1, 1], (rows, n)), e).astype(np.float32))
    norm_and_check(x.cuda().to(DT[dtype]), torch.from_numpy(rng.uniform(0.5, 2, n).astype(np.float32)).cuda(), eps, out)


@pytest.mark.parametrize("out", ["f32", "i8"])
def test_norm_sums_of_any_size(out):
    rng = np.random.default_rng(9)
    x, r = (torch.from_numpy(np.ldexp(rng.normal(size=(6, 500)), np.array([[-100], [0], [64], [100], [-64], [120]])).astype(np.float32)).cuda()
            for _ in range(2))
    norm_and_check(x, torch.ones(500, device="cuda"), 0.0, out, residual=r)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("rows,n", [(2, 300), (2500, 1001)])
def test_norm_infinities_behind_zero_weights(rows, n, bad):
    """A row is not finite wherever its infinity stands, also where the weight is 0."""
    x, w = torch.ones((rows, n), device="cuda"), torch.ones(n, device="cuda")
    w[n // 2] = 0
    x[rows - 1, n // 2] = bad
    y, sc = torch.full((rows, n), 9, dtype=torch.int8, device="cuda"), torch.zeros(rows, device="cuda")
    wq.wq_rmsnorm_dev(x, w, 1e-6, y, y_scale=sc)
    assert sc[rows - 1].isnan() and not y[rows - 1].any()
    assert (y[:-1, : n // 2] == 127).all() and (y[:-1, n // 2] == 0).all() and (sc[:-1] > 0).all()


@pytest.mark.parametrize("pairing", [0, 1])
@pytest.mark.parametrize("theta,rot,sections", [(1e4, 128, [64]), (1e6, 64, [16, 16]), (3.0, 8, [4])])
def test_rope_of_far_positions(pairing, theta, rot, sections):
    """Every int32 position: within 8 u (|a| + |b|) + u |y|, the bound for near ones. The reference's angles, in 80 bits,
    are within 2^31 * 2^-64 * 2 turns."""
    rng = np.random.default_rng(rot)
    T = 400
    x = torch.from_numpy(rng.normal(size=(T, 2, rot)).astype(np.float32)).cuda()
    pos = rng.integers(-(1 << 31), 1 << 31, (len(sections), T)).astype(np.int32)
    pos[:, :4] = [(1 << 31) - 1, -(1 << 31), (1 << 24) + 1, 0]
    y = torch.empty_like(x)
    wq.wq_rope_dev(wq.wq_rope_create(rot, pairing, theta, sections), x, torch.from_numpy(pos).cuda(), y)
    x64 = f64(x)
    want = ref.rope(x64, pos, rot, pairing, theta, sections)
    i = np.arange(rot // 2)
    a, b = (i, i + rot // 2) if pairing == 0 else (2 * i, 2 * i + 1)
    mag = np.zeros_like(x64)
    mag[..., a] = mag[..., b] = np.abs(x64[..., a]) + np.abs(x64[..., b])
    assert (np.abs(f64(y) - want) <= 8 * U * mag + 1.01 * U * np.abs(want)).all()
