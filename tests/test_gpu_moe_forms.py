"""Every form in which the expert layer's products run: operands, waves along a row, tiles of outputs a block, phases of
activations, forms of scales. Each test asks for the plan first (wq_describe_moe, on 256 CUs) and holds the result to the bounds
of the arithmetic."""
from __future__ import annotations

import re

import numpy as np
import pytest

import moe_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("no GPU", allow_module_level=True)

import gpu_util as gu  # noqa: E402
import weight_only_quantized_matmul_amd as wq  # noqa: E402
from test_gpu_moe_ranges import Layer, choose, matrix  # noqa: E402

SPREAD = {ref.I8: 74.0, ref.I4: 4.6, ref.I2: 1.2}
STEP = {ref.I8: 128, ref.I4: 256, ref.I2: 512}  # columns of 128 bytes
# one scale a row, groups of whole halves of a step, groups that are not
SCALES = [(ref.I8, 0), (ref.I8, 64), (ref.I8, 192), (ref.I4, 0), (ref.I4, 64), (ref.I4, 128), (ref.I2, 0), (ref.I2, 64), (ref.I2, 256)]


@pytest.fixture(autouse=True)
def _init():
    gu.reinit_with_env(WQ_FAULT=None, WQ_MEM_LIMIT_BYTES=None)
    yield
    torch.cuda.synchronize()


def plan(layer, T, k, stride=None):
    """The numbers of a plan: {"in": {"operands": ...}, "out": {...}, "plan": ...}."""
    text = wq.wq_describe_moe(layer.moe, wq.WQ_DT_F32, T, k, stride)
    m = re.fullmatch(r"in (.*) out (.*) plan=(\d) copy=(\d) workspace=(\d+)", text)
    side = lambda s: {a: b if "-" in b else int(b) for a, b in (f.split("=") for f in s.split())}  # noqa: E731
    return {"in": side(m[1]), "out": side(m[2]), "plan": int(m[3]), "copy": int(m[4])}


def layer_of(rng, fmt, gs, D, F, O, sets, E=None):
    return Layer([[matrix(rng, fmt, r, c, gs, 1 / (SPREAD[fmt] * np.sqrt(c))) for r, c in ((F, D), (F, D), (O, F))] for _ in range(sets)], E)


def phases(p, side):
    return int(p[side]["phases"].split("-")[1])


@pytest.mark.parametrize("steps,waves", [(2, 1), (6, 2), (17, 4)])
@pytest.mark.parametrize("side", ["in", "out"])
@pytest.mark.parametrize("fmt,gs", SCALES)
def test_operands_and_waves(fmt, gs, side, steps, waves):
    """One, two, four (three) and eight operands with one, two and four waves along rows whose last step is not full; expert 0 has
    a row of every token: all that are taken at a time, and more."""
    rng = np.random.default_rng(51)
    long = STEP[fmt] * (steps - 1) + 77
    D, F, O = (long - 1, 70, 40) if side == "in" else (72, long, 40)
    layer = layer_of(rng, fmt, gs, D, F, O, 3)
    turned = gs > 0 and fmt != ref.I8 and gs % (STEP[fmt] // 2) != 0
    for T, operands, dtype, apart in ((4, 1, "f32", 0), (3, 1, "f16", 1), (8, 2, "f32", 0), (7, 2, "bf16", 1), (14, 4, "bf16", 0), (40, 8, "f32", 1)):
        p = plan(layer, T, 2, D + apart)
        assert p[side]["waves"] == waves and p[side]["tiles"] == 1 and p["plan"] == (operands >= 4 or apart)
        assert p[side]["operands"] == (3 if turned and operands >= 4 else operands)
        ids, w = choose(rng, T, 2, 2)
        ids[:, 1], ids[:, 0] = ids[:, 0] + 1, 0
        layer.check(rng.normal(0, 1, (T, D)).astype(np.float32), ids, w, "%s fmt %d gs %d operands %d waves %d" % (side, fmt, gs, operands, waves), dtype, apart)
    if steps == 17:  # all rows of an operand: more than one phase of activations
        assert phases(plan(layer, 4, 2), side) > 1 or fmt == ref.I8
        assert all(phases(plan(layer, T, 2), side) > 1 for T in (8, 14, 40))
    layer.free()


# (tokens, chosen, experts): one operand without a plan and with one, two without and with
MANY = [(4, 32, 1024, 1, 0), (9, 32, 1024, 1, 1), (8, 32, 64, 2, 0), (17, 32, 256, 2, 1)]


@pytest.mark.parametrize("T,k,E,operands,planned", MANY)
@pytest.mark.parametrize("side", ["in", "out"])
@pytest.mark.parametrize("fmt,gs", SCALES)
def test_blocks_of_several_tiles(fmt, gs, side, T, k, E, operands, planned):
    """Many experts: a block takes several tiles of outputs, the last one's outputs end inside a tile; an expert with all rows
    that are taken at a time."""
    rng = np.random.default_rng(52)
    D, F, O = (STEP[fmt] + 36, 1610, 40) if side == "in" else (40, STEP[fmt] + 33, 3300)
    layer = layer_of(rng, fmt, gs, D, F, O, 2, E)
    p = plan(layer, T, k)
    assert p[side]["tiles"] > 1 and p[side]["waves"] == 1 and p[side]["operands"] == operands and p["plan"] == planned
    ids, w = choose(rng, T, E - 1, k)
    ids[:, 1:], ids[:, 0] = ids[:, 1:] + 1, 0
    layer.check(rng.normal(0, 1, (T, D)).astype(np.float32), ids, w / k, "%s fmt %d gs %d tiles %d" % (side, fmt, gs, p[side]["tiles"]))
    layer.free()


@pytest.mark.parametrize("T,k,E,operands,planned", [MANY[0], MANY[2], MANY[3]])
@pytest.mark.parametrize("side", ["in", "out"])
@pytest.mark.parametrize("fmt,gs", [(ref.I8, 0), (ref.I8, 64), (ref.I4, 0), (ref.I4, 64), (ref.I2, 0), (ref.I2, 256)])
def test_blocks_of_several_tiles_in_phases(fmt, gs, side, T, k, E, operands, planned):
    """Several tiles of outputs whose rows' activations come in several phases: they are brought anew for every tile."""
    rng = np.random.default_rng(53)
    long = STEP[fmt] * {ref.I8: 25, ref.I4: 13, ref.I2: 7}[fmt] + 20  # more than one phase of four rows
    D, F, O = (long, 1610, 24) if side == "in" else (24, long, 3300)
    layer = layer_of(rng, fmt, gs, D, F, O, 1, E)
    p = plan(layer, T, k)
    assert p[side]["tiles"] > 1 and phases(p, side) > 1 and p[side]["operands"] == operands
    ids, w = choose(rng, T, E - 1, k)
    ids[:, 1:], ids[:, 0] = ids[:, 1:] + 1, 0
    ids[:, 12:] = -1  # (so much of the reference's work)
    layer.check(rng.normal(0, 1, (T, D)).astype(np.float32), ids, w / k, "%s fmt %d gs %d tiles %d phases %d" % (side, fmt, gs, p[side]["tiles"], phases(p, side)))
    layer.free()


def test_plans():
    """The text of a plan, and its refusals."""
    rng = np.random.default_rng(54)
    layer = layer_of(rng, ref.I4, 0, 100, 60, 40, 4)
    text = wq.wq_describe_moe(layer.moe, wq.WQ_DT_F32, 1, 2)
    assert text.startswith("in operands=1 waves=1 tiles=1 rows=4 phases=1-1 out operands=1 waves=1 tiles=1 rows=4 phases=1-1 plan=0 copy=0 workspace=")
    assert " plan=1 copy=1 " in wq.wq_describe_moe(layer.moe, wq.WQ_DT_BF16, 1, 2, x_stride=101)
    for args, code in (((wq.WQ_DT_I8, 1, 1), wq.WQ_E_INVAL), ((wq.WQ_DT_F32, 0, 1), wq.WQ_E_INVAL), ((wq.WQ_DT_F32, 1, 0), wq.WQ_E_INVAL),
                       ((wq.WQ_DT_F32, 1, 1, -1), wq.WQ_E_INVAL), ((wq.WQ_DT_F32, wq.WQ_MOE_MAX_ROWS, 2), wq.WQ_E_UNSUPPORTED)):
        with pytest.raises(wq.WqError) as e:
            wq.wq_describe_moe(layer.moe, *args)
        assert e.value.code == code
    layer.free()
