"""Numbers that do not fit a C int, in the binding of the calls between a decoder layer's products (no GPU)."""
from __future__ import annotations

import pytest

import weight_only_quantized_matmul_amd as wq


@pytest.mark.parametrize("rot,pairing,sections", [((1 << 32) + 8, 0, [4]), (8, 1 << 32, [4]), (8, 0, [(1 << 32) + 4]),
                                                  (8, 0, [5, -1 - (1 << 32)])])
def test_rope_create_takes_no_number_modulo_2_to_the_32(rot, pairing, sections):
    with pytest.raises(wq.WqError):
        wq.wq_rope_create(rot, pairing, 1e4, sections)


def test_c_ints():
    assert [wq._int(v) for v in (-1, 0, 7, (1 << 31) - 1, 1 << 31, 1 << 70, -2, -(1 << 40))] == [
        -1, 0, 7, (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1, -1, -1]
