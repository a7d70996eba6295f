"""Pins of the float64 oracle of the operators around the block against exact
rational arithmetic, closed forms and brute-force loops."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import block


def test_layer_norm_against_fractions():
    x = [[3, -1, 4, 1, -5, 9], [2, 2, 2, 2, 2, 2]]
    for row, got in zip(x, block.norm(x, "layer", eps=0.25)):
        f = [Fraction(v) for v in row]
        mean = sum(f) / 6
        var = sum((v - mean) ** 2 for v in f) / 6
        assert got == pytest.approx([float(v - mean) / math.sqrt(float(var) + 0.25) for v in f], abs=1e-15)


def test_rms_norm_closed_form_and_scale_invariance():
    x = np.array([[3.0, 4.0]])
    assert block.norm(x, "rms", eps=0.0)[0] == pytest.approx([3 / math.sqrt(12.5), 4 / math.sqrt(12.5)])
    assert block.norm(8 * x, "rms", eps=0.0) == pytest.approx(block.norm(x, "rms", eps=0.0))
    assert block.norm(x, "rms", weight=[2, 0], bias=[0, 7], eps=0.0)[0] == pytest.approx([6 / math.sqrt(12.5), 7])


def test_layer_norm_ignores_an_offset():
    g = np.random.default_rng(1)
    x = g.standard_normal((3, 50))
    assert block.norm(x + 5.0) == pytest.approx(block.norm(x), abs=1e-12)


def test_modulation_and_gate_row_by_row():
    g = np.random.default_rng(2)
    n, y = g.standard_normal((6, 4)), g.standard_normal((6, 4))
    sc, sh, ga = (g.standard_normal((3, 4)) for _ in range(3))
    index = np.array([0, 2, -1, 1, 3, 2], np.int32)               # -1 and 3 are padding
    i = block.rows_of(6, 3, index)
    h, o = block.modulate(n, i, sc, sh), block.gated(n, y, i, ga)
    for r, k in enumerate(index):
        if 0 <= k < 3:
            assert h[r] == pytest.approx(n[r] * (1 + sc[k]) + sh[k])
            assert o[r] == pytest.approx(n[r] + ga[k] * y[r])
        else:
            assert not h[r].any() and (o[r] == n[r]).all()
    assert block.rows_of(5, 3, group=2).tolist() == [0, 0, 1, 1, 2]


def test_epilogue_order():
    v = np.array([[1.0, -2.0]])
    out = block.epilogue(v, np.array([0]), bias=[0.5, 0.5], act="silu", gate=[[2.0, 3.0]], residual=[[10.0, 20.0]])
    want = [10 + 2 * 1.5 / (1 + math.exp(-1.5)), 20 + 3 * -1.5 / (1 + math.exp(1.5))]
    assert out[0] == pytest.approx(want)
    assert block.activation([1.0], "gelu")[0] == pytest.approx(0.5 * (1 + math.tanh(math.sqrt(2 / math.pi) * 1.044715)))
    assert block.epilogue(v, np.array([-1]), residual=[[10.0, 20.0]])[0].tolist() == [10.0, 20.0]
    assert block.epilogue(v, np.array([-1]))[0].tolist() == [0.0, 0.0]
