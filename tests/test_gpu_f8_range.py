"""8-bit matrices of values at the top of f32's range, where a code's value may be 2^128."""
import numpy as np
import pytest
import torch

import mixed_gemm_amd as mg
from oracle import f8 as of8
from tests.f8_util import codes, scales, value

pytestmark = pytest.mark.gpu

BORDER = {"e4m3": 2.0 ** 128 * (1 - 2.0 ** -5), "e5m2": 2.0 ** 128 * (1 - 2.0 ** -4)}


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_values_that_round_to_two_to_the_128(fmt):
    b = np.float32(BORDER[fmt])
    X = np.zeros((4, 160), np.float32)
    X[0, :3] = b, 1.0, -1e30                                          # a tie, to the even code: 2^128
    X[1, :3] = np.nextafter(b, np.float32(0)), 1.0, -1e30             # below it: finite
    X[2, 130] = -np.finfo(np.float32).max
    X[3] = 3.0e38
    x = mg.f8_checkpoint(torch.from_numpy(X).cuda(), fmt)
    q, s = of8.quantize(X, fmt)
    assert np.array_equal(codes(x), q) and np.array_equal(scales(x), s)
    exact = value(x)
    assert exact[0, 0] == 2.0 ** 128 and exact[2, 130] == -2.0 ** 128 and exact[1, 0] < 2.0 ** 128
    for dtype in (torch.float32, torch.bfloat16):
        back = mg.f8_restore(x, dtype).double().cpu().numpy()
        assert np.array_equal(back, np.where(np.abs(exact) >= 2.0 ** 128, np.copysign(np.inf, exact), exact))
    xt = mg.F8.empty(160, 32, fmt)
    mg.mg_f8_transpose(x, xt)
    want = of8.t(np.where(np.abs(exact) >= 2.0 ** 128, np.inf, exact), fmt)
    assert np.array_equal(value(xt)[:, :4], want, equal_nan=True)
