"""The MXFP4 oracle against hand-worked values and the format's own rules (CPU)."""
import numpy as np
import pytest

from oracle import mxfp4 as O


def test_worked_block():
    x = np.zeros((1, 32))
    x[0, :8] = [7.9, 5.0, -2.5, 1.75, 0.75, -0.25, 0.2500001, 4.9]
    codes, scales = O.quantize(x)
    assert codes.shape == (1, 1, 128) and scales.shape == (1, 1, 8)
    assert scales[0, 0].tolist() == [127, 0, 0, 0, 0, 0, 0, 0]      # floor(log2 7.9) - 2 = 0
    # 7.9 -> 6 (7), 5 ties to 4 (6), -2.5 ties to -2 (4 | 8), 1.75 ties to 2 (4), .75 ties to 1 (2),
    # -.25 ties to -0 (8), just above .25 -> .5 (1), 4.9 -> 4 (6)
    assert codes[0, 0, :4].tolist() == [0x67, 0x4C, 0x82, 0x61]
    assert O.dequantize(codes, scales, 32)[0, :8].tolist() == [6, 4, -2, 2, 1, -0.0, 0.5, 4]


def test_scale_bytes():
    assert O.scale_byte([1.0, 0.999, 4.0, 0.0, np.inf, np.nan, 2.0 ** -140, 3.0e38]).tolist() == [
        125, 124, 127, 0, 255, 255, 0, 252]


def test_every_value_of_the_format_round_trips():
    for e in (-126, -3, 0, 60, 125):
        x = np.concatenate((O.E2M1, -O.E2M1, np.zeros(16)))[None] * 2.0 ** e
        assert np.array_equal(O.held(x), x)


@pytest.mark.parametrize("shape", [(1, 1), (3, 31), (5, 33), (2, 257), (4, 512)])
def test_error_bound_and_idempotence(shape):
    x = np.random.default_rng(sum(shape)).standard_normal(shape)
    y = O.held(x)
    p = O.panels(shape[1])
    top = np.zeros((shape[0], p * 256))
    top[:, :shape[1]] = np.abs(x)
    unit = np.exp2(np.floor(np.log2(np.maximum(top.reshape(shape[0], -1, 32).max(-1), 1e-300))) - 2)
    unit = np.repeat(unit, 32, axis=1)[:, :shape[1]]
    # half the widest step (2 units), or the distance from 8 down to 6
    assert np.all(np.abs(y - x) <= 2 * unit)
    assert np.array_equal(O.held(y), y)


def test_non_finite_blocks_and_signed_zeros():
    x = np.ones((1, 96))
    x[0, 40] = np.inf
    x[0, 64:] = -0.0
    codes, scales = O.quantize(x)
    assert scales[0, 0, :3].tolist() == [125, 255, 0]
    y = O.dequantize(codes, scales, 96)
    assert np.array_equal(y[0, :32], np.ones(32)) and np.all(np.isnan(y[0, 32:64]))
    assert np.all(y[0, 64:] == 0) and np.all(np.signbit(y[0, 64:]))
