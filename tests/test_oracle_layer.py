"""Pins of oracle/layer.py: Philox's published answers, E4M3 against torch's
type, gradients against differences."""
import numpy as np
import pytest
import torch

from oracle import layer as L


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_philox_known_answers(counter, key, want):
    """The vectors that the generator's authors publish with it."""
    assert tuple(int(v[0]) for v in L.philox(counter, key)) == want


def test_drop_bits_are_even_and_independent_of_width():
    a, b = L.drop_bits(40, 333, 7, 9), L.drop_bits(40, 64, 7, 9)
    assert np.array_equal(a[:, :64], b)
    assert not np.array_equal(a, L.drop_bits(40, 333, 7, 10)) and not np.array_equal(a, L.drop_bits(40, 333, 8, 9))
    assert not np.array_equal(a, L.drop_bits(40, 333, 7, 9 + (1 << 32)))
    # 13320 draws of a uniform 16-bit number: the mean within five deviations
    assert abs(a.mean() - 32767.5) < 5 * 65536 / np.sqrt(12 * a.size)


def test_e4m3_is_torchs():
    v = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(L.e4m3_values(), v)
    x = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * np.exp2(np.random.default_rng(1).integers(-12, 8, 20000)).astype(np.float32)
    x = np.clip(np.concatenate([x, (v[1:] + v[:-1]) / 2]).astype(np.float32), -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = L.nearest_e4m3(np.abs(x)) | (np.signbit(x).astype(np.uint8) << 7)
    assert np.array_equal(got, want)


def test_mx8_blocks():
    x = np.zeros((3, 300))
    x[0, :32] = np.linspace(-511, 511, 32)       # up to 512 occurs, 448 is held
    x[1, 40] = np.nan
    x[2, 299] = 2.0 ** -140
    codes, scales = L.mx8_quantize(x)
    assert codes.shape == (2, 3, 256) and scales.shape == (2, 3, 8)
    assert scales[0, 0, 0] == 127 and codes[0, 0, 31] == 0x7E and codes[0, 0, 0] == 0xFE
    assert scales[0, 1, 1] == 255 and not codes[0, 1].any()
    assert scales[1, 2, 1] == 0 and codes[1, 2, 43] == 0
    back = L.mx8_dequantize(codes, scales, 300)
    assert np.isnan(back[1, 32:64]).all() and np.isfinite(back[0]).all() and back.shape == (3, 300)
    rng = np.random.default_rng(3)
    y = rng.standard_normal((5, 70)) * np.exp2(rng.integers(-30, 30, (5, 70)))
    held = L.mx8_dequantize(*L.mx8_quantize(y), 70)
    assert np.array_equal(L.mx8_dequantize(*L.mx8_quantize(held), 70), held)


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(5)
    h, w, dy = rng.standard_normal((4, 9)), rng.standard_normal(9), rng.standard_normal((4, 9))
    dh, dw = L.norm_backward(dy, h, w, 1e-3)
    f = lambda a, b: float(np.sum(dy * L.norm(a, b, 1e-3)))  # noqa: E731
    step = 1e-5
    for i in np.ndindex(4, 9):
        e = np.zeros((4, 9))
        e[i] = step
        assert abs((f(h + e, w) - f(h - e, w)) / (2 * step) - dh[i]) < 1e-8
    for c in range(9):
        e = np.zeros(9)
        e[c] = step
        assert abs((f(h, w + e) - f(h, w - e)) / (2 * step) - dw[c]) < 1e-8
