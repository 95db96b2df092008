"""Pins of the 8-bit activation oracle (CPU)."""
import numpy as np
import torch

from oracle import a8_oracle as a8
from oracle import awq_oracle as o


def test_e4m3_rounding_matches_the_format():
    """Every e4m3 value maps to itself, and midpoints and random values round as torch's conversion."""
    bits = np.arange(256, dtype=np.uint8)
    vals = torch.from_numpy(bits).view(torch.float8_e4m3fn).double().numpy()
    vals = vals[np.isfinite(vals)]
    assert np.array_equal(a8.round_e4m3(vals), vals)
    pos = np.unique(np.abs(vals))
    mid = (pos[1:] + pos[:-1]) / 2
    v = np.concatenate([mid, -mid, np.random.default_rng(0).uniform(-448, 448, 10000).astype(np.float32)])
    want = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(a8.round_e4m3(v.astype(np.float32).astype(np.float64)), want)


def test_codes_below_16_are_linear_in_e4m3():
    """A byte b < 16 read as e4m3 is b 2^-9: a 4-bit code needs no conversion."""
    v = torch.arange(16, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, np.arange(16) * 2.0 ** -9)


def test_norm_by_hand():
    x, r = np.array([[1.0, 2.0]]), np.array([[2.0, 2.0]])
    h, y = a8.rmsnorm(x, r, np.array([1.0, 2.0]), 0.5)
    assert np.array_equal(h, [[3.0, 4.0]])
    assert np.allclose(y, [[3 / np.sqrt(13.0), 8 / np.sqrt(13.0)]], rtol=1e-15)
    assert np.allclose(a8.row_scale(y, "int8"), [8 / np.sqrt(13.0) / 127])


def test_product_is_the_dequantized_product():
    rng = np.random.default_rng(1)
    art = o.pack((rng.standard_normal((5, 256)) / 16).astype(np.float32), np.ones(256, np.float32))
    x = rng.integers(-127, 128, (3, 256)).astype(np.float64)
    sc = rng.uniform(0.1, 1, 3)
    Y, mag, absmag = a8.w4a8(x, sc, art)
    want = (x * sc[:, None]) @ o.dequant_artefact(art["qweight"], art["scales"], art["zeros"]).astype(np.float64).T
    assert np.allclose(Y, want, rtol=1e-12, atol=1e-12)
    assert np.all(absmag >= mag) and np.all(mag >= np.abs(Y) - 1e-12)
