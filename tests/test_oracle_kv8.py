"""Pins of the 64-bit restatement of the 8-bit KV cache: the code values, rounding by brute force, the exponent
rule, and attention against a dense softmax."""
import numpy as np
import pytest
import torch

from oracle import kv8 as O


def test_code_values_are_e4m3():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    v = O.e4m3_values()
    assert np.array_equal(np.isnan(t), np.isnan(v)) and np.array_equal(t[~np.isnan(t)], v[~np.isnan(v)])


def test_rounding_is_the_nearest_code_ties_to_even():
    g = np.random.default_rng(0)
    grid = np.unique(O.e4m3_values()[~np.isnan(O.e4m3_values())])
    mid = (grid[1:] + grid[:-1]) / 2
    y = np.concatenate([g.normal(size=3000) * 2.0 ** g.integers(-12, 9, 3000), mid, grid, [500.0, -1e9]])
    got = O.e4m3_values()[O.nearest_codes(y)]
    best = np.min(np.abs(np.clip(y, -448, 448)[:, None] - grid[None, :]), axis=1)
    assert np.array_equal(np.abs(np.clip(y, -448, 448) - got), best)
    tied = O.nearest_codes(mid)
    assert np.all(tied % 2 == 0)


def test_exponent_is_the_smallest_that_covers():
    g = np.random.default_rng(1)
    x = g.normal(size=(500, 64)) * 2.0 ** g.integers(-30, 30, 500)[:, None]
    _, b = O.quantise(x)
    e = b.astype(int) - O.BIAS
    top = np.abs(x).max(-1)
    assert np.all(top <= 448 * 2.0 ** e) and np.all(top > 448 * 2.0 ** (e - 1))
    z = np.zeros((1, 64))
    assert O.quantise(z)[1][0] == O.E_LO + O.BIAS
    z[0, 3] = np.inf
    assert O.quantise(z)[1][0] == O.BAD and np.isnan(O.dequantise(*O.quantise(z))).all()


def test_reading_and_writing_again_keeps_values():
    g = np.random.default_rng(2)
    x = O.dequantise(*O.quantise(g.normal(size=(2000, 64)) * np.exp(2 * g.normal(size=(2000, 1)))))
    assert np.array_equal(O.dequantise(*O.quantise(x)), x)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_against_a_dense_softmax(d):
    g = np.random.default_rng(3)
    q, K, V = g.normal(size=(5, d)), g.normal(size=(33, d)), g.normal(size=(33, d))
    see = g.random((5, 33)) < 0.5
    see[2] = False
    out, _, _ = O.attend(q, K, V, see, d ** -0.5)
    s = torch.from_numpy(q @ K.T * d ** -0.5).masked_fill(~torch.from_numpy(see), -np.inf)
    want = torch.nan_to_num(torch.softmax(s, -1)) @ torch.from_numpy(V)
    assert np.allclose(out, want.numpy(), rtol=0, atol=1e-13) and not out[2].any()
