"""Pins of the oracle of the gated product, the adapters and dropout: gradients
against central differences of its own forwards, special cases with known
answers, and the generator's published test vectors."""

import math

import numpy as np
import pytest

from oracle import mlp


def _differences(loss, values, grads, tol=1e-7):
    for v, g in zip(values, grads):
        for i in np.ndindex(v.shape):
            old, d = v[i], 1e-5
            v[i] = old + d
            up = loss()
            v[i] = old - d
            down = loss()
            v[i] = old
            assert abs((up - down) / (2 * d) - g[i]) <= tol * max(1.0, abs(g[i]))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_gradient_against_differences(act):
    rng = np.random.default_rng(0)
    x, wg, wu = rng.standard_normal((3, 5)), rng.standard_normal((4, 5)), rng.standard_normal((4, 5))
    ag, au, dh = (rng.standard_normal((3, 4)) for _ in range(3))
    _, gate, up = mlp.gated_linear(x, wg, wu, act, ag, au)
    g = mlp.gated_linear_backward(dh, x, wg, wu, gate, up, act)
    _differences(lambda: (mlp.gated_linear(x, wg, wu, act, ag, au)[0] * dh).sum(), (x, wg, wu, ag, au),
                 (g["dx"], g["d_w_gate"], g["d_w_up"], g["d_gate"], g["d_up"]))


def test_activations():
    f, d = mlp.activation([0.0, 1.0, -40.0], "silu")
    assert f[0] == 0 and d[0] == 0.5 and abs(f[1] - 1 / (1 + math.exp(-1))) < 1e-15
    assert abs(f[2] / (-40 * math.exp(-40)) - 1) < 1e-12
    f, d = mlp.activation([0.0, 1.0, -10.0], "gelu")
    assert f[0] == 0 and d[0] == 0.5 and abs(f[1] - 0.8413447460685429) < 1e-15
    assert abs(f[2] / (-10 * 7.619853024160495e-24) - 1) < 1e-9  # Phi(-10)


def test_lora_gradient_against_differences():
    rng = np.random.default_rng(1)
    T, K, N, R, E = 5, 4, 3, 2, 3
    x, a, b = rng.standard_normal((T, K)), rng.standard_normal((E, R, K)), rng.standard_normal((E, N, R))
    index, scale = np.array([2, -1, 0, 2, 7]), np.array([0.5, 3.0, 2.0])
    dy = rng.standard_normal((T, N))
    out, v = mlp.lora(x, a, b, index, scale)
    assert not out[[1, 4]].any() and not v[[1, 4]].any()
    assert np.allclose(out[0], 2.0 * b[2] @ a[2] @ x[0], rtol=1e-13)
    dx, da, db = mlp.lora_backward(dy, x, v, a, b, index, scale)
    assert not da[1].any() and not db[1].any() and not dx[[1, 4]].any()
    _differences(lambda: (mlp.lora(x, a, b, index, scale)[0] * dy).sum(), (x, a, b), (dx, da, db))


def test_philox_known_answers():
    """The published known-answer vectors of Philox4x32-10."""
    f = 0xFFFFFFFF
    assert mlp.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert mlp.philox([f] * 4, [f] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert mlp.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_factors():
    n = 20000
    f = mlp.dropout_factor(n, 0.3, 5)
    # the share of zeros: five standard deviations of a binomial
    assert abs((f == 0).mean() - 0.3) < 5 * math.sqrt(0.3 * 0.7 / n)
    assert np.unique(f).tolist() == [0.0, 65536.0 / (65536 - 19661)]
    assert (mlp.dropout_factor(64, 0.0, 5) == 1).all() and not mlp.dropout_factor(64, 1.0, 5).any()
    assert np.array_equal(mlp.dropout_factor(50, 0.3, 5, first=13), f[13:63])
    assert not np.array_equal(mlp.dropout_factor(64, 0.3, 5, offset=1), f[:64])
