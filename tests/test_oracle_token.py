"""Pins of the oracle of embedding, dropout and log probabilities: the generator's
published answers, closed forms, and gradients against differences (CPU)."""

import numpy as np
import pytest

from oracle import token as K


def test_philox_known_answers():
    """Known answers published with the generator (Salmon et al., SC 2011; four 32-bit words, 10 rounds)."""
    ones = 0xFFFFFFFF
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((ones,) * 4, (ones, ones), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        got = K.philox4x32(np.array([counter], dtype=np.uint64), key)[0]
        assert tuple(int(w) for w in got) == want


def test_keep_rates_and_streams():
    n = 1 << 18
    for p in (0.0, 0.1, 0.5, 1.0):
        k = K.keep(n, 0, p, 99, 3)
        q = K.drop_steps(p) / 65536
        # standard deviation of the mean of n draws, six of them
        assert abs((~k).mean() - q) <= 6 * np.sqrt(q * (1 - q) / n)
    a = K.keep(n, 0, 0.5, 99, 3)
    for other in (K.keep(n, 1, 0.5, 99, 3), K.keep(n, 0, 0.5, 100, 3), K.keep(n, 0, 0.5, 99, 4),
                  K.keep(n, 0, 0.5, 99 + (1 << 32), 3), K.keep(n, 0, 0.5, 99, 3 + (1 << 32))):
        assert abs((a == other).mean() - 0.5) < 6 * 0.5 / np.sqrt(n)


def test_embedding_gradient_is_the_transpose():
    rng = np.random.default_rng(3)
    V, H, T = 7, 5, 23
    w, dout = rng.normal(size=(V, H)), rng.normal(size=(T, H))
    tokens = rng.integers(-2, V + 2, T)
    g, mag, n = K.embedding_backward(dout, tokens, V, 1.5)
    assert np.isclose((K.embedding(w, tokens, 1.5) * dout).sum(), (w * g).sum())
    assert (mag >= np.abs(g) - 1e-12).all() and n.sum() == ((tokens >= 0) & (tokens < V)).sum()


@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_logprob_closed_forms(scale):
    rng = np.random.default_rng(5)
    x = rng.normal(size=(4, 9)) * 3
    lp, lse = K.log_softmax(x, scale)
    assert np.allclose(np.exp(lp).sum(1), 1.0) and np.allclose(lse, np.log(np.exp(scale * x).sum(1)))
    u = K.log_softmax(np.full((1, 8), 2.5), scale)[0]
    assert np.allclose(K.entropy(u), np.log(8))
    x[1, :] = -np.inf
    x[2, 3:] = -np.inf
    lp, lse = K.log_softmax(x, scale)
    assert np.isneginf(lse[1]) and np.isneginf(lp[1]).all() and K.entropy(lp)[1] == 0
    assert np.isclose(np.exp(lp[2, :3]).sum(), 1)
    assert K.token_logprob(lp, np.array([9, 0, 5, -1])).tolist() == [0.0, -np.inf, -np.inf, 0.0]


def test_alternatives_order():
    x = np.array([[1.0, 3.0, 3.0, -np.inf, np.nan, 2.0], [np.nan] * 6])
    ids, val = K.alternatives(x[:1], np.zeros((1, 6)), 6)
    assert ids.tolist() == [[1, 2, 5, 0, 3, -1]]
    ids, _ = K.alternatives(np.array([[-0.0, 0.0, -1.0]]), np.zeros((1, 3)), 2)
    assert ids.tolist() == [[0, 1]]


@pytest.mark.parametrize("scale", [1.0, 1.3])
def test_logprob_gradient_against_differences(scale):
    rng = np.random.default_rng(8)
    T, V = 3, 6
    x, t = rng.normal(size=(T, V)), np.array([2, -1, 5])
    a, b = rng.normal(size=T), rng.normal(size=T)

    def loss(x_):
        lp, _ = K.log_softmax(x_, scale)
        return (a * K.token_logprob(lp, t) + b * K.entropy(lp)).sum()

    lp, lse = K.log_softmax(x, scale)
    g = K.token_logprob_backward(x, t, lse, a, scale, K.entropy(lp), b)
    for _ in range(5):
        v = rng.normal(size=x.shape)
        h = 1e-6
        assert abs((loss(x + h * v) - loss(x - h * v)) / (2 * h) - (g * v).sum()) < 1e-7


def test_log_softmax_of_equal_large_values():
    for v in (-1e30, 1e30, -1e300):
        lp, lse = K.log_softmax(np.full((1, 8), v))
        assert np.allclose(lp, -np.log(8), atol=1e-15) and lse[0] == v
