"""CPU pins of the layer operators' oracle: the 8-bit format against torch's e4m3
type, backward passes against differences, block tables against hand counts."""

import numpy as np
import pytest
import torch

import collective_communication_reduction_amd as gc
from oracle import layer as L


def test_e4m3_codes_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = L.e4m3_table()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


def test_e4m3_rounding_matches_torch_on_every_tie():
    t = np.sort(L.e4m3_table()[:127])
    mids = (t[1:] + t[:-1]) / 2
    v = np.concatenate([t, mids, mids * (1 + 2.0 ** -20), mids * (1 - 2.0 ** -20)])
    v = np.concatenate([v, -v])
    want = torch.from_numpy(v).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(L.encode_e4m3(v), want)


@pytest.mark.parametrize("a,e", [(0.0, -117), (448.0, 0), (np.nextafter(448.0, 500), 1), (1.75, -8), (1.7500001, -7),
                                 (1.0, -8), (2.0, -7), (1e-40, -117), (float(np.finfo(np.float32).max), 120)])
def test_block_exponent(a, e):
    assert L.block_exponent(a) == e
    if -117 < e < 120:
        assert a <= 448 * 2.0 ** e and (a == 0 or a > 448 * 2.0 ** (e - 1))


def test_round_trip_error_is_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(20, 100)) * 10.0 ** rng.integers(-6, 6, size=(20, 100))
    p = L.pack8(x)
    assert p.shape[1] == L.row_bytes(100) == gc.gc_mx8_row_bytes(100) == 112
    e = np.repeat(p[:, 100:104].astype(int) - 127, 32, axis=1)[:, :100]
    assert np.all(np.abs(L.unpack8(p, 100) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (e - 10.0)))
    assert not p[:, 104:].any()


@pytest.mark.parametrize("n", [1, 31, 32, 33, 480, 4096, 11008])
def test_row_bytes(n):
    assert gc.gc_mx8_row_bytes(n) == L.row_bytes(n) and L.row_bytes(n) % 16 == 0
    assert L.row_bytes(n) - n - -(-n // 32) in range(16)


def _difference(f, a, d, h=1e-6):
    return (f(a + h * d) - f(a - h * d)) / (2 * h)


def test_norm_backward_against_differences():
    rng = np.random.default_rng(1)
    s, w, dy, ds = rng.normal(size=(5, 12)), rng.normal(size=12), rng.normal(size=(5, 12)), rng.normal(size=(5, 12))
    eps = 1e-3
    loss = lambda s_, w_: (L.rms_norm(s_, w_, eps)[0] * dy).sum() + (s_ * ds).sum()  # noqa: E731
    dx, dw = L.rms_norm_backward(dy, s, w, L.rms_norm(s, w, eps)[1], ds)
    for _ in range(4):
        v, u = rng.normal(size=s.shape), rng.normal(size=w.shape)
        assert abs(_difference(lambda a: loss(a, w), s, v) - (dx * v).sum()) < 1e-7
        assert abs(_difference(lambda a: loss(s, a), w, u) - (dw * u).sum()) < 1e-7


def test_ffn_backward_against_differences():
    rng = np.random.default_rng(2)
    T, H, F = 6, 5, 7
    x, wg, wu, wd = rng.normal(size=(T, H)), rng.normal(size=(F, H)), rng.normal(size=(F, H)), rng.normal(size=(H, F))
    dy = rng.normal(size=(T, H))
    g, u, _, _ = L.ffn(x, wg, wu, wd)
    b = L.ffn_backward(dy, x, g, u, wg, wu, wd)
    loss = lambda *a: (L.ffn(*a)[3] * dy).sum()  # noqa: E731
    args = [x, wg, wu, wd]
    for i, k in enumerate(("dx", "dwg", "dwu", "dwd")):
        v = rng.normal(size=args[i].shape)
        got = _difference(lambda a: loss(*args[:i], a, *args[i + 1:]), args[i], v)
        assert abs(got - (b[k] * v).sum()) < 1e-6


def test_blocks_clamp_malformed_tables():
    s = np.zeros((2, 2, 3), dtype=np.int64)
    s[0, 0] = [2, -5, 3]
    s[1, 0] = [1, 0, 1 << 50]
    s[0, 1] = [0, 4, 0]
    assert L.blocks(s, [10, 3]) == [(0, 0, 0, 3), (0, 1, 3, 0), (0, 2, 3, 7), (1, 0, 0, 0), (1, 1, 0, 3), (1, 2, 3, 0)]
