"""Dropouts of several layers over several steps: only the sum of offset and step tells masks apart, and offsets spaced
as the interface says keep every layer's mask of every step its own."""

import itertools
import os

import numpy as np
import pytest
import torch

from oracle import token as K

N, P, SEED, LAYERS, STEPS = 4096, 0.5, 1234567, 4, 5


def _apart(masks):
    """Every two masks agree in half of their elements, within six standard deviations."""
    return all(abs((a == b).mean() - 0.5) <= 6 * 0.5 / np.sqrt(N) for a, b in itertools.combinations(masks, 2))


def _spacings():
    spaced = [(layer << 40, step) for step in range(STEPS) for layer in range(LAYERS)]
    counted = [(layer, step * LAYERS) for step in range(STEPS) for layer in range(LAYERS)]
    return spaced, counted


def test_spaced_sums_give_masks_of_their_own():
    for calls in _spacings():
        assert _apart([K.keep(N, 0, P, SEED, offset + step) for offset, step in calls])
    # sums that meet: layer 1 of a step has the mask of layer 0 of the next
    assert np.array_equal(K.keep(N, 0, P, SEED, 0 + 1), K.keep(N, 0, P, SEED, 1 + 0))


def test_the_header_says_how():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "gc.h"), encoding="utf-8") as f:
        text = " ".join(f.read().replace("*", " ").split())
    assert "different offsets or steps" not in text
    assert "share a mask exactly where their sums" in text


@pytest.mark.gpu
def test_kernel_masks_of_layers_and_steps():
    import collective_communication_reduction_amd as gc
    x, y = torch.ones(N, device="cuda"), torch.empty(N, device="cuda")

    def mask(offset, step):
        gc.gc_dropout([x], [N], P, SEED, [y], offset=offset, step=torch.tensor([step], device="cuda"))
        return (y != 0).cpu().numpy()
    for calls in _spacings():
        masks = [mask(*c) for c in calls]
        assert _apart(masks)
        assert all(np.array_equal(m, K.keep(N, 0, P, SEED, sum(c))) for m, c in zip(masks, calls))
    assert np.array_equal(mask(0, 1), mask(1, 0))
