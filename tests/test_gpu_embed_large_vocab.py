"""The embedding gradient of long ranks over large vocabularies: the sort by two digits of 11 bits in pieces of 1024
tokens, several workgroups for each digit."""

import numpy as np
import pytest
import torch

import collective_communication_reduction_amd as gc
from oracle import token as K
from tests.gpu_util import DEV
from tests.test_gpu_embed import HALF, U, _dev, _f64, _rows, _tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,V,H", [([2600], (1 << 20) + 1, 3), ([5000, 1], 1 << 22, 2), ([3100, 2049, 0], (1 << 21) + 12345, 4)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_large_vocabulary_in_pieces(tokens, V, H, accumulate):
    rng = np.random.default_rng(V + len(tokens))
    dout = [_rows(rng, (n, H), "bf16") for n in tokens]
    # a few frequent tokens at both ends and in the middle, the rest anywhere; padding
    ids = [np.where(rng.random(n) < 0.5, rng.choice([0, 2047, 2048, V // 2, V - 1], n), _tokens(rng, n, V, "uniform")).astype(np.int32)
           for n in tokens]
    dw = [torch.full((V, H), 3.0, device=DEV) for _ in tokens]
    scratch = torch.empty(gc.gc_embedding_backward_scratch_bytes(tokens, V, H), dtype=torch.uint8, device=DEV)
    gc.gc_embedding_backward(dout, [_dev(i) for i in ids], tokens, V, H, dw, scratch, accumulate=accumulate)
    for r in range(len(tokens)):
        want, mag, terms = K.embedding_backward(_f64(dout[r]), ids[r], V)
        base = 3.0 if accumulate else 0.0
        tol = (terms[:, None] + 3) * U * (mag + base) + HALF["fp32"] * np.abs(want + base) * (1 + 2 ** -8)
        assert (np.abs(_f64(dw[r]) - want - base) <= tol).all(), r
