"""The embedding gradient added to what the weight's gradient holds: every column of every row gets its sum, also in rows
whose last 16-byte unit overlaps the one before it and whose sums are joined from several runs of tokens."""

import numpy as np
import pytest
import torch

import collective_communication_reduction_amd as gc
from oracle import token as K
from tests.gpu_util import DEV
from tests.test_gpu_embed import HALF, TYPES, U, _dev, _f64, _rows, _tokens, guarded, untouched

pytestmark = pytest.mark.gpu

HIDDEN = [9, 10, 11, 12, 13, 14, 15, 17, 99, 1001, 4095, 4097, 4100]


def _check(tokens, V, H, dtype, gt, offset, kind, accumulate):
    rng = np.random.default_rng(H * 5 + offset + len(tokens))
    dout = [_rows(rng, (n, H), dtype, 1.0, offset) for n in tokens]
    ids = [_tokens(rng, n, V, kind) for n in tokens]
    dw = [guarded((V, H), TYPES[gt], offset, fill=3) for _ in tokens]
    old = [_rows(rng, (V, H), gt, 2.0, offset) for _ in tokens]
    for d, o in zip(dw, old):
        d[1].copy_(o)
    scratch = torch.empty(gc.gc_embedding_backward_scratch_bytes(tokens, V, H), dtype=torch.uint8, device=DEV)
    gc.gc_embedding_backward(dout, [_dev(i) for i in ids], tokens, V, H, [d[1] for d in dw], scratch, scale=1.75, accumulate=accumulate)
    for r, n in enumerate(tokens):
        want, mag, terms = K.embedding_backward(_f64(dout[r]), ids[r], V, 1.75)
        if accumulate:
            want, mag = want + _f64(old[r]), mag + np.abs(_f64(old[r]))
        # n - 1 additions, the product, the addition to what was there; one rounding to the gradient's type
        tol = (terms[:, None] + 3) * U * mag + HALF[gt] * np.abs(want) * (1 + 2 ** -8)
        wrong = np.argwhere(np.abs(_f64(dw[r][1]) - want) > tol)
        assert not len(wrong), (r, sorted({int(c) for _, c in wrong}))
        if accumulate:
            assert torch.equal(dw[r][1][_dev(terms == 0)], old[r][_dev(terms == 0)])
        assert untouched(dw[r][0], offset, V * H, fill=3)


@pytest.mark.parametrize("H", HIDDEN)
@pytest.mark.parametrize("tokens,V,kind", [([2600], 7, "one"), ([700, 30], 90, "zipf")])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("accumulate", [False, True])
def test_every_column_bf16(tokens, V, H, kind, offset, accumulate):
    _check(tokens, V, H, "bf16", "bf16", offset, kind, accumulate)


@pytest.mark.parametrize("H", [5, 6, 7, 9, 13, 4097])
@pytest.mark.parametrize("dtype,gt", [("bf16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32")])
def test_every_column_other_types(H, dtype, gt):
    _check([2600], 7, H, dtype, gt, 1, "one", True)


def test_micro_batches_add_up():
    """Three calls that add; a token's ten rows lie in three runs of eight sorted tokens: the end of one, a whole one, the start of one."""
    V, H, n = 4, 12, 17
    dw = torch.zeros(V, H, dtype=torch.bfloat16, device=DEV)
    ids = torch.tensor([0] * 7 + [2] * 10, dtype=torch.int32, device=DEV)
    dout = torch.ones(n, H, dtype=torch.bfloat16, device=DEV)
    scratch = torch.empty(gc.gc_embedding_backward_scratch_bytes([n], V, H), dtype=torch.uint8, device=DEV)
    for _ in range(3):
        gc.gc_embedding_backward([dout], [ids], [n], V, H, [dw], scratch, accumulate=True)
    # small whole numbers: exact in bf16 up to 256
    assert (dw[2] == 30).all() and (dw[0] == 21).all() and (dw[[1, 3]] == 0).all()
