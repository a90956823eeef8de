"""Log probabilities on 9 to 60 ranks, which have kernels of their own: every kind of row, ties, bans and empty rows among
them, with the bounds of the tests on fewer ranks."""

import pytest

from tests import test_gpu_logprob as few

pytestmark = pytest.mark.gpu

MANY = [
    # ranks' rows, vocabulary, padding columns, type, element offset
    ([1 + s % 2 for s in range(60)], 300, 4, "bf16", 0), ([3, 0, 2] * 3, 1003, 5, "bf16", 1), ([2] * 9, 33000, 0, "fp32", 0),
    ([s % 3 for s in range(34)], 70000, 0, "bf16", 0), ([1] * 16, 5, 0, "fp32", 0), ([2] * 12, 4096, 0, "fp32", 0),
]


@pytest.mark.parametrize("rows,V,pad,dtype,offset", MANY)
@pytest.mark.parametrize("kind", few.KINDS)
def test_many_ranks(rows, V, pad, dtype, offset, kind):
    few.test_token_logprob(rows, V, pad, dtype, offset, kind)
