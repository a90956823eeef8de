"""The streamed forward of few rows: one expert's rows in several turns, and both sides of its limits."""

import numpy as np
import pytest

from tests import test_gpu_ffn as F

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,H,I", [
    ([[31, 0, 0, 0, 0, 0, 0, 1]], 4104, 1032), ([[0, 0, 32, 0, 0, 0, 0, 0]], 264, 2056), ([[17, 0, 0], [0, 9, 6]], 520, 264),
    ([[0, 0, 33, 0, 0, 0, 0, 0]], 264, 520), ([[16] + [0] * 63], 136, 72), ([[16] + [0] * 63 + [16]], 136, 72),
    ([[0] * 200 + [300, 1, 0, 2]], 136, 264)])
@pytest.mark.parametrize("x_t", ["bf16", "mx8"])
def test_rows_on_few_of_the_experts(counts, H, I, x_t):
    st = F.make(np.random.default_rng(H + I), counts, H, I, spare=0)
    xv, y, saved = F.run_forward(st, x_t, None)
    F.check_forward(st, xv, y, saved, None)
