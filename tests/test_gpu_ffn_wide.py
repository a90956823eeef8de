"""The experts at the largest inter that gc.h allows: 16 experts of 8 x 2^20."""

import numpy as np
import pytest
import torch

from tests import test_gpu_ffn as F
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("saved_t", [None, "bf16"])
def test_largest_inter(saved_t):
    H, I, E = 8, 1 << 20, 16
    counts = [[0] * 5 + [3] + [0] * 9 + [2]]
    rng = np.random.default_rng(1)
    st = F.make(rng, counts, H, 8)
    st["F"] = I
    g = torch.Generator(device=DEV).manual_seed(2)
    for k, sh, sc in (("w_gate", (E, I, H), H), ("w_up", (E, I, H), H), ("w_down", (E, H, I), I)):
        st[k] = [torch.empty(*sh, dtype=torch.bfloat16, device=DEV).normal_(0, sc ** -0.5, generator=g)]
    xv, y, saved = F.run_forward(st, "bf16", saved_t)
    F.check_forward(st, xv, y, saved, saved_t)
    if saved_t:
        dy = [F._bf16(rng, (r, H)) for r in st["rows"]]
        gate_up = [t.cpu() for t in saved]
        xv, sv, dx, dw = F.run_backward(st, "bf16", "bf16", "bf16", gate_up, dy)
        F.check_backward(st, xv, sv, dy, dx, dw, "bf16")
