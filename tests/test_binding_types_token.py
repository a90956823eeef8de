"""CPU tests of the binding's checks of the tensors that embedding, dropout and log probabilities take (stand-in
device tensors): another type than the call reads, or too small a tensor, is refused by name before the library sees
its address."""

import pytest
import torch

import collective_communication_reduction_amd as gc
from tests.test_binding_types import BF, F32, FLOATS, I32, I64, T, U8, refused, tensors

N, V, H = 3, 10, 64
NAN = float("nan")             # a scale that the library refuses: nothing is launched


def test_embedding():
    spec = {"weight": (V * H, BF), "tokens": (N, I32), "out": (N * H, BF)}
    refused(gc.gc_embedding, spec, {"tokens": (I64, F32), "out": FLOATS}, ntokens=[N], vocab=V, hidden=H, scale=NAN, stream=0)
    spec = {"dout": (N * H, BF), "tokens": (N, I32), "dweight": (V * H, F32)}
    refused(gc.gc_embedding_backward, spec, {"tokens": (I64,), "dout": (torch.float16, I64)}, ntokens=[N], vocab=V, hidden=H, scale=NAN,
            scratch=T(1 << 20, U8), dtype="bf16", stream=0)


def test_dropout():
    spec = {"x": (N, F32), "y": (N, F32), "residual": (N, F32)}
    refused(gc.gc_dropout, spec, {"y": (torch.float64, I64), "residual": (torch.float64, I64)}, counts=[N], p=2.0, seed=1, stream=0)
    for step in (T(1, F32), T(1, torch.float64)):
        with pytest.raises(ValueError, match="^step: "):
            gc.gc_dropout(**tensors(spec), counts=[N], p=2.0, seed=1, step=step, stream=0)


def test_token_logprob():
    spec = {"logits": (N * V, BF), "targets": (N, I32), "logprob": (N, F32), "entropy": (N, F32), "lse": (N, F32),
            "top_ids": (2 * N, I32), "top_logprob": (2 * N, F32), "dlogprob": (N, F32), "dentropy": (N, F32), "dlogits": (N * V, BF)}
    rest = dict(ntokens=[N], vocab=V, scratch=T(1 << 20, U8), top=2, scale=NAN, stream=0)
    wide = (torch.float64, I64)
    refused(gc.gc_token_logprob, spec, {**{k: wide for k in ("logprob", "entropy", "lse", "top_logprob", "dlogprob", "dentropy")},
                                        "targets": (I64,), "top_ids": (I64,), "dlogits": FLOATS}, **rest)
    spec = {k: spec[k] for k in ("logits", "targets", "lse", "entropy", "dlogprob", "dentropy", "dlogits")}
    refused(gc.gc_token_logprob_backward, spec, {"lse": wide, "dlogits": FLOATS}, ntokens=[N], vocab=V, scale=NAN, stream=0)


@pytest.mark.parametrize("short", ["logits", "targets", "top_ids", "dlogits"])
def test_short_tensors(short):
    size = {"logits": N * (V + 2), "targets": N, "top_ids": 3 * N, "dlogits": N * (V + 2)}
    size[short] -= 1
    with pytest.raises(ValueError, match=f"^{short}\\[0\\]: "):
        gc.gc_token_logprob([T(size["logits"], BF)], [N], V, T(1 << 20, U8), targets=[T(size["targets"], I32)], logprob=[T(N, F32)], top=3,
                            top_ids=[T(size["top_ids"], I32)], top_logprob=[T(3 * N, F32)], dlogprob=[T(N, F32)],
                            dlogits=[T(size["dlogits"], BF)], stride=V + 2, scale=NAN, stream=0)
