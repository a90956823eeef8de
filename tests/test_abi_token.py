"""CPU tests of the ABI of embedding, dropout and log probabilities: every refusal comes
before the first HIP call, so stand-in addresses are enough; sizes of scratch."""

import pytest

import collective_communication_reduction_amd as gc

GIB = 1 << 30
OK, BAD, UNSUP = gc.GC_OK, gc.GC_ERR_INVALID_ARG, gc.GC_ERR_UNSUPPORTED


def _status(fn, *a, **k):
    try:
        fn(*a, **k)
    except gc.GcError as e:
        return e.status
    return OK


class Slots:
    """Stand-in device addresses, far apart from one another and from those of every other Slots."""
    at = 1 << 41

    def one(self, off=0):
        Slots.at += 64 * GIB
        return Slots.at + off

    def list(self, n, off=0):
        return [self.one(off) for _ in range(n)]


def _embed(n=2, **over):
    m = Slots()
    k = dict(weight=m.list(n), tokens=m.list(n), ntokens=[3] * n, vocab=100, hidden=64, out=m.list(n), scale=1.0,
             dtype="bf16", stream=0)
    k.update(over)
    return _status(gc.gc_embedding, **k)


def test_embedding_validation():
    m = Slots()
    a, b = m.list(2), m.list(2)
    assert _embed(ntokens=[0, 0], weight=[None, None]) == OK
    assert _embed(ntokens=[3, -1]) == BAD and _embed(vocab=0) == BAD and _embed(hidden=0) == BAD
    assert _embed(vocab=(1 << 22) + 1) == UNSUP and _embed(hidden=(1 << 31) + 1) == UNSUP
    assert _embed(ntokens=[1 << 30, 1 << 30]) == UNSUP
    for s in (float("nan"), float("inf")):
        assert _embed(scale=s) == BAD
    assert _embed(dtype="int32") == UNSUP and _embed(dtype="mx8") == UNSUP and _embed(dtype=9) == BAD
    assert _embed(weight=[a[0], None]) == BAD and _embed(tokens=[a[0], a[1] + 2]) == BAD
    assert _embed(weight=a, out=a) == BAD and _embed(out=[b[0], b[0] + 128]) == BAD
    assert _embed(out=[b[0] + 1, b[1]]) == BAD
    assert _embed(weight=[(1 << 64) - 64] * 2) == BAD                     # wraps
    assert _embed(n=65) == UNSUP and _embed(n=0) == BAD


def _embed_bwd(n=2, **over):
    m = Slots()
    k = dict(dout=m.list(n), tokens=m.list(n), ntokens=[3] * n, vocab=100, hidden=64, dweight=m.list(n), scratch=m.one(),
             scratch_bytes=1 << 20, dtype="bf16", dw_dtype="fp32", stream=0)
    k.update(over)
    return _status(gc.gc_embedding_backward, **k)


def test_embedding_backward_validation():
    m = Slots()
    a, b = m.list(2), m.list(2)
    need = gc.gc_embedding_backward_scratch_bytes([3, 3], 100, 64)
    assert need > 0
    assert _embed_bwd(scratch_bytes=need - 1) == BAD
    assert _embed_bwd(scratch=m.one(64)) == BAD and _embed_bwd(scratch=None) == BAD
    assert _embed_bwd(ntokens=[-1, 1]) == BAD and _embed_bwd(hidden=0) == BAD and _embed_bwd(vocab=0) == BAD
    assert _embed_bwd(vocab=(1 << 22) + 1) == UNSUP
    assert _embed_bwd(dtype="int32") == UNSUP and _embed_bwd(dw_dtype="mx8") == UNSUP and _embed_bwd(dw_dtype=7) == BAD
    assert _embed_bwd(scale=float("inf")) == BAD
    assert _embed_bwd(dout=a, dweight=a) == BAD and _embed_bwd(dweight=[b[0], b[0]]) == BAD
    assert _embed_bwd(dweight=[b[0], None]) == BAD
    assert _embed_bwd(dweight=[b[0] + 2, b[1]]) == BAD                     # fp32: 4 bytes
    assert _embed_bwd(dweight=b, scratch=(b[0] + 255) // 256 * 256) == BAD
    assert gc.gc_embedding_backward_scratch_bytes([-1], 100, 64) == 0
    assert gc.gc_embedding_backward_scratch_bytes([1], 0, 64) == 0


def _drop(n=2, **over):
    m = Slots()
    k = dict(x=m.list(n), counts=[1000] * n, p=0.1, seed=1, y=m.list(n), residual=m.list(n), step=m.one(), dtype="bf16",
             stream=0)
    k.update(over)
    return _status(gc.gc_dropout, **k)


def test_dropout_validation():
    m = Slots()
    a, b = m.list(2), m.list(2)
    assert _drop(counts=[0, 0], x=[None, None]) == OK
    for p in (-0.1, 1.01, float("nan")):
        assert _drop(p=p) == BAD
    assert _drop(counts=[-1, 1]) == BAD and _drop(counts=[1, (1 << 40) + 1]) == BAD
    assert _drop(dtype="int32") == UNSUP and _drop(dtype="mx8") == UNSUP and _drop(dtype=8) == BAD
    assert _drop(x=[a[0], None]) == BAD and _drop(residual=[a[0] + 1, a[1]]) == BAD
    assert _drop(step=m.one(4)) == BAD
    assert _drop(x=a, y=[a[1], a[0]]) == BAD                              # another rank's
    assert _drop(x=a, y=[a[0] + 64, b[1]]) == BAD                         # shifted
    assert _drop(residual=a, x=a, y=b, step=b[0] + 8) == BAD              # the step inside an output
    assert _drop(y=[b[0], b[0]]) == BAD
    assert _drop(n=65) == UNSUP


def _lp(n=2, **over):
    m = Slots()
    k = dict(logits=m.list(n), ntokens=[3] * n, vocab=100, scratch=m.one(), targets=m.list(n), logprob=m.list(n),
             entropy=m.list(n), lse=m.list(n), top=4, top_ids=m.list(n), top_logprob=m.list(n), dlogprob=m.list(n),
             dentropy=m.list(n), dlogits=m.list(n), stride=104, scale=1.0, scratch_bytes=1 << 20, dtype="bf16", stream=0)
    k.update(over)
    return _status(gc.gc_token_logprob, **k)


def test_token_logprob_validation():
    m = Slots()
    a, b = m.list(2), m.list(2)
    assert _lp(ntokens=[0, 0], logits=[None, None]) == OK
    assert _lp(ntokens=[0, -1]) == BAD and _lp(vocab=0) == BAD and _lp(stride=99) == BAD
    assert _lp(top=-1) == BAD and _lp(top=65) == UNSUP and _lp(vocab=3, stride=3) == BAD      # top past the vocabulary
    assert _lp(vocab=(1 << 31) + 1, stride=(1 << 31) + 1) == UNSUP
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert _lp(scale=s) == BAD
    assert _lp(dtype="int32") == UNSUP and _lp(dtype=9) == BAD
    assert _lp(targets=None) == BAD and _lp(logprob=None) == BAD
    assert _lp(top_ids=None) == BAD and _lp(top_logprob=[a[0], None]) == BAD
    assert _lp(dlogprob=None) == BAD and _lp(dlogits=None) == BAD
    assert _lp(dlogits=None, dlogprob=None) == BAD                        # dentropy alone
    assert _lp(targets=None, logprob=None) == BAD                         # a gradient needs targets
    assert _lp(logits=a, dlogits=[a[1], a[0]]) == BAD and _lp(logits=a, dlogits=[a[0] + 208, b[0]]) == BAD
    assert _lp(entropy=a, lse=a) == BAD and _lp(logits=a, lse=a) == BAD
    assert _lp(lse=[a[0] + 2, a[1]]) == BAD and _lp(logits=[b[0] + 1, b[1]]) == BAD
    assert _lp(scratch=m.one(128)) == BAD and _lp(scratch=None) == BAD
    need = gc.gc_token_logprob_scratch_bytes([3, 3], 100, 4)
    assert need > 0 and _lp(scratch_bytes=need - 1) == BAD
    assert gc.gc_token_logprob_scratch_bytes([3], 100, 65) == 0
    assert _lp(n=65) == UNSUP


def _lp_bwd(n=2, **over):
    m = Slots()
    k = dict(logits=m.list(n), ntokens=[3] * n, vocab=100, lse=m.list(n), targets=m.list(n), dlogprob=m.list(n),
             dlogits=m.list(n), entropy=m.list(n), dentropy=m.list(n), stride=104, dtype="fp32", stream=0)
    k.update(over)
    return _status(gc.gc_token_logprob_backward, **k)


def test_token_logprob_backward_validation():
    m = Slots()
    a, b = m.list(2), m.list(2)
    assert _lp_bwd(ntokens=[0, 0]) == OK
    for k in ("lse", "targets", "dlogprob", "dlogits", "entropy", "logits"):
        assert _lp_bwd(**{k: None}) == BAD, k
        assert _lp_bwd(**{k: [a[0], None]}) == BAD, k
    assert _lp_bwd(stride=50) == BAD and _lp_bwd(scale=0.0) == BAD and _lp_bwd(dtype="mx8") == UNSUP
    assert _lp_bwd(logits=a, dlogits=[a[0] + 416, b[1]]) == BAD
    assert _lp_bwd(lse=b, dlogits=b) == BAD


@pytest.mark.parametrize("vocab,ntokens", [(1, [0]), (2048, [5]), (2049, [5, 0]), (1 << 22, [1 << 20, 3])])
def test_embedding_scratch_sizes(vocab, ntokens):
    need = gc.gc_embedding_backward_scratch_bytes(ntokens, vocab, 64)
    assert need % 256 == 0 and need >= 8 * sum(ntokens)
