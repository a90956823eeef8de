"""CPU tests of the layer operators' ABI: every refusal comes before the first HIP
call, so stand-in addresses are enough; sizes of 8-bit rows and scratch."""

import ctypes

import pytest

import collective_communication_reduction_amd as gc

BASE = 0x7F0000000000
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
    at = 1 << 40

    def one(self, off=0):
        Slots.at += 64 * GIB
        return Slots.at + off

    def list(self, n, off=0):
        return [self.one(off) for _ in range(n)]


# ------------------------------------------------------------------ 8-bit rows

def test_mx8_validation():
    for fn in (gc.gc_mx8_pack, gc.gc_mx8_unpack):
        m = Slots()
        a, b = m.list(2), m.list(2)
        assert _status(fn, a, [0, 0], 64, b, dtype="bf16", stream=0) == OK          # nothing to do
        assert _status(fn, a, [1, -1], 64, b, dtype="bf16", stream=0) == BAD
        assert _status(fn, a, [1, 1], 0, b, dtype="bf16", stream=0) == BAD
        assert _status(fn, a, [1, 1], 64, b, dtype=7, stream=0) == BAD
        assert _status(fn, a, [1, 1], 64, b, dtype="int32", stream=0) == UNSUP
        assert _status(fn, a, [1, 1], 64, b, dtype="mx8", stream=0) == UNSUP
        assert _status(fn, a, [1, 1], (1 << 31) + 1, b, dtype="bf16", stream=0) == UNSUP
        assert _status(fn, a, [1 << 31, 0], 8, b, dtype="bf16", stream=0) == UNSUP
        assert _status(fn, a, [1 << 30, 1 << 30], 8, b, dtype="bf16", stream=0) == UNSUP   # 2^31 rows in all
        assert _status(fn, [None, a[1]], [1, 1], 64, b, dtype="bf16", stream=0) == BAD
        assert _status(fn, a, [1, 1], 64, a, dtype="bf16", stream=0) == BAD          # in place
        assert _status(fn, a, [1, 1], 64, [b[0], b[0] + 16], dtype="bf16", stream=0) == BAD
        assert _status(fn, [], [], 64, [], dtype="bf16", stream=0) == BAD
        assert _status(fn, a * 33, [1] * 66, 64, b * 33, dtype="bf16", stream=0) == UNSUP
    m = Slots()
    a, b = m.list(1), m.list(1)
    assert _status(gc.gc_mx8_pack, a, [1], 64, [b[0] + 8], dtype="bf16", stream=0) == BAD   # 8-bit rows: 16 bytes
    assert _status(gc.gc_mx8_pack, [a[0] + 1], [1], 64, b, dtype="bf16", stream=0) == BAD
    assert _status(gc.gc_mx8_unpack, [a[0] + 4], [1], 64, b, dtype="bf16", stream=0) == BAD
    assert _status(gc.gc_mx8_pack, [(1 << 64) - 64], [4], 64, b, dtype="bf16", stream=0) == BAD   # wraps


def test_mx8_row_bytes():
    assert [gc.gc_mx8_row_bytes(n) for n in (0, 1, 15, 31, 32, 4096)] == [0, 16, 16, 32, 48, 4224]
    assert gc.gc_mx8_row_bytes((1 << 31) + 1) == 0


# ------------------------------------------------------------------ norm

def _norm(m=None, n=2, **over):
    m = m or Slots()
    k = dict(x=m.list(n), weight=m.list(n), ntokens=[3] * n, hidden=64, y=m.list(n), residual=m.list(n),
             sum_out=m.list(n), rstd=m.list(n), eps=1e-6, dtype="bf16", y_dtype="bf16", stream=0)
    k.update(over)
    return _status(gc.gc_rms_norm, **k)


def test_norm_validation():
    m = Slots()
    x, res, y = m.list(2), m.list(2), m.list(2)
    assert _norm(ntokens=[0, 0]) == OK
    assert _norm(ntokens=[3, -1]) == BAD
    assert _norm(hidden=0) == BAD
    assert _norm(hidden=(1 << 31) + 1) == UNSUP
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _norm(eps=eps) == BAD
    assert _norm(dtype=9) == BAD and _norm(y_dtype=9) == BAD
    assert _norm(dtype="int32", y_dtype="int32") == UNSUP
    assert _norm(dtype="bf16", y_dtype="fp32") == UNSUP
    assert _norm(dtype="mx8", y_dtype="mx8") == UNSUP
    assert _norm(ntokens=[1 << 30, 1 << 30]) == UNSUP
    assert _norm(x=[None, 16]) == BAD
    assert _norm(x=x, y=x) == BAD                                    # y over x
    assert _norm(x=x, sum_out=[x[1], x[0]]) == BAD                   # another rank's x
    assert _norm(x=x, sum_out=[x[0] + 128, x[1]]) == BAD             # shifted
    assert _norm(residual=res, sum_out=res, y=res) == BAD
    assert _norm(y=[y[0], y[0]]) == BAD
    assert _norm(y=[y[0] + 8, y[1]], y_dtype="mx8") == BAD
    assert _norm(x=[x[0] + 1, x[1]]) == BAD


def _norm_bwd(n=2, **over):
    m = Slots()
    k = dict(dy=m.list(n), sum=m.list(n), weight=m.list(n), rstd=m.list(n), ntokens=[3] * n, hidden=64, dx=m.list(n),
             dweight=m.list(n), scratch=m.one(), scratch_bytes=1 << 20, dsum=m.list(n), dtype="bf16", stream=0)
    k.update(over)
    return _status(gc.gc_rms_norm_backward, **k)


def test_norm_backward_validation():
    m = Slots()
    a, b = m.list(2), m.list(2)
    assert _norm_bwd(scratch_bytes=255) == BAD
    assert _norm_bwd(scratch=m.one(64)) == BAD
    assert _norm_bwd(scratch=None) == BAD
    assert _norm_bwd(ntokens=[-1, 1]) == BAD and _norm_bwd(hidden=0) == BAD
    assert _norm_bwd(dtype="int32") == UNSUP and _norm_bwd(dtype=5) == BAD
    assert _norm_bwd(dx=a, sum=a) == BAD
    assert _norm_bwd(dx=a, dy=[a[1], a[0]]) == BAD
    assert _norm_bwd(dweight=[b[0], b[0] + 4]) == BAD
    assert _norm_bwd(dweight=[None, b[0]]) == BAD
    assert _norm_bwd(dweight=[a[0], b[0]], dy=[a[0], a[1]]) == BAD
    need = gc.gc_rms_norm_backward_scratch_bytes([1000, 10], 4096)
    assert need % 256 == 0 and need > 0
    assert gc.gc_rms_norm_backward_scratch_bytes([1000, -1], 4096) == 0
    assert gc.gc_rms_norm_backward_scratch_bytes([10], 0) == 0


# ------------------------------------------------------------------ combine gradient

def _combine(n=2, **over):
    m = Slots()
    k = dict(dout=m.list(n), expert_out=m.list(n), expert_rows=[6] * n, dest=m.list(n), weights=m.list(n),
             ntokens=[3] * n, topk=2, hidden=64, dtype="bf16", dexpert=m.list(n), dweights=m.list(n), stream=0)
    k.update(over)
    return _status(gc.gc_moe_combine_backward, **k)


def test_combine_backward_validation():
    m = Slots()
    a = m.list(2)
    assert _combine(ntokens=[0, 0], expert_rows=[0, 0]) == OK
    assert _combine(topk=0) == BAD and _combine(topk=9) == UNSUP
    assert _combine(hidden=0) == BAD and _combine(dtype="int32") == UNSUP and _combine(dtype="mx8") == UNSUP
    assert _combine(ntokens=[3, -1]) == BAD and _combine(expert_rows=[-6, 6]) == BAD
    assert _combine(ntokens=[1 << 29, 1 << 29]) == UNSUP             # 2^31 routes
    assert _combine(expert_out=a, dexpert=a) == BAD
    assert _combine(dexpert=[a[0], a[0] + 64]) == BAD
    assert _combine(dest=[a[0] + 4, a[1]]) == BAD
    assert _combine(weights=[a[0] + 2, a[1]]) == BAD
    assert _combine(dweights=[None, a[1]]) == BAD


# ------------------------------------------------------------------ experts

def _ffn(backward=False, n=2, **over):
    m = Slots()
    k = dict(x=m.list(n), rows=[5] * n, splits=m.one(), experts_per_rank=2, hidden=64, inter=32, w_gate=m.list(n),
             w_up=m.list(n), w_down=m.list(n), scratch=m.one(), scratch_bytes=1 << 30, saved=m.list(n), x_dtype="bf16",
             saved_dtype="bf16", stream=0)
    if backward:
        k.update(dy=m.list(n), dx=m.list(n), dw_gate=m.list(n), dw_up=m.list(n), dw_down=m.list(n), dw_dtype="bf16")
    else:
        k.update(y=m.list(n))
    k.update(over)
    return _status(gc.gc_moe_ffn_backward if backward else gc.gc_moe_ffn, **k)


@pytest.mark.parametrize("backward", [False, True])
def test_ffn_validation(backward):
    f = lambda **k: _ffn(backward, **k)  # noqa: E731
    m = Slots()
    a = m.list(2)
    out = "dx" if backward else "y"
    if not backward:
        assert f(rows=[0, 0]) == OK
        assert f(rows=[0, 0], saved=None) == OK
    else:
        assert f(saved=None) == BAD
    assert f(rows=[5, -1]) == BAD and f(rows=[1 << 30, 1 << 30]) == UNSUP
    assert f(experts_per_rank=0) == BAD and f(experts_per_rank=4097) == UNSUP
    assert f(hidden=0) == BAD and f(inter=0) == BAD
    assert f(hidden=68) == UNSUP and f(inter=36) == UNSUP            # multiples of 8
    assert f(hidden=(1 << 20) + 8) == UNSUP
    assert f(inter=40, saved_dtype="mx8") == UNSUP                   # 8-bit checkpoints: multiples of 32
    assert f(x_dtype="fp32") == UNSUP and f(x_dtype="int32") == UNSUP and f(x_dtype=11) == BAD
    assert f(saved_dtype="fp32") == UNSUP and f(saved_dtype=11) == BAD
    assert f(splits=None) == BAD and f(splits=m.one(4)) == BAD
    assert f(scratch=None) == BAD and f(scratch=m.one(128)) == BAD
    need = gc.gc_moe_ffn_scratch_bytes([5, 5], 2, 64, 32, backward=backward)
    assert f(scratch_bytes=need - 1) == BAD
    for k in ("x", "w_gate", "w_up", "w_down", "saved", out):
        assert f(**{k: [a[0] + 8, a[1]]}) == BAD, k                  # 16-byte alignment
        assert f(**{k: [None, a[1]]}) == BAD, k
    assert f(x=a, **{out: a}) == BAD
    assert f(w_gate=a, **{out: a}) == BAD
    assert f(**{out: [a[0], a[0] + 16]}) == BAD
    if backward:
        assert f(dw_dtype="int32") == UNSUP and f(dw_dtype="mx8") == UNSUP and f(dw_dtype=12) == BAD
        assert f(w_gate=a, dw_gate=a) == BAD
        assert f(dw_gate=a, dw_up=a) == BAD
        assert f(dy=a, dx=a) == BAD
        assert f(saved=a, dx=a) == BAD
    else:
        assert f(saved=a, y=a) == BAD


def test_ffn_scratch_bytes():
    s = gc.gc_moe_ffn_scratch_bytes
    assert s([5], 0, 64, 32) == 0 and s([-1], 1, 64, 32) == 0 and s([5], 1, 60, 32) == 0 and s([5], 1, 64, 32, x_dtype="fp32") == 0
    f, b = s([1000, 24], 4, 512, 256), s([1000, 24], 4, 512, 256, backward=True)
    assert f % 256 == 0 and f >= 1024 * 256 * 2                      # h
    assert b - f == 1024 * 256 * 4                                   # dgate and dup
    assert s([1000, 24], 4, 512, 256, x_dtype="mx8") - f == 1024 * 512 * 2   # x decoded


def test_short_tensors_are_refused_by_the_binding():
    """The binding checks every tensor's bytes (here a stand-in device tensor)."""
    class T:
        is_cuda = True
        device = type("D", (), {"type": "cuda", "index": 0})()

        def __init__(self, n, es=2):
            self.n, self.es = n, es

        def is_contiguous(self):
            return True

        def numel(self):
            return self.n

        def element_size(self):
            return self.es

        def data_ptr(self):
            return BASE
    ok = T(3 * 64)
    with pytest.raises(ValueError, match="residual"):
        gc.gc_rms_norm([ok], [T(64)], [3], 64, [T(3 * 64)], residual=[T(3 * 64 - 1)], dtype="bf16", y_dtype="bf16", stream=0)
    with pytest.raises(ValueError, match="packed"):
        gc.gc_mx8_pack([ok], [3], 64, [T(3 * 80 - 1, 1)], dtype="bf16", stream=0)
    with pytest.raises(ValueError, match="w_up"):
        gc.gc_moe_ffn([ok], [3], T(1, 8), 1, 64, 32, [T(2048)], [T(2047)], [T(2048)], [ok], T(1 << 20, 1),
                      x_dtype="bf16", stream=0)
    with pytest.raises(ValueError, match="splits"):
        gc.gc_moe_ffn([ok], [3], T(1, 4), 1, 64, 32, [T(2048)], [T(2048)], [T(2048)], [ok], T(1 << 20, 1),
                      x_dtype="bf16", stream=0)


def test_pointer_arrays_pass_through():
    arr = (ctypes.c_void_p * 1)(BASE)
    assert _status(gc.gc_mx8_pack, arr, [0], 64, arr, dtype="bf16", stream=0) == OK
