"""CPU tests of the binding's check of tensor types (stand-in device tensors): a tensor of another type than the
call reads is refused by name before the library sees its address."""

import pytest
import torch

import collective_communication_reduction_amd as gc

BF, F32, U8, I32, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64
AT = [(1 << 40) + 2]         # 8-bit rows at such addresses are refused by the library: nothing is launched


class T:
    """A contiguous device tensor of n elements that exists by its address alone."""
    is_cuda = True
    device = type("D", (), {"type": "cuda", "index": 0})()

    def __init__(self, n, dtype):
        self.n, self.dtype, self.at = n, dtype, AT[0]
        AT[0] += 1 << 34

    def is_contiguous(self):
        return True

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return self.at


def tensors(spec):
    return {k: [T(*v)] for k, v in spec.items()}


def refused(call, spec, wrong, **fixed):
    """The call passes the checks with the right types (the library then refuses its eps, sizes or scratch: nothing is
    launched) and is refused by the binding, naming the argument, with each wrong one."""
    with pytest.raises(gc.GcError):
        call(**tensors(spec), **fixed)
    for k, types in wrong.items():
        for t in types:
            with pytest.raises(ValueError, match=rf"^{k}(\[0\])?: a tensor of"):
                call(**tensors({**spec, k: (spec[k][0], t)}), **fixed)


FLOATS = (F32, torch.float64, torch.float16, I64)      # as wide as bf16 or wider
N = 3 * 64


def test_norm():
    spec = {"x": (N, BF), "weight": (N, BF), "y": (N, BF), "residual": (N, BF), "sum_out": (N, BF), "rstd": (N, F32)}
    refused(gc.gc_rms_norm, spec, {**{k: FLOATS for k in ("weight", "residual", "sum_out")}, "rstd": (torch.float64, I64)},
            ntokens=[3], hidden=64, eps=-1.0, y_dtype="bf16", stream=0)
    refused(gc.gc_rms_norm, spec, {"y": FLOATS, "x": FLOATS}, ntokens=[3], hidden=64, eps=-1.0, dtype="bf16", y_dtype="bf16", stream=0)
    refused(gc.gc_rms_norm, {**spec, "y": (2 * N, U8)}, {"y": (BF, F32)}, ntokens=[3], hidden=64, eps=-1.0, y_dtype="mx8", stream=0)
    spec = {"dy": (N, F32), "sum": (N, F32), "weight": (N, F32), "rstd": (N, F32), "dx": (N, F32), "dweight": (N, F32), "dsum": (N, F32)}
    refused(gc.gc_rms_norm_backward, spec, {k: (torch.float64, I64) for k in spec if k != "dy"}, ntokens=[3], hidden=64,
            scratch=1 << 39, scratch_bytes=0, stream=0)


def test_8bit_rows():
    refused(gc.gc_mx8_pack, {"x": (N, BF), "packed": (4 * N, U8)}, {"packed": (BF, F32, I64)}, rows=[3], n=64, stream=0)
    refused(gc.gc_mx8_unpack, {"packed": (4 * N, U8), "out": (N, F32)}, {"packed": (BF, F32), "out": (torch.float64,)}, rows=[3], n=64, dtype="fp32", stream=0)
    with pytest.raises(ValueError, match="packed"):
        gc.gc_mx8_pack([T(N, BF)], [3], 64, [T(N, BF)], stream=0)


def test_combine_gradient():
    spec = {"dout": (N, BF), "expert_out": (2 * N, BF), "dest": (12, I32), "weights": (6, F32), "dexpert": (2 * N, BF), "dweights": (6, F32)}
    for k, types in {"dout": FLOATS, "expert_out": FLOATS, "dexpert": FLOATS, "dest": (F32, I64), "weights": (torch.float64, I64),
                     "dweights": (torch.float64,)}.items():
        for t in types:
            with pytest.raises(ValueError, match=rf"^{k}\[0\]: a tensor of"):
                gc.gc_moe_combine_backward(**tensors({**spec, k: (spec[k][0], t)}), expert_rows=[6], ntokens=[3], topk=2, hidden=64,
                                           dtype="bf16", stream=0)


def test_experts():
    w = 2 * 64 * 32
    spec = {"x": (N, BF), "w_gate": (w, BF), "w_up": (w, BF), "w_down": (w, BF), "y": (N, BF), "saved": (N, BF)}
    fixed = dict(rows=[3], splits=T(2, I64), experts_per_rank=2, hidden=64, inter=32, scratch=1 << 39, scratch_bytes=0, stream=0)
    refused(gc.gc_moe_ffn, spec, {k: FLOATS for k in ("w_gate", "w_up", "w_down", "y")}, **fixed)
    refused(gc.gc_moe_ffn, spec, {"saved": FLOATS, "x": FLOATS}, x_dtype="bf16", saved_dtype="bf16", **fixed)
    with pytest.raises(ValueError, match="^splits: a tensor of"):
        gc.gc_moe_ffn(**tensors(spec), **{**fixed, "splits": T(4, torch.float64)})
    spec = {**spec, "dy": (N, BF), "dx": (N, BF), "dw_gate": (w, F32), "dw_up": (w, F32), "dw_down": (w, F32)}
    del spec["y"]
    refused(gc.gc_moe_ffn_backward, spec, {**{k: FLOATS for k in ("w_gate", "w_up", "w_down", "dy", "dx")},
                                           **{k: (torch.float64,) for k in ("dw_up", "dw_down")}}, **fixed)
    with pytest.raises(ValueError, match=r"^dw_up\[0\]"):     # another type than dw_gate's, though large enough
        gc.gc_moe_ffn_backward(**tensors({**spec, "dw_gate": (w, BF), "dw_up": (w, F32), "dw_down": (w, BF)}), **fixed)


def test_raw_bits_and_empty_tensors_pass():
    """Integer tensors count as raw bits, a buffer of which nothing is read may be of any type."""
    for bits in (torch.int16, torch.uint16):
        with pytest.raises(gc.GcError):
            gc.gc_rms_norm([T(N, bits)], [T(N, bits)], [3], 64, [T(2 * N, U8)], eps=-1.0, dtype="bf16", y_dtype="bf16", stream=0)
    with pytest.raises(gc.GcError):
        gc.gc_mx8_pack([T(N, torch.int32)], [3], 64, [T(2 * N, torch.int8)], dtype="fp32", stream=0)
    gc.gc_rms_norm([T(0, BF)], [T(64, F32)], [0], 64, [T(0, F32)], y_dtype="bf16", stream=0)
