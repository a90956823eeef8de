"""CPU tests of the binding's pointer lists: addresses of any integer type, tensors behind the ranks a call uses."""

import enum

import pytest

import collective_communication_reduction_amd as gc


class Region(enum.IntEnum):
    A = 1 << 40
    B = 1 << 41


class Address(int):
    pass


@pytest.mark.parametrize("a,b", [(Region.A, Region.B), (Address(1 << 40), Address(1 << 41)), (1 << 40, Region.B)])
def test_addresses_of_integer_subclasses(a, b):
    gc.gc_all_gather([a], [b], count=0, dtype="fp32", stream=0)                       # nothing to do: no launch
    gc.gc_mx8_pack([a], [0], 64, [b], dtype="bf16", stream=0)
    with pytest.raises(gc.GcError):
        gc.gc_mx8_pack([a], [1], 64, [a], dtype="bf16", stream=0)                     # the address arrives: in place
    arr = gc.gc_pointers([a, b, None])
    assert [arr[0], arr[1], arr[2]] == [int(a), int(b), None]


def test_a_list_longer_than_the_ranks():
    gc.gc_mx8_pack([1 << 40, None, Region.A], [0], 64, [1 << 41, 1 << 42], dtype="bf16", stream=0)


def test_a_host_tensor_is_refused_as_before():
    import torch
    with pytest.raises(ValueError, match="device"):
        gc.gc_mx8_pack([torch.zeros(64)], [1], 64, [1 << 40], dtype="fp32", stream=0)
    with pytest.raises(ValueError, match=r"x\[1\]"):
        gc.gc_mx8_pack([1 << 40, torch.zeros(64)], [1], 64, [1 << 41], dtype="fp32", stream=0)
