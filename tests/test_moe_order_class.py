"""MoEOrder built from tensors that are not what moe_sort gives, without a GPU: refused, since the kernels read int32
through plain pointers."""

import pytest
import torch

from mxfp8_block_scaled_amd import api


def parts(T=5, topk=2, E=3):
    return (torch.zeros(T, topk, dtype=torch.int32), torch.zeros(T * topk, dtype=torch.int32),
            torch.zeros(E + 1, dtype=torch.int32))


def test_accepted():
    o = api.MoEOrder(*parts())
    assert (o.T, o.topk, o.E) == (5, 2, 3)
    o = api.MoEOrder(*parts(T=0))
    assert (o.T, o.topk, o.E) == (0, 2, 3)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_other_types(which):
    for dtype in (torch.int64, torch.int16, torch.float32, torch.uint8):
        p = list(parts())
        p[which] = p[which].to(dtype)
        with pytest.raises(ValueError, match="int32"):
            api.MoEOrder(*p)


def test_other_shapes():
    rows, slots, offsets = parts()
    for bad in ((rows.view(-1), slots, offsets), (rows, slots[:-1], offsets), (rows, rows, offsets),
                (rows, torch.zeros(12, dtype=torch.int32), offsets), (rows, slots, offsets[:1]), (rows, slots, offsets[:0]),
                (rows, slots, offsets.view(2, 2)), (rows, slots, offsets[0])):
        with pytest.raises(ValueError, match="int32"):
            api.MoEOrder(*bad)


def test_strided():
    wide, slots, offsets = torch.zeros(5, 4, dtype=torch.int32), *parts()[1:]
    for bad in ((wide[:, ::2], slots, offsets), (wide[:, :2], slots, offsets),
                (parts()[0], torch.zeros(20, dtype=torch.int32)[::2], offsets),
                (parts()[0], slots, torch.zeros(8, dtype=torch.int32)[::2])):
        with pytest.raises(ValueError, match="contiguous"):
            api.MoEOrder(*bad)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_other_devices(which):
    p = list(parts())
    p[which] = p[which].to("meta")
    with pytest.raises(ValueError, match="operands on"):
        api.MoEOrder(*p)


def test_not_tensors():
    for p in ((None, *parts()[1:]), (parts()[0].tolist(), *parts()[1:])):
        with pytest.raises(ValueError):
            api.MoEOrder(*p)
