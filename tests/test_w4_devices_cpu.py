"""The parts of a 4-bit weight are on one device: their addresses go to one
kernel.  (Stand-ins with a device index; no GPU.)"""
import pytest
import torch

from routed_grouped_gemm_routing_gb300.block import W4Experts, W4Linear


class OnDevice:
    """What the constructors ask of a CUDA tensor."""

    is_cuda = True

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index

    def get_device(self):
        return self.index

    def contiguous(self):
        return self


def _parts(*lead, K, group, devices):
    return (OnDevice((*lead, K // 2), torch.uint8, devices[0]), OnDevice((*lead, K // group), torch.bfloat16, devices[1]))


def test_codes_and_scales_on_one_device():
    W4Linear(*_parts(8, K=128, group=32, devices=(1, 1)), 32)
    with pytest.raises(ValueError):
        W4Linear(*_parts(8, K=128, group=32, devices=(0, 1)), 32)


def test_experts_on_one_device():
    def make(d):
        return W4Experts(*_parts(2, 256, K=256, group=64, devices=d[:2]), *_parts(2, 256, K=128, group=64, devices=d[2:]), 64)

    make((1, 1, 1, 1))
    for d in ((0, 1, 0, 0), (0, 0, 1, 1), (0, 0, 0, 1)):
        with pytest.raises(ValueError):
            make(d)
