"""Expert ids of a given routing, of every integer type: nothing here touches a device."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300.layer import _expert_ids

INTEGERS = [torch.uint8, torch.int8, torch.int16, torch.int32, torch.int64, torch.uint16, torch.uint32, torch.uint64]


@pytest.mark.parametrize("dtype", INTEGERS)
@pytest.mark.parametrize("E", [1, 8, 100, 127, 128, 255, 256, 1024])
def test_ids_of_any_integer_type(dtype, E):
    top = min(torch.iinfo(dtype).max, 2 ** 63 - 1)
    low = max(torch.iinfo(dtype).min, -2 ** 63)
    ids = sorted({i for i in (low, -2 ** 32 + 1, -2, -1, 0, 1, 7, 100, 127, 128, 255, 256, 1023, E - 1, E, E + 1, 2 ** 31, 2 ** 32,
                              2 ** 32 + 1, top) if low <= i <= top})
    got = _expert_ids(torch.tensor(ids, dtype=torch.int64).to(dtype), E)
    assert got.dtype is torch.int32
    for i, g in zip(ids, got.tolist()):
        assert g == i if 0 <= i < E else not 0 <= g < E, (i, g)


def test_the_largest_of_64_bits_without_a_sign():
    ids = torch.tensor([2 ** 64 - 1, 2 ** 63, 5], dtype=torch.uint64)
    got = _expert_ids(ids, 8).tolist()
    assert not 0 <= got[0] < 8 and not 0 <= got[1] < 8 and got[2] == 5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float64, torch.complex64])
def test_other_types_are_refused(dtype):
    with pytest.raises(TypeError):
        _expert_ids(torch.zeros(2, 2, dtype=dtype), 8)
