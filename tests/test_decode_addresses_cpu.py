"""The addresses that a decoding layer hands to the library, taken down by a stand-in
for it: the weights' own at each call, none that has been freed.  Nothing here touches
a device."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import layer as L

BF = torch.bfloat16
NAMES = ("router", "W1", "W2", "S1", "S2")


class OnDevice(torch.Tensor):
    """A host tensor that says it is on cuda:0."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


class Library:
    def __init__(self):
        self.calls = []

    def moe_decode_forward(self, shape, x, *args):
        self.calls.append(args[:5])
        return 0


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(B, "lib", lambda: lib)
    monkeypatch.setattr(B, "moe_decode_workspace", lambda s: 256)
    monkeypatch.setattr(B, "_here", lambda stream: (0, 0))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return lib


def _tensor(*shape):
    return torch.zeros(shape, dtype=BF).as_subclass(OnDevice)


def _layer():
    w = dict(router=_tensor(64, 8), W1=_tensor(8, 64, 128), W2=_tensor(8, 64, 64), S1=_tensor(64, 128), S2=_tensor(64, 64))
    return w, L.DecodeLayer(w["router"], w["W1"], w["W2"], 2, w["S1"], w["S2"])


def _call(layer, form):
    if form == "strided":
        return layer(_tensor(6, 64)[::2])
    return layer(_tensor(3, 64), return_routing=form == "routing")


@pytest.mark.parametrize("form", ["plain", "routing"])
@pytest.mark.parametrize("name", NAMES)
def test_a_weight_that_is_made_again_is_read_where_it_lies(library, form, name):
    w, layer = _layer()
    _call(layer, form)
    assert list(library.calls[-1]) == [w[n].data_ptr() for n in NAMES]
    storage, size = w[name].untyped_storage(), w[name].untyped_storage().nbytes()
    before = w[name].data_ptr()
    storage.resize_(0)
    held = [torch.zeros(size // 2, dtype=BF) for _ in range(4)]  # whatever takes the place that it had
    storage.resize_(size)
    _call(layer, form)
    assert list(library.calls[-1]) == [w[n].data_ptr() for n in NAMES]
    del held
    assert before and w[name].data_ptr()


@pytest.mark.parametrize("form", ["plain", "routing", "strided"])
@pytest.mark.parametrize("name", NAMES)
def test_a_weight_that_has_been_freed_is_refused(library, form, name):
    w, layer = _layer()
    w[name].untyped_storage().resize_(0)
    with pytest.raises(RuntimeError, match=name):
        _call(layer, form)
    assert not library.calls


def test_a_layer_without_some_weights(library):
    w, _ = _layer()
    layer = L.DecodeLayer(None, w["W1"], w["W2"], 2)
    assert layer._addresses() == [None, w["W1"].data_ptr(), w["W2"].data_ptr(), None, None]
    layer = L.DecodeLayer(w["router"], w["W1"], w["W2"], 2)
    _call(layer, "plain")
    assert list(library.calls[-1]) == [w["router"].data_ptr(), w["W1"].data_ptr(), w["W2"].data_ptr(), None, None]
