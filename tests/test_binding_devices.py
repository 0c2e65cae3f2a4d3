"""The binding's device and stream handling of the cache operators, on the CPU (stand-ins for CUDA tensors)."""
import pytest
import torch


@pytest.fixture(scope="module")
def T():
    from two_level_sparse_quest_b200 import build

    build.build()
    from two_level_sparse_quest_b200 import tls

    return tls


def fake_cuda(index):
    """A tensor that says it lies on cuda:index."""
    class Fake(torch.Tensor):
        def get_device(self):
            return index

        def data_ptr(self):
            return 0x1000 + 256 * index

    return torch.zeros(4, 4).as_subclass(Fake)


def test_tensors_of_another_device_are_refused(T, monkeypatch):
    monkeypatch.setattr(T, "_current_device", lambda: 1)
    here, there = fake_cuda(1), fake_cuda(0)
    assert T._dptrs(here, None, 0x20, here) == [0x1100, None, 0x20, 0x1100]
    for args in ((there,), (here, there), (there, here)):
        with pytest.raises(ValueError, match="current device is cuda:1"):
            T._dptrs(*args)
    with pytest.raises(ValueError, match="CUDA tensor"):
        T._dptrs(here, torch.zeros(2))
    with pytest.raises(ValueError, match="contiguous"):
        T._dptrs(here.t())
    with pytest.raises(TypeError):
        T._dptrs(1.5)


def test_stream_argument(T):
    class Stream:
        cuda_stream = 77

    assert T._stream(5) == 5 and T._stream(Stream()) == 77
