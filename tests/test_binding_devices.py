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


def test_binding_does_without_the_private_names_of_a_cuda_build():
    """A build of torch without torch._C._cuda_getDevice and _cuda_getCurrentRawStream (CPU builds have neither): the
    binding is imported, and its device and stream come from torch.cuda's public calls."""
    import os
    import subprocess
    import sys

    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from two_level_sparse_quest_b200 import tls as T
class Stream:
    cuda_stream = 77
torch.cuda.is_initialized = lambda: True
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda device=None: Stream()
assert T._current_device() == 3 and T._raw_stream(3) == 77 and T._stream(None) == 77 and T._stream(5) == 5
print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
