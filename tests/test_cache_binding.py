"""What the binding of the cache takes from torch, with a library that records
its calls in place of the real one (nothing is launched)."""
import importlib.util

import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
import ancestral_draft_sampling_gb300.cache as binding
from ancestral_draft_sampling_gb300 import _lib
from tests.test_cache_abi import host_cache


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args, torch.cuda.current_device()))
            return 0
        return call


class Stream:
    def __init__(self, device, number):
        self.device_index, self.cuda_stream = device, number


@pytest.fixture
def fake(monkeypatch):
    """Two devices, device 0 current, device i's current stream is 100 + i."""
    now = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.old, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.old

    def index_of(device):
        if device is None:
            return now[0]
        return device if isinstance(device, int) else torch.device(device).index
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(index_of(device), 100 + index_of(device)))
    monkeypatch.setattr(torch.cuda, "device", lambda device: Device(index_of(device)))
    lib = Recorder()
    monkeypatch.setattr(_lib, "load", lambda: lib)
    return lib


@pytest.mark.parametrize("missing", [(), ("_cuda_getDevice",), ("_cuda_getCurrentRawStream",),
                                     ("_cuda_getDevice", "_cuda_getCurrentRawStream")])
@pytest.mark.parametrize("index", [0, 1])
def test_calls_without_torchs_private_functions(fake, monkeypatch, missing, index):
    """Where a torch has no such function the public one stands in."""
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
        if name not in missing:
            public = (torch.cuda.current_device if name == "_cuda_getDevice"
                      else lambda i: torch.cuda.current_stream(i).cuda_stream)
            monkeypatch.setattr(torch._C, name, public, raising=False)
    spec = importlib.util.spec_from_file_location("ancestral_draft_sampling_gb300.cache_again", binding.__file__)
    cache = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(cache)
    c = host_cache()
    c.index = index
    cache._call(c, "dspark_cache_init", None)
    cache._call(c, "dspark_cache_init", Stream(index, 7))
    assert [(name, args[-1], device) for name, args, device in fake.calls] == [
        ("dspark_cache_init", 100 + index, index), ("dspark_cache_init", 7, index)]


@pytest.mark.parametrize("index", [0, 1])
def test_the_error_word_is_read_on_its_own_device(fake, index):
    """On the stream that the calls on that device run on, whichever device is
    the current one: another device's stream is not ordered behind them."""
    class Buffer:
        device = torch.device("cuda", index)

        def get_device(self):
            return index

        def data_ptr(self):
            return 4096

    class Held:
        buffer = Buffer()
    assert dspark.read_device_error(Held()) == 0
    assert dspark.read_device_error(Held(), stream=Stream(index, 7)) == 0
    assert [(name, args[0], args[2], device) for name, args, device in fake.calls] == [
        ("dspark_read_device_error", 4096, 100 + index, index), ("dspark_read_device_error", 4096, 7, index)]
