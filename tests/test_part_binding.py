"""On which device and stream the calls that read part of the cache are made,
with a library that records its calls (nothing is launched)."""
import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.test_cache_abi import host_cache
from tests.test_cache_binding import Stream, fake  # noqa: F401


class Workspace:
    nbytes = 1 << 20

    class buffer:
        device = 1

        @classmethod
        def get_device(cls):
            return cls.device

        @staticmethod
        def data_ptr():
            return 4096


def all_calls(c, stream=None, workspace=Workspace):
    i32 = torch.int32
    one, q = torch.zeros(1, dtype=i32), torch.zeros(1, 3, 4, 8)
    b, out, lse = torch.zeros(1, 6, 2, 2, 8), torch.zeros(1, 3, 4, 8), torch.zeros(1, 3, 4)
    pages, start = torch.zeros(1, 3, 2, 5, dtype=i32), torch.zeros(2, dtype=i32)
    kw = dict(stream=stream)
    more = dict(kw, out=out, lse=lse, workspace=workspace)
    return (lambda: dspark.cache_bounds(c, one, one, bounds=b, **kw),
            lambda: dspark.select_pages(c, 0, b, q, one, 5, pages=pages, workspace=workspace, **kw),
            lambda: dspark.sparse_attention(c, 0, q, one, pages, **more),
            lambda: dspark.prefix_attention(c, 0, q, one, start, one, **more))


@pytest.fixture
def on_device(fake, monkeypatch):  # noqa: F811
    """A cache whose tensors, and all others, say that they are on device 1."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", torch.cuda.current_device, raising=False)
    import ancestral_draft_sampling_gb300.cache as binding
    monkeypatch.setattr(binding, "_device", torch.cuda.current_device)
    monkeypatch.setattr(binding, "_stream_of", lambda i: torch.cuda.current_stream(i).cuda_stream)
    monkeypatch.setattr(binding, "_functions", {})
    c = host_cache()
    c.index = 1
    return fake, c


def test_calls_go_to_the_caches_device(on_device):
    """Its current stream, whichever device is the current one; or the stream given."""
    lib, c = on_device
    for stream, number in ((None, 101), (Stream(1, 7), 7)):
        lib.calls.clear()
        for call in all_calls(c, stream):
            call()
        assert [(name, args[-1], device) for name, args, device in lib.calls] == [
            (f"dspark_{name}", number, 1) for name in ("cache_bounds", "select_pages", "sparse_attention",
                                                       "prefix_attention")]


def test_a_workspace_on_another_device_is_refused(on_device):
    lib, c = on_device

    class Far(Workspace):
        class buffer(Workspace.buffer):
            device = 0
    for call in all_calls(c, workspace=Far)[1:]:
        with pytest.raises(ValueError):
            call()
    assert lib.calls == []


def test_tensors_on_another_device_are_refused(on_device, monkeypatch):
    lib, c = on_device
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    for call in all_calls(c):
        with pytest.raises(ValueError):
            call()
    assert lib.calls == []
