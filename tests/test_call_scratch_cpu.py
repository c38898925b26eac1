"""Which stream's pool a call's own scratch comes from, with CUDA and the library's calls stood in for (no GPU)."""
import contextlib
import math

import pytest
import torch

from depth_wise_attention_attnres_gb300 import binding, build

P = 1 << 24  # a stand-in pointer, never followed


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


class _FakeStream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class _FakeTensor:
    def __init__(self, *size):
        self.shape, self.dtype = size, torch.float32

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        strides = tuple(math.prod(self.shape[k + 1:]) for k in range(len(self.shape)))
        return strides if i is None else strides[i]

    is_cuda, device = True, torch.device("cuda", 0)

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return P

    def record_stream(self, stream):
        pass


@pytest.fixture
def allocations(monkeypatch, lib):
    """The streams that were current when the binding allocated, with CUDA and the library's calls stood in for."""
    current, seen = [_FakeStream(77)], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    class Calls:
        def __getattr__(self, name):
            return getattr(lib, name) if name.endswith("_scratch_floats") else lambda *args: 0

    def empty(n, **kw):
        seen.append(current[-1].cuda_stream)
        return _FakeTensor(n)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "Stream", _FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", _FakeStream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: _FakeStream(0))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda device: current[-1].cuda_stream)
    monkeypatch.setattr(binding, "_lib", Calls())
    return seen


def _scratch_calls():
    row, gain, one = _FakeTensor(4, 16), _FakeTensor(16), _FakeTensor(1)
    part, per = _FakeTensor(4, 4, 16), _FakeTensor(4, 16)
    return [
        lambda **kw: binding.attnres_gated_residual_bwd(row, gain, 1e-6, None, 1, 0, 1.0, row, gain, 1e-6, row, row, row,
                                                        row, **kw),
        lambda **kw: binding.attnres_rmsnorm_bwd(row, gain, 1e-6, row, row, row, gain, **kw),
        lambda **kw: binding.attnres_grad_norm([row, gain], one, **kw),
        lambda **kw: binding.attnres_grad_clip([row, gain], 1.0, one, **kw),
        lambda **kw: binding.attnres_block_bwd(part, part, 2, 2, per, per, 1e-6, part, row, part, per, per, **kw),
    ]


@pytest.mark.parametrize("call", range(5))
def test_scratch_comes_from_the_pool_of_the_calls_stream(allocations, call):
    """A block of another stream's pool may still be in use by work queued there, so a call that allocates its own
    scratch takes it while its stream is the current one: a Stream, a handle (0: the default stream), or none given."""
    run = _scratch_calls()[call]
    for stream, handle in ((None, 77), (_FakeStream(5), 5), (9, 9), (0, 0)):
        allocations.clear()
        run(stream=stream)
        assert allocations == [handle]
    allocations.clear()
    run(stream=_FakeStream(5), scratch=_FakeTensor(1 << 20))
    assert allocations == []
