"""A call on a stream of its own takes, clears and gives back its memory on that stream (no GPU
needed: tensors and streams are stand-ins that record where they were made)."""
import contextlib
import types

import pytest
import torch

from block_sparse_online_b200 import solattn

DEV = torch.device("cuda", 0)
CURRENT = types.SimpleNamespace(device=DEV, cuda_stream=11)
SIDE = types.SimpleNamespace(device=DEV, cuda_stream=22)


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on the GPU."""
    is_cuda = True
    device = DEV

    def get_device(self):
        return 0

    def record_stream(self, s):
        self.used_on = s


def on_gpu(x):
    return x.as_subclass(OnGpu)


@pytest.fixture
def log(monkeypatch):
    """Streams that were current when memory was taken, and that the library launched on."""
    active, seen = [CURRENT], {"alloc": [], "clear": [], "launch": []}

    @contextlib.contextmanager
    def stream(s):
        active.append(s)
        try:
            yield
        finally:
            active.pop()

    def made(fn):
        def call(*a, device=None, **kw):
            seen["alloc"].append(active[-1].cuda_stream)
            return on_gpu(fn(*a, **kw))
        return call

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("workspace_size"):
                    return 1024
                h = next(a for a in reversed(args) if getattr(a, "value", a) in (11, 22))
                seen["launch"].append(getattr(h, "value", h))
                return 0
            return call

    real_empty, real_like, real_zero = torch.empty, torch.empty_like, torch.Tensor.zero_
    monkeypatch.setattr(torch, "empty", made(real_empty))
    monkeypatch.setattr(torch, "empty_like", made(lambda x, **kw: real_empty(x.shape, dtype=x.dtype)))
    monkeypatch.setattr(OnGpu, "zero_", lambda x: (seen["clear"].append(active[-1].cuda_stream), real_zero(x))[1], raising=False)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "set_stream", lambda s: active.__setitem__(-1, s))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: active[-1])
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(solattn, "_current_device", lambda: 0)
    monkeypatch.setattr(solattn, "_raw_stream", lambda i: active[-1].cuda_stream)
    monkeypatch.setattr(solattn, "_lib", Library())
    monkeypatch.setattr(solattn, "_fast", None)
    return seen


def rows(*shape, dtype=torch.bfloat16):
    return on_gpu(torch.zeros(*shape, dtype=dtype))


def ints(*x):
    return on_gpu(torch.tensor(x, dtype=torch.int32))


def paged_cache():
    return solattn.PagedCache(rows(3, 2, 16, 64), rows(3, 2, 16, 64))


CALLS = {
    "cross": lambda s: solattn.solattn_cross(rows(1, 2, 5, 64), rows(1, 2, 7, 64), rows(1, 2, 7, 64), stream=s),
    "cross_positional": lambda s: solattn.solattn_cross(rows(1, 2, 5, 64), rows(1, 2, 7, 64), rows(1, 2, 7, 64), None, None, None, s),
    "paged": lambda s: solattn.solattn_paged_forward(rows(4, 2, 64), paged_cache(), ints(0, 1)[None], ints(0, 4), ints(9), 4, stream=s),
    "append": lambda s: solattn.solattn_cache_append(paged_cache(), rows(4, 2, 64), rows(4, 2, 64), ints(0, 1)[None], ints(0, 4),
                                                     ints(9), stream=s),
    "read": lambda s: solattn.solattn_cache_read(paged_cache(), ints(0, 1)[None], ints(0, 4), ints(9), rows(4, 2, 64), rows(4, 2, 64),
                                                 stream=s),
    "forward": lambda s: solattn.solattn_forward(*[rows(1, 1, 64, 64)] * 3, 64, 64, 6.0, stream=s),
    "gaussian": lambda s: solattn.solattn_forward_gaussian(*[rows(1, 1, 64, 64)] * 3, 64, 64, 1.0, stream=s),
    "ex": lambda s: solattn.solattn_forward_ex(*[rows(1, 1, 64, 64)] * 3, 64, 64, stream=s),
    "noalloc": lambda s: solattn.solattn_forward_noalloc(*[rows(1, 1, 64, 64)] * 3, 64, 64, 6.0, stream=s),
    "pool": lambda s: solattn.solattn_pool(rows(1, 1, 64, 64), 64, stream=s),
    "route_keep": lambda s: solattn.solattn_route_keep(*[rows(1, 1, 1, 64, dtype=torch.float32)] * 2, 64, 64, 64, 1.0, stream=s),
}
FRESH = {"cross", "cross_positional", "paged", "forward", "gaussian", "ex", "noalloc", "pool", "route_keep"}  # return new tensors


@pytest.mark.parametrize("name", CALLS)
def test_memory_belongs_to_the_stream_of_the_launch(name, log):
    result = CALLS[name](SIDE)
    assert log["launch"] == [22]
    assert log["alloc"] and set(log["alloc"]) == {22}
    assert set(log["clear"]) <= {22}
    if name in FRESH:  # and the result may be dropped on the caller's stream
        first = result[0] if isinstance(result, tuple) else result
        assert first.used_on is CURRENT


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_all_is_on_the_current_one(name, log):
    CALLS[name](None)
    assert log["launch"] == [11] and set(log["alloc"]) == {11} and set(log["clear"]) <= {11}


@pytest.mark.parametrize("current", [0, 1])
def test_the_current_stream_is_put_back(log, monkeypatch, current):
    """After the call and after a refusal, whichever device is current."""
    monkeypatch.setattr(solattn, "_current_device", lambda: current)
    CALLS["cross"](SIDE)
    assert torch.cuda.current_stream() is CURRENT
    with pytest.raises(ValueError):
        solattn.solattn_cross(rows(1, 2, 5, 64), rows(1, 2, 7, 64), rows(1, 2, 8, 64), stream=SIDE)
    assert torch.cuda.current_stream() is CURRENT


def test_a_stream_of_another_device_is_refused(log):
    with pytest.raises(ValueError):
        CALLS["cross"](types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=22))
