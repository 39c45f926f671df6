"""Which stream's memory a call uses, without a GPU: torch's CUDA streams and
the library's entry points are stand-ins that record what they are given."""

import contextlib
import types

import pytest
import torch

from flow_matching_action_dm0_b200 import ActionExpert
from flow_matching_action_dm0_b200 import _lib as L


class FakeStream:
    def __init__(self, address, device_index=0):
        self.cuda_stream, self.device_index = address, device_index


class FakeTensor:
    """A dense CUDA tensor of GPU 0 as the handle looks at it."""
    is_cuda = True

    def __init__(self, world, shape, dtype, pool):
        self.world, self.shape, self.dtype, self.pool = world, torch.Size(shape), dtype, pool
        self.used_on = []

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def get_device(self):
        return 0

    def new_empty(self, shape, dtype=None):
        return FakeTensor(self.world, shape, dtype or self.dtype, self.world.current[-1].cuda_stream)

    def record_stream(self, s):
        self.used_on.append(s.cuda_stream)


@pytest.fixture
def world(monkeypatch):
    """One GPU whose current stream is 17; calls go to `calls`."""
    w = types.SimpleNamespace(current=[FakeStream(17)], calls={})

    @contextlib.contextmanager
    def stream(s):
        w.current.append(s)
        yield
        w.current.pop()

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.current[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda address, device=None: FakeStream(address))
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None:
                        FakeTensor(w, shape, dtype, w.current[-1].cuda_stream))
    for name in ("rtv_get_prefix_kv_quantized", "rtv_set_prefix_kv_quantized", "rtv_denoise_shared", "rtv_denoise"):
        monkeypatch.setattr(L, name, lambda *a, _n=name: w.calls.setdefault(_n, []).append(a))
    ex = object.__new__(ActionExpert)
    ex.device, ex.h, ex._keep = 0, None, []
    ex.cfg = types.SimpleNamespace(n_layers=2, n_kv_heads=1, head_dim=64, chunk_len=5, action_dim=3, state_dim=4)
    w.ex = ex
    return w


SIDE = 34
GIVEN = [(lambda: FakeStream(SIDE), SIDE), (lambda: SIDE, SIDE), (lambda: None, 17), (lambda: 0, 0)]


@pytest.mark.parametrize("stream,address", GIVEN)
def test_a_parked_prefix_is_allocated_for_the_stream_that_writes_it(world, stream, address):
    codes, scales = world.ex.get_prefix_kv_quantized(6, 1, stream=stream())
    assert world.calls["rtv_get_prefix_kv_quantized"][0][-1] == address
    assert codes.pool == address and scales.pool == address
    assert len(world.current) == 1


@pytest.mark.parametrize("stream,address", GIVEN)
def test_an_installed_prefix_is_kept_until_its_stream_has_read_it(world, stream, address):
    first, second = ([FakeTensor(world, (2, 2, 1, 1, 6, 64), torch.uint8, 5),
                      FakeTensor(world, (2, 2, 1, 1, 6), torch.float32, 5)] for _ in range(2))
    world.ex.set_prefix_kv_quantized(*first, stream=stream())
    world.ex.set_prefix_kv_quantized(*second, stream=FakeStream(51))
    assert [c[-1] for c in world.calls["rtv_set_prefix_kv_quantized"]] == [address, 51]
    assert [t.used_on for t in first + second] == [[address]] * 2 + [[51]] * 2


@pytest.mark.parametrize("stream,address", GIVEN)
def test_candidate_chunks_are_allocated_for_the_stream_that_writes_them(world, stream, address):
    noise = FakeTensor(world, (2, 5, 3), torch.float32, 17)
    state = FakeTensor(world, (4,), torch.float32, 17)
    out = world.ex.denoise_shared(noise, state, 2, stream=stream())
    assert world.calls["rtv_denoise_shared"][0][-1] == address and out.pool == address
    assert noise.used_on == state.used_on == [address]
    assert world.ex.denoise(noise, state, 2, stream=stream()).pool == address


def test_a_stream_of_another_gpu_is_refused(world):
    with pytest.raises(ValueError):
        world.ex.get_prefix_kv_quantized(6, 1, stream=FakeStream(SIDE, device_index=1))
    assert not world.calls


def test_the_default_stream_is_the_contexts_gpus(world, monkeypatch):
    """With another GPU current, every call still goes to a stream of the context's."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: FakeStream(
        91 if device is None else 17, 1 if device is None else 0))
    pair = (FakeTensor(world, (2, 2, 1, 1, 6, 64), torch.uint8, 5), FakeTensor(world, (2, 2, 1, 1, 6), torch.float32, 5))
    world.ex.set_prefix_kv_quantized(*pair)
    world.ex.get_prefix_kv_quantized(6, 1)
    world.ex.denoise_shared(FakeTensor(world, (2, 5, 3), torch.float32, 17),
                            FakeTensor(world, (4,), torch.float32, 17), 2)
    assert [c[0][-1] for c in world.calls.values()] == [17, 17, 17]


@pytest.mark.parametrize("stream,address", GIVEN[:2])
def test_what_a_cache_operator_is_given_is_kept_until_its_stream_has_used_it(world, monkeypatch, stream, address):
    from flow_matching_action_dm0_b200 import CacheOps, QuantizedKV
    kept, went = [], []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: kept.append((id(self), s.cuda_stream)))
    described = types.SimpleNamespace(batch=1, dtype=0, n_tokens=1, n_heads=1, head_dim=64)
    for name in ("_rows", "_cache"):
        monkeypatch.setattr(CacheOps, name, lambda self, *a, **kw: described)
    monkeypatch.setattr(CacheOps, "_queries", lambda self, q, out, lse, scale: (described, out, lse))
    monkeypatch.setattr(CacheOps, "_workspace", lambda self, *a: (None, 0, None))
    for name in ("_ints", "_bools"):
        monkeypatch.setattr(CacheOps, name, lambda self, *a: None)
    monkeypatch.setattr(CacheOps, "_stream", lambda self: torch.cuda.current_stream(0).cuda_stream)
    for name in ("rtv_kv_write", "rtv_kv_read", "rtv_cross_attention", "rtv_shared_attention"):
        monkeypatch.setattr(L, name, lambda *a: went.append(a[-1]))
    ops = object.__new__(CacheOps)
    ops.device, ops.h, ops._torch_device = 0, None, torch.device("cuda", 0)
    t = [torch.zeros(1) for _ in range(8)]
    cache = QuantizedKV(*t[:4])
    for call, given in ((lambda s: ops.write(cache, t[4], t[5], start=t[6], count=t[7], stream=s), t),
                        (lambda s: ops.read(cache, lens=t[4], out=(t[5], t[6]), stream=s), t[:7]),
                        (lambda s: ops.cross_attention(t[4], cache, lens=t[5], out=t[6], lse=t[7], stream=s), t),
                        (lambda s: ops.shared_attention(t[0], (t[1], t[2]), (t[3], t[4]), prefix_mask=t[5],
                                                        own_lens=t[6], out=t[7], stream=s), t)):
        kept.clear()
        call(stream())
        assert went.pop() == address
        assert sorted(kept) == sorted((id(x), address) for x in given)
        assert len(world.current) == 1
