"""CPU: the paged SRFT cache's calls run with the cache's device current, whatever device is when they are made."""
import types

import pytest

torch = pytest.importorskip("torch")
hq = pytest.importorskip("kv_quantization_tile_amd")

DEVICE = torch.device("cuda", 1)


class OnDevice:
    """A host tensor that says it lies on DEVICE."""
    is_cuda, device = True, DEVICE

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture
def world(monkeypatch):
    """Device 0 is current; the calls that reach the library, with the device that is current then and their stream."""
    now, calls = [0], []

    class Current:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    def entry(name):
        def call(*a):
            if not name.endswith("size"):
                calls.append((name, now[0], a[-1]))
            return hq.HQ_OK
        return call

    names = ("hq_kv_append", "hq_kv_read", "hq_kv_attend_workspace_size", "hq_kv_attend", "hq_kv_evict")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Current)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
    monkeypatch.setattr(hq, "_empty", lambda shape, dtype, device, stream: OnDevice(torch.empty(shape, dtype=dtype)))
    monkeypatch.setattr(hq, "lib", lambda: types.SimpleNamespace(**{n: entry(n) for n in names}))
    return now, calls


def calls_of(stream=None):
    i32 = lambda *s: OnDevice(torch.zeros(*s, dtype=torch.int32))  # noqa: E731
    cache = OnDevice(torch.zeros(4, 2, 64 * hq.hq_kv_token_bytes(4), dtype=torch.uint8))
    k, slots = OnDevice(torch.zeros(3, 2, 128, dtype=torch.bfloat16)), OnDevice(torch.zeros(3, dtype=torch.int64))
    hq.hq_kv_append(cache, k, k, slots, stream=stream)
    hq.hq_kv_read(cache, slots, stream=stream)
    hq.hq_kv_attend(cache, k, i32(3, 1), i32(3), stream=stream)
    hq.hq_kv_evict(cache, i32(3, 1), i32(3), OnDevice(torch.zeros(3, 2, 64)), 16, 1, 1, i32(3, 1), stream=stream)


@pytest.mark.parametrize("current", [0, 1])
def test_the_caches_device_is_current_in_every_call(world, current):
    now, calls = world
    now[0] = current
    calls_of()
    calls_of(types.SimpleNamespace(device=DEVICE, cuda_stream=77))
    assert [c[0] for c in calls] == ["hq_kv_append", "hq_kv_read", "hq_kv_attend", "hq_kv_evict"] * 2
    assert all(c[1] == 1 for c in calls) and now[0] == current
    assert [c[2] for c in calls] == [1001] * 4 + [77] * 4


def test_a_stream_of_another_device_is_refused(world):
    with pytest.raises(ValueError):
        calls_of(types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=77))
    assert not world[1]
