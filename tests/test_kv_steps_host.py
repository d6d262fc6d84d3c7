"""CPU checks of places, prompts and drafts: bad arguments are refused on the host before any device call, and the Python
calls run with their tensors' device current."""
import ctypes
import types

import numpy as np
import pytest

import kv_quantization_tile_amd as hq
import steps_reference as ref
from test_kv_host import BAD_CACHES, OK, E, attend_args, cache

torch = pytest.importorskip("torch")


def reserve(**kw):
    a = dict(table=OK, lens=OK, counts=OK, free=OK, free_count=OK, seqs=4, table_width=8, pages=100, page=64, tokens=50, slots=OK, positions=OK,
             q_start=OK, granted=OK)
    return hq.lib().hq_kv_reserve(ctypes.byref(hq.HqKvReserveArgs(**a | kw)), None)


def accept(c, **kw):
    a = dict(table=OK, lens=OK, q_start=None, tokens=OK, target=OK, parents=OK, total_q=8, seqs=2, table_width=8, max_q=4, path=OK, accepted=OK,
             next=OK, change=OK)
    return hq.lib().hq_kv_accept(ctypes.byref(c), ctypes.byref(hq.HqKvAcceptArgs(**a | kw)), None)


def tree(c, a, parents=OK, ws=OK, size=1 << 30):
    return hq.lib().hq_kv_attend_tree(ctypes.byref(c), ctypes.byref(a), parents, ws, size, None)


def prompt(**kw):
    two = ctypes.c_int64 * 2
    a = dict(q=OK, k=OK, v=OK, out=OK, dtype=1, out_dtype=1, q_stride=two(1024, 128), k_stride=two(256, 128), v_stride=two(256, 128), rows=10,
             q_heads=8, heads=2, seqs=2, start=OK, scale=0.1, softcap=0.0, causal=1, window=0)
    kw = {x: two(*y) if x.endswith("stride") else y for x, y in kw.items()}
    return hq.lib().hq_attend_prompt(ctypes.byref(hq.HqAttendPromptArgs(**a | kw)), None)


@pytest.mark.parametrize("kw", [
    dict(page=8), dict(page=48), dict(page=8192), dict(page=0), dict(table=None), dict(lens=None), dict(counts=None), dict(free=None),
    dict(free_count=None), dict(slots=None), dict(q_start=None), dict(granted=None), dict(table=OK + 2), dict(lens=OK + 1), dict(counts=OK + 2),
    dict(free=OK + 2), dict(free_count=OK + 1), dict(slots=OK + 4), dict(positions=OK + 2), dict(q_start=OK + 2), dict(granted=OK + 2),
    dict(tokens=(1 << 31) + 1), dict(pages=1 << 31), dict(table_width=1 << 26), dict(seqs=1 << 29), dict(seqs=0xFFFFFFFF, table_width=0),
])
def test_reserve_refusals(kw):
    assert reserve(**kw) == E


def test_reserve_null():
    assert hq.lib().hq_kv_reserve(None, None) == E


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches(kw):
    c = cache(**kw)
    assert accept(c) == E and tree(c, attend_args()) == E


@pytest.mark.parametrize("kw", [
    dict(max_q=257), dict(total_q=(1 << 31) + 1), dict(total_q=7), dict(table_width=1 << 26), dict(seqs=1 << 28), dict(lens=None), dict(accepted=None),
    dict(next=None), dict(change=None), dict(path=None), dict(table=None), dict(tokens=None), dict(target=None), dict(parents=None),
    dict(table=OK + 2), dict(lens=OK + 2), dict(q_start=OK + 2), dict(tokens=OK + 1), dict(target=OK + 2), dict(parents=OK + 2), dict(path=OK + 2),
    dict(accepted=OK + 2), dict(next=OK + 2), dict(change=OK + 2),
])
def test_accept_refusals(kw):
    assert accept(cache(), **kw) == E


def test_tree_workspace():
    L, c, size = hq.lib(), cache(), ctypes.c_size_t(0)
    call = lambda a, s=size: L.hq_kv_attend_tree_workspace_size(ctypes.byref(c), ctypes.byref(a), ctypes.byref(s) if s is not None else None)  # noqa: E731
    assert call(attend_args(), None) == E and call(attend_args(causal=0)) == E and call(attend_args(max_q=257, total_q=4 * 257)) == E
    for q in (1, 4, 7, 16, 33, 200):
        a = attend_args(max_q=q, total_q=4 * q, max_len=40000, table_width=700)
        assert call(a) == hq.HQ_OK and size.value % 256 == 0
        assert tree(c, a, size=size.value - 1) == E


def test_accept_of_nothing():
    assert hq.lib().hq_kv_accept(ctypes.byref(cache()), None, None) == E
    assert accept(cache(), seqs=0, total_q=0, lens=None, accepted=None, next=None, change=None, path=None, table=None) == hq.HQ_OK


@pytest.mark.parametrize("kw", [dict(causal=0), dict(weights=OK, weights_stride=512), dict(max_q=257, total_q=4 * 257), dict(total_q=5),
                                dict(scale=float("nan")), dict(q=None), dict(max_len=(1 << 30) + 1)])
def test_tree_refusals(kw):
    assert tree(cache(), attend_args(**kw)) == E


def test_tree_parents():
    assert tree(cache(), attend_args(), parents=None) == E and tree(cache(), attend_args(), parents=OK + 2) == E
    assert hq.lib().hq_kv_attend_tree(ctypes.byref(cache()), None, OK, OK, 1 << 30, None) == E
    a = attend_args(max_len=40000, table_width=700)
    assert tree(cache(), a, size=16) == E and tree(cache(), a, ws=None) == E and tree(cache(), a, ws=OK + 16) == E
    assert tree(cache(), attend_args(total_q=0), parents=None, ws=None, size=0) == hq.HQ_OK


@pytest.mark.parametrize("kw", [
    dict(dtype=0), dict(dtype=2), dict(out_dtype=2), dict(heads=0), dict(q_heads=0), dict(q_heads=7), dict(q_heads=65536, heads=1), dict(rows=(1 << 30) + 1),
    dict(rows=1 << 26), dict(scale=float("nan")), dict(scale=float("inf")), dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
    dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(start=None), dict(q=OK + 8), dict(k=OK + 2), dict(v=OK + 4), dict(out=OK + 8),
    dict(start=OK + 2), dict(q_stride=(1024, 129)), dict(k_stride=(257, 128)), dict(v_stride=(260, 128)),
    dict(k_stride=(1 << 23, 128)), dict(v_stride=(-256, 128)),
])
def test_prompt_refusals(kw):
    assert prompt(**kw) == E


def test_prompt_of_nothing():
    assert hq.lib().hq_attend_prompt(None, None) == E
    assert prompt(rows=0, q=None, k=None, v=None, out=None, start=None) == hq.HQ_OK and prompt(seqs=0, start=None) == hq.HQ_OK


def test_python_refuses_host_tensors():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        hq.hq_kv_reserve(i32(2, 4), i32(2), i32(2), i32(9), i32(1), 16, 5)
    with pytest.raises(TypeError):
        hq.hq_attend_prompt(x, x, x, i32(2))
    with pytest.raises(TypeError):
        hq.hq_kv_accept(hq.hq_kv_cache(4, 2, device="cpu"), i32(2, 1), i32(2), i32(4), i32(4), i32(4))


# ---- the device that is current ---------------------------------------------------------------------

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

    names = ("hq_kv_reserve", "hq_kv_attend_tree_workspace_size", "hq_kv_attend", "hq_kv_attend_tree", "hq_kv_accept", "hq_attend_prompt")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Current)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
    monkeypatch.setattr(hq, "_empty", lambda shape, dtype, device, stream: OnDevice(torch.empty(shape, dtype=dtype)))
    monkeypatch.setattr(hq, "lib", lambda: types.SimpleNamespace(**{n: entry(n) for n in names}))
    return now, calls


def calls_of(stream=None):
    i32 = lambda *s: OnDevice(torch.zeros(*s, dtype=torch.int32))  # noqa: E731
    c = OnDevice(torch.zeros(4, 2, 64 * hq.hq_kv_token_bytes(4), dtype=torch.uint8))
    q = OnDevice(torch.zeros(3, 2, 128, dtype=torch.bfloat16))
    hq.hq_kv_reserve(i32(3, 4), i32(3), i32(3), i32(9), i32(1), 16, 5, stream=stream)
    hq.hq_kv_attend(c, q, i32(3, 1), i32(3), parents=i32(3), stream=stream)
    hq.hq_kv_accept(c, i32(3, 1), i32(3), i32(3), i32(3), i32(3), stream=stream)
    hq.hq_attend_prompt(q, q, q, i32(4), stream=stream)


@pytest.mark.parametrize("current", [0, 1])
def test_the_tensors_device_is_current_in_every_call(world, current):
    now, calls = world
    now[0] = current
    calls_of()
    calls_of(types.SimpleNamespace(device=DEVICE, cuda_stream=77))
    assert [c[0] for c in calls] == ["hq_kv_reserve", "hq_kv_attend_tree", "hq_kv_accept", "hq_attend_prompt"] * 2
    assert all(c[1] == 1 for c in calls) and now[0] == current
    assert [c[2] for c in calls] == [1001] * 4 + [77] * 4


def test_a_stream_of_another_device_is_refused(world):
    with pytest.raises(ValueError):
        calls_of(types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=77))
    assert not world[1]


# ---- the reference itself ---------------------------------------------------------------------------


def test_reference_places():
    table, lens, free = np.array([[3, -1, -1], [1, 0, -1]], np.int32), np.array([16, 20], np.int32), np.array([2, 4, 5, -1, -1, -1], np.int32)
    out = ref.reserve(table, lens, [1, -10], free, 3, 16, 2)
    # sequence 1 gives page 0 back, sequence 0 takes it
    assert out[0].tolist() == [0, -1] and out[1].tolist() == [16, 0] and out[2].tolist() == [0, 1, 1] and out[3].tolist() == [1, -10] and out[4] == 3
    assert table.tolist() == [[3, 0, -1], [1, -1, -1]] and lens.tolist() == [17, 10]


def test_reference_trees():
    parents = [-1, 0, 0, 2, 9, 3]
    assert ref.chain(parents, 5) == [0, 2, 3, 5] and ref.chain(parents, 4) == [4]
    see = ref.tree_sees(parents, 8, 6)
    assert np.flatnonzero(see[5]).tolist() == [0, 1, 2, 4, 5, 7] and np.flatnonzero(see[4]).tolist() == [0, 1, 6]
    assert np.flatnonzero(ref.tree_sees(parents, 8, 6, 3)[1]).tolist() == [1, 2, 3]
    assert ref.accept_path([7, 5, 5, 1], [5, 2, 1, 0], [-1, 0, 0, 2]) == [0, 1]
    assert ref.accept_path([7, 4, 5, 1], [5, 2, 1, 0], [-1, 0, 0, 2]) == [0, 2, 3]
    assert ref.accept_path([], [], []) == []
