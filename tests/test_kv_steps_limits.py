"""CPU checks of places, prompts and drafts at the limits of their sizes: what a call cannot take is refused on the host, and not cut
to what it can."""
import ctypes
import types

import pytest

import kv_quantization_tile_amd as hq
from test_kv_steps_host import DEVICE, E, OnDevice, prompt, world  # noqa: F401

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("seqs", [1 << 31, 0xFFFFFFFF])
def test_prompt_sequences(seqs):
    """A workgroup looks for its tile over all sequences, 64 at a time: an index past them has to fit 32 bits."""
    assert prompt(seqs=seqs) == E


def i32(*shape, device="cpu"):
    return OnDevice(torch.empty(*shape, dtype=torch.int32, device=device))


def far(*shape):
    return i32(*shape, device="meta")  # of a size, without memory


CACHE = OnDevice(torch.zeros(4, 2, 64 * hq.hq_kv_token_bytes(4), dtype=torch.uint8))
ROWS = OnDevice(torch.zeros(3, 2, 128, dtype=torch.bfloat16))
WIDE = 2 ** 32 + 16  # 16 to a 32-bit field


@pytest.mark.parametrize("call", [
    lambda: hq.hq_attend_prompt(ROWS, ROWS, ROWS, far(WIDE + 1)),
    lambda: hq.hq_kv_reserve(far(1, WIDE), i32(1), i32(1), i32(9), i32(1), 16, 5),
    lambda: hq.hq_kv_reserve(i32(1, 4), i32(1), i32(1), far(WIDE), i32(1), 16, 5),
    lambda: hq.hq_kv_reserve(far(WIDE, 4), far(WIDE), far(WIDE), i32(9), i32(1), 16, 5, q_start=far(WIDE + 1), granted=far(WIDE)),
    lambda: hq.hq_kv_accept(CACHE, far(1, WIDE), i32(1), i32(3), i32(3), i32(3)),
    lambda: hq.hq_kv_attend(CACHE, ROWS, far(1, WIDE), i32(1), max_len=100),
    lambda: hq.hq_kv_attend(CACHE, ROWS, far(1, WIDE), i32(1), max_len=100, parents=i32(3)),
    lambda: hq.hq_kv_attend(CACHE, ROWS, far(WIDE, 1), far(WIDE), q_start=far(WIDE + 1)),
    lambda: hq.hq_kv_evict(CACHE, far(1, WIDE), i32(1), OnDevice(torch.zeros(1, 2, 8)), 4, 1, 1, i32(1, 1)),
    lambda: hq.hq_kv_evict(CACHE, i32(1, 1), i32(1), OnDevice(torch.zeros(1, 2, 8)), 4, 1, 1, far(1, WIDE)),
])
def test_sizes_past_32_bits_are_not_cut(world, call):  # noqa: F811
    with pytest.raises(ValueError):
        call()
    assert not world[1]


# ---- drafts ---------------------------------------------------------------------------------------


def drafts(n, seqs=1, **kw):
    q = OnDevice(torch.zeros(n, 2, 128, dtype=torch.bfloat16))
    return hq.hq_kv_attend(CACHE, q, i32(seqs, 1), i32(seqs), parents=i32(n), **kw)


def test_drafts_that_would_not_be_computed(world):  # noqa: F811
    """Without q_start the drafts of a sequence are known: more than 256 are refused, unless max_q says which are asked for."""
    drafts(256)
    drafts(3 * 256, seqs=3)
    drafts(300, max_q=256)
    drafts(300, seqs=2, q_start=i32(3))
    assert len(world[1]) == 4
    for n, seqs in ((257, 1), (3 * 257, 3), (1 << 16, 1)):
        with pytest.raises(ValueError):
            drafts(n, seqs)
    assert len(world[1]) == 4


def test_a_failed_call_names_itself(world, monkeypatch):  # noqa: F811
    """An error of a tree's call, or of its workspace's size, names the C entry that failed."""
    for failing in ("hq_kv_attend_tree", "hq_kv_attend_tree_workspace_size"):
        L = types.SimpleNamespace(**{n: lambda *a: hq.HQ_OK for n in ("hq_kv_attend_tree", "hq_kv_attend_tree_workspace_size")})
        setattr(L, failing, lambda *a: E)
        monkeypatch.setattr(hq, "lib", lambda: L)
        monkeypatch.setattr(hq, "strerror", lambda code: str(code))
        with pytest.raises(hq.HqError, match="hq_kv_attend_tree"):
            drafts(4)
