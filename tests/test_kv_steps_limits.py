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
