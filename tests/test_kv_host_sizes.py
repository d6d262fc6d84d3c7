"""CPU: what attention over the paged SRFT cache asks for.  A batch is sized by the queries it has, not by its longest
sequence's in every place; sizes that the kernels take are not refused."""
import ctypes

import pytest

import kv_quantization_tile_amd as hq

MIB = 1 << 20


def workspace(seqs, total_q, max_q, max_len=32768, heads=8, group=4, page=64, bits=4, offsets=True, weights=False):
    """Bytes, or the error."""
    c = hq.HqKvCache(data=1 << 20, pages=1 << 20, heads=heads, page=page, bits=bits)
    a = hq.HqKvAttendArgs(q=1 << 20, out=1 << 20, q_dtype=1, out_dtype=1, q_stride_token=heads * group * 128, q_stride_head=128, total_q=total_q,
                          q_heads=heads * group, seqs=seqs, max_q=max_q, max_len=max_len, q_start=1 << 20 if offsets else None, table=1 << 20,
                          table_width=-(-max_len // page), lens=1 << 20, scale=0.1, weights=1 << 20 if weights else None, weights_stride=max_len)
    size = ctypes.c_size_t(0)
    rc = hq.lib().hq_kv_attend_workspace_size(ctypes.byref(c), ctypes.byref(a), ctypes.byref(size))
    return rc if rc != hq.HQ_OK else size.value


def rows_bytes(total_q, weights):
    """The transformed rows in one or two binary16 parts, their factors and statistics, 32 heads."""
    return total_q * 32 * (256 * (2 if weights else 1) + 8)


# split outputs of 512 tiles of 256 rows and of 2048 tiles of 16 rows
SPLIT = 512 * 256 * 520 + 2048 * 16 * 520


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("seqs,total_q,max_q", [
    (128, 2175, 2048),        # 127 single tokens beside a chunk
    (64, 575, 512),
    (256, 255 + 8192, 8192),
    (256, 255 + 32768, 32768),
    (1024, 1023 + 32768, 32768),
])
def test_a_chunk_beside_single_tokens(seqs, total_q, max_q, weights):
    got = workspace(seqs, total_q, max_q, weights=weights)
    assert 0 < got <= rows_bytes(total_q, weights) + SPLIT + MIB, got / MIB


@pytest.mark.parametrize("seqs", [64, 256, 1024])
def test_single_tokens_without_a_bound_on_their_number(seqs):
    """max_q as the count of all queries, which is what a call without it takes."""
    assert 0 < workspace(seqs, seqs, seqs) <= rows_bytes(seqs, False) + SPLIT + MIB


def test_equal_sequences_take_what_they_took():
    """Where all tiles are full the split outputs are those of 1536 tiles at most (with what rounding up adds)."""
    for seqs, m in ((1, 2048), (4, 512), (8, 129)):
        for offsets in (False, True):
            assert 0 < workspace(seqs, seqs * m, m, offsets=offsets) <= rows_bytes(seqs * m, False) + 2048 * 256 * 520 + 2048 * 16 * 520 + MIB


@pytest.mark.parametrize("kw", [dict(softcap=3e38), dict(softcap=1e-39), dict(scale=3e38), dict(scale=-2.0 ** 127), dict(softcap=-1e-40)])
def test_factors_that_binary32_cannot_hold_in_log2_units(kw):
    """log2(e) times the scale or the cap, or its reciprocal, would be infinite or lose its bits: refused, not computed."""
    c = hq.HqKvCache(data=1 << 20, pages=8, heads=2, page=64, bits=4)
    a = dict(q=1 << 20, out=1 << 20, q_dtype=1, out_dtype=1, q_stride_token=1024, q_stride_head=128, total_q=4, q_heads=8, seqs=4, max_q=1, max_len=512,
             table=1 << 20, table_width=8, lens=1 << 20, scale=0.1)
    # without a workspace nothing is launched whatever the factors: a good call is told from a refused one by none being asked for
    good = hq.HqKvAttendArgs(**a | dict(total_q=0))
    assert hq.lib().hq_kv_attend(ctypes.byref(c), ctypes.byref(good), None, 0, None) == hq.HQ_OK
    bad = hq.HqKvAttendArgs(**a | dict(total_q=0) | kw)
    assert hq.lib().hq_kv_attend(ctypes.byref(c), ctypes.byref(bad), None, 0, None) == hq.HQ_ERR_INVALID_ARG


def test_sizes_past_a_launch_are_refused():
    for kw in (dict(seqs=1 << 24, total_q=1 << 24, max_q=1), dict(seqs=1, total_q=1 << 30, max_q=1 << 30), dict(seqs=1, total_q=1 << 27, max_q=1 << 27)):
        assert workspace(**kw) == hq.HQ_ERR_INVALID_ARG
    # the weights' launch, a thread a token, counts only where weights are asked for
    assert workspace(2048, 2048, 1, max_len=1 << 20) > 0
    assert workspace(2048, 2048, 1, max_len=1 << 20, weights=True) == hq.HQ_ERR_INVALID_ARG
