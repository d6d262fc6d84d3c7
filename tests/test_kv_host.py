"""CPU checks of the paged SRFT cache: the page layout's arithmetic, and that bad arguments are refused on the host
before any device call."""
import ctypes

import numpy as np
import pytest

import kv_quantization_tile_amd as hq
import kv_reference as ref

OK = 1 << 20
E = hq.HQ_ERR_INVALID_ARG


def cache(**kw):
    a = dict(data=OK, pages=8, heads=2, page=64, bits=4, seed=0, lambda_k=None, lambda_v=None)
    a.update(kw)
    return hq.HqKvCache(**a)


def lam(value):
    return ctypes.cast((ctypes.c_float * 128)(*([1.0] * 127 + [value])), ctypes.c_void_p)


BAD_CACHES = [dict(bits=5), dict(bits=0), dict(page=8), dict(page=48), dict(page=8192), dict(heads=0), dict(heads=70000),
              dict(data=None), dict(data=OK + 8), dict(pages=1 << 31)]


def append(c, k=OK, v=OK, dtype=1, tokens=4, strides=(256, 128, 256, 128), slots=OK):
    st = (ctypes.c_int64 * 4)(*strides) if strides else None
    return hq.lib().hq_kv_append(ctypes.byref(c), k, v, dtype, tokens, st, slots, None)


def read(c, slots=OK, tokens=4, k=OK, v=OK, dtype=1):
    return hq.lib().hq_kv_read(ctypes.byref(c), slots, tokens, k, v, dtype, None)


def attend_args(**kw):
    a = dict(q=OK, out=OK, q_dtype=1, out_dtype=1, q_stride_token=1024, q_stride_head=128, total_q=4, q_heads=8, seqs=4, max_q=1,
             max_len=512, q_start=None, table=OK, table_width=8, lens=OK, scale=0.1, softcap=0.0, causal=1, window=0, weights=None,
             weights_stride=0)
    a.update(kw)
    return hq.HqKvAttendArgs(**a)


def attend(c, a, ws=OK, size=1 << 30):
    return hq.lib().hq_kv_attend(ctypes.byref(c), ctypes.byref(a), ws, size, None)


def evict(c, **kw):
    a = dict(table=OK, lens=OK, weights=OK, weights_stride=512, seqs=2, table_width=8, max_len=512, budget=128, sink=4, recent=16,
             dst_table=OK, dst_width=2, kept=OK, new_lens=OK, new_weights=None)
    a.update(kw)
    return hq.lib().hq_kv_evict(ctypes.byref(c), ctypes.byref(hq.HqKvEvictArgs(**a)), None)


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(kw):
    c = cache(**kw)
    assert append(c) == E and read(c) == E and attend(c, attend_args()) == E and evict(c) == E


@pytest.mark.parametrize("value", [0.0, -1.0, float("nan"), float("inf")])
def test_bad_lambda_is_refused(value):
    for c in (cache(lambda_k=lam(value)), cache(lambda_v=lam(value))):
        assert append(c) == E and read(c) == E and attend(c, attend_args()) == E


def test_append_and_read_refusals():
    c = cache()
    assert append(c, k=None) == E and append(c, v=None) == E and append(c, slots=None) == E and append(c, strides=None) == E
    assert append(c, dtype=2) == E and append(c, k=OK + 1) == E and append(c, dtype=0, v=OK + 2) == E and append(c, slots=OK + 4) == E
    assert append(c, tokens=(1 << 31) + 1) == E
    assert append(c, tokens=1 << 31) == E                      # a launch of more than 2^32 threads
    assert append(c, k=None, v=None, slots=None, tokens=0) == hq.HQ_OK
    assert append(cache(pages=0, data=None)) == hq.HQ_OK       # no page: nothing to write
    assert read(c, slots=None) == E and read(c, k=None, v=None) == E and read(c, k=OK + 8) == E and read(c, dtype=7) == E
    assert read(c, tokens=1 << 31) == E and read(c, tokens=0, slots=None, k=None, v=None) == hq.HQ_OK


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(lens=None), dict(table=None), dict(q=OK + 1), dict(q_dtype=0, q=OK + 2), dict(out=OK + 8),
    dict(lens=OK + 2), dict(table=OK + 1), dict(q_start=OK + 2), dict(weights=OK + 1, weights_stride=512), dict(q_dtype=2),
    dict(out_dtype=-1), dict(q_heads=0), dict(q_heads=7), dict(total_q=5), dict(max_len=(1 << 30) + 1), dict(table_width=1 << 26),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(softcap=-1.0), dict(softcap=float("inf")), dict(softcap=float("nan")),
    dict(weights=OK, weights_stride=511), dict(seqs=1 << 30, total_q=1 << 30), dict(max_q=1 << 30),
])
def test_attend_refusals(kw):
    assert attend(cache(), attend_args(**kw)) == E


def test_attend_workspace():
    c, a, size = cache(), attend_args(), ctypes.c_size_t(0)
    L = hq.lib()
    assert L.hq_kv_attend_workspace_size(ctypes.byref(c), ctypes.byref(a), None) == E
    assert L.hq_kv_attend_workspace_size(ctypes.byref(c), None, ctypes.byref(size)) == E
    assert L.hq_kv_attend_workspace_size(None, ctypes.byref(a), ctypes.byref(size)) == E
    assert L.hq_kv_attend_workspace_size(ctypes.byref(c), ctypes.byref(a), ctypes.byref(size)) == hq.HQ_OK
    assert size.value > 0 and size.value % 256 == 0
    assert attend(c, a, size=size.value - 1) == E and attend(c, a, ws=None) == E and attend(c, a, ws=OK + 16) == E
    for nothing in (dict(total_q=0), dict(seqs=0, total_q=0), dict(max_q=0)):
        assert attend(c, attend_args(**nothing), ws=None, size=0) == hq.HQ_OK


@pytest.mark.parametrize("kw", [
    dict(lens=None), dict(new_lens=None), dict(weights=None), dict(table=None), dict(kept=None), dict(dst_table=None),
    dict(lens=OK + 1), dict(kept=OK + 2), dict(new_weights=OK + 1), dict(sink=100, recent=29), dict(budget=129), dict(max_len=513),
    dict(max_len=(1 << 30) + 1, weights_stride=1 << 31), dict(table_width=1 << 26), dict(seqs=1 << 30),
])
def test_evict_refusals(kw):
    assert evict(cache(), **kw) == E


def test_evict_of_nothing():
    assert evict(cache(), seqs=0, lens=None, new_lens=None, kept=None) == hq.HQ_OK


def test_python_refusals():
    torch = pytest.importorskip("torch")
    for kw in (dict(bits=3), dict(page=8), dict(page=24), dict(page=8192)):
        with pytest.raises(ValueError):
            hq.hq_kv_cache(4, 2, device="cpu", **kw)
    c = hq.hq_kv_cache(4, 2, device="cpu")
    assert c.shape == (4, 2, 64 * hq.hq_kv_token_bytes(4))
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):  # a host tensor
        hq.hq_kv_append(c, x, x, torch.zeros(3, dtype=torch.int64))


def test_reference_pages_round_trip(orc):
    """The reference's page views name every byte once, and its transform is the oracle's."""
    for bits in (4, 8):
        c = np.arange(2 * 3 * 32 * hq.hq_kv_token_bytes(bits), dtype=np.uint64).astype(np.uint8).reshape(2, 3, -1)
        views = ref.parts(c, bits)
        assert sum(v.nbytes for v in views) == c.nbytes
        assert all(np.shares_memory(v, c) for v in views)
    x = np.random.default_rng(3).standard_normal(128).astype(np.float32)
    got = orc.srft_forward(x, 11)
    # 12 roundings a coordinate on values up to the vector's norm
    assert np.abs(ref.transform(orc, 11) @ x - got).max() <= 12 * 2.0 ** -24 * np.linalg.norm(x)
