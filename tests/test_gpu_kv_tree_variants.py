"""GPU: every kernel that a tree of drafted tokens may go through, against the definition in binary64: operands in registers (up to
16 rows a tile, and 32) and through LDS (64 rows a tile, and 128), at 4 and 8 bits, with caps, lambdas, windows, one split and many,
values of any size, tokens that take no part, and a cache past 2^32 bytes.

`plan` repeats the rule by which the library chooses among them; the workspace that it asks for has to be that plan's, so that a test
says which kernel it has run."""
import ctypes

import numpy as np
import pytest

import kv_reference
import steps_reference as ref

torch = pytest.importorskip("torch")
hq = pytest.importorskip("kv_quantization_tile_amd")

from test_gpu_kv_tree import SEED, Case, dev, host, say, some_tree  # noqa: E402

pytestmark = pytest.mark.gpu

D, WORK = 128, 1 << 24


def up(n, m):
    return -(-n // m) * m


def plan(seqs, heads, group, total, max_q, max_len, window=0):
    """(rows of a tile, splits, workspace bytes)."""
    rows, sh = min(max_q, total) * group, seqs * heads
    seen = window + min(max_q, total) + 15
    span = min(seen, max_len) if window else max_len
    tile = 16 if rows <= 16 else 32 if rows <= 32 or sh * rows * span <= WORK else 64 if rows <= 64 else 128
    items = sh * -(-rows // tile)
    splits = max(1, min(-(-{16: 2048, 32: 512, 64: 1536, 128: 512}[tile] // items), -(-span // 512)))
    chunk = up(-(-span // splits), 128)
    splits = max(1, -(-span // chunk))
    parts, held = items * splits * tile if splits > 1 else 0, total * group * heads + 16 if tile > 32 else 0
    return tile, splits, sum(up(n, 256) for n in (parts * 8, parts * D * 4, held * 4, held * 2 * D))


def planned(c, max_len, max_q=None):
    """The plan of a case's call, which the library's workspace agrees with."""
    heads, group, max_q = c.cache.shape[1], c.q.shape[1] // c.cache.shape[1], max_q or max(c.q_lens)
    tile, splits, size = plan(len(c.lens), heads, group, sum(c.q_lens), max_q, max_len, c.window)
    cache = hq.HqKvCache(256, c.cache.shape[0], heads, c.page, c.bits, SEED, None, None)
    a = hq.HqKvAttendArgs(q=256, out=256, q_dtype=0, out_dtype=0, q_stride_token=group * heads * D, q_stride_head=D, total_q=sum(c.q_lens),
                          q_heads=heads * group, seqs=len(c.lens), max_q=max_q, max_len=max_len, q_start=256, table=256,
                          table_width=c.table.shape[1], lens=256, scale=0.1, causal=1, window=c.window)
    got = ctypes.c_size_t()
    assert hq.lib().hq_kv_attend_tree_workspace_size(ctypes.byref(cache), ctypes.byref(a), ctypes.byref(got)) == hq.HQ_OK
    assert got.value == size
    return tile, splits


def attend(c, large=False):
    """steps_reference.attend's outputs and bounds, a (sequence, head) at a time.  A token whose K scales are -0 takes no part.  With
    `large` scales about, scales of the same 16 tokens are off by up to 2^-18, a value by up to that times its code."""
    T, cache = kv_reference.transform(c.orc, SEED), host(c.cache)
    lam_k, lam_v = (np.ones(D) if x is None else x.astype(np.float64) for x in c.lam)
    heads, hq_heads = cache.shape[1], c.q.shape[1]
    out, tol, at = np.zeros(c.q.shape), np.zeros(c.q.shape[:2]), 0
    for b, (n, see) in enumerate(zip(c.lens, c.sees)):
        m = len(see)
        # the sequence's pages alone
        row = c.table[b, :-(-n // c.page)]
        named = (row >= 0) & (row < len(cache))
        pages = cache[np.where(named, row, 0)]
        row = np.where(named, np.arange(len(row)), -1)
        ks = kv_reference.parts(pages, c.bits)[1].view(np.uint16)
        for a in range(heads if m else 0):
            k, v, there = kv_reference.coordinates(pages, c.bits, row, n, a, lam_k, lam_v)
            t = np.arange(n)
            there = there & (ks[t // c.page, a, t % c.page, 0] != 0x8000)
            k, v, w = k[there], v[there], see[:, there]
            for j in range(a * hq_heads // heads, (a + 1) * hq_heads // heads):
                y = c.q[at:at + m, j].astype(np.float64) @ T.T * c.kw["scale"]
                s = y @ k.T
                big = np.where(w, np.abs(y) @ np.abs(k).T, 0).max(-1, initial=0)
                cap = c.kw["softcap"]
                if cap:
                    s = cap * np.tanh(s / cap)
                s = np.where(w, s, -np.inf)
                e = np.exp(s - np.maximum(s.max(-1, initial=-np.inf), -1e300)[:, None])
                p = e / np.maximum(e.sum(-1), 1e-300)[:, None]
                out[at:at + m, j] = (p @ v) @ T
                eps = (2.0 ** -10 + 2.0 ** -17) * big + 2.0 ** -20 * (big + cap)
                rel = np.exp(2 * eps) * (1 + 2.0 ** -20) - 1
                most = np.where(w, np.abs(v).max(-1, initial=0), 0).max(-1, initial=0)
                tol[at:at + m, j] = (rel + 3 * 2.0 ** -11 + 2.0 ** -17) * np.linalg.norm(p @ np.abs(v), axis=-1) + \
                    2.0 ** -33 * w.sum(-1) * most * np.sqrt(D)
                if large:
                    tol[at:at + m, j] += 2.0 ** -18 * (7 if c.bits == 4 else 127) * lam_v.max() * np.sqrt(D)
        at += m
    return out, tol


def within(got, want, tol):
    """With the transform back's 12 binary32 roundings."""
    got = host(got).astype(np.float64)
    err, bound = np.linalg.norm(got - want, axis=-1), tol + 2.0 ** -20 * np.linalg.norm(want, axis=-1)
    assert np.isfinite(got).all() and (err <= bound).all(), np.max(err / np.maximum(bound, 1e-30))


# (rows of a tile: shape, and the most tokens announced, from which the library takes the kernel)
SHAPES = {
    16: (dict(lens=[300, 77], q_lens=[4, 3], group=4), 300),
    32: (dict(lens=[300, 77], q_lens=[13, 9], group=2), 300),
    "32_of_80": (dict(lens=[300, 150], q_lens=[40, 33], group=2), 300),
    64: (dict(lens=[1300, 150], q_lens=[30, 17], group=2), 1 << 18),
    "64_one_head": (dict(lens=[700, 150], q_lens=[7, 2], group=7, heads=1, page=64), 1 << 20),
    128: (dict(lens=[1300, 150], q_lens=[40, 33], group=2), 1 << 18),
    "128_tiles": (dict(lens=[700], q_lens=[200], group=1, heads=1, page=32), 1 << 20),
}


def shape(name, **kw):
    d, max_len = SHAPES[name]
    return dict(d) | kw, max_len, name if isinstance(name, int) else int(name.split("_")[0])


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lam,softcap", [(False, 0.0), (True, 0.0), (False, 15.0), (True, 20.0)])
def test_every_kernel(orc, name, bits, lam, softcap):
    say(f"case: tree, {name} rows a tile, {bits} bits, lambda {lam}, cap {softcap}")
    kw, max_len, tile = shape(name, bits=bits, lam=lam, softcap=softcap)
    c = Case(orc, **kw)
    assert planned(c, max_len)[0] == tile
    got = c.run(max_len=max_len)
    within(got, *attend(c))
    assert torch.equal(c.run(max_len=max_len), got)
    # the batch's queries as the bound on a sequence's: another plan, the same rows
    within(c.run(max_len=max_len, max_q=None), *attend(c))


# ---- one split: rows stored without a join -----------------------------------------------------------


def wide(seqs, long, most, lens, **kw):
    """A batch of mostly single drafts, a few sequences with up to `most`."""
    g = np.random.default_rng(seqs)
    m = np.ones(seqs, int)
    m[g.choice(seqs, long, replace=False)] = np.linspace(most, 2, long).astype(int)
    n = np.maximum(g.integers(*lens, seqs), 1)
    n[m > 1] = lens[1]
    return dict(lens=n.tolist(), q_lens=m.tolist(), seed=seqs, **kw)


@pytest.mark.parametrize("tile,max_len,kw", [
    (64, 320, wide(768, 9, 20, (0, 70), heads=2, group=2)),
    (64, 320, wide(768, 9, 20, (0, 70), heads=2, group=2, bits=8, lam=True, softcap=12.0)),
    (128, 500, wide(256, 9, 40, (0, 200), heads=2, group=2)),
    (128, 500, wide(256, 9, 40, (0, 200), heads=2, group=2, bits=8, lam=True, softcap=12.0)),
    (32, 128, wide(300, 9, 13, (0, 100), heads=2, group=2, lam=True)),
    (16, 128, wide(1100, 9, 8, (0, 50), heads=2, group=2, lam=True, bits=8)),
])
def test_one_split(orc, tile, max_len, kw):
    say(f"case: tree, one split, {tile} rows a tile, {len(kw['lens'])} sequences, {kw.get('bits', 4)} bits")
    c = Case(orc, **kw)
    assert planned(c, max_len) == (tile, 1)
    within(c.run(max_len=max_len), *attend(c))


# ---- windows -----------------------------------------------------------------------------------------


@pytest.mark.parametrize("tile,kw", [
    # the window ends among the held tokens, at another one for every depth
    (64, wide(64, 6, 32, (600, 700), heads=8, group=2, window=500, page=64)),
    (64, wide(64, 6, 32, (600, 700), heads=8, group=2, window=500, page=64, bits=8, softcap=20.0)),
    (128, dict(lens=[1500], q_lens=[256], heads=8, group=8, window=800, page=64)),
    (128, dict(lens=[900, 1400], q_lens=[100, 256], heads=8, group=4, window=777, page=64, bits=8, lam=True)),
    # it ends among the drafts: ancestors drop out
    (64, wide(420, 6, 64, (0, 90), heads=8, group=1, window=2)),
    (64, wide(420, 6, 64, (0, 90), heads=8, group=1, window=1, bits=8)),
    (128, wide(120, 6, 256, (0, 300), heads=2, group=1, window=3)),
    (128, wide(120, 6, 250, (0, 300), heads=2, group=1, window=23, bits=8, lam=True)),
    (32, dict(lens=[400, 50], q_lens=[30, 30], group=2, window=23, bits=8)),
    (16, dict(lens=[700, 31], q_lens=[8, 8], group=2, window=5, bits=8)),
])
def test_windows(orc, tile, kw):
    say(f"case: tree, window {kw['window']}, {tile} rows a tile, {len(kw['lens'])} sequences, {kw.get('bits', 4)} bits")
    c = Case(orc, **kw)
    assert planned(c, max(c.lens))[0] == tile
    got = c.run()
    within(got, *attend(c))
    assert torch.equal(c.run(), got)


# ---- values of any size ------------------------------------------------------------------------------


class Scaled(Case):
    """A case whose keys and values are taken times `k` and `v` (numbers, or one per slot), with the scores' scale undoing
    the largest of `k`."""

    def __init__(self, orc, *, k, v, **kw):
        super().__init__(orc, **kw)
        slots = torch.arange(self.cache.shape[0] * self.page, device="cuda")
        old = hq.hq_kv_read(self.cache, slots, out_dtype=torch.float32, **self.fmt)
        new = [x * dev(np.full(slots.shape, f, np.float32))[:, None, None] for x, f in zip(old, (k, v))]
        hq.hq_kv_append(self.cache, *new, slots, **self.fmt)
        self.kw["scale"] = float(128 ** -0.5 / np.max(k))


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("which", ["keys", "values", "both", "some"])
def test_large_values(orc, which, bits, name):
    """Scales up to the largest there are (65504), everywhere or at one token in ten: nothing overflows, bounds as ever."""
    say(f"case: tree over large {which}, {bits} bits, {name} rows a tile")
    kw, max_len, tile = shape(name, bits=bits)
    page = kw.get("page", 16)
    slots = (sum(-(-n // page) for n in kw["lens"]) + 2) * page
    g = np.random.default_rng(5)
    some = [np.where(g.random(slots) < 0.1, 1e7, 1.0) for _ in range(2)]
    k, v = {"keys": (1e7, 1), "values": (1, 1e7), "both": (1e7, 1e7), "some": some}[which]
    c = Scaled(orc, k=k, v=v, **kw)
    assert planned(c, max_len)[0] == tile
    _, ks, _, vs = kv_reference.parts(host(c.cache), bits)
    assert max(ks.max(), vs.max()) == 65504
    for cap in (0.0, 20.0):
        c.kw["softcap"] = cap
        within(c.run(max_len=max_len), *attend(c, which == "some"))


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("bits", [4, 8])
def test_stale_scales_past_a_length(orc, name, bits):
    """What lies past a length in its last page, the largest scales there are, infinite and NaN ones, leaves what is before it as it
    was, to the bit."""
    say(f"case: tree beside stale scales, {bits} bits, {name} rows a tile")
    kw, max_len, tile = shape(name, bits=bits)
    c = Scaled(orc, k=1e-4, v=1e-4, **kw)
    assert planned(c, max_len)[0] == tile
    want, clean = c.run(max_len=max_len), host(c.cache)
    for word in (0x7BFF, 0x7C00, 0x7E00, 0xFE00, 0x8000):
        stale = clean.copy()
        _, ks, _, vs = kv_reference.parts(stale, bits)
        for b, n in enumerate(c.lens):
            for t in range(n, up(n, c.page)):
                pg = c.table[b, t // c.page]
                ks.view(np.uint16)[pg, :, t % c.page] = vs.view(np.uint16)[pg, :, t % c.page // 4, :, t % c.page % 4] = word
        c.cache = dev(stale)
        assert torch.equal(c.run(max_len=max_len), want)


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("bits", [4, 8])
def test_tokens_that_take_no_part(orc, name, bits):
    """Absent pages, and tokens whose K scales are -0 (as an eviction and an acceptance leave them), drafts among them."""
    say(f"case: tree, tokens that take no part, {bits} bits, {name} rows a tile")
    kw, max_len, tile = shape(name, bits=bits)
    c = Case(orc, **kw)
    assert planned(c, max_len)[0] == tile
    g, raw = np.random.default_rng(3), host(c.cache)
    ks = kv_reference.parts(raw, bits)[1].view(np.uint16)
    for b, (n, m) in enumerate(zip(c.lens, c.q_lens)):
        for t in {0, n - 1, n - m, n - m - 1, *g.integers(0, n, n // 5).tolist()}:
            ks[c.table[b, t // c.page], :, t % c.page] = 0x8000
    c.table[0, 2] = -1
    c.cache = dev(raw)
    within(c.run(max_len=max_len), *attend(c))
    c.table[:] = -1
    assert not c.run(max_len=max_len).any()


@pytest.mark.parametrize("name", SHAPES)
def test_nan_vectors_at_8_bits(orc, name):
    """A vector that was not finite reaches the drafts that see it, and no other."""
    say(f"case: tree, NaN vectors, 8 bits, {name} rows a tile")
    kw, max_len, _ = shape(name, bits=8)
    c = Case(orc, **kw)
    clean, group, b = host(c.run(max_len=max_len)), kw["group"], len(c.lens) - 1
    n, m, first = c.lens[b], c.q_lens[b], sum(c.q_lens[:b])
    for t in (n - m + m // 2, n - m - 1):
        slot = dev(np.array([c.table[b, t // c.page] * c.page + t % c.page], np.int64))
        for side in range(2):
            held = c.cache.clone()
            pair = list(hq.hq_kv_read(c.cache, slot, out_dtype=torch.float32, **c.fmt))
            pair[side][:, 0] = float("nan")
            hq.hq_kv_append(c.cache, *pair, slot, **c.fmt)
            got, sees = host(c.run(max_len=max_len)), c.sees[b][:, t]
            assert sees.any() and np.isnan(got[first:first + m, :group][sees]).all()
            got[first:first + m, :group][sees] = clean[first:first + m, :group][sees]
            # the vectors that were finite were written again, from what they decode to
            assert np.isfinite(got).all()
            c.cache = held


# ---- far offsets -------------------------------------------------------------------------------------


def test_cache_past_32_bits():
    """Pages beyond 2^32 bytes: attention and acceptance give what they give in a small cache."""
    say("case: tree and acceptance, a cache of 5 GiB")
    g = np.random.default_rng(1)
    heads, page, n, m, width = 8, 64, 1000, 40, 16
    small = torch.randint(0, 256, (width, heads, page * hq.hq_kv_token_bytes(4)), dtype=torch.uint8, device="cuda")
    for s in kv_reference.parts(host(small), 4)[1::2]:
        assert s.shape[0] == width
    raw = host(small).copy()
    for s in kv_reference.parts(raw, 4)[1::2]:
        s[:] = g.uniform(0.05, 0.3, s.shape)
    for x in kv_reference.parts(raw, 4)[::2]:  # codes are -7..7
        x &= 0x77
    small = dev(raw)
    pages = 5 * 2 ** 30 // small[0].numel()
    large = hq.hq_kv_cache(pages, heads, page)
    at = np.array([pages - 1 - 2 * i for i in range(width // 2)] + list(range(width // 2)), np.int32)
    large[dev(at).long()] = small
    i32 = lambda x: dev(np.array(x, np.int32))  # noqa: E731
    table, far, lens, parents = i32([list(range(width))]), dev(at[None]), i32([n]), i32(some_tree(g, m))
    q = torch.randn(m, heads * 2, D, device="cuda").to(torch.bfloat16)
    for max_len in (None, 1 << 18):  # in registers, through LDS
        assert plan(1, heads, 2, m, m, max_len or n)[0] == (128 if max_len else 32)
        a, b = (hq.hq_kv_attend(c, q, t, lens, parents=parents, max_len=max_len) for c, t in ((small, table), (large, far)))
        assert torch.isfinite(a).all() and torch.equal(a, b)
    tokens, target = i32(g.integers(0, 2, m)), i32(g.integers(0, 2, m))
    a, b = (hq.hq_kv_accept(c, t, lens, tokens, target, parents) for c, t in ((small, table), (large, far)))
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(large[dev(at).long()], small)


def test_steps_reference_agrees(orc):
    """The definition above is steps_reference.attend's."""
    say("case: tree, the two forms of the definition")
    for kw in (dict(lens=[200, 3, 40], q_lens=[9, 4, 20], lam=True, softcap=9.0), dict(lens=[90], q_lens=[30], window=7)):
        c = Case(orc, **kw)
        for x, y in zip(attend(c), ref.attend(orc, host(c.cache), c.q, c.table, c.lens, c.sees, c.bits, SEED, *c.lam, **c.kw)):
            assert np.allclose(x, y, rtol=1e-9, atol=1e-12)


# ---- graphs, and calls at once ------------------------------------------------------------------------


@pytest.mark.parametrize("name", [64, 128])
def test_graphs_through_lds(orc, name):
    """Captured with launches of their own for rows and joins, replayed on other queries, trees, lengths and pages."""
    say(f"case: tree graph, {name} rows a tile")
    kw, max_len, tile = shape(name, window=0)
    c = Case(orc, **kw)
    assert planned(c, max_len)[0] == tile
    q, table, lens, parents, start = (dev(x) for x in (c.q, c.table, np.array(c.lens, np.int32), c.parents, c.start))
    call = lambda: hq.hq_kv_attend(c.cache, q, table, lens, q_start=start, max_q=max(c.q_lens), max_len=max_len, parents=parents, **c.kw, **c.fmt)  # noqa: E731
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    g = np.random.default_rng(2)
    for i in range(4):
        q.normal_()
        parents.copy_(torch.tensor(sum((some_tree(g, m) for m in c.q_lens), []), dtype=torch.int32))
        lens.copy_(torch.tensor([n - 37 * i for n in c.lens], dtype=torch.int32))
        table.copy_(dev(c.table[::-1].copy() if i == 2 else c.table))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, call())


def test_calls_at_once(orc):
    """Trees of every kernel and prompts on streams of their own, their launches among one another's, give what they give alone."""
    say("case: trees and prompts on several streams")
    cases = [(Case(orc, **shape(name)[0]), shape(name)[1]) for name in SHAPES]
    rows = [torch.randn(n, 6, D, device="cuda").to(torch.bfloat16) for n in (700, 300)]
    starts = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 100, 101, 700], list(range(0, 301, 3)))]
    calls = [lambda s, c=c, n=n: c.run(max_len=n, stream=s) for c, n in cases]
    calls += [lambda s, x=x, st=st: hq.hq_attend_prompt(x[:, :4], x[:, 4:5], x[:, 5:], st, stream=s) for x, st in zip(rows, starts)]
    want = [f(None) for f in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for f, s in zip(calls, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):  # the case's own buffers too
                got.append(f(s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
