"""GPU: a tree of drafted tokens over the paged SRFT cache: attention against its definition in binary64 (steps_reference.attend
gives each output row's error bound), and the acceptance of drafts, byte for byte."""
import numpy as np
import pytest

import kv_reference
import steps_reference as ref

torch = pytest.importorskip("torch")
hq = pytest.importorskip("kv_quantization_tile_amd")

pytestmark = pytest.mark.gpu

SEED = 21


def say(msg):
    print(msg, flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.cpu().numpy()


def some_tree(g, m):
    """Chains, bushes and some drafts without a draft before them."""
    p = [-1]
    for i in range(1, m):
        p.append(int(g.choice([i - 1, max(0, i - 2), int(g.integers(0, i)), -1], p=[0.5, 0.2, 0.25, 0.05])))
    return p[:m]


class Case:
    def __init__(self, orc, lens, q_lens, heads=2, group=2, page=16, bits=4, window=0, softcap=0.0, lam=False, scale=128 ** -0.5,
                 seed=0, trees=None):
        g = np.random.default_rng(seed + sum(lens))
        self.orc, self.lens, self.q_lens, self.bits, self.window, self.page = orc, lens, q_lens, bits, window, page
        self.kw = dict(softcap=softcap, scale=scale)
        self.lam = [g.uniform(0.5, 2.0, 128).astype(np.float32) if lam else None for _ in range(2)]
        used = [-(-n // page) for n in lens]
        pages = sum(used) + 2
        order = g.permutation(pages).astype(np.int32)
        self.table = np.full((len(lens), max(used) + 1), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        self.cache = hq.hq_kv_cache(pages, heads, page, bits)
        k, v = (dev(g.standard_normal((pages * page, heads, 128)).astype(np.float32)) for _ in range(2))
        self.fmt = dict(bits=bits, seed=SEED, lam_k=self.lam[0], lam_v=self.lam[1])
        hq.hq_kv_append(self.cache, k, v, torch.arange(pages * page, device="cuda"), **self.fmt)
        self.trees = trees or [some_tree(g, m) for m in q_lens]
        self.sees = [ref.tree_sees(t, n, m, window) for t, n, m in zip(self.trees, lens, q_lens)]
        q = g.standard_normal((sum(q_lens), heads * group, 128)).astype(np.float32)
        kh, at = host(k), 0
        for b, (n, m) in enumerate(zip(lens, q_lens)):
            for i in range(m):
                # the last that it sees, drafts that it does not, and a held token at the window's edge
                seen = np.flatnonzero(self.sees[b][i])
                for t in {n - m + i, n - m + i - 1, n - m + i + 1, seen[0] if len(seen) else 0, seen[0] - 1 if len(seen) else 0, n - 1}:
                    if 0 <= t < n:
                        q[at + i] += 0.4 * np.repeat(kh[self.table[b, t // page] * page + t % page], group, 0)
            at += m
        self.q = q
        self.start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.parents = np.array(sum((list(t) for t in self.trees), []), np.int32)

    def run(self, q=None, out_dtype=torch.float32, **kw):
        q = dev(self.q) if q is None else q
        out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
        a = dict(q_start=dev(self.start), max_q=max(self.q_lens), max_len=max(self.lens), out=out, window=self.window, parents=dev(self.parents),
                 **self.kw, **self.fmt) | kw
        return hq.hq_kv_attend(self.cache, q, dev(self.table), dev(np.array(self.lens, np.int32)), **a)

    def want(self):
        return ref.attend(self.orc, host(self.cache), self.q, self.table, self.lens, self.sees, self.bits, SEED, *self.lam, **self.kw)

    def check(self):
        want, tol = self.want()
        got = host(self.run()).astype(np.float64)
        # the transform back: 12 binary32 roundings
        err, bound = np.linalg.norm(got - want, axis=-1), tol + 2.0 ** -20 * np.linalg.norm(want, axis=-1)
        assert np.isfinite(got).all()
        assert (err <= bound).all(), np.max(err / np.maximum(bound, 1e-30))


CASES = {
    "one_draft": dict(lens=[100, 1, 33], q_lens=[1, 1, 1]),
    "few_rows": dict(lens=[200, 130, 9], q_lens=[4, 3, 4], group=4),
    "few_rows_8bit_cap": dict(lens=[257, 640], q_lens=[5, 2], heads=3, group=1, page=32, bits=8, softcap=20.0),
    "eight_drafts": dict(lens=[301], q_lens=[8], group=4),
    "sixteen": dict(lens=[200, 77], q_lens=[16, 9], group=1),
    "drafts_alone": dict(lens=[8, 20, 64], q_lens=[8, 20, 64]),
    "more_drafts_than_tokens": dict(lens=[2, 0, 1, 30], q_lens=[4, 3, 1, 40], group=3),
    "mid": dict(lens=[400, 300], q_lens=[13, 13], group=2, lam=True),
    "mid_window": dict(lens=[400, 50], q_lens=[30, 30], group=2, window=23),
    "window_of_drafts": dict(lens=[300, 200], q_lens=[40, 8], group=1, window=2),
    "window_one": dict(lens=[90, 200], q_lens=[5, 33], group=2, window=1),
    "window_few": dict(lens=[700, 31], q_lens=[4, 4], window=33, page=128),
    "tile_128": dict(lens=[350, 260, 700], q_lens=[40, 1, 33], heads=1, group=3, page=64),
    "tile_256": dict(lens=[900, 140], q_lens=[130, 7], heads=1, group=2, page=32, lam=True),
    "all_256": dict(lens=[600], q_lens=[256], heads=1, group=1, page=64, bits=8),
    "tiles": dict(lens=[530], q_lens=[200], heads=1, group=4, page=16, bits=8, window=100),
    "splits": dict(lens=[1300, 2700], q_lens=[9, 20], heads=1, group=2, page=64),
    "splits_few": dict(lens=[3300, 700], q_lens=[7, 8], heads=1, group=2, page=64),
    "splits_window": dict(lens=[3300, 1700], q_lens=[20, 8], heads=1, group=2, page=64, window=1500),
    "cap_many": dict(lens=[260], q_lens=[100], heads=2, group=1, softcap=15.0, bits=8, page=256),
    "mixed": dict(lens=[300, 77, 150, 400], q_lens=[130, 1, 8, 129], heads=1, group=2, page=32),
    "odd_group": dict(lens=[300, 277], q_lens=[11, 5], heads=2, group=7, page=32),
    "group_8": dict(lens=[500, 277], q_lens=[7, 64], heads=1, group=8, page=32),
    "negative_scale": dict(lens=[70, 64], q_lens=[3, 30], scale=-0.11),
}


@pytest.mark.parametrize("name", CASES)
def test_against_definition(orc, name):
    say(f"case: tree {name} {CASES[name]}")
    Case(orc, **CASES[name]).check()


@pytest.mark.parametrize("lens,m,group", [([200, 150], 8, 2), ([400, 300], 60, 2), ([300, 1100], 17, 1), ([300, 2000], 17, 4)])
def test_a_chain_is_causal(orc, lens, m, group):
    """Drafts that follow one another see what causal queries see; all of them on the held tokens, those and themselves."""
    say(f"case: tree chain {lens} {m}")
    for window in (0, 25):
        c = Case(orc, lens, [m, m], group=group, window=window, trees=[list(range(-1, m - 1))] * 2)
        c.check()
        # kv_reference's causal attention is another definition of the same
        want, tol, _, _ = kv_reference.attend(orc, host(c.cache), c.q, c.table, c.lens, c.q_lens, c.bits, SEED, window=window)
        err = np.linalg.norm(host(c.run()).astype(np.float64) - want, axis=-1)
        assert (err <= tol + 2.0 ** -20 * np.linalg.norm(want, axis=-1)).all()
    Case(orc, lens, [m, m], group=group, trees=[[-1] * m] * 2).check()


def test_parents_out_of_range(orc):
    """A parent that is not before its draft counts as none."""
    say("case: tree bad parents")
    for m in (5, 40):
        c = Case(orc, [150], [m], trees=[[-1, 0, 1, 2, 3] + [3] * (m - 5)])
        c.parents[:5] = [0, 0, 1, 7, -(1 << 31)]
        c.trees = [c.parents.tolist()]
        c.parents[m - 1] = c.trees[0][m - 1] = (1 << 31) - 1
        c.sees = [ref.tree_sees(c.trees[0], 150, m)]
        assert not c.sees[0][3, 150 - m:150 - m + 3].any()
        c.check()


@pytest.mark.parametrize("name", ["few_rows", "mid", "tile_128", "splits", "splits_few"])
def test_types_strides_and_repeats(orc, name):
    say(f"case: tree types and strides {name}")
    c = Case(orc, **CASES[name])
    q = dev(c.q).to(torch.bfloat16)
    first = c.run(q)
    assert torch.equal(c.run(q.float()), first) and torch.equal(c.run(q, out_dtype=torch.bfloat16), first.to(torch.bfloat16))
    row = torch.full((q.shape[0], 2 * q.shape[1] * 128 + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    for off in (0, 1, 8):
        view = row[:, off:off + q.shape[1] * 128].unflatten(1, (q.shape[1], 128))
        view.copy_(q)
        assert torch.equal(c.run(view), first)
    assert torch.equal(c.run(q.transpose(0, 1).contiguous().transpose(0, 1)), first)


@pytest.mark.parametrize("group,m", [(2, 3), (2, 13), (2, 40), (1, 140)])
def test_absent_pages_and_nan_vectors(orc, group, m):
    """Absent pages hide their tokens, drafts among them; a vector that was not finite reaches the drafts that see it alone."""
    say(f"case: tree absent pages and NaN, group {group}, {m} drafts")
    c = Case(orc, [190, 170], [m, m], heads=2, group=group)
    c.table[0, 2], c.table[0, 11], c.table[1, 0] = -1, c.cache.shape[0], 1 << 30
    c.check()
    clean = host(c.run())
    bad = 170 - m + m // 2  # a draft of the second sequence
    for side in range(2):
        slot = dev(np.array([c.table[1, bad // 16] * 16 + bad % 16], np.int64))
        held = c.cache.clone()
        pair = list(hq.hq_kv_read(c.cache, slot, out_dtype=torch.float32, **c.fmt))
        pair[side][:, 1] = float("nan")
        hq.hq_kv_append(c.cache, *pair, slot, **c.fmt)
        got, sees = host(c.run()), c.sees[1][:, bad]
        assert sees.any() and np.isnan(got[m:, group:][sees]).all()
        got[m:, group:][sees] = clean[m:, group:][sees]
        # the other side's vector was written again, from what it decodes to
        assert np.isfinite(got).all()
        c.cache = held
    assert np.array_equal(host(c.run()), clean)


def test_offsets_and_cuts(orc):
    say("case: tree offsets")
    c = Case(orc, [100, 100, 100], [6, 6, 6], heads=1, group=2)
    full = c.run()
    assert torch.equal(c.run(q_start=None, max_q=None, max_len=None), full)
    out = c.run(max_q=2)
    assert torch.isnan(out[2:6]).all() and torch.equal(out[:2], full[:2]) and torch.equal(out[6:8], full[6:8])
    out = c.run(q_start=dev(np.array([-5, 6, 6, 999], np.int32)))
    assert torch.equal(out[:6], full[:6])
    c.lens = [100, 1 << 30, -4]
    out = c.run(max_len=100)
    assert torch.equal(out[:12], full[:12]) and not out[12:].any()


def test_streams_and_graphs(orc):
    """A step of drafts (append, attend, accept) captured and replayed on other inputs gives what the eager calls give."""
    say("case: tree graph")
    c = Case(orc, [120, 90], [9, 9], heads=2, group=2)
    eager = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=side)
    side.synchronize()
    assert torch.equal(got, eager)
    q, table, lens, parents = dev(c.q), dev(c.table), dev(np.array(c.lens, np.int32)), dev(c.parents)
    k, v = (torch.randn(18, 2, 128, device="cuda") for _ in range(2))
    slots = dev(np.array([c.table[b, t // 16] * 16 + t % 16 for b, n in enumerate(c.lens) for t in range(n - 9, n)], np.int64))
    tokens, target = (torch.zeros(18, dtype=torch.int32, device="cuda") for _ in range(2))

    def step(cache):
        hq.hq_kv_append(cache, k, v, slots, **c.fmt)
        out = hq.hq_kv_attend(cache, q, table, lens, parents=parents, max_len=120, **c.fmt)
        return (out, *hq.hq_kv_accept(cache, table, lens, tokens, target, parents))

    one, two = c.cache.clone(), c.cache.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(one)
    one.copy_(c.cache)
    g = np.random.default_rng(5)
    for i in range(4):
        for x in (k, v, q):
            x.normal_()
        parents.copy_(torch.tensor(some_tree(g, 9) + some_tree(g, 9), dtype=torch.int32))
        tokens.copy_(torch.from_numpy(g.integers(0, 3, 18).astype(np.int32)))
        target.copy_(torch.from_numpy(g.integers(0, 3, 18).astype(np.int32)))
        graph.replay()
        want = step(two)
        assert all(torch.equal(a, b) for a, b in zip(held, want)) and torch.equal(one, two)


def test_refusals(orc):
    say("case: tree refuses")
    cache = hq.hq_kv_cache(4, 2)
    q = torch.zeros(2, 4, 128, device="cuda", dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(cache=cache, q=q, table=i32(2, 1), lens=i32(2), parents=i32(2))
    hq.hq_kv_attend(**good)
    for bad in (dict(parents=i32(3)), dict(parents=i32(2).long()), dict(parents=i32(2).cpu()), dict(causal=False), dict(max_q=257),
                dict(weights=torch.zeros(2, 2, 64, device="cuda"))):
        with pytest.raises(ValueError):
            hq.hq_kv_attend(**good | bad)
    ok = dict(cache=cache, table=i32(2, 1), lens=i32(2), tokens=i32(4), target=i32(4), parents=i32(4))
    hq.hq_kv_accept(**ok)
    for bad in (dict(lens=i32(2).long()), dict(table=i32(3, 1)), dict(target=i32(3)), dict(parents=i32(4).long()), dict(max_q=257), dict(q_start=i32(2)),
                dict(max_q=-1), dict(path=i32(2, 3)), dict(change=i32(3))):
        with pytest.raises(ValueError):
            hq.hq_kv_accept(**ok | bad)
    with pytest.raises(hq.HqError):  # not as many drafts each
        hq.hq_kv_accept(**ok | dict(tokens=i32(3), target=i32(3), parents=i32(3)))


# ---- acceptance --------------------------------------------------------------------------------


def accept_case(g, lens, q_lens, vocabulary):
    trees = [some_tree(g, m) for m in q_lens]
    return trees, [g.integers(0, vocabulary, m).tolist() for m in q_lens], [g.integers(0, vocabulary, m).tolist() for m in q_lens]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("lens,q_lens,vocabulary", [
    ([40], [1], 2), ([40, 17, 90], [8, 8, 8], 2), ([100, 65], [64, 65], 1), ([300, 256, 2], [256, 100, 0], 2), ([50] * 20, [11] * 20, 3),
    ([64, 130], [30, 63], 1),
])
def test_accept(lens, q_lens, vocabulary, page, bits):
    """Paths, counts and every byte of the cache: chains over pages' ends, whole trees, drafts that are all the tokens."""
    say(f"case: accept {lens} {q_lens}, page {page}, {bits} bits")
    g = np.random.default_rng(sum(lens) + page)
    heads, used = 3, [-(-n // page) for n in lens]
    pages = sum(used) + 1
    cache = torch.randint(0, 256, hq.hq_kv_cache(pages, heads, page, bits).shape, dtype=torch.uint8, device="cuda")
    order = g.permutation(pages).astype(np.int32)
    table, at = np.full((len(lens), max(used)), -1, np.int32), 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    trees, tokens, target = accept_case(g, lens, q_lens, vocabulary)
    flat = lambda x: dev(np.array(sum(x, []), np.int32))  # noqa: E731
    start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    want = host(cache).copy()
    paths = [ref.accept_path(*x) for x in zip(tokens, target, trees)]
    for b, p in enumerate(paths):
        ref.move(want, bits, table[b], lens[b], q_lens[b], p, page)
    path, accepted, nxt, change = (host(x) for x in hq.hq_kv_accept(cache, dev(table), dev(np.array(lens, np.int32)), flat(tokens), flat(target), flat(trees),
                                                                     q_start=dev(start), max_q=max(q_lens), bits=bits))
    for b, p in enumerate(paths):
        assert path[b].tolist() == p + [-1] * (max(q_lens) - len(p)) and accepted[b] == len(p) and change[b] == len(p) - q_lens[b]
        assert nxt[b] == (target[b][p[-1]] if p else -1)
    assert np.array_equal(host(cache), want)


def test_accept_ties_absent_pages_and_cuts():
    """The first of two equal children; absent pages at either end; bad parents; more drafts than tokens; max_q."""
    say("case: accept edges")
    page, bits, heads = 16, 4, 2
    cache = torch.randint(0, 256, hq.hq_kv_cache(12, heads, page, bits).shape, dtype=torch.uint8, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tree, tok, tgt = [-1, 0, 0, 2, 2, 4, 9, -7], [9, 5, 7, 7, 7, 8, 8, 8], [7, 7, 7, 1, 8, 3, 8, 8]
    assert ref.accept_path(tok, tgt, tree) == [0, 2, 3]
    for table, n in (([0, 1, 2], 40), ([0, -1, 2], 36), ([3, 5, 99], 35), ([4, 6, 7], 3), ([4, 6, 7], 0), ([8, 9, 10], 1000)):
        want = host(cache).copy()
        held = min(n, 48)
        ref.move(want, bits, table, held, 8, [0, 2, 3], page)
        out = hq.hq_kv_accept(cache, i32(*table).view(1, 3), i32(n), i32(*tok), i32(*tgt), i32(*tree))
        assert [x.tolist() for x in out] == [[[0, 2, 3, -1, -1, -1, -1, -1]], [3], [1], [-5]]
        assert np.array_equal(host(cache), want)
    before = cache.clone()
    out = hq.hq_kv_accept(cache, i32(0, 1, 2).view(1, 3), i32(40), i32(*tok), i32(*tgt), i32(*tree), max_q=2)
    assert [x.tolist() for x in out] == [[[0, -1]], [1], [7], [-7]] and torch.equal(cache, before)
    out = hq.hq_kv_accept(cache, i32(0, 1, 2).view(1, 3), i32(40), i32(), i32(), i32())
    assert [x.tolist() for x in out] == [[[]], [0], [-1], [0]] and torch.equal(cache, before)
    none = cache[:0]
    out = hq.hq_kv_accept(none, i32(0, 1, 2).view(1, 3), i32(40), i32(*tok), i32(*tgt), i32(*tree))
    assert out[1].tolist() == [3]


# ---- operands through LDS ------------------------------------------------------------------------

WORK = 1 << 24  # rows x tokens from which operands go through LDS


@pytest.mark.parametrize("name", ["mid", "tile_128", "tile_256", "all_256", "tiles", "cap_many", "mixed", "group_8", "splits", "more_drafts_than_tokens"])
def test_much_work(orc, name):
    """The kernels for much work, which max_len announces, on the same inputs; whole and in splits."""
    say(f"case: tree through LDS, {name}")
    kw = dict(CASES[name])
    if kw.pop("window", 0):
        kw["lens"] = [1200]
    c = Case(orc, **kw)
    rows = len(c.lens) * c.cache.shape[1] * max(c.q_lens) * c.q.shape[1] // c.cache.shape[1]
    want, tol = c.want()
    bound = tol + 2.0 ** -20 * np.linalg.norm(want, axis=-1)
    for max_len in (WORK // rows + 600, 1 << 24):  # more than WORK; the second: one split holds all
        got = c.run(max_len=max_len)
        err = np.linalg.norm(host(got).astype(np.float64) - want, axis=-1)
        assert np.isfinite(host(got)).all() and (err <= bound).all(), np.max(err / np.maximum(bound, 1e-30))
        assert torch.equal(c.run(max_len=max_len), got)


def test_much_work_window(orc):
    """A window's edge in the kernels for much work, against those for little: the same operands, so rows differ by the weights'
    roundings, 2 2^-11 in either, and by the order of sums (below 2^-10 for scores up to 64): 2^-8 of the longest value."""
    say("case: tree through LDS, window")
    c = Case(orc, [5000], [64], heads=8, group=8, window=4500, page=64)
    assert 8 * 512 * (4500 + 64 + 15) > WORK >= 8 * 64 * 4600
    slots = dev(np.array([c.table[0, t // 64] * 64 + t % 64 for t in range(5000)], np.int64))
    longest = float(hq.hq_kv_read(c.cache, slots, out_dtype=torch.float32, **c.fmt)[1].norm(dim=-1).max())
    much, little = c.run(), c.run(max_q=8)
    assert torch.isfinite(much).all() and float((much[:8] - little[:8]).norm(dim=-1).max()) <= 2.0 ** -8 * longest


@pytest.mark.parametrize("group,m", [(2, 20), (2, 40), (1, 140)])
def test_much_work_absent_pages_and_nan(orc, group, m):
    say(f"case: tree through LDS, absent pages and NaN, group {group}, {m} drafts")
    c = Case(orc, [190, 170], [m, m], heads=2, group=group)
    c.table[0, 2], c.table[0, 11], c.table[1, 0] = -1, c.cache.shape[0], 1 << 30
    want, tol = c.want()
    clean = host(c.run(max_len=1 << 24))
    assert (np.linalg.norm(clean - want, axis=-1) <= tol + 2.0 ** -20 * np.linalg.norm(want, axis=-1)).all()
    bad = 170 - m + m // 2
    slot = dev(np.array([c.table[1, bad // 16] * 16 + bad % 16], np.int64))
    for side in range(2):
        held = c.cache.clone()
        pair = list(hq.hq_kv_read(c.cache, slot, out_dtype=torch.float32, **c.fmt))
        pair[side][:, 1] = float("nan")
        hq.hq_kv_append(c.cache, *pair, slot, **c.fmt)
        got, sees = host(c.run(max_len=1 << 24)), c.sees[1][:, bad]
        assert np.isnan(got[m:, group:][sees]).all()
        got[m:, group:][sees] = 0
        assert np.isfinite(got).all()
        c.cache = held
