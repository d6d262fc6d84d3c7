"""GPU: attention over the paged SRFT cache at the edges of what a call may ask: fewer queries computed than a sequence has,
small and large cached values, batches that are mostly single tokens,
tokens that an eviction kept without having them, and scores of any size.

Bounds are kv_reference.attend's; cases are those of test_gpu_kv_attend."""
import numpy as np
import pytest

import kv_reference as ref

torch = pytest.importorskip("torch")
hq = pytest.importorskip("kv_quantization_tile_amd")

from test_gpu_kv_attend import SEED, Case, dev, host, say  # noqa: E402

pytestmark = pytest.mark.gpu


def within(got, want, tol):
    """Rows of outputs against the definition, with the transform back's 12 binary32 roundings."""
    err = np.linalg.norm(got.astype(np.float64) - want, axis=-1)
    bound = tol + 2.0 ** -20 * np.linalg.norm(want, axis=-1)
    assert np.isfinite(got).all() and (err <= bound).all(), np.max(err / np.maximum(bound, 1e-30))


@pytest.mark.parametrize("lens,q_lens,group,max_q,kw", [
    ([120, 90], [2, 2], 2, 1, {}),
    ([120, 90, 4], [6, 5, 9], 2, 5, dict(window=33)),
    ([300, 260], [40, 33], 2, 5, dict(page=64)),                # few rows of sequences with many
    ([300, 260], [40, 33], 2, 20, dict(bits=8)),
    ([700, 400], [150, 1], 2, 140, dict(window=77, lam=True)),  # single tokens beside cut chunks
    ([300, 260], [30, 30], 3, 7, dict(causal=False)),
    ([300, 260], [30, 30], 3, 2, dict(causal=False, window=20)),
])
def test_fewer_queries_than_a_sequence_has(orc, lens, q_lens, group, max_q, kw):
    """The first max_q queries of a sequence stand where they stand among all of them; the others are not written, and
    add no weight."""
    say(f"case: attend {q_lens} queries on {lens} tokens, max_q {max_q}, {kw}")
    c = Case(orc, lens, q_lens, heads=2, group=group, **kw)
    for precise in (False, True):
        want, tol, _, _ = c.want(precise)
        w = torch.zeros(len(lens), 2, max(lens), device="cuda") if precise else None
        forms = [c.run(weights=w, max_q=max_q)]
        if len(set(q_lens)) == 1 and not precise:
            forms.append(c.run(q_start=None, max_q=max_q))
        first = np.concatenate([np.arange(m) < max_q for m in q_lens])
        for out in map(host, forms):
            within(out[first], want[first], tol[first])
            assert np.isnan(out[~first]).all()
    if not c.kw["causal"]:
        return
    # causal, the computed queries are all the queries of a sequence that ends with them
    cut = [max(m - max_q, 0) for m in q_lens]
    _, _, ww, wtol = ref.attend(orc, host(c.cache), c.q[first], c.table, [max(n - x, 0) for n, x in zip(lens, cut)],
                                [m - x for m, x in zip(q_lens, cut)], c.bits, SEED, *c.lam, precise=True, **c.kw)
    got = host(w).astype(np.float64)
    top = ww.shape[2]
    assert (np.abs(got[..., :top] - ww) <= wtol + 2.0 ** -23 * ww).all() and not got[..., top:].any()


class Scaled(Case):
    """A case whose keys and values are taken times `k` and `v` (numbers, or one per slot), with the scores' scale undoing
    the largest of `k`."""

    def __init__(self, orc, *a, k, v, **kw):
        super().__init__(orc, *a, **kw)
        slots = torch.arange(self.cache.shape[0] * kw.get("page", 16), device="cuda")
        old = hq.hq_kv_read(self.cache, slots, out_dtype=torch.float32, **self.fmt)
        new = [x * dev(np.full(slots.shape, f, np.float32))[:, None, None] for x, f in zip(old, (k, v))]
        hq.hq_kv_append(self.cache, *new, slots, **self.fmt)
        self.scale = float(128 ** -0.5 / np.max(k))


SHAPES = {"single": dict(lens=[300, 77], q_lens=[1, 1], group=4), "many": dict(lens=[150, 200], q_lens=[40, 33], group=2),
          "tile_256": dict(lens=[300, 40], q_lens=[130, 1], heads=1, group=2, page=32)}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("size", [1e-1, 1e-2, 1e-3, 1e-4, 1e-5])
def test_small_values(orc, size, bits, shape):
    """Operands are off by half a step of binary16 however small the cached vectors are: the bounds are those of unit ones."""
    say(f"case: attend over values of {size}, {bits} bits, {shape}")
    Scaled(orc, bits=bits, k=size, v=size, **SHAPES[shape]).check()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("which", ["keys", "values", "both", "some"])
def test_large_values(orc, which, bits, shape):
    """Scales up to the largest there are (65504), everywhere or at one token in ten: nothing overflows, bounds as ever."""
    say(f"case: attend over large {which}, {bits} bits, {shape}")
    page = SHAPES[shape].get("page", 16)
    slots = (sum(-(-n // page) for n in SHAPES[shape]["lens"]) + 2) * page
    g = np.random.default_rng(5)
    some = [np.where(g.random(slots) < 0.1, 1e7, 1.0) for _ in range(2)]
    k, v = {"keys": (1e7, 1), "values": (1, 1e7), "both": (1e7, 1e7), "some": some}[which]
    c = Scaled(orc, bits=bits, k=k, v=v, **SHAPES[shape])
    _, ks, _, vs = ref.parts(host(c.cache), bits)
    assert max(ks.max(), vs.max()) == 65504
    c.check()
    c.kw["softcap"] = 20.0
    c.check()


@pytest.mark.parametrize("shape", SHAPES)
def test_large_scales_past_a_length(orc, shape):
    """What lies past a length in its last page, the largest scales there are, leaves small values before it as exact."""
    say(f"case: attend beside stale large scales, {shape}")
    c = Scaled(orc, bits=8, k=1e-4, v=1e-4, **SHAPES[shape])
    w = [torch.zeros(len(c.lens), c.cache.shape[1], max(c.lens), device="cuda") for _ in range(2)]
    want = c.run(), c.run(weights=w[0])
    stale = host(c.cache)
    _, ks, vc, vs = ref.parts(stale, 8)
    page = ks.shape[2]
    for b, n in enumerate(c.lens):
        for t in range(n, -(-n // page) * page):
            pg = c.table[b, t // page]
            ks.view(np.uint16)[pg, :, t % page] = vs.view(np.uint16)[pg, :, t % page // 4, :, t % page % 4] = 0x7BFF
    c.cache = dev(stale)
    assert torch.equal(c.run(), want[0]) and torch.equal(c.run(weights=w[1]), want[1]) and torch.equal(*w)


def mixture(seed, seqs, long):
    """Lengths and query counts of a continuous batch: mostly single tokens, some sequences idle, a few chunks."""
    g = np.random.default_rng(seed)
    m = g.choice([0, 1, 1, 1, 1, 5, 17, 40], seqs)
    m[g.integers(seqs)] = long
    lens = m + g.integers(0, 200, seqs)
    lens[g.integers(seqs)] = 1400
    return lens.tolist(), m.tolist()


@pytest.mark.parametrize("seed,seqs,long,kw", [
    (1, 9, 150, dict(heads=2, group=2)),
    (2, 70, 90, dict(heads=1, group=4, page=64)),       # more sequences than a wavefront looks at together
    (3, 130, 33, dict(heads=1, group=1, bits=8, page=32)),
    (4, 12, 300, dict(heads=1, group=3, window=70)),
    (5, 5, 140, dict(heads=3, group=2, softcap=20.0, lam=True)),
    (6, 300, 70, dict(heads=1, group=2, causal=False, page=128)),
])
def test_continuous_batches(orc, seed, seqs, long, kw):
    say(f"case: attend a continuous batch of {seqs} sequences, a chunk of {long}, {kw}")
    lens, m = mixture(seed, seqs, long)
    c = Case(orc, lens, m, **kw)
    c.check()
    bounded = c.run()
    # without bounds on queries or lengths: another cut of the same work
    want, tol, _, _ = c.want()
    within(host(c.run(max_q=None, max_len=None)), want, tol)
    within(host(bounded), want, tol)


def test_many_sequences_beside_a_chunk_of_32768():
    """Each sequence's rows are those of the sequence alone, bit for bit (lengths of one split)."""
    say("case: attend 255 single tokens and a chunk of 32768 queries, 8 heads")
    seqs, heads, group, page, chunk = 256, 8, 4, 64, 32768
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    lens = torch.randint(1, 400, (seqs,), generator=g, device="cuda").to(torch.int32)
    lens[77] = 410
    used = [-(-n // page) for n in lens.tolist()]
    cache = hq.hq_kv_cache(sum(used), heads, page)
    slots = torch.arange(sum(used) * page, device="cuda")
    k, v = (torch.randn(slots.numel(), heads, 128, generator=g, device="cuda") for _ in range(2))
    hq.hq_kv_append(cache, k, v, slots)
    first = np.concatenate([[0], np.cumsum(used)[:-1]])
    table = dev((first[:, None] + np.arange(max(used))).astype(np.int32))
    m = np.ones(seqs, np.int64)
    m[77] = chunk
    start = np.concatenate([[0], np.cumsum(m)]).astype(np.int32)
    q = torch.randn(int(start[-1]), heads * group, 128, generator=g, device="cuda").bfloat16()
    for max_q in (chunk, None):
        out = hq.hq_kv_attend(cache, q, table, lens, q_start=dev(start), max_q=max_q, max_len=410)
        a, b = int(start[77]), int(start[78])
        assert torch.equal(out[a:b], hq.hq_kv_attend(cache, q[a:b], table[77:78], lens[77:78], max_len=410))
        assert not out[a:b - 410].any() and bool(out[b - 410:b].any(-1).all())
        alone = hq.hq_kv_attend(cache, torch.cat([q[:a], q[b:]]), torch.cat([table[:77], table[78:]]), torch.cat([lens[:77], lens[78:]]), max_len=410)
        assert torch.equal(torch.cat([out[:a], out[b:]]), alone)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("group,m", [(2, 1), (2, 40), (2, 140)])
def test_absent_tokens_that_an_eviction_keeps(orc, monkeypatch, group, m, bits):
    """Tokens of absent pages that stay (first, last or within the budget) take no part after the move either, whatever their
    new slots held, nor after a second move."""
    say(f"case: attend after an eviction that keeps absent tokens, group {group}, {m} queries, {bits} bits")
    c = Case(orc, [250, 230], [m, m], heads=2, group=group, bits=bits)
    c.table[0, 0] = c.table[0, 7] = c.table[1, 3] = c.table[1, 14] = -1
    pages, want_pages, budget = c.cache.shape[0], 12, 180
    cache = torch.cat([c.cache, c.cache[torch.randint(0, pages, (48,), device="cuda")]])  # fresh pages hold other tokens
    lens = dev(np.array(c.lens, np.int32))
    weights = torch.rand(2, 2, 250, device="cuda")
    dst = pages + np.arange(24, dtype=np.int32).reshape(2, 12)
    kept, left, wk = hq.hq_kv_evict(cache, dev(c.table), lens, weights, budget, 20, 30, dev(dst), bits=bits)
    assert left.tolist() == [budget, budget]
    old = [[ref.coordinates(host(c.cache), bits, c.table[b], c.lens[b], h, np.ones(128), np.ones(128)) for h in range(2)] for b in range(2)]

    def moved(kept):
        def of(_, __, row, n, head, ___, ____):
            k, v, there = old[row][head]
            at = kept[row, head, :n]
            return k[at], v[at], there[at]
        return of

    kh = host(kept)
    assert any(not old[b][h][2][kh[b, h]].all() for b in range(2) for h in range(2))
    second = pages + 24 + np.arange(24, dtype=np.int32).reshape(2, 12)
    kept2, left2, _ = hq.hq_kv_evict(cache, dev(dst), left, wk, 150, 20, 30, dev(second), bits=bits)
    kh2 = np.take_along_axis(kh, host(kept2), 2)
    for table, n, index in ((dst, budget, kh), (second, 150, kh2)):
        monkeypatch.setattr(ref, "coordinates", moved(index))
        for precise in (False, True):
            want, tol, ww, wtol = ref.attend(orc, cache, c.q, [0, 1], [n, n], [m, m], bits, SEED, scale=c.scale, precise=precise)
            w = torch.zeros(2, 2, n, device="cuda") if precise else None
            out = torch.full(c.q.shape, float("nan"), device="cuda")
            hq.hq_kv_attend(cache, dev(c.q), dev(table), torch.full_like(left, n), max_len=n, bits=bits, seed=SEED, weights=w, out=out)
            within(host(out), want, tol)
            if precise:
                got = host(w).astype(np.float64)
                assert (np.abs(got - ww) <= wtol + 2.0 ** -23 * ww).all()
                assert all((got[b, h][~old[b][h][2][index[b, h]]] == 0).all() for b in range(2) for h in range(2))
    slots = dev((dst[0, 0] * 16 + np.arange(16)).astype(np.int64))  # the first tokens of the first sequence were absent
    assert not any(x.any() for x in hq.hq_kv_read(cache, slots, bits=bits, seed=SEED))


@pytest.mark.parametrize("m", [1, 40, 140])
def test_large_scores_pick_one_token(orc, m):
    """Where the best score of a row leads by more than its error allows, the row is that token's value."""
    say(f"case: attend with scores of thousands, {m} queries")
    c = Case(orc, [256, 190], [m, m], heads=1, group=2)
    c.q *= 1000
    T = ref.transform(orc, SEED)
    runs = [host(c.run()), host(c.run(weights=torch.zeros(2, 1, 256, device="cuda")))]
    rows = 0
    for b, n in enumerate(c.lens):
        k, v, _ = ref.coordinates(host(c.cache), 4, c.table[b], n, 0, np.ones(128), np.ones(128))
        for i in range(m):
            for j in range(2):
                seen = n - m + i + 1
                y = c.q[b * m + i, j].astype(np.float64) @ T.T * c.scale
                s, size = k[:seen] @ y, (np.abs(k[:seen]) @ np.abs(y)).max()
                best = int(np.argmax(s))
                lead = s[best] - np.max(np.delete(s, best))
                # scores are off by (2^-10 + 2^-17) of their sum of magnitudes; e^-20 of 256 others is below 2^-20
                if lead <= 2 * (2.0 ** -10 + 2.0 ** -17) * size + 20:
                    continue
                rows += 1
                for out in runs:
                    want = v[best] @ T
                    assert np.linalg.norm(out[b * m + i, j] - want) <= (3 * 2.0 ** -11 + 2.0 ** -17) * np.linalg.norm(v[best])
    assert rows >= m  # of 4 m


@pytest.mark.parametrize("m", [1, 40, 140])
@pytest.mark.parametrize("size", [-1e3, -1e28, -1e34, 1e34])
def test_scores_far_from_zero(orc, size, m):
    """Equal scores of any size, far below zero too, average the values that a row sees."""
    say(f"case: attend with scores about {size}, {m} queries")
    c = Case(orc, [150, 190], [m, m], heads=1, group=2)
    slots = torch.arange(c.cache.shape[0] * 16, device="cuda")
    key = torch.ones(slots.numel(), 1, 128, device="cuda")
    v = hq.hq_kv_read(c.cache, slots, out_dtype=torch.float32, **c.fmt)[1]
    hq.hq_kv_append(c.cache, key, v, slots, **c.fmt)
    c.q[:] = size
    T = ref.transform(orc, SEED)
    for w in (None, torch.zeros(2, 1, 190, device="cuda")):
        got = host(c.run(weights=w))
        for b, n in enumerate(c.lens):
            _, v, _ = ref.coordinates(host(c.cache), 4, c.table[b], n, 0, np.ones(128), np.ones(128))
            for i in range(m):
                v_seen = v[:n - m + i + 1]
                want = v_seen.mean(0) @ T
                bound = (3 * 2.0 ** -11 + 2.0 ** -17) * np.linalg.norm(np.abs(v_seen).mean(0))
                assert (np.linalg.norm(got[b * m + i] - want, axis=-1) <= bound).all()


@pytest.mark.parametrize("softcap", [2.0 ** -125, 1e-20, 1e20, 2.0 ** 125])
@pytest.mark.parametrize("m", [1, 40])
def test_caps_of_any_size(orc, m, softcap):
    """A cap far above the scores leaves them, one far below makes them equal; one that binary32 cannot hold is refused."""
    say(f"case: attend with a cap of {softcap}, {m} queries")
    c = Case(orc, [150, 190], [m, m], heads=1, group=2, softcap=softcap)
    if softcap > 1:
        c.kw["softcap"] = 0.0
    want, tol, _, _ = c.want()
    c.kw["softcap"] = softcap
    within(host(c.run()), want, tol)
    for kw in (dict(softcap=3e38), dict(softcap=1e-39), dict(scale=3e38)):
        with pytest.raises(hq.HqError):
            c.run(**kw)
