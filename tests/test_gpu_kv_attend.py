"""GPU: attention over the paged SRFT cache against its definition in binary64.

kv_reference.attend gives, with each output row, the error that the kernel's roundings may make (derived there from half
steps of binary16 and binary32).  Masks are tested where a mistake shows: every query looks for the keys just
inside and just outside what it may see, so one token too many or too few moves its row by far more than that."""
import numpy as np
import pytest

import kv_reference as ref

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


class Case:
    """A filled cache, a table over shuffled pages and queries that look for tokens at the edges of what they see."""

    def __init__(self, orc, lens, q_lens, heads=2, group=2, page=16, bits=4, causal=True, window=0, softcap=0.0, lam=False,
                 scale=None, f32=True, seed=0):
        g = np.random.default_rng(1000 + seed)
        self.orc, self.lens, self.q_lens, self.bits = orc, lens, q_lens, bits
        self.kw = dict(causal=causal, window=window, softcap=softcap)
        self.scale = 128 ** -0.5 if scale is None else scale
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
        total, hq_heads = sum(q_lens), heads * group
        q = g.standard_normal((total, hq_heads, 128)).astype(np.float32)
        kh = host(k)
        at = 0
        for b, (n, m) in enumerate(zip(lens, q_lens)):
            for i in range(m):
                pos = n - m + i
                for t in (pos, pos + 1, pos - window, pos - window + 1) if window else (pos, pos + 1, n - 1):
                    if 0 <= t < n:
                        at_slot = self.table[b, t // page] * page + t % page
                        q[at + i] += 0.4 * np.repeat(kh[at_slot], group, 0)
            at += m
        if not f32:
            q = dev(q).to(torch.bfloat16).float().cpu().numpy()
        self.q = q
        self.start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)

    def run(self, q=None, weights=None, out_dtype=torch.float32, **kw):
        q = dev(self.q) if q is None else q
        out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
        a = dict(q_start=dev(self.start), max_q=max(self.q_lens), max_len=max(self.lens), weights=weights, out=out, scale=self.scale,
                 **self.kw, **self.fmt) | kw
        return hq.hq_kv_attend(self.cache, q, dev(self.table), dev(np.array(self.lens, np.int32)), **a)

    def want(self, precise=False):
        return ref.attend(self.orc, host(self.cache), self.q, self.table, self.lens, self.q_lens, self.bits, SEED, *self.lam,
                          scale=self.scale, precise=precise, **self.kw)

    def check(self, weights=True):
        """Outputs, with and without the weights, against the definition; then the weights."""
        for precise in (False, True) if weights else (False,):
            want, tol, ww, wtol = self.want(precise)
            w = None
            if precise:
                w0 = np.random.default_rng(3).random((len(self.lens), self.cache.shape[1], max(self.lens) + 5)).astype(np.float32)
                w = dev(w0)
            got = host(self.run(weights=w)).astype(np.float64)
            # the transform back: 12 binary32 roundings
            err, bound = np.linalg.norm(got - want, axis=-1), tol + 2.0 ** -20 * np.linalg.norm(want, axis=-1)
            assert np.isfinite(got).all()
            assert (err <= bound).all(), (precise, np.max(err / np.maximum(bound, 1e-30)))
            if precise:
                top = max(self.lens)
                wg = host(w).astype(np.float64)
                # the sum with what was there is rounded once
                bound = wtol + 2.0 ** -23 * (w0[..., :top] + ww)
                assert (np.abs(wg[..., :top] - w0[..., :top] - ww) <= bound).all()
                assert np.array_equal(host(w)[..., top:], w0[..., top:])
                for b, n in enumerate(self.lens):
                    assert np.array_equal(host(w)[b, :, n:], w0[b, :, n:])


CASES = {
    # single tokens: lengths about a block, a split and a page; an empty sequence
    "single_short": dict(lens=[1, 15, 16, 17, 0, 33], q_lens=[1] * 6),
    "single_long": dict(lens=[300, 1, 1111], q_lens=[1] * 3, heads=1, group=7, page=64, lam=True),
    "single_8bit_cap": dict(lens=[257, 640], q_lens=[1] * 2, heads=3, group=1, page=32, bits=8, softcap=20.0),
    "single_window": dict(lens=[700, 31, 5], q_lens=[1] * 3, window=33, page=128),
    "few_rows": dict(lens=[200, 130], q_lens=[4, 2], group=4, bits=8, lam=True),
    "more_queries_than_tokens": dict(lens=[2, 0, 1], q_lens=[4, 3, 1], group=3),
    "few_rows_everything": dict(lens=[100], q_lens=[5], group=3, causal=False),
    # many rows: tiles of 128 and of 256, several of them, splits of the tokens
    "rows_of_a_wavefront": dict(lens=[40, 17], q_lens=[17, 17], group=1),
    "tile_128": dict(lens=[150, 60, 700], q_lens=[33, 1, 16], heads=1, group=3, page=64),
    "tile_256": dict(lens=[300, 140], q_lens=[130, 7], heads=1, group=2, page=32, lam=True),
    "tiles": dict(lens=[530], q_lens=[303], heads=1, group=2, page=16, bits=8),
    "splits": dict(lens=[1300, 700], q_lens=[9, 20], heads=1, group=2, page=64),
    "window_many": dict(lens=[400, 150], q_lens=[140, 100], heads=1, group=1, window=37, page=64),
    "cap_many": dict(lens=[260], q_lens=[100], heads=2, group=1, softcap=15.0, bits=8, page=256),
    "everything_many": dict(lens=[90, 200], q_lens=[90, 35], heads=1, group=2, causal=False),
    "window_without_causal": dict(lens=[90, 200], q_lens=[40, 35], heads=1, group=2, causal=False, window=20),
    "many_queries_than_tokens": dict(lens=[7, 0, 64], q_lens=[20, 18, 64], heads=1, group=2),
    # tiles of up to 16 rows beside full ones: single tokens, and what is left of 256 or 128 rows
    "mixed": dict(lens=[300, 77, 150, 400], q_lens=[130, 1, 8, 129], heads=1, group=2, page=32, lam=True),
    "mixed_window_cap": dict(lens=[200, 33, 180], q_lens=[66, 2, 65], heads=2, group=2, window=50, softcap=25.0, bits=8),
    "mixed_splits": dict(lens=[1400, 900], q_lens=[44, 1], heads=1, group=3, page=256),
    "negative_scale": dict(lens=[70, 64], q_lens=[1, 1], scale=-0.11),
    "zero_scale": dict(lens=[70, 64], q_lens=[20, 1], scale=0.0),
}


@pytest.mark.parametrize("name", CASES)
def test_against_definition(orc, name):
    say(f"case: attend {name} {CASES[name]}")
    Case(orc, **CASES[name]).check()


@pytest.mark.parametrize("name", ["single_long", "few_rows", "tile_128", "tile_256", "splits"])
def test_types_strides_and_repeats(orc, name):
    """bfloat16 queries inside wider rows, aligned or not; bfloat16 outputs are the binary32 ones rounded; equal calls give
    equal bits, weights among them."""
    say(f"case: attend types and strides {name}")
    c = Case(orc, **CASES[name] | dict(f32=False))
    q, w = dev(c.q), lambda: torch.zeros(len(c.lens), c.cache.shape[1], max(c.lens), device="cuda")  # noqa: E731
    first = c.run(q)
    for dt in (torch.bfloat16, torch.float32):
        for off in (0, 1, 8):
            row = torch.full((q.shape[0], 2 * q.shape[1] * 128 + 16), float("nan"), dtype=dt, device="cuda")
            view = row[:, off:off + q.shape[1] * 128].unflatten(1, (q.shape[1], 128))
            view.copy_(q)
            assert torch.equal(c.run(view), first)
            assert torch.equal(c.run(view, out_dtype=torch.bfloat16), first.to(torch.bfloat16))
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(c.run(heads_first), first)
    wa, wb = w(), w()
    assert torch.equal(c.run(q, weights=wa), c.run(q, weights=wb)) and torch.equal(wa, wb)


@pytest.mark.parametrize("group,m", [(2, 1), (2, 40), (2, 140)])
def test_absent_pages_and_stale_slots(orc, group, m):
    """Table entries outside the cache hide their tokens; slots past a length, and absent pages' stand-ins, may hold NaN."""
    say(f"case: attend absent pages, group {group}, {m} queries")
    c = Case(orc, [150, 170], [m, m], heads=1, group=group)
    c.table[0, 2], c.table[0, 5], c.table[1, 0], c.table[1, 10] = -1, c.cache.shape[0], 1 << 30, -(1 << 31)
    held = c.cache.clone()
    bad = host(c.cache)
    for pg in range(bad.shape[0]):  # every slot that no sequence holds, page 0 included if it is free
        use = [(b, i) for b in range(2) for i in range(-(-c.lens[b] // 16)) if c.table[b, i] == pg]
        kc, ks, vc, vs = ref.parts(bad, 4)
        at = c.lens[use[0][0]] - 16 * use[0][1] if use else 0
        for t in range(max(at, 0), 16):
            ks.view(np.uint16)[pg, :, t] = vs.view(np.uint16)[pg, :, t // 4, :, t % 4] = 0x7E00 if t % 2 else 0xFC00
    c.cache = dev(bad)
    got = host(c.run())
    c.check()
    c.cache = held
    assert np.array_equal(got, host(c.run()))


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("m", [1, 40, 140])
def test_nan_vectors_reach_the_rows_that_see_them(orc, m, softcap):
    """Vectors that were not finite when appended have NaN scales: rows that see one are NaN, no other row is."""
    say(f"case: attend NaN vectors, {m} queries, cap {softcap}")
    for side in range(2):
        c = Case(orc, [200], [m], heads=2, group=2, softcap=softcap)
        t = 200 - max(m // 2, 1)  # seen by the later half of the queries
        x = torch.full((1, 2, 128), float("nan"), device="cuda")
        x[:, 0] = 0.5  # head 0's vector is fine
        slot = dev(np.array([c.table[0, t // 16] * 16 + t % 16], np.int64))
        old = hq.hq_kv_read(c.cache, slot, out_dtype=torch.float32, **c.fmt)
        pair = [o.clone() for o in old]
        pair[side] = x
        hq.hq_kv_append(c.cache, pair[0], pair[1], slot, **c.fmt)
        for w in (None, torch.zeros(1, 2, 200, device="cuda")):
            bad = np.isnan(host(c.run(weights=w)))
            pos = 200 - m + np.arange(m)
            assert not bad[:, :2].any()
            assert np.array_equal(bad[:, 2:].all(-1), np.repeat((pos >= t)[:, None], 2, 1)) and np.array_equal(bad.any(-1), bad.all(-1))


def test_extreme_queries(orc):
    """Zero and subnormal queries average what they see; NaN queries are NaN and alone in it; large scores pick one token."""
    say("case: attend extreme queries")
    for m in (1, 40, 200):
        c = Case(orc, [256, 256, 256, 256], [m] * 4, heads=1, group=2)
        c.q[:m] = 0
        c.q[m:2 * m] = 1e-41 * np.sign(c.q[m:2 * m])
        c.q[3 * m:] *= 1000
        want = c.want()[0]
        clean = host(c.run())
        flat = np.linalg.norm(clean[:2 * m] - want[:2 * m], axis=-1)
        assert (flat <= 4 * 2.0 ** -11 * np.linalg.norm(want[:2 * m], axis=-1) * np.sqrt(256)).all()
        c.q[2 * m:3 * m] = np.nan
        got = host(c.run())
        assert np.isnan(got[2 * m:3 * m]).all()
        got[2 * m:3 * m] = clean[2 * m:3 * m]
        assert np.array_equal(got, clean)
        assert np.isfinite(clean).all()


def test_query_offsets(orc):
    """q_start may leave rows out, name none, or be missing; max_q and max_len cut."""
    say("case: attend q_start forms")
    c = Case(orc, [100, 100, 100], [2, 2, 2], heads=1, group=2)
    full = c.run()
    assert torch.equal(c.run(q_start=None, max_q=None, max_len=None), full)
    out = c.run(q_start=dev(np.array([0, 0, 2, 2], np.int32)))  # the first two queries are the second sequence's
    assert torch.isnan(out[2:]).all() and torch.isfinite(out[:2]).all()
    out = c.run(q_start=dev(np.array([-5, 2, 2, 999], np.int32)))  # offsets are cut to the queries there are
    assert torch.equal(out[:2], full[:2])
    out = c.run(max_q=1)
    assert torch.isnan(out[1::2]).all() and torch.isfinite(out[0::2]).all()
    c.lens = [64, 64, 64]
    short = c.run()
    c.lens = [100, 1 << 30, 100]
    assert torch.equal(c.run(max_len=64), short)
    c.lens = [-3, 64, 64]
    out = c.run(max_len=64)
    assert not out[:2].any() and torch.equal(out[2:], short[2:])


def test_equal_sequences_without_offsets(orc):
    """Without q_start the last tile of each sequence may be a light one: the same rows as with offsets."""
    say("case: attend equal sequences, light last tiles")
    for m, group in ((130, 2), (44, 3), (86, 3)):
        c = Case(orc, [300, 260], [m, m], heads=1, group=group)
        w = [torch.zeros(2, 1, 300, device="cuda") for _ in range(2)]
        assert torch.equal(c.run(q_start=None, max_q=None), c.run())
        assert torch.equal(c.run(q_start=None, weights=w[0]), c.run(weights=w[1])) and torch.equal(*w)


def test_no_pages_and_empty_calls():
    say("case: attend without pages, queries or sequences")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(40, 2, 128, device="cuda")
    lens = torch.full((2,), 50, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, 2, 64 * hq.hq_kv_token_bytes(4), dtype=torch.uint8, device="cuda")
    w = torch.zeros(2, 2, 64, device="cuda")
    for qq in (q, q[:2]):
        assert not hq.hq_kv_attend(none, qq, i32(2, 1), lens, weights=w).any() and not w.any()
    cache = hq.hq_kv_cache(2, 2)
    assert hq.hq_kv_attend(cache, q[:0], i32(2, 1), lens).shape == (0, 2, 128)
    assert hq.hq_kv_attend(cache, q[:0], i32(0, 1), lens[:0]).shape == (0, 2, 128)
    assert not hq.hq_kv_attend(cache, q, i32(2, 0), lens).any()
    assert not hq.hq_kv_attend(cache, q, i32(2, 1), i32(2)).any()


def test_refusals():
    say("case: attend refuses")
    cache = hq.hq_kv_cache(4, 2)
    q = torch.zeros(2, 4, 128, device="cuda", dtype=torch.bfloat16)
    table, lens = (torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((2, 1), (2,)))
    good = dict(cache=cache, q=q, table=table, lens=lens)
    for bad in (dict(q=q[:, :3]), dict(q=q[..., :64]), dict(q=q[..., ::2]), dict(q=q[0]), dict(table=table.long()), dict(lens=lens.cpu()),
                dict(q_start=lens), dict(weights=torch.zeros(2, 2, 64, device="cuda", dtype=torch.float64)), dict(window=-1), dict(max_q=-1),
                dict(weights=torch.zeros(2, 64, device="cuda")), dict(out=torch.zeros(2, 4, 64, device="cuda")), dict(max_len=1 << 32),
                dict(ws=torch.zeros(4096, device="cuda"))):
        with pytest.raises(ValueError):
            hq.hq_kv_attend(**good | bad)
    for bad in (dict(q=q.half()), dict(out=torch.zeros(2, 4, 128, device="cuda", dtype=torch.float16))):
        with pytest.raises(TypeError):
            hq.hq_kv_attend(**good | bad)
    for bad in (dict(softcap=-1.0), dict(scale=float("nan")), dict(weights=torch.zeros(2, 2, 63, device="cuda"), max_len=64),
                dict(ws=torch.zeros(128, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(hq.HqError):
            hq.hq_kv_attend(**good | bad)


@pytest.mark.parametrize("m", [1, 40])
def test_other_streams_and_graphs(orc, m):
    """A call on another stream, and a captured step (append, attend with weights, evict) replayed on new inputs, give the
    eager results."""
    say(f"case: streams and graphs, {m} queries")
    c = Case(orc, [120, 90], [m, m], heads=2, group=2)
    eager = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=side)
    side.synchronize()
    assert torch.equal(got, eager)

    q = dev(c.q)
    table, lens, start = dev(c.table), dev(np.array(c.lens, np.int32)), dev(c.start)
    pages = c.cache.shape[0]
    big = torch.cat([c.cache, torch.zeros_like(c.cache[:4])])
    dst = torch.arange(pages, pages + 4, dtype=torch.int32, device="cuda").view(2, 2)
    k, v = (torch.randn(2, 2, 128, device="cuda") for _ in range(2))
    slots = dev(np.array([c.table[b, (n - 1) // 16] * 16 + (n - 1) % 16 for b, n in enumerate(c.lens)], np.int64))

    def step(cache, weights):
        hq.hq_kv_append(cache, k, v, slots, **c.fmt)
        out = hq.hq_kv_attend(cache, q, table, lens, q_start=start, max_q=m, max_len=120, weights=weights, **c.kw, **c.fmt)
        return (out, *hq.hq_kv_evict(cache, table, lens, weights, 32, 2, 4, dst, max_len=120))

    cache, weights = big.clone(), torch.zeros(2, 2, 128, device="cuda")
    step(cache, weights)  # the first call of each kernel is eager
    cache.copy_(big)
    weights.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(cache, weights)
    e_cache, e_weights = big.clone(), torch.zeros_like(weights)
    for i in range(4):
        for x in (k, v, q):
            x.normal_()
        graph.replay()
        want = step(e_cache, e_weights)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        assert torch.equal(cache, e_cache) and torch.equal(weights, e_weights)


def test_pages_past_4_gib(orc):
    say("case: attend over the last pages of a cache of more than 4 GiB")
    for m in (1, 40):
        c = Case(orc, [200, 64], [m, m], heads=8, group=1, page=64)
        small, n = c.run(), c.cache.shape[0]
        w = [torch.zeros(2, 8, 200, device="cuda") for _ in range(2)]
        precise = c.run(weights=w[0])
        pages = 50000
        cache = torch.zeros(pages, *c.cache.shape[1:], dtype=torch.uint8, device="cuda")
        assert cache.numel() > 1 << 32
        cache[-n:] = c.cache
        c.cache = cache
        c.table = np.where(c.table >= 0, c.table + pages - n, -1).astype(np.int32)
        assert torch.equal(c.run(), small)
        assert torch.equal(c.run(weights=w[1]), precise) and torch.equal(w[0], w[1])


def test_long_sequences_split_and_join(orc):
    """33 thousand tokens: a needle in each split's range is found, and the weights of a row sum to one."""
    say("case: attend 33333 tokens")
    n, page = 33333, 256
    pages = -(-n // page)
    for m, group in ((1, 4), (5, 4), (33, 4)):
        cache = hq.hq_kv_cache(pages, 1, page)
        g = torch.Generator(device="cuda")
        g.manual_seed(m)
        k, v = (torch.randn(pages * page, 1, 128, generator=g, device="cuda") for _ in range(2))
        hq.hq_kv_append(cache, k, v, torch.arange(pages * page, device="cuda"), seed=SEED)
        k2, v2 = hq.hq_kv_read(cache, torch.arange(pages * page, device="cuda"), seed=SEED, out_dtype=torch.float32)
        at = torch.randint(0, n - m, (m * group,), generator=g, device="cuda")
        q = (k2[at, 0] * 3).view(m, group, 128)
        w = torch.zeros(1, 1, n, device="cuda")
        out = hq.hq_kv_attend(cache, q, torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                              torch.tensor([n], dtype=torch.int32, device="cuda"), seed=SEED, weights=w,
                              out=torch.empty(m, group, 128, device="cuda"))
        s = (q.double().view(-1, 128) @ k2[:n, 0].double().t().contiguous()) / 128 ** 0.5
        s = torch.softmax(torch.where(torch.arange(n, device="cuda") <= (n - m + torch.arange(m * group, device="cuda") // group)[:, None],
                                      s, torch.full_like(s, -float("inf"))), -1)
        want = (s @ v2[:n, 0].double()).view(m, group, 128)
        # scores up to 3 |k|^2 / 11.3, about 50, off by 2^-16.8 of sum |q_c k_c|: weights off by 2^-9; values by 3 2^-11
        assert float((out - want).norm() / want.norm()) < 2.0 ** -8
        assert float((w[0, 0] - s.sum(0)).abs().max()) < m * group * 2.0 ** -9
        assert abs(float(w.double().sum()) - m * group) < m * group * 2.0 ** -12
