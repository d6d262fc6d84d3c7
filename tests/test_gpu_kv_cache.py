"""GPU: appending to, reading from and evicting from the paged SRFT cache.

Codes, scales and decoded values equal the flat codec's oracle bit for bit; eviction moves whole numbers and bytes, so
everything here is compared exactly."""
import numpy as np
import pytest

import kv_reference as ref
import synth

torch = pytest.importorskip("torch")
hq = pytest.importorskip("kv_quantization_tile_amd")

pytestmark = pytest.mark.gpu

NAN16 = 0x7E00


def say(msg):
    print(msg, flush=True)


def host(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def slots_of(n, pages, page, seed, skip):
    g = np.random.default_rng(seed)
    s = g.permutation(pages * page)[:n].astype(np.int64)
    if skip:  # none, before the cache, after it, far after it
        for i, bad in zip(g.permutation(n)[:4], (-1, -(1 << 40), pages * page, 1 << 50)):
            s[i] = bad
    return s


def expected(orc, x, seed, bits, lam):
    """Codes [tokens][heads][16][E] and scales' bits [tokens][heads][16] of device x [tokens][heads][128]."""
    x = x.contiguous()
    a = x.view(torch.int16).cpu().numpy().view(np.uint16) if x.dtype == torch.bfloat16 else x.cpu().numpy()
    c, s = orc.srft_encode(a, seed, bits, lam)
    return c.reshape(x.shape[0], x.shape[1], 16, bits), s.reshape(x.shape[0], x.shape[1], 16)


@pytest.mark.parametrize("bits,page,heads,tokens,dtype,fused,lam,skip", [
    (4, 16, 1, 1, "bf16", False, False, False),
    (4, 64, 8, 5, "bf16", True, True, True),
    (8, 32, 3, 67, "bf16", True, False, True),
    (4, 16, 2, 130, "f32", False, True, False),
    (8, 256, 4, 1001, "f32", True, True, True),
    (4, 4096, 2, 301, "bf16", False, False, True),
])
def test_append_and_read_bit_exact(orc, bits, page, heads, tokens, dtype, fused, lam, skip):
    say(f"case: append {tokens} tokens, {heads} heads, page {page}, {bits} bits, {dtype}, fused {fused}, lambda {lam}, skip {skip}")
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    r = np.random.default_rng(tokens)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    if fused:  # keys and values inside wider rows, their starts off the 16-byte grid in one case
        off = 1 if tokens == 1001 else 0
        row = torch.randn(tokens, 4 * heads * 128 + 3, generator=g, device="cuda").to(dt)
        k = row[:, off:off + heads * 128].unflatten(1, (heads, 128))
        v = row[:, off + 2 * heads * 128:off + 3 * heads * 128].unflatten(1, (heads, 128))
    else:  # K with the heads outside
        k = torch.randn(heads, tokens, 128, generator=g, device="cuda").to(dt).transpose(0, 1)
        v = torch.randn(tokens, heads, 128, generator=g, device="cuda").to(dt)
    lams = [r.uniform(0.5, 2.0, 128).astype(np.float32) if lam else None for _ in range(2)]
    pages = -(-tokens // page) + 2
    slots = slots_of(tokens, pages, page, tokens, skip and tokens > 4)
    cache = torch.full((pages, heads, page * hq.hq_kv_token_bytes(bits)), 0x5A, dtype=torch.uint8, device="cuda")
    sl = torch.from_numpy(slots).cuda()
    hq.hq_kv_append(cache, k, v, sl, bits=bits, seed=7, lam_k=lams[0], lam_v=lams[1])
    want = np.full(cache.shape, 0x5A, np.uint8)
    kc, ks, vc, vs = ref.parts(want, bits)
    live = (slots >= 0) & (slots < pages * page)
    kx, vx = expected(orc, k, 7, bits, lams[0]), expected(orc, v, 7, bits, lams[1])
    for i in np.nonzero(live)[0]:
        pg, t = divmod(int(slots[i]), page)
        kc[pg, :, t], ks.view(np.uint16)[pg, :, t] = kx[0][i], kx[1][i]
        vc[pg, :, t // 4, :, t % 4], vs.view(np.uint16)[pg, :, t // 4, :, t % 4] = vx[0][i], vx[1][i]
    assert np.array_equal(host(cache), want)
    for od in ("bf16", "f32"):
        out = hq.hq_kv_read(cache, sl, bits=bits, seed=7, lam_k=lams[0], lam_v=lams[1],
                            out_dtype=torch.bfloat16 if od == "bf16" else torch.float32)
        for y, x, lm in ((out[0], kx, lams[0]), (out[1], vx, lams[1])):
            w = orc.srft_decode(x[0].reshape(-1, 16 * bits), x[1].reshape(-1, 16), tokens * heads * 128, 7, bits, lm, out_dtype=od)
            w = w.reshape(tokens, -1).copy()
            w[~live] = 0
            assert np.array_equal(host(y), w.view(np.uint8).reshape(host(y).shape))


def test_append_edge_vectors(orc):
    say("case: append zero, NaN, infinite, huge and tiny vectors")
    g = np.random.default_rng(8)
    rows = [np.zeros(128), g.standard_normal(128), g.standard_normal(128), np.full(128, 3e36), g.standard_normal(128) * 1e6,
            g.standard_normal(128) * 1e-38, g.standard_normal(128) * 1e-6]
    rows[1][17], rows[2][0] = np.nan, np.inf
    x = torch.from_numpy(np.stack(rows).astype(np.float32))[:, None].cuda()
    for bits in (4, 8):
        cache = hq.hq_kv_cache(1, 1, 16, bits)
        hq.hq_kv_append(cache, x, x.flip(0), torch.arange(7, device="cuda"), bits=bits, seed=3)
        kc, ks, vc, vs = ref.tokens_of(host(cache), bits)
        for (c, s), (gc, gs) in zip((expected(orc, x, 3, bits, None), expected(orc, x.flip(0), 3, bits, None)), ((kc, ks), (vc, vs))):
            assert np.array_equal(gc[0, 0, :7], c[:, 0]) and np.array_equal(gs.view(np.uint16)[0, 0, :7], s[:, 0])
        assert (ks.view(np.uint16)[0, 0, 1:3] == NAN16).all()


def test_append_of_nothing_and_refusals():
    say("case: empty calls and refused tensors")
    cache = hq.hq_kv_cache(2, 2)
    x = torch.zeros(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    hq.hq_kv_append(cache, x, x, none)
    assert [t.shape[0] for t in hq.hq_kv_read(cache, none)] == [0, 0]
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    s = torch.arange(3, device="cuda")
    for bad in (lambda: hq.hq_kv_append(cache, k[:2], k, s), lambda: hq.hq_kv_append(cache, k, k.float(), s),
                lambda: hq.hq_kv_append(cache, k, k, s.int()), lambda: hq.hq_kv_append(cache, k, k, s[:2]),
                lambda: hq.hq_kv_append(cache, k[..., ::2], k[..., ::2], s), lambda: hq.hq_kv_append(cache, k, k, s, bits=8, lam_k=[1.0]),
                lambda: hq.hq_kv_append(cache[:, :, :-1], k, k, s), lambda: hq.hq_kv_append(cache[..., :1000].contiguous(), k, k, s),
                lambda: hq.hq_kv_read(cache, s.cpu())):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(TypeError):
        hq.hq_kv_append(cache, k.half(), k.half(), s)
    with pytest.raises(hq.HqError):
        hq.hq_kv_append(cache, k, k, s, lam_k=np.full(128, -1.0))


def evict_case(seed, seqs, heads, top, page, bits, kind):
    g = np.random.default_rng(seed)
    w = np.exp(2.0 * g.standard_normal((seqs, heads, top)) - 4).astype(np.float32)
    if kind == "ties":
        w = np.round(w * 4).astype(np.float32) / 4
    if kind == "equal":
        w[:] = 0.25
    if kind == "odd":  # signs, zeros of either sign, infinities, NaN
        w *= np.where(g.random(w.shape) < 0.3, -1, 1)
        for value in (0.0, -0.0, np.inf, -np.inf, np.nan):
            w[g.random(w.shape) < 0.08] = value
    return w


@pytest.mark.parametrize("bits,page,heads,lens,budget,sink,recent,kind", [
    (4, 16, 1, [1], 1, 0, 0, "plain"),
    (4, 16, 2, [40, 0, 17, 16], 16, 2, 3, "plain"),
    (8, 32, 3, [1000, 1025, 31], 100, 4, 32, "ties"),
    (4, 64, 2, [5000, 4097], 1024, 0, 0, "equal"),
    (4, 16, 2, [700, 2049], 333, 1, 7, "odd"),
    (8, 64, 1, [130, 500], 128, 64, 64, "plain"),     # sink and recent fill the budget
    (4, 16, 1, [50, 3], 64, 4, 4, "ties"),            # nothing to evict
    (4, 16, 2, [20, 5], 0, 0, 0, "plain"),            # nothing stays
    (4, 128, 2, [20000], 7777, 4, 1000, "ties"),
    (4, 256, 1, [40000, 7], 3000, 4, 100, "odd"),     # more tokens than keys are held
    (8, 64, 1, [33000], 32900, 1, 1, "equal"),
])
def test_evict_exact(bits, page, heads, lens, budget, sink, recent, kind):
    say(f"case: evict {lens} to {budget} (sink {sink}, recent {recent}), page {page}, {bits} bits, weights {kind}")
    top, seqs = max(lens), len(lens)
    w = evict_case(budget, seqs, heads, top + 3, page, bits, kind)
    used = [-(-n // page) for n in lens]
    width, dw = max(used) + 1, max(1, -(-budget // page))
    first = sum(used) + 1
    g = np.random.default_rng(1)
    order = g.permutation(first)
    table = np.full((seqs, width), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    dst = first + np.arange(seqs * dw, dtype=np.int32).reshape(seqs, dw)
    before = g.integers(0, 256, (first + seqs * dw, heads, page * hq.hq_kv_token_bytes(bits))).astype(np.uint8)
    cache = torch.from_numpy(before).cuda()
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    kept, left, wk = hq.hq_kv_evict(cache, dev(table), dev(np.array(lens, np.int32)), dev(w), budget, sink, recent, dev(dst), bits=bits)
    want, left_want = ref.evict(w, lens, budget, sink, recent)
    assert np.array_equal(left.cpu().numpy(), left_want) and np.array_equal(kept.cpu().numpy(), want)
    after = before.copy()
    src, to = ref.tokens_of(before, bits), ref.parts(after, bits)
    ww = np.zeros(want.shape, np.float32)
    for b in range(seqs):
        for a in range(heads):
            m = left_want[b]
            t, j = want[b, a, :m], np.arange(m)
            ww[b, a, :m] = w[b, a, t]
            s, d = (table[b, t // page], a, t % page), (dst[b, j // page], a)
            to[0][d + (j % page,)], to[1].view(np.uint16)[d + (j % page,)] = src[0][s], src[1].view(np.uint16)[s]
            quad = (j % page // 4, slice(None), j % page % 4)
            to[2][d + quad], to[3].view(np.uint16)[d + quad] = src[2][s], src[3].view(np.uint16)[s]
    assert np.array_equal(host(wk), ww.view(np.uint8).reshape(host(wk).shape))
    assert np.array_equal(host(cache), after)


def test_evict_absent_pages_and_refusals():
    say("case: evict with absent pages; refused arguments")
    cache = torch.randint(0, 256, (6, 1, 16 * hq.hq_kv_token_bytes(4)), dtype=torch.uint8, device="cuda")
    before = host(cache).copy()
    table = torch.tensor([[0, -1, 99]], dtype=torch.int32, device="cuda")
    dst = torch.tensor([[4, -5]], dtype=torch.int32, device="cuda")
    lens, w = torch.tensor([48], dtype=torch.int32, device="cuda"), torch.ones(1, 1, 48, device="cuda")
    kept, left, _ = hq.hq_kv_evict(cache, table, lens, w, 20, 0, 2, dst)
    assert kept[0, 0].tolist() == [*range(18), 46, 47] and left.tolist() == [20]
    after = host(cache)
    assert np.array_equal(after[:4], before[:4]) and np.array_equal(after[5:], before[5:])
    a, b = ref.tokens_of(after, 4), ref.tokens_of(before, 4)
    assert all(np.array_equal(x[4, 0, :16], y[0, 0, :16]) for x, y in zip([z.view(np.uint8) for z in a], [z.view(np.uint8) for z in b]))
    for bad in (dict(budget=33), dict(budget=-1), dict(sink=-1), dict(max_len=-1)):
        kw = dict(budget=20, sink=0, recent=2) | bad
        with pytest.raises(ValueError):
            hq.hq_kv_evict(cache, table, lens, w, kw["budget"], kw["sink"], kw["recent"], dst, max_len=kw.get("max_len"))
    with pytest.raises(hq.HqError):
        hq.hq_kv_evict(cache, table, lens, w, 20, 15, 6, dst)


def test_pages_past_4_gib():
    say("case: append, read and evict in the last pages of a cache of more than 4 GiB")
    page, heads, pages = 64, 8, 50000
    cache = torch.zeros(pages, heads, page * hq.hq_kv_token_bytes(4), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    n = 100
    k, v = (torch.randn(n, heads, 128, device="cuda") for _ in range(2))
    slots = (pages - 4) * page + torch.arange(n, device="cuda")
    hq.hq_kv_append(cache, k, v, slots, seed=5)
    small = hq.hq_kv_cache(4, heads, page)
    hq.hq_kv_append(small, k, v, torch.arange(n, device="cuda"), seed=5)
    assert torch.equal(cache[-4:], small) and not bool(cache[:-4].any())
    for a, b in zip(hq.hq_kv_read(cache, slots, seed=5), hq.hq_kv_read(small, torch.arange(n, device="cuda"), seed=5)):
        assert torch.equal(a, b)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    w = torch.rand(1, heads, n, device="cuda")
    hq.hq_kv_evict(cache, i32([pages - 4, pages - 3]), i32(n), w, 64, 2, 2, i32([pages - 1]))
    hq.hq_kv_evict(small, i32([0, 1]), i32(n), w, 64, 2, 2, i32([3]))
    assert torch.equal(cache[-4:], small)


def test_append_into_a_synthetic_layer_equals_flat_codec(orc):
    """The SRFT workload's own layer (8 heads of 4096 tokens): the cache holds the flat codec's codes and scales."""
    say("case: a synthetic KV layer through the cache and the flat codec")
    x = torch.from_numpy(synth.kv(2, 0, tokens=4096).reshape(8, 4096, 128).view(np.int16)).view(torch.bfloat16).cuda()
    cache = hq.hq_kv_cache(64, 8, 64, 4)
    kv = x.transpose(0, 1)
    hq.hq_kv_append(cache, kv, kv, torch.arange(4096, device="cuda"), seed=9)
    c, s = hq.hq_srft_encode(x, seed=9, bits=4)
    for codes, scales in (ref.tokens_of(host(cache), 4)[:2], ref.tokens_of(host(cache), 4)[2:]):
        flat = codes.swapaxes(0, 1).reshape(8 * 4096, 64)
        assert np.array_equal(flat, c.cpu().numpy())
        assert np.array_equal(scales.view(np.uint16).swapaxes(0, 1).reshape(-1, 16), s.cpu().numpy().view(np.uint16))


@pytest.mark.parametrize("bits,page,heads,tokens,dtype,lam", [
    (4, 64, 8, 8203, "bf16", (False, False)),
    (8, 16, 4, 32801, "f32", (True, True)),
    (4, 256, 8, 16387, "bf16", (True, False)),
    (8, 32, 16, 8199, "bf16", (False, True)),
    (4, 16, 1, 65537, "f32", (False, False)),
])
def test_many_tokens_equal_few_at_a_time(bits, page, heads, tokens, dtype, lam):
    """Enough vectors for a thread to take one each: the bytes and values of calls too small for that, which are tested
    against the oracle; vectors that are not finite, and slots outside the cache, among them."""
    say(f"case: {tokens} tokens in one call and in many, {heads} heads, page {page}, {bits} bits, {dtype}, lambda {lam}")
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    row = torch.randn(tokens, 3 * heads * 128, generator=g, device="cuda").to(dt)
    k, v = row[:, heads * 128:2 * heads * 128].unflatten(1, (heads, 128)), row[:, 2 * heads * 128:].unflatten(1, (heads, 128))
    k[17, 0, 5], v[tokens - 1, heads - 1, 127], k[300] = float("nan"), float("inf"), 0
    r = np.random.default_rng(tokens)
    fmt = dict(bits=bits, seed=13, lam_k=r.uniform(0.5, 2.0, 128).astype(np.float32) if lam[0] else None,
               lam_v=r.uniform(0.5, 2.0, 128).astype(np.float32) if lam[1] else None)
    pages = -(-tokens // page) + 2
    slots = torch.from_numpy(slots_of(tokens, pages, page, tokens, True)).cuda()
    one, many = (torch.full((pages, heads, page * hq.hq_kv_token_bytes(bits)), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(2))
    hq.hq_kv_append(one, k, v, slots, **fmt)
    step = 1000
    vectors = heads * (1 if lam[0] or lam[1] else 2)  # of a launch and token
    assert step * vectors < 1 << 17 <= tokens * vectors
    for i in range(0, tokens, step):
        hq.hq_kv_append(many, k[i:i + step], v[i:i + step], slots[i:i + step], **fmt)
    assert torch.equal(one, many)
    for od in (torch.bfloat16, torch.float32):
        whole = hq.hq_kv_read(one, slots, out_dtype=od, **fmt)
        for i in range(0, tokens, step):
            part = hq.hq_kv_read(one, slots[i:i + step], out_dtype=od, **fmt)
            for a, b in zip(whole, part):
                assert np.array_equal(host(a[i:i + step]), host(b))
