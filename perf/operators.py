"""Cases, plain forms and 64-bit values of the paged SRFT cache's operators.

A layer's paged cache is one uint8 tensor [pages][kv heads][page bytes]; a page holds P tokens (P a multiple of
16) of one KV head, D = 128 coordinates each, in the SRFT codec's form at `bits` = 4 or 8: a vector x is stored as
y = pack(F diag(s) x) / lambda, 16 groups of 8 coordinates with a binary16 scale Delta each and signed codes.
With E = 4 or 8 bytes per group's 8 codes, the page holds, in this order:

    K codes  [P][16][E]        K scales [P][16] binary16
    V codes  [P/4][16][4][E]   V scales [P/4][16][4] binary16   (blocks of four tokens, group by group)

4-bit codes lie two a byte, the even coordinate in the low nibble.  Token t of sequence b is slot t % P of page
table[b][t / P].  The operators:

  append + read  new tokens' K and V are transformed, quantised and written to their slots; slots are read back
  attend         softmax attention of new queries over the cache, optionally adding each key's weight to `weights`
  evict          the tokens of most accumulated weight (with the first and the last ones) move to fresh pages
"""
import math
import random

import numpy as np
import torch

own = False

D, GROUPS = 128, 16


# ---- the cases -------------------------------------------------------------------------------------


def listed():
    return [
        # one decode step's new token of four sequences in a layer of 8 KV heads: latency counts
        dict(name="append_4_tokens", op="append", tokens=4, heads=8, page=16, bits=4, f32=False, fused=False, lam=False, skip=False),
        # the new tokens of a large batch, out of a fused projection's rows, some slots inactive, calibrated scales
        dict(name="append_333_fused_8bit", op="append", tokens=333, heads=8, page=64, bits=8, f32=False, fused=True, lam=True, skip=True),
        # a whole prompt of one layer's cache
        dict(name="append_prompt_32768", op="append", tokens=32768, heads=8, page=64, bits=4, f32=False, fused=True, lam=False, skip=False),
        # a short conversation's next token
        dict(name="decode_1x301", op="attend", seqs=1, len=301, ragged=False, q=1, mixed=False, heads=8, group=4, page=16, bits=4,
             causal=True, window=0, softcap=0.0, weights=False, lam=False),
        # one long document's next token: the cache's length is all there is to split
        dict(name="decode_1x32768", op="attend", seqs=1, len=32768, ragged=False, q=1, mixed=False, heads=8, group=4, page=64, bits=4,
             causal=True, window=0, softcap=0.0, weights=True, lam=False),
        # a batch of ragged long sequences: more bytes than the card's caches hold
        dict(name="decode_16x32768_ragged", op="attend", seqs=16, len=32768, ragged=True, q=1, mixed=False, heads=8, group=4, page=64, bits=4,
             causal=True, window=0, softcap=0.0, weights=False, lam=True),
        # a wide batch at 8 bits with capped scores, as models with a soft cap decode
        dict(name="decode_64x4001_cap_8bit", op="attend", seqs=64, len=4001, ragged=True, q=1, mixed=False, heads=4, group=2, page=32, bits=8,
             causal=True, window=0, softcap=30.0, weights=False, lam=False),
        # a chunk of a long prompt beside sequences that decode, with the accumulated weight an eviction needs
        dict(name="mixed_8xq129x5003_weights", op="attend", seqs=8, len=5003, ragged=True, q=129, mixed=True, heads=8, group=4, page=64, bits=4,
             causal=True, window=0, softcap=0.0, weights=True, lam=False),
        # a whole prompt
        dict(name="prompt_1x8192", op="attend", seqs=1, len=8192, ragged=False, q=8192, mixed=False, heads=8, group=4, page=64, bits=4,
             causal=True, window=0, softcap=0.0, weights=False, lam=False),
        # one conversation over its budget by a page
        dict(name="evict_1x1040_to_1024", op="evict", seqs=1, len=1040, ragged=False, budget=1024, sink=4, recent=128, heads=8, page=16, bits=4),
        # a batch of long prompts cut down to a quarter
        dict(name="evict_4x32768_to_8192", op="evict", seqs=4, len=32768, ragged=True, budget=8192, sink=4, recent=1024, heads=8, page=64, bits=4),
        # many middling sequences at 8 bits
        dict(name="evict_32x4097_to_1000_8bit", op="evict", seqs=32, len=4097, ragged=True, budget=1000, sink=1, recent=32, heads=4, page=32, bits=8),
    ]


def draw(rng):
    def between(lo, hi):  # over the logarithm
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    op = rng.choice(["append", "attend", "attend", "attend", "evict"])
    c = dict(op=op, heads=rng.choice([1, 2, 4, 8]), page=rng.choice([16, 32, 64, 128, 256]), bits=rng.choice([4, 4, 8]))
    if op == "append":
        c.update(tokens=between(1, 32768), f32=rng.random() < 0.3, fused=rng.random() < 0.5, lam=rng.random() < 0.5, skip=rng.random() < 0.5)
        return c
    c["seqs"], c["ragged"] = between(1, 64), rng.random() < 0.7
    most = (1 << 18) // c["seqs"]  # cached tokens in all
    c["len"] = between(1, min(32768, most))
    if op == "evict":
        c["budget"] = between(1, c["len"])
        c["sink"] = rng.randint(0, min(4, c["budget"]))
        c["recent"] = rng.randint(0, (c["budget"] - c["sink"]) // 2)
        return c
    c["group"] = rng.choice([1, 2, 3, 4, 7, 8])
    rows = (1 << 30) // (c["seqs"] * c["len"] * c["heads"] * c["group"])  # a quarter of the longest prompt's scores
    c["q"] = 1 if rng.random() < 0.5 else between(1, max(1, min(c["len"], rows, 4096)))
    c["mixed"] = c["q"] > 1 and rng.random() < 0.3
    c.update(causal=rng.random() < 0.8, window=between(1, c["len"]) if rng.random() < 0.25 else 0,
             softcap=rng.choice([0.0, 0.0, 20.0, 50.0]), weights=rng.random() < 0.3, lam=rng.random() < 0.3)
    return c


def seq_lens(case):
    n, top = case["seqs"], case["len"]
    return [max(1, top - int((b * 0.6180339887 % 1.0) * 0.75 * top)) if case["ragged"] else top for b in range(n)]


def query_lens(case):
    return [1 if case["mixed"] and b % 2 else min(case["q"], n) for b, n in enumerate(seq_lens(case))]


def token_bytes(case):
    return 2 * (GROUPS * case["bits"] + 32)  # K and V of one token and head


def work(case):
    h = case["heads"]
    if case["op"] == "append":
        n = case["tokens"] * h
        return {"bytes": n * (2 * D * ((4 if case["f32"] else 2) + 2) + 2 * token_bytes(case)) + 8 * case["tokens"], "flops": n * 2 * (3186 + 3028)}
    lens = seq_lens(case)
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": h * (4 * sum(lens) + kept * (2 * token_bytes(case) + 8)), "flops": h * sum(lens)}
    pairs = seen = rows = 0
    for n, m in zip(lens, query_lens(case)):
        pos = np.arange(n - m, n)
        hi = pos + 1 if case["causal"] else np.full(m, n)
        lo = np.maximum(0, pos + 1 - case["window"]) if case["window"] else np.zeros(m, np.int64)
        pairs += int(np.maximum(0, hi - lo).sum())
        seen += int(hi.max() - lo.min())
        rows += m
    return {"bytes": seen * h * (token_bytes(case) + (8 if case["weights"] else 0)) + rows * h * case["group"] * D * 4,
            "flops": 4 * D * pairs * h * case["group"]}


# ---- the transform ---------------------------------------------------------------------------------

SEED = 11  # of the sign diagonal


def sign_diagonal(seed):
    """+-1 from bit i % 32 of word i / 32 of Philox4x32-10 (key = seed, counter 0)."""
    c, k0, k1, m = [0, 0, 0, 0], seed & 0xFFFFFFFF, seed >> 32, 0xFFFFFFFF
    for _ in range(10):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k0, p1 & m, (p0 >> 32) ^ c[3] ^ k1, p0 & m]
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return np.array([-1.0 if c[i // 32] >> (i % 32) & 1 else 1.0 for i in range(D)])


def transform_matrix(seed):
    """T of pack(F diag(s) x) = T x: rows X_0, X_64, then sqrt 2 (Re X_k, Im X_k), all over sqrt 128."""
    n = np.arange(D)
    rows = [np.ones(D), np.cos(np.pi * n)]
    for k in range(1, D // 2):
        a = 2 * np.pi * (k * n % D) / D
        rows += [np.sqrt(2) * np.cos(a), -np.sqrt(2) * np.sin(a)]
    return np.stack(rows) / np.sqrt(D) * sign_diagonal(seed)


# ---- pages -----------------------------------------------------------------------------------------


def parts(cache, bits):
    """K codes [pages][heads][P][16][E], K scales [..][P][16], V codes [..][P/4][16][4][E], V scales [..][P/4][16][4]."""
    n, h, size = cache.shape
    p = size // (2 * (GROUPS * bits + 32))
    a, b = p * GROUPS * bits, p * 32
    half = lambda t: t.view(torch.float16)  # noqa: E731
    return (cache[:, :, :a].unflatten(2, (p, GROUPS, bits)), half(cache[:, :, a:a + b]).unflatten(2, (p, GROUPS)),
            cache[:, :, a + b:2 * a + b].unflatten(2, (p // 4, GROUPS, 4, bits)), half(cache[:, :, 2 * a + b:]).unflatten(2, (p // 4, GROUPS, 4)))


def codes_of(raw, bits):
    """int codes [..][16][8] of bytes [..][16][E]."""
    if bits == 8:
        return raw.view(torch.int8)
    return torch.stack([raw << 4, raw], -1).view(torch.int8).flatten(-2) >> 4


def bytes_of(codes, bits):
    if bits == 8:
        return codes.to(torch.int8).view(torch.uint8)
    c = codes.to(torch.int16) & 15
    return (c[..., 0::2] | c[..., 1::2] << 4).to(torch.uint8)


def quantised(x, T, lam, bits):
    """Codes [..][16][8] and binary16 scales [..][16] of vectors x [..][128]."""
    top = 7 if bits == 4 else 127
    y = (torch.matmul(x, T.t().contiguous()) / lam).unflatten(-1, (GROUPS, 8))
    scale = (y.abs().amax(-1) / top).clamp(max=65504.0).to(torch.float16)
    d = scale.to(y.dtype).unsqueeze(-1)
    return torch.where(d > 0, torch.round(y * (1 / d)), torch.zeros_like(y)).clamp(-top, top), scale


def filled(cache, bits, T, lams, g):
    """Writes a KV workload into every slot: N(0, 1) values, four channels of each K head ten times as large."""
    kc, ks, vc, vs = parts(cache, bits)
    pages, h, p = ks.shape[:3]
    loud = torch.ones(h, 1, D, device="cuda")
    loud.scatter_(2, torch.rand(h, 1, D, generator=g, device="cuda").argsort(-1)[..., :4], 10.0)
    step = max(1, (1 << 27) // (h * p * D))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        c, s = quantised(torch.randn(n, h, p, D, generator=g, device="cuda") * loud, T, lams[0], bits)
        kc[i:i + n], ks[i:i + n] = bytes_of(c, bits), s
        c, s = quantised(torch.randn(n, h, p, D, generator=g, device="cuda"), T, lams[1], bits)
        vc[i:i + n] = bytes_of(c, bits).unflatten(2, (p // 4, 4)).transpose(3, 4)
        vs[i:i + n] = s.unflatten(2, (p // 4, 4)).transpose(3, 4)
    return loud


# ---- what a program has in hand --------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = random.Random(seed)
    h, p, bits = case["heads"], case["page"], case["bits"]
    lam = [None, None]
    if case.get("lam"):
        lam = [np.array([r.uniform(0.5, 2.0) for _ in range(D)], np.float32) for _ in range(2)]
    lams = [torch.ones(D, device="cuda") if a is None else torch.from_numpy(a).cuda() for a in lam]
    T64 = torch.from_numpy(transform_matrix(SEED)).cuda()
    st = dict(case=case, lam=lam, lams=lams, T=T64.float())

    def pool(pages):
        return torch.zeros(pages, h, p * token_bytes(case), dtype=torch.uint8, device="cuda")

    if case["op"] == "append":
        n = case["tokens"]
        pages = -(-n // p) + 3
        dt = torch.float32 if case["f32"] else torch.bfloat16
        if case["fused"]:  # rows of a fused projection: queries, keys, values
            row = torch.randn(n, 6 * h * D, generator=g, device="cuda").to(dt)
            k, v = row[:, 4 * h * D:5 * h * D].unflatten(1, (h, D)), row[:, 5 * h * D:].unflatten(1, (h, D))
        else:
            k, v = (torch.randn(n, h, D, generator=g, device="cuda").to(dt) for _ in range(2))
        k.mul_((1 + 9 * (torch.rand(h, D, generator=g, device="cuda") < 0.03)).to(dt))
        slots = torch.randperm(pages * p, generator=g, device="cuda")[:n] if n < 4096 else \
            (torch.randperm(pages, generator=g, device="cuda")[:, None] * p + torch.arange(p, device="cuda")).flatten()[:n].contiguous()
        if case["skip"]:
            slots[torch.rand(n, generator=g, device="cuda") < 0.1] = -1
        return dict(st, cache=pool(pages), k=k, v=v, slots=slots)

    lens = seq_lens(case)
    used = [-(-n // p) for n in lens]
    kept_pages = -(-case["budget"] // p) if case["op"] == "evict" else 0
    first = sum(used) + 2
    cache = pool(first + kept_pages * len(lens))
    loud = filled(cache[:first], bits, st["T"], lams, g)
    order = torch.randperm(first, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(used)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    st.update(cache=cache, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), max_len=max(lens))
    if case["op"] == "evict":
        w = torch.exp(2.5 * torch.randn(len(lens), h, max(lens), generator=g, device="cuda") - 6).to(torch.bfloat16).float()  # ties occur
        dst = first + torch.arange(len(lens) * kept_pages, dtype=torch.int32, device="cuda").view(len(lens), kept_pages)
        return dict(st, weights=w, dst=dst, first=first)

    m = query_lens(case)
    start = np.concatenate([[0], np.cumsum(m)]).astype(np.int32)
    hq = h * case["group"]
    rows = torch.randn(int(start[-1]), (hq + 2 * h) * D, generator=g, device="cuda").to(torch.bfloat16)
    q = rows[:, :hq * D].unflatten(1, (hq, D))  # beside the new keys and values, as a fused projection leaves them
    # a few keys of its sequence that each query looks for
    kc, ks = parts(cache, bits)[:2]
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(m, device="cuda"))[:, None]
    tok = (torch.rand(int(start[-1]), hq, generator=g, device="cuda") * st["lens"][seq]).long()
    pg, head = table[seq, tok // p].long(), torch.arange(hq, device="cuda") // case["group"]
    y = codes_of(kc[pg, head, tok % p], bits).float() * ks[pg, head, tok % p].float()[..., None]
    q += (0.7 * torch.matmul(y.flatten(-2) * lams[0], st["T"]) / loud[head, 0] ** 1.5).to(torch.bfloat16)
    st.update(q=q, start=torch.from_numpy(start).cuda(), max_q=max(m))
    if case["weights"]:
        st["weights"] = torch.rand(len(lens), h, max(lens), generator=g, device="cuda")
    return st


# ---- one pass --------------------------------------------------------------------------------------


def run(st):
    return {"append": run_append, "attend": run_attend, "evict": run_evict}[st["case"]["op"]](st)


def run_append(st):
    c, bits = st["case"], st["case"]["bits"]
    cache, slots = st["cache"], st["slots"]
    if own:
        import kv_quantization_tile_amd as hq
        hq.hq_kv_append(cache, st["k"], st["v"], slots, bits=bits, seed=SEED, lam_k=st["lam"][0], lam_v=st["lam"][1])
        return hq.hq_kv_read(cache, slots, bits=bits, seed=SEED, lam_k=st["lam"][0], lam_v=st["lam"][1])
    kc, ks, vc, vs = parts(cache, bits)
    live = slots >= 0
    at = slots[live]
    pg, t = at // c["page"], at % c["page"]
    codes, scale = quantised(st["k"][live].float(), st["T"], st["lams"][0], bits)
    kc[pg, :, t], ks[pg, :, t] = bytes_of(codes, bits), scale
    codes, scale = quantised(st["v"][live].float(), st["T"], st["lams"][1], bits)
    vc[pg, :, t // 4, :, t % 4], vs[pg, :, t // 4, :, t % 4] = bytes_of(codes, bits), scale
    pg, t = slots.clamp(min=0) // c["page"], slots.clamp(min=0) % c["page"]

    def back(raw, scale, lam):
        y = (codes_of(raw, bits).float() * scale.float()[..., None]).flatten(-2) * lam
        return torch.where(live[:, None, None], torch.matmul(y, st["T"]), torch.zeros_like(y)).to(torch.bfloat16)

    return back(kc[pg, :, t], ks[pg, :, t], st["lams"][0]), back(vc[pg, :, t // 4, :, t % 4], vs[pg, :, t // 4, :, t % 4], st["lams"][1])


def run_attend(st):
    c, bits, table, lens = st["case"], st["case"]["bits"], st["table"], st["lens"]
    weights = st.get("weights")
    if own:
        import kv_quantization_tile_amd as hq
        out = hq.hq_kv_attend(st["cache"], st["q"], table, lens, q_start=st["start"], max_q=st["max_q"], max_len=st["max_len"], bits=bits,
                              seed=SEED, lam_k=st["lam"][0], lam_v=st["lam"][1], causal=c["causal"], window=c["window"],
                              softcap=c["softcap"], weights=weights)
        return out if weights is None else (out, weights)
    kc, ks, vc, vs = parts(st["cache"], bits)
    h, grp, pages = c["heads"], c["group"], table.clamp(min=0).long()
    n, width = table.shape
    top = st["max_len"]
    # keys and values of the padded sequences, [seqs][heads][top][128]
    y = codes_of(kc[pages], bits).float() * ks[pages].float()[..., None]
    k = torch.matmul(y.transpose(1, 2).reshape(n, h, width * c["page"], D)[:, :, :top] * st["lams"][0], st["T"])
    y = codes_of(vc[pages], bits).float() * vs[pages].float()[..., None]
    v = torch.matmul(y.transpose(4, 5).transpose(1, 2).reshape(n, h, width * c["page"], D)[:, :, :top] * st["lams"][1], st["T"])
    # queries of a sequence as rows, [seqs][heads][max_q * group][128]
    start, m = st["start"][:-1].long(), (st["start"][1:] - st["start"][:-1]).long()
    i = torch.arange(st["max_q"], device="cuda")
    have = i < m[:, None]
    at = torch.where(have, start[:, None] + i, torch.zeros_like(i))
    q = st["q"][at].float().unflatten(2, (h, grp)).permute(0, 2, 1, 3, 4).reshape(n, h, -1, D)
    s = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(1 / math.sqrt(D))
    if c["softcap"]:
        s = s.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    pos = lens[:, None] - m[:, None] + i
    hi = torch.where(have, torch.minimum(pos + 1, lens[:, None]) if c["causal"] else lens[:, None].expand_as(pos), torch.zeros_like(pos))
    lo = pos + 1 - c["window"] if c["window"] else torch.zeros_like(pos)
    t = torch.arange(top, device="cuda")
    hidden = ((t >= hi[..., None]) | (t < lo[..., None])).repeat_interleave(grp, 1)[:, None]
    s.masked_fill_(hidden, -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = s.sum(-1, keepdim=True)
    s.div_(torch.where(total > 0, total, torch.ones_like(total)))
    o = torch.matmul(s, v).unflatten(2, (-1, grp)).permute(0, 2, 1, 3, 4).reshape(n, -1, h * grp, D)
    out = torch.empty(st["q"].shape, dtype=torch.bfloat16, device="cuda")
    out[at[have]] = o[have].to(torch.bfloat16)
    if weights is None:
        return out
    weights += s.sum(2)
    return out, weights


def run_evict(st):
    c, bits, table, lens, w = st["case"], st["case"]["bits"], st["table"], st["lens"], st["weights"]
    if own:
        import kv_quantization_tile_amd as hq
        kept, left, wk = hq.hq_kv_evict(st["cache"], table, lens, w, c["budget"], c["sink"], c["recent"], st["dst"], bits=bits, max_len=st["max_len"])
        return kept, left, wk, st["cache"][st["first"]:]
    n, h, top = w.shape
    p, budget = c["page"], c["budget"]
    t = torch.arange(top, device="cuda")
    ends = (t < c["sink"]) | (t >= (lens - c["recent"])[:, None])
    key = torch.where(ends[:, None], torch.full_like(w, math.inf), w)
    key = torch.where((t < lens[:, None])[:, None], key, torch.full_like(w, -math.inf))
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    left = torch.minimum(lens, torch.full_like(lens, budget))
    j = torch.arange(budget, device="cuda")
    inside = (j[:best.shape[-1]] < left[:, None])[:, None].expand_as(best)
    got = torch.where(inside, best, torch.full_like(best, top)).sort(-1).values
    at = torch.where(got < top, got, torch.zeros_like(got))
    kept = torch.full((n, h, budget), -1, dtype=torch.int32, device="cuda")
    wk = torch.zeros(n, h, budget, device="cuda")
    kept[..., :at.shape[-1]] = torch.where(got < top, got, torch.full_like(got, -1)).to(torch.int32)
    wk[..., :at.shape[-1]] = torch.where(got < top, w.gather(2, at), torch.zeros_like(at, dtype=torch.float32))
    b, head, j = torch.nonzero(got < top, as_tuple=True)
    src = at[b, head, j]
    sp, so, dp, do = table[b, src // p].long(), src % p, st["dst"][b, j // p].long(), j % p
    kc, ks, vc, vs = parts(st["cache"], bits)
    kc[dp, head, do] = kc[sp, head, so]
    ks[dp, head, do] = ks[sp, head, so]
    vc[dp, head, do // 4, :, do % 4] = vc[sp, head, so // 4, :, so % 4]
    vs[dp, head, do // 4, :, do % 4] = vs[sp, head, so // 4, :, so % 4]
    return kept, left, wk, st["cache"][st["first"]:]


# ---- the same in 64 bits, from the definition ------------------------------------------------------


def spectrum(x, signs):
    """pack(F diag(s) x) by the discrete Fourier transform."""
    X = torch.fft.rfft(x * signs, norm="ortho")
    y = torch.view_as_real(X[..., 1:-1]).flatten(-2) * math.sqrt(2)
    return torch.cat([X[..., :1].real, X[..., -1:].real, y], -1)


def from_spectrum(y, signs):
    inner = torch.view_as_complex((y[..., 2:] / math.sqrt(2)).unflatten(-1, (-1, 2)).contiguous())
    X = torch.cat([y[..., :1] + 0j, inner, y[..., 1:2] + 0j], -1)
    return torch.fft.irfft(X, n=D, norm="ortho") * signs


def exact(case, seed):
    st = prepare(case, seed)
    bits, p, h = case["bits"], case["page"], case["heads"]
    signs = torch.from_numpy(sign_diagonal(SEED)).cuda()
    lam = [a.double() for a in st["lams"]]
    if case["op"] == "append":
        top = 2 ** (bits - 1) - 1

        def there_and_back(x, lam):
            y = (spectrum(x.double(), signs) / lam).unflatten(-1, (GROUPS, 8))
            d = torch.clamp(y.abs().amax(-1, keepdim=True) / top, max=65504.0).half().double()
            q = torch.where(d > 0, torch.clamp(torch.round(y / d), -top, top), torch.zeros_like(y))
            return from_spectrum((q * d).flatten(-2) * lam, signs) * (st["slots"] >= 0)[:, None, None]

        return there_and_back(st["k"], lam[0]), there_and_back(st["v"], lam[1])
    if case["op"] == "evict":
        w, kept = st["weights"].cpu().numpy().astype(np.float64), []
        wk = torch.zeros(case["seqs"], h, case["budget"], dtype=torch.float64)
        for b, n in enumerate(seq_lens(case)):
            m = min(n, case["budget"])
            fixed = np.zeros(n, bool)
            fixed[:case["sink"]] = True
            fixed[max(0, n - case["recent"]):] = True
            for a in range(h):
                rank = np.lexsort((np.arange(n), -w[b, a, :n], ~fixed))[:m]  # fixed ones, then by weight, then by index
                wk[b, a, :m] = torch.from_numpy(w[b, a, np.sort(rank)])
        return None, None, wk.cuda(), None

    kc, ks, vc, vs = parts(st["cache"], bits)
    grp, lens, m, table = case["group"], seq_lens(case), query_lens(case), st["table"].long()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    weights = st["weights"].double() if case["weights"] else None
    at = 0
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        pg, off = table[b, t // p], t % p
        for a in range(h):
            k = from_spectrum((codes_of(kc[pg, a, off], bits).double() * ks[pg, a, off].double()[..., None]).flatten(-2) * lam[0], signs)
            v = from_spectrum((codes_of(vc[pg, a, off // 4, :, off % 4], bits).double() * vs[pg, a, off // 4, :, off % 4].double()[..., None])
                              .flatten(-2) * lam[1], signs)
            for i in range(0, m[b], 1024):
                rows = slice(at + i, at + min(m[b], i + 1024))
                q = st["q"][rows, a * grp:(a + 1) * grp].double()
                s = torch.matmul(q, k.t().contiguous()) / math.sqrt(D)
                if case["softcap"]:
                    s = case["softcap"] * torch.tanh(s / case["softcap"])
                pos = (n - m[b] + i + torch.arange(q.shape[0], device="cuda"))[:, None, None]
                see = (t <= pos) if case["causal"] else (t >= 0).expand(q.shape[0], 1, n)
                if case["window"]:
                    see = see & (t > pos - case["window"])
                s = torch.softmax(torch.where(see, s, torch.full_like(s, -math.inf)), -1)
                out[rows, a * grp:(a + 1) * grp] = torch.matmul(s, v)
                if weights is not None:
                    weights[b, a, :n] += s.sum((0, 1))
        at += m[b]
    return out if weights is None else (out, weights)
