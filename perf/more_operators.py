"""Cases, plain forms and 64-bit values of the operators around the paged SRFT cache: places, prompts and drafts.

A layer's paged cache is one uint8 tensor [pages][kv heads][page bytes]; a page holds P tokens (P a multiple of
16) of one KV head, D = 128 coordinates each, in the SRFT codec's form at `bits` = 4 or 8: a vector x is stored as
y = pack(F diag(s) x) / lambda, 16 groups of 8 coordinates with a binary16 scale Delta each and signed codes.
With E = 4 or 8 bytes per group's 8 codes, the page holds, in this order:

    K codes  [P][16][E]        K scales [P][16] binary16
    V codes  [P/4][16][4][E]   V scales [P/4][16][4] binary16   (blocks of four tokens, group by group)

Token t of sequence b is slot t % P of page table[b][t / P].  The operators:

  reserve  sequences grow and shrink: pages come from and go to a stack of free ones; the new tokens' slots
  prompt   softmax attention within packed prompts, on the keys and values themselves
  tree     softmax attention of drafted tokens over the cache: each sees the cached ones and its own ancestors
  accept   the drafted tokens that the model would have chosen move to the sequence's end in the cache
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
        # the next token of four sequences: latency counts
        dict(name="reserve_4_tokens", op="reserve", seqs=4, new=1, len=1000, page=16, mixed=False, short=False),
        # a batch that takes in prompts while others decode, draft or end, from a pool that runs out
        dict(name="reserve_333_prompts", op="reserve", seqs=333, new=211, len=4096, page=64, mixed=True, short=True),
        # a handful of short prompts
        dict(name="prompt_3x100_ragged", op="prompt", seqs=3, len=100, ragged=True, heads=8, group=4, causal=True, window=0, softcap=0.0, fused=True),
        # packed prompts of middling length, no two alike
        dict(name="prompt_16x2048_ragged", op="prompt", seqs=16, len=2048, ragged=True, heads=8, group=4, causal=True, window=0, softcap=0.0, fused=True),
        # odd group and length, capped scores, a sliding window
        dict(name="prompt_2x4001_window_cap", op="prompt", seqs=2, len=4001, ragged=False, heads=4, group=7, causal=True, window=1024, softcap=30.0, fused=False),
        # one long document
        dict(name="prompt_1x16384", op="prompt", seqs=1, len=16384, ragged=False, heads=8, group=4, causal=True, window=0, softcap=0.0, fused=True),
        # a short conversation's drafts
        dict(name="tree_1x301_q8", op="tree", seqs=1, len=301, ragged=False, q=8, heads=8, group=4, page=16, bits=4, window=0, softcap=0.0, lam=False),
        # a long document's drafts: the cache's length is all there is to split
        dict(name="tree_1x32768_q64", op="tree", seqs=1, len=32768, ragged=False, q=64, heads=8, group=4, page=64, bits=4, window=0, softcap=0.0, lam=False),
        # a ragged batch of long sequences, a few drafts each
        dict(name="tree_16x8192_q16_ragged", op="tree", seqs=16, len=8192, ragged=True, q=16, heads=8, group=4, page=64, bits=4, window=0, softcap=0.0, lam=True),
        # a wide batch at 8 bits with capped scores
        dict(name="tree_64x2001_q13_cap_8bit", op="tree", seqs=64, len=2001, ragged=True, q=13, heads=4, group=2, page=32, bits=8, window=0, softcap=30.0, lam=False),
        # one sequence's few drafts
        dict(name="accept_1x8", op="accept", seqs=1, len=301, ragged=False, q=8, keep=4, heads=8, page=16, bits=4),
        # a wide batch's large trees
        dict(name="accept_64x64_8bit", op="accept", seqs=64, len=1025, ragged=True, q=64, keep=9, heads=8, page=64, bits=8),
    ]


def draw(rng):
    def between(lo, hi):  # over the logarithm
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    op = rng.choice(["reserve", "prompt", "prompt", "tree", "tree", "tree", "accept"])
    c = dict(op=op)
    if op == "reserve":
        c.update(seqs=between(1, 512), page=rng.choice([16, 32, 64, 128, 256]), mixed=rng.random() < 0.6, short=rng.random() < 0.3)
        c["new"] = between(1, min(4096, (1 << 17) // c["seqs"]))
        c["len"] = between(1, 8192)
        return c
    c.update(seqs=between(1, 64), heads=rng.choice([1, 2, 4, 8]), ragged=rng.random() < 0.7)
    if op == "accept":
        c.update(page=rng.choice([16, 32, 64, 128, 256]), bits=rng.choice([4, 4, 8]), len=between(1, 2048))
        c["q"] = between(1, min(256, c["len"]))
        c["keep"] = rng.randint(1, min(c["q"], 16))
        return c
    c.update(group=rng.choice([1, 2, 3, 4, 7, 8]), softcap=rng.choice([0.0, 0.0, 20.0, 50.0]))
    if op == "prompt":
        most = math.isqrt((1 << 33) // (c["seqs"] * c["heads"] * c["group"]))  # the scores of the longest listed one
        c["len"] = between(1, min(16384, most))
        c.update(causal=rng.random() < 0.8, fused=rng.random() < 0.5)
    else:
        c["len"] = between(1, min(32768, (1 << 18) // c["seqs"]))
        rows = (1 << 29) // (c["seqs"] * c["len"] * c["heads"] * c["group"])
        c["q"] = between(1, max(1, min(c["len"], rows, 256)))
        c.update(page=rng.choice([16, 32, 64, 128, 256]), bits=rng.choice([4, 4, 8]), lam=rng.random() < 0.3)
    c["window"] = between(1, c["len"]) if rng.random() < 0.25 else 0
    return c


def seq_lens(case):
    n, top = case["seqs"], case["len"]
    return [max(1, top - int((b * 0.6180339887 % 1.0) * 0.75 * top)) if case.get("ragged") else top for b in range(n)]


def draft_lens(case):
    return [min(case["q"], n) for n in seq_lens(case)]


def reserve_counts(case):
    """The change of each sequence's length: prompts (most of the new tokens), single tokens, drafts, ends and rejected drafts."""
    r, n = random.Random(3), case["seqs"]
    if not case["mixed"]:
        return [case["new"]] * n
    return [1 + r.randrange(2 * case["new"]) if b % 4 == 0 else 1 if b % 4 == 1 else 8 if b % 4 == 2 else r.choice([-case["len"], -r.randint(0, 7)]) for b in range(n)]


def reserve_lens(case, seed):
    """Tokens that each sequence holds before: none where a prompt comes in."""
    r = random.Random(seed)
    return [0 if case["mixed"] and b % 4 == 0 else r.randint(1, case["len"]) for b in range(case["seqs"])]


def token_bytes(case):
    return 2 * (GROUPS * case["bits"] + 32)  # K and V of one token and head


def pairs_of(case, n):
    """Visible (query, token) pairs of a prompt of n tokens."""
    i = np.arange(n)
    hi = i + 1 if case["causal"] else np.full(n, n)
    lo = np.maximum(0, i + 1 - case["window"]) if case["window"] else np.zeros(n, np.int64)
    return int(np.maximum(0, hi - lo).sum())


def work(case):
    if case["op"] == "reserve":
        lens, counts, p = reserve_lens(case, 0), reserve_counts(case), case["page"]
        pages = sum(abs(-(-max(0, n + c) // p) + -n // p) for n, c in zip(lens, counts))
        tokens = sum(max(c, 0) for c in counts)
        return {"bytes": 2 * (20 * case["seqs"] + 12 * tokens + 8 * pages), "flops": 0}
    h, lens = case["heads"], seq_lens(case)
    if case["op"] == "accept":
        moved = sum(min(case["keep"], m) - 1 for m in draft_lens(case))
        return {"bytes": 2 * moved * h * token_bytes(case) + 12 * sum(draft_lens(case)) + 16 * case["seqs"], "flops": 0}
    if case["op"] == "prompt":
        rows = sum(lens)
        return {"bytes": rows * h * (2 + 2 * case["group"]) * D * 2, "flops": 4 * D * h * case["group"] * sum(pairs_of(case, n) for n in lens)}
    pairs = seen = rows = 0
    for n, m in zip(lens, draft_lens(case)):
        held = min(n - m, case["window"]) if case["window"] else n - m
        pairs += m * held + 4 * m  # a few ancestors each
        seen += held + m
        rows += m
    return {"bytes": seen * h * token_bytes(case) + rows * h * case["group"] * D * 4, "flops": 4 * D * pairs * h * case["group"]}


# ---- the transform and the pages -------------------------------------------------------------------

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
    k = np.arange(1, D // 2)[:, None]
    a = 2 * np.pi * (k * n % D) / D
    rows = np.sqrt(2) * np.stack([np.cos(a), -np.sin(a)], 1).reshape(-1, D)
    return np.concatenate([np.ones((1, D)), np.cos(np.pi * n)[None], rows]) / np.sqrt(D) * sign_diagonal(seed)


def parts(cache, bits):
    """K codes [pages][heads][P][16][E], K scales [..][P][16], V codes [..][P/4][16][4][E], V scales [..][P/4][16][4]."""
    size = cache.shape[2]
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


# ---- what a program has in hand --------------------------------------------------------------------


def some_tree(r, m):
    """Parents of m drafted tokens: the first follows the cached ones, the others an earlier draft, mostly a late one."""
    return [-1] + [max(0, i - 1 - int(r.expovariate(0.4))) for i in range(1, m)]


def filled(pages, case, g):
    """A cache whose every slot holds random codes, with scales that give values the spread of a KV workload."""
    h, p, bits = case["heads"], case["page"], case["bits"]
    cache = torch.empty(pages, h, p * token_bytes(case), dtype=torch.uint8, device="cuda")
    cache.random_(0, 256, generator=g)
    kc, ks, vc, vs = parts(cache, bits)
    if bits == 8:  # codes are -127..127
        kc.masked_fill_(kc == 128, 0)
        vc.masked_fill_(vc == 128, 0)
    else:  # -7..7: a nibble of 8 becomes 0
        for c in (kc, vc):
            c.copy_(torch.where(c >> 4 == 8, c & 15, c))
            c.copy_(torch.where(c & 15 == 8, c & 240, c))
    top = 7.0 if bits == 4 else 127.0
    for s in (ks, vs):
        s.copy_((0.4 + 1.6 * torch.rand(s.shape, generator=g, device="cuda")) / top)
    return cache


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = random.Random(seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    st = dict(case=case)
    if case["op"] == "reserve":
        lens, counts, p = reserve_lens(case, seed), reserve_counts(case), case["page"]
        up = lambda n: -(-n // p)  # noqa: E731
        used = [up(n) for n in lens]
        need = sum(up(n + c) - up(n) for n, c in zip(lens, counts) if c > 0)
        spare = need // 2 if case["short"] else need + 5
        total = sum(up(case["len"]) + up(max(c, 0)) + 1 for c in counts) + 5
        pages = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        width = up(case["len"] + max(max(counts), 0)) + 1
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(width, device="cuda") < i32(used)[:, None]] = pages[:sum(used)]
        free = torch.full_like(pages, -1)
        free[:spare] = pages[sum(used):sum(used) + spare]
        return dict(st, table=table, lens=i32(lens), counts=i32(counts), free=free, free_count=i32([spare]), tokens=sum(max(c, 0) for c in counts) + 3,
                    back=sum(min(-c, case["len"]) for c in counts if c < 0))
    h, lens = case["heads"], seq_lens(case)
    if case["op"] == "prompt":
        total, grp = sum(lens), case["group"]
        if case["fused"]:  # rows of a fused projection: queries, keys, values
            row = torch.randn(total, (grp + 2) * h * D, generator=g, device="cuda").to(torch.bfloat16)
            q, k, v = row[:, :grp * h * D].unflatten(1, (grp * h, D)), row[:, grp * h * D:(grp + 1) * h * D].unflatten(1, (h, D)), row[:, (grp + 1) * h * D:].unflatten(1, (h, D))
        else:
            q, k, v = (torch.randn(total, n, D, generator=g, device="cuda").to(torch.bfloat16) for n in (grp * h, h, h))
        loud = (1 + 9 * (torch.rand(h, D, generator=g, device="cuda") < 0.03)).to(torch.bfloat16)
        # each query looks for a token of its sequence
        start = np.concatenate([[0], np.cumsum(lens)])
        first = torch.repeat_interleave(torch.from_numpy(start[:-1]).cuda(), i32(lens).long(), output_size=total)
        at = first + (torch.rand(total, generator=g, device="cuda") * (torch.arange(total, device="cuda") - first + 1)).long()
        q += 0.5 * k[at].repeat_interleave(grp, 1)
        k.mul_(loud)
        return dict(st, q=q, k=k, v=v, start=i32(start.tolist()))

    p, bits = case["page"], case["bits"]
    m = draft_lens(case)
    used = [-(-n // p) for n in lens]
    cache = filled(sum(used) + 2, case, g)
    order = torch.randperm(sum(used) + 2, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(used)), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(max(used), device="cuda") < i32(used)[:, None]] = order[:sum(used)]
    start = np.concatenate([[0], np.cumsum(m)]).tolist()
    trees = [some_tree(r, n) for n in m]
    st.update(cache=cache, table=table, lens=i32(lens), start=i32(start), max_q=max(m), max_len=max(lens))
    if case["op"] == "accept":
        tokens, target = [], []
        for t, n in zip(trees, m):
            keep = min(case["keep"], n)
            path = [0] + sorted(r.sample(range(1, n), keep - 1))
            tok, tgt = [r.randrange(32000) for _ in range(n)], [32000 + r.randrange(99) for _ in range(n)]
            for a, b in zip(path, path[1:]):
                t[b], tgt[a] = a, tok[b]
            tokens += tok
            target += tgt
        return dict(st, tokens=i32(tokens), target=i32(target), parents=i32(sum(trees, [])))
    lam = [np.array([r.uniform(0.5, 2.0) for _ in range(D)], np.float32) if case["lam"] else None for _ in range(2)]
    lams = [torch.ones(D, device="cuda") if a is None else torch.from_numpy(a).cuda() for a in lam]
    T = torch.from_numpy(transform_matrix(SEED)).cuda().float()
    hq = h * case["group"]
    rows = torch.randn(start[-1], (hq + 2 * h) * D, generator=g, device="cuda").to(torch.bfloat16)
    q = rows[:, :hq * D].unflatten(1, (hq, D))  # beside the new keys and values, as a fused projection leaves them
    # a key of its sequence that each query looks for
    kc, ks = parts(cache, bits)[:2]
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), i32(m).long(), output_size=start[-1])[:, None]
    tok = (torch.rand(start[-1], hq, generator=g, device="cuda") * st["lens"][seq]).long()
    pg, head = table[seq, tok // p].long(), torch.arange(hq, device="cuda") // case["group"]
    y = (codes_of(kc[pg, head, tok % p], bits).float() * ks[pg, head, tok % p].float()[..., None]).flatten(-2)
    q += (0.7 * torch.matmul(y * lams[0], T)).to(torch.bfloat16)
    return dict(st, q=q, parents=i32(sum(trees, [])), lam=lam, lams=lams, T=T)


# ---- one pass --------------------------------------------------------------------------------------


def run(st):
    return {"reserve": run_reserve, "prompt": run_prompt, "tree": run_tree, "accept": run_accept}[st["case"]["op"]](st)


def run_reserve(st):
    """A step's change, and the change that takes it back."""
    if own:
        import kv_quantization_tile_amd as hq
        reserve = hq.hq_kv_reserve
    else:
        reserve = plain_reserve
    table, lens, free, count, page = st["table"], st["lens"], st["free"], st["free_count"], st["case"]["page"]
    there = reserve(table, lens, st["counts"], free, count, page, st["tokens"])
    back = reserve(table, lens, there[3].neg(), free, count, page, st["back"])
    return there, back, table, lens, free, count


def plain_reserve(table, lens, counts, free, free_count, page, tokens):
    seqs, width = table.shape
    pages = free.numel()
    up = lambda n: (n + page - 1) // page  # noqa: E731
    old, c = lens.long().clamp(0, width * page), counts.long()
    j = torch.arange(width, device=table.device)
    # pages that go back: the last of the last sequence first
    shrunk = torch.where(c < 0, (old + c).clamp(min=0), old)
    gone = (j >= up(shrunk)[:, None]) & (j < up(old)[:, None])
    pushed = (gone & (table >= 0) & (table < pages)).flatten()
    rank = pushed.cumsum(0)
    at = free_count.long().clamp(0, pages) + pushed.sum() - rank
    stack = torch.cat([free, free.new_zeros(1)])
    stack[torch.where(pushed & (at < pages), at, torch.full_like(at, pages))] = table.flatten()
    table[:] = torch.where(gone, torch.full_like(table, -1), table)
    held = (free_count.long().clamp(0, pages) + pushed.sum()).clamp(max=pages)
    # pages that are taken: the first sequence's first, as far as they go
    fits = (c > 0) & (old + c <= width * page)
    need = torch.where(fits, up(old + c) - up(old), torch.zeros_like(c))
    can = fits & (need.cumsum(0) <= held)
    taken = can[:, None] & (j >= up(old)[:, None]) & (j < up(old + c)[:, None])
    at = (held - taken.flatten().cumsum(0)).clamp(min=0).view_as(taken)
    table[:] = torch.where(taken, stack[at], table)
    free[:] = stack[:pages]
    free_count[:] = (held - taken.sum()).to(torch.int32)
    change = torch.where(c < 0, shrunk - old, torch.where(can, c, torch.zeros_like(c)))
    lens[:] = torch.where(change != 0, old + change, lens.long()).to(torch.int32)
    # the new tokens
    start = torch.cat([c.new_zeros(1), c.clamp(min=0).cumsum(0)])
    i = torch.arange(tokens, device=table.device)
    b = torch.searchsorted(start, i, right=True) - 1
    here = b < seqs
    b = b.clamp(max=seqs - 1)
    t = torch.where(here, old[b] + i - start[b], torch.zeros_like(i))
    entry = table[b, (t // page).clamp(max=width - 1)].long()
    fine = here & can[b] & (entry >= 0) & (entry < pages)
    slots = torch.where(fine, entry * page + t % page, torch.full_like(t, -1))
    return slots, t.to(torch.int32), start.to(torch.int32), change.to(torch.int32)


def softmax_(s):
    """exp(s) over its sum along the last dimension; a row of -inf gives 0."""
    s = s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = s.sum(-1, keepdim=True)
    return s.div_(torch.where(total > 0, total, torch.ones_like(total)))


def padded(x, start, top):
    """x [rows][heads][128] by sequences: [seqs][heads][top][128] in 32 bits, and where a row is in x, and whether it is there."""
    first, m = start[:-1].long(), (start[1:] - start[:-1]).long()
    i = torch.arange(top, device="cuda")
    have = i < m[:, None]
    at = torch.where(have, first[:, None] + i, torch.zeros_like(i))
    return x[at].float().mul_(have[..., None, None]).transpose(1, 2).contiguous(), at, have


def run_prompt(st):
    c, start = st["case"], st["start"]
    if own:
        import kv_quantization_tile_amd as hq
        return hq.hq_attend_prompt(st["q"], st["k"], st["v"], start, causal=c["causal"], window=c["window"], softcap=c["softcap"])
    h, grp, top = c["heads"], c["group"], max(seq_lens(c))
    q, at, have = padded(st["q"], start, top)
    k, v = padded(st["k"], start, top)[0], padded(st["v"], start, top)[0]
    s = torch.matmul(q.unflatten(1, (h, grp)), k.transpose(2, 3).contiguous()[:, :, None]).mul_(1 / math.sqrt(D))
    if c["softcap"]:
        s = s.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    i = torch.arange(top, device="cuda")
    hidden = ~have[:, None, :].expand(-1, top, -1)
    if c["causal"]:
        hidden = hidden | (i > i[:, None])
    if c["window"]:
        hidden = hidden | (i <= i[:, None] - c["window"])
    s = softmax_(s.masked_fill_(hidden[:, None, None], -math.inf))
    o = torch.matmul(s, v[:, :, None]).flatten(1, 2).transpose(1, 2)
    out = torch.empty(st["q"].shape, dtype=torch.bfloat16, device="cuda")
    out[at[have]] = o[have].to(torch.bfloat16)
    return out


def ancestors(parents, start, m):
    """[seqs][m][m]: whether draft j is draft i or an ancestor of it."""
    first, n = start[:-1].long(), (start[1:] - start[:-1]).long()
    i = torch.arange(m, device="cuda")
    have = i < n[:, None]
    p = torch.where(have, parents[torch.where(have, first[:, None] + i, torch.zeros_like(i))].long(), torch.full_like(i, -1))
    up = (p[..., None] == i).float() + torch.eye(m, device="cuda")
    for _ in range(max(1, (m - 1).bit_length())):  # chains of twice the length
        up = torch.matmul(up, up).clamp_(max=1)
    return up > 0, p, have


def run_tree(st):
    c, bits, table, lens = st["case"], st["case"]["bits"], st["table"], st["lens"]
    if own:
        import kv_quantization_tile_amd as hq
        return hq.hq_kv_attend(st["cache"], st["q"], table, lens, q_start=st["start"], max_q=st["max_q"], max_len=st["max_len"], bits=bits,
                               seed=SEED, lam_k=st["lam"][0], lam_v=st["lam"][1], window=c["window"], softcap=c["softcap"], parents=st["parents"])
    kc, ks, vc, vs = parts(st["cache"], bits)
    h, grp, pages, m = c["heads"], c["group"], table.clamp(min=0).long(), st["max_q"]
    n, width = table.shape
    top = st["max_len"]
    # keys and values of the padded sequences, [seqs][heads][top][128]
    y = codes_of(kc[pages], bits).float() * ks[pages].float()[..., None]
    k = torch.matmul(y.transpose(1, 2).reshape(n, h, width * c["page"], D)[:, :, :top] * st["lams"][0], st["T"])
    y = codes_of(vc[pages], bits).float() * vs[pages].float()[..., None]
    v = torch.matmul(y.transpose(4, 5).transpose(1, 2).reshape(n, h, width * c["page"], D)[:, :, :top] * st["lams"][1], st["T"])
    q, at, have = padded(st["q"], st["start"], m)
    s = torch.matmul(q.unflatten(1, (h, grp)).flatten(2, 3), k.transpose(2, 3).contiguous()).mul_(1 / math.sqrt(D))
    if c["softcap"]:
        s = s.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    # drafts lie behind the held tokens; draft i stands as far behind them as it has ancestors
    up = ancestors(st["parents"], st["start"], m)[0]
    depth = up.sum(-1) - 1
    held = lens.long() - (st["start"][1:] - st["start"][:-1])
    t = torch.arange(top, device="cuda")
    j = t - held[:, None]
    of = j.clamp(0, m - 1)
    see = torch.where((j >= 0)[:, None], up.gather(2, of[:, None].expand(n, m, top)), torch.ones_like(up[:, :, :1])) & (t < lens[:, None])[:, None] & have[..., None]
    if c["window"]:
        pos = t + torch.where(j >= 0, depth.gather(1, of) - j, torch.zeros_like(j))
        see = see & (pos[:, None] > (held[:, None] + depth)[..., None] - c["window"])
    s = softmax_(s.unflatten(2, (grp, m)).masked_fill_(~see[:, None, None], -math.inf))
    o = torch.matmul(s.flatten(2, 3), v).unflatten(2, (grp, m)).flatten(1, 2).transpose(1, 2)
    out = torch.empty(st["q"].shape, dtype=torch.bfloat16, device="cuda")
    out[at[have]] = o[have].to(torch.bfloat16)
    return out


def run_accept(st):
    c, bits, table, lens, m, p = st["case"], st["case"]["bits"], st["table"], st["lens"], st["max_q"], st["case"]["page"]
    tokens, target, start = st["tokens"], st["target"], st["start"]
    if own:
        import kv_quantization_tile_amd as hq
        got = hq.hq_kv_accept(st["cache"], table, lens, tokens, target, st["parents"], q_start=start, max_q=m, bits=bits)
        return (*got, st["cache"])
    up, parent, have = ancestors(st["parents"], start, m)
    i = torch.arange(m, device="cuda")
    at = torch.where(have, start[:-1, None].long() + i, torch.zeros_like(i))
    tok, tgt = tokens[at], target[at]
    # a draft is right after its parent if it is what the parent's target asks for and no earlier child is
    right = have & (parent >= 0) & (tok == tgt.gather(1, parent.clamp(min=0)))
    earlier = (right[:, None, :] & (parent[:, None, :] == parent[..., None]) & (i < i[:, None])).any(-1)
    right = right & ~earlier
    right[:, 0] = have[:, 0]
    good = have & (~up | right[:, None, :]).all(-1) & up[:, :, 0]
    path = torch.where(good, i, torch.full_like(i, m)).sort(-1).values
    count = good.sum(-1)
    last = path.gather(1, (count - 1).clamp(min=0)[:, None])[:, 0].clamp(max=m - 1)
    nxt = torch.where(count > 0, tgt.gather(1, last[:, None])[:, 0], torch.full_like(count, -1, dtype=torch.int32))
    held = lens.long() - have.sum(-1)
    b, k = torch.nonzero(path < m, as_tuple=True)
    src, dst = held[b] + path[b, k], held[b] + k
    sp, so, dp, do = table[b, src // p].long(), src % p, table[b, dst // p].long(), dst % p
    kc, ks, vc, vs = parts(st["cache"], bits)
    kc[dp, :, do] = kc[sp, :, so]
    ks[dp, :, do] = ks[sp, :, so]
    vc[dp, :, do // 4, :, do % 4] = vc[sp, :, so // 4, :, so % 4]
    vs[dp, :, do // 4, :, do % 4] = vs[sp, :, so // 4, :, so % 4]
    path = torch.where(path < m, path, torch.full_like(path, -1)).to(torch.int32)
    return path, count.to(torch.int32), nxt, (count - have.sum(-1)).to(torch.int32), st["cache"]


# ---- the same in 64 bits, from the definition ------------------------------------------------------


def from_spectrum(y, signs):
    """diag(s) F^-1 unpack(y), by the inverse discrete Fourier transform."""
    inner = torch.view_as_complex((y[..., 2:] / math.sqrt(2)).unflatten(-1, (-1, 2)).contiguous())
    X = torch.cat([y[..., :1] + 0j, inner, y[..., 1:2] + 0j], -1)
    return torch.fft.irfft(X, n=D, norm="ortho") * signs


def attend64(q, k, v, see, softcap):
    """Rows q [rows][heads][128] over k, v [tokens][128] in 64 bits; see [rows][tokens]."""
    s = torch.matmul(q, k.t().contiguous()) / math.sqrt(D)
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    return torch.matmul(torch.softmax(torch.where(see[:, None], s, torch.full_like(s, -math.inf)), -1), v)


def exact(case, seed):
    if case["op"] in ("reserve", "accept"):  # whole numbers alone
        return None
    st = prepare(case, seed)
    grp, h, lens = case["group"], case["heads"], seq_lens(case)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    if case["op"] == "prompt":
        for n in lens:
            t = torch.arange(n, device="cuda")
            for a in range(h):
                k, v = st["k"][at:at + n, a].double(), st["v"][at:at + n, a].double()
                for i in range(0, n, 1024):
                    rows = slice(at + i, at + min(n, i + 1024))
                    pos = (i + torch.arange(rows.stop - rows.start, device="cuda"))[:, None]
                    see = (t <= pos) if case["causal"] else (t >= 0).expand(len(pos), n)
                    if case["window"]:
                        see = see & (t > pos - case["window"])
                    out[rows, a * grp:(a + 1) * grp] = attend64(st["q"][rows, a * grp:(a + 1) * grp].double(), k, v, see, case["softcap"])
            at += n
        return out
    bits, p = case["bits"], case["page"]
    signs = torch.from_numpy(sign_diagonal(SEED)).cuda()
    lam = [a.double() for a in st["lams"]]
    kc, ks, vc, vs = parts(st["cache"], bits)
    parents = st["parents"].tolist()
    for b, (n, m) in enumerate(zip(lens, draft_lens(case))):
        # which tokens a draft sees, walked up the tree
        see = np.zeros((m, n), bool)
        for i in range(m):
            chain, j = [], i
            while j >= 0:
                chain.append(n - m + j)
                j = parents[at + j]
            seen = list(range(n - m)) + chain[::-1]
            see[i, seen[-case["window"]:] if case["window"] else seen] = True
        see = torch.from_numpy(see).cuda()
        t = torch.arange(n, device="cuda")
        pg, off = st["table"][b, t // p].long(), t % p
        for a in range(h):
            k = from_spectrum((codes_of(kc[pg, a, off], bits).double() * ks[pg, a, off].double()[..., None]).flatten(-2) * lam[0], signs)
            v = from_spectrum((codes_of(vc[pg, a, off // 4, :, off % 4], bits).double() * vs[pg, a, off // 4, :, off % 4].double()[..., None])
                              .flatten(-2) * lam[1], signs)
            heads = slice(a * grp, (a + 1) * grp)
            out[at:at + m, heads] = attend64(st["q"][at:at + m, heads].double(), k, v, see, case["softcap"])
        at += m
    return out
