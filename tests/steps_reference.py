"""Places, prompts and drafts in NumPy, from their definitions: the page stack, attention within packed prompts, attention of a
tree of drafts over the paged cache (binary64, with error bounds), and the acceptance of drafts.  Shares no code with the package."""
import numpy as np

import kv_reference as ref

D = 128


# ---- places ------------------------------------------------------------------------------------


def reserve(table, lens, counts, free, free_count, page, tokens):
    """Updates table, lens, free (arrays) and returns (slots, positions, q_start, granted, free_count)."""
    seqs, width = table.shape
    pages = len(free)
    up = lambda n: -(-n // page)  # noqa: E731
    stack = [int(x) for x in free[:min(max(free_count, 0), pages)]]
    old = [min(max(int(n), 0), width * page) for n in lens]
    granted = np.zeros(seqs, np.int32)
    for b in reversed(range(seqs)):
        if counts[b] < 0:
            new = max(0, old[b] + int(counts[b]))
            granted[b] = new - old[b]
            for j in reversed(range(up(new), up(old[b]))):
                if 0 <= table[b, j] < pages and len(stack) < pages:
                    stack.append(int(table[b, j]))
                table[b, j] = -1
    full = False
    for b in range(seqs):
        if counts[b] <= 0 or old[b] + int(counts[b]) > width * page:
            continue
        need = up(old[b] + int(counts[b])) - up(old[b])
        full = full or need > len(stack)
        if not full:
            granted[b] = counts[b]
            for j in range(up(old[b]), up(old[b]) + need):
                table[b, j] = stack.pop()
    start = np.concatenate([[0], np.cumsum([max(int(c), 0) for c in counts])])
    slots, positions = np.full(tokens, -1, np.int64), np.zeros(tokens, np.int32)
    for b in range(seqs):
        for i in range(int(start[b]), min(int(start[b + 1]), tokens)):
            t = old[b] + i - int(start[b])
            positions[i] = t
            if granted[b] > 0 and 0 <= table[b, t // page] < pages:
                slots[i] = int(table[b, t // page]) * page + t % page
        if granted[b]:
            lens[b] = old[b] + granted[b]
    left = len(stack)
    free[:left] = stack
    return slots, positions, np.minimum(start, 2 ** 31 - 1).astype(np.int32), granted, left


# ---- prompts -----------------------------------------------------------------------------------


def prompt(q, k, v, start, scale=D ** -0.5, causal=True, window=0, softcap=0.0):
    """Outputs [rows][q heads][128] and, for each output row, the error of its 2-norm that the kernel's roundings may make:

      a score: a sum of 128 exact products in binary32      2^-17 A, A = scale sum |q_c k_c|
      its scale, and the cap's tanh (off by 2^-21)           2^-22 A + 2^-21 cap
      exp2 of y <= 0 in binary32, |y| < 150 where it is not 0  2^-16 of the weight
      a weight as bf16, in the product and in the sum       2 2^-8 of it
      a sum over n tokens in binary32                       n 2^-24 of sum p |v|
    """
    out, tol = np.zeros(q.shape), np.zeros(q.shape[:2])
    group = q.shape[1] // k.shape[1]
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    for b in range(len(start) - 1):
        n = start[b + 1] - start[b]
        rows = slice(start[b], start[b + 1])
        if n == 0:
            continue
        t, i = np.arange(n), np.arange(n)[:, None]
        see = (t <= i) if causal else np.ones((n, n), bool)
        if window:
            see = see & (t > i - window)
        for j in range(q.shape[1]):
            kk, vv = k[rows, j // group], v[rows, j // group]
            s = q[rows, j] @ kk.T * scale
            big = np.where(see, np.abs(q[rows, j]) @ np.abs(kk).T * abs(scale), 0).max(-1)
            if softcap:
                s = softcap * np.tanh(s / softcap)
            s = np.where(see, s, -np.inf)
            e = np.exp(s - s.max(-1, keepdims=True))
            p = e / e.sum(-1, keepdims=True)
            out[rows, j] = p @ vv
            eps = (2.0 ** -17 + 2.0 ** -22) * big + 2.0 ** -21 * softcap
            rel = np.exp(2 * eps) * (1 + 2.0 ** -16) - 1 + 2.0 ** -7 + n * 2.0 ** -24
            tol[rows, j] = rel * np.linalg.norm(p @ np.abs(vv), axis=-1)
    return out, tol


# ---- drafts ------------------------------------------------------------------------------------


def chain(parents, i):
    """Draft i and its ancestors, first to last."""
    path = []
    while i >= 0:
        path.append(i)
        i = parents[i] if 0 <= parents[i] < i else -1
    return path[::-1]


def tree_sees(parents, n, m, window=0):
    """[m][n]: which of a sequence's n tokens each of its m drafts sees."""
    see = np.zeros((m, n), bool)
    for i in range(m):
        seen = list(range(max(n - m, 0))) + [n - m + j for j in chain(parents, i)]
        if window:
            seen = seen[-window:]
        see[i, [t for t in seen if t >= 0]] = True
    return see


def attend(orc, cache, q, table, lens, sees, bits, seed, lam_k=None, lam_v=None, scale=D ** -0.5, softcap=0.0):
    """Outputs [queries][q heads][128] of queries that see what `sees` (a [queries][tokens] array a sequence) says, and the error
    that the kernel's roundings may make (the terms are kv_reference.attend's)."""
    T = ref.transform(orc, seed)
    lam_k = np.ones(D) if lam_k is None else np.asarray(lam_k, np.float64)
    lam_v = np.ones(D) if lam_v is None else np.asarray(lam_v, np.float64)
    h, hq = cache.shape[1], q.shape[1]
    out, tol = np.zeros(q.shape), np.zeros(q.shape[:2])
    at = 0
    with np.errstate(invalid="ignore", over="ignore"):
        for b, (n, see) in enumerate(zip(lens, sees)):
            m = len(see)
            for j in range(hq):
                k, v, there = ref.coordinates(cache, bits, table[b], n, j // (hq // h), lam_k, lam_v)
                y = q[at:at + m, j].astype(np.float64) @ T.T * scale
                for i in range(m):
                    w = see[i] & there
                    if not w.any():
                        continue
                    s = k[w] @ y[i]
                    big = (np.abs(k[w]) @ np.abs(y[i])).max()
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                    e = np.exp(s - s.max())
                    p = e / e.sum()
                    out[at + i, j] = (p @ v[w]) @ T
                    eps = (2.0 ** -10 + 2.0 ** -17) * big + 2.0 ** -20 * (big + softcap)
                    rel = np.exp(2 * eps) * (1 + 2.0 ** -20) - 1
                    tol[at + i, j] = (rel + 3 * 2.0 ** -11 + 2.0 ** -17) * np.linalg.norm(p @ np.abs(v[w])) + \
                        2.0 ** -33 * w.sum() * np.abs(v[w]).max() * np.sqrt(D)
            at += m
    return out, tol


def accept_path(tokens, target, parents):
    """The accepted drafts of one sequence."""
    path = [0] if len(tokens) else []
    while path:
        i = path[-1]
        nxt = [j for j in range(i + 1, len(tokens)) if parents[j] == i and tokens[j] == target[i]]
        if not nxt:
            break
        path.append(nxt[0])
    return path


def move(cache, bits, table, n, m, path, page):
    """Moves a sequence's accepted drafts in `cache` (an array), as accept does."""
    raw = ref.parts(cache, bits)
    kc, ks, vc, vs = raw[0], raw[1].view(np.uint16), raw[2], raw[3].view(np.uint16)
    pages, width = cache.shape[0], len(table)

    def at(t):
        ok = 0 <= t < width * page and 0 <= table[t // page] < pages
        return (int(table[t // page]), t % page) if ok else None

    held = []
    for j in path:
        a = at(n - m + j)
        if a is None:
            z = np.zeros_like
            held.append((z(kc[0, :, 0]), np.full_like(ks[0, :, 0], 0x8000), z(vc[0, :, 0, :, 0]), z(vs[0, :, 0, :, 0])))
        else:
            p, o = a
            held.append((kc[p, :, o].copy(), ks[p, :, o].copy(), vc[p, :, o // 4, :, o % 4].copy(), vs[p, :, o // 4, :, o % 4].copy()))
    for i, (j, x) in enumerate(zip(path, held)):
        a = at(n - m + i)
        if a is not None and i != j:
            p, o = a
            kc[p, :, o], ks[p, :, o], vc[p, :, o // 4, :, o % 4], vs[p, :, o // 4, :, o % 4] = x
