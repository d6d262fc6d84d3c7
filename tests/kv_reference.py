"""The paged SRFT cache in NumPy, binary64, from its definition: page layout, the transform, attention with its
error bound, and eviction.  Shares no code with the package."""
import numpy as np

D, GROUPS = 128, 16


def signs(orc, seed):
    """The sign diagonal: the first coordinate of unit vector i is s_i / sqrt 128."""
    return np.array([np.sign(orc.srft_forward(row, seed)[0]) for row in np.eye(D, dtype=np.float32)], np.float64)


def transform(orc, seed):
    """T of pack(F diag(s) x) = T x, orthogonal."""
    s, n = signs(orc, seed), np.arange(D)
    rows = [np.ones(D), (-1.0) ** n]
    for k in range(1, D // 2):
        a = 2 * np.pi * (k * n % D) / D
        rows += [np.sqrt(2) * np.cos(a), -np.sqrt(2) * np.sin(a)]
    return np.stack(rows) / np.sqrt(D) * s


def parts(cache, bits):
    """Views of a uint8 cache [pages][heads][page bytes]: K codes [pages][heads][P][16][E], K scales [..][P][16], V codes
    [..][P/4][16][4][E], V scales [..][P/4][16][4] (scales as binary16)."""
    n, h, size = cache.shape
    p = size // (2 * (16 * bits + 32))
    a, b = p * 16 * bits, p * 32
    kc, ks, vc, vs = cache[..., :a], cache[..., a:a + b], cache[..., a + b:2 * a + b], cache[..., 2 * a + b:]
    return (kc.reshape(n, h, p, 16, bits), ks.view(np.float16).reshape(n, h, p, 16),
            vc.reshape(n, h, p // 4, 16, 4, bits), vs.view(np.float16).reshape(n, h, p // 4, 16, 4))


def tokens_of(cache, bits):
    """Codes and scales token by token: K codes [pages][heads][P][16][E], K scales [..][16], V codes, V scales."""
    kc, ks, vc, vs = parts(cache, bits)
    n, h, p = ks.shape[:3]
    return kc, ks, vc.swapaxes(3, 4).reshape(n, h, p, 16, bits), vs.swapaxes(3, 4).reshape(n, h, p, 16)


def ints(raw, bits):
    """Signed codes [..][16][8] of bytes [..][16][E]."""
    if bits == 8:
        return raw.view(np.int8).astype(np.int64)
    u = raw.astype(np.int64)
    c = np.stack([u & 15, u >> 4], -1).reshape(raw.shape[:-1] + (8,))
    return c - 16 * (c > 7)


def coordinates(cache, bits, table_row, n, head, lam_k, lam_v):
    """Transformed coordinates of a sequence's n tokens, with lambda: K [n][128], V [n][128], and which are there."""
    kc, ks, vc, vs = tokens_of(cache, bits)
    pages, p = cache.shape[0], ks.shape[2]
    t = np.arange(n)
    pg = np.asarray(table_row)[t // p] if n else np.zeros(0, int)
    there = (pg >= 0) & (pg < pages)
    at = (np.where(there, pg, 0), head, t % p)
    k = (ints(kc[at], bits) * ks[at].astype(np.float64)[..., None]).reshape(n, D) * lam_k
    v = (ints(vc[at], bits) * vs[at].astype(np.float64)[..., None]).reshape(n, D) * lam_v
    return k, v, there


def attend(orc, cache, q, table, lens, q_lens, bits, seed, lam_k=None, lam_v=None, scale=D ** -0.5, causal=True, window=0,
           softcap=0.0, precise=False):
    """Outputs [queries][q heads][128] and weights [seqs][heads][max len], and for each output row and weight the error
    that the kernel's roundings may make (an error of the row's 2-norm; one of each weight):

      a score of 16-bit factors     query and key coordinates are each off by 2^-11: 2^-10 A, A = scale sum |q_c k_c|
      the same in two parts         lo parts off by 2^-11 of 2^-11, their product left out: 3 2^-22 A
      sums of 128 products, binary32     2^-17 A in either; the transform's 12 roundings and the cap's tanh: 2^-20 (A + cap)
      a softmax weight, scores off by e  exp(2 e) - 1, times 1 + 2^-20 for exp2 and the sums
      a weight as binary16          2^-11 in the product, 2^-11 in the sum; below its range 2^-33 of the largest a token
      a value coordinate            2^-11
    """
    T = transform(orc, seed)
    lam_k = np.ones(D) if lam_k is None else np.asarray(lam_k, np.float64)
    lam_v = np.ones(D) if lam_v is None else np.asarray(lam_v, np.float64)
    h, hq, top = cache.shape[1], q.shape[1], max([0, *lens])
    out, tol = np.zeros(q.shape), np.zeros(q.shape[:2])
    weights, wtol = np.zeros((len(lens), h, top)), np.zeros((len(lens), h, top))
    at = 0
    with np.errstate(invalid="ignore", over="ignore"):
        for b, (n, m) in enumerate(zip(lens, q_lens)):
            for j in range(hq):
                a = j // (hq // h)
                k, v, there = coordinates(cache, bits, table[b], n, a, lam_k, lam_v)
                y = q[at:at + m, j].astype(np.float64) @ T.T * scale
                pos = n - m + np.arange(m)[:, None]
                t = np.arange(n)
                see = there & ((t <= pos) if causal else np.ones((m, n), bool))
                if window:
                    see &= t > pos - window
                for i in range(m):
                    w = see[i]
                    if not w.any():
                        continue
                    s = k[w] @ y[i]
                    big = (np.abs(k[w]) @ np.abs(y[i])).max()
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                    e = np.exp(s - s.max())
                    p = e / e.sum()
                    out[at + i, j] = (p @ v[w]) @ T
                    eps = (3 * 2.0 ** -22 if precise else 2.0 ** -10) * big + 2.0 ** -17 * big + 2.0 ** -20 * (big + softcap)
                    rel = np.exp(2 * eps) * (1 + 2.0 ** -20) - 1
                    tol[at + i, j] = (rel + 3 * 2.0 ** -11 + 2.0 ** -17) * np.linalg.norm(p @ np.abs(v[w])) + \
                        2.0 ** -33 * w.sum() * np.abs(v[w]).max() * np.sqrt(D)
                    weights[b, a, :n][w] += p
                    wtol[b, a, :n][w] += p * rel + 2.0 ** -40
            at += m
    return out, tol, weights, wtol


def evict(weights, lens, budget, sink, recent):
    """Indices that stay [seqs][heads][budget] (-1 past the end) and the new lengths."""
    n, h, _ = weights.shape
    kept, left = np.full((n, h, budget), -1, np.int32), np.zeros(n, np.int32)
    for b in range(n):
        m = left[b] = min(lens[b], budget)
        t = np.arange(lens[b])
        fixed = (t < sink) | (t >= lens[b] - recent)
        for a in range(h):
            w = weights[b, a, :lens[b]].astype(np.float64)
            w = np.where(np.isnan(w), -np.inf, w)
            last = np.isnan(weights[b, a, :lens[b]])  # NaN after -inf
            kept[b, a, :m] = np.sort(np.lexsort((t, -w, last, ~fixed))[:m])
    return kept, left
