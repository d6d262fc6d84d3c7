"""One attention layer of a decoder over the paged SRFT cache: prompts in, tokens out, with a bounded cache.

A batch of prompts of different lengths is appended and attended in one call; then each sequence decodes
token by token.  Softmax weights accumulate per cached token, and whenever a sequence's cache passes `high`
tokens the batch is cut back to the `budget` tokens of most accumulated weight (the first and the most recent
ones always stay), which move to fresh pages; the old pages return to the pool.  The layer's projections are
random; positions are not encoded, so a token may move within the cache.

    python examples/paged_cache.py [--steps N] [--bits 4|8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kv_quantization_tile_amd as hq  # noqa: E402


class PagedLayer:
    def __init__(self, seqs, q_heads=8, kv_heads=2, page=16, high=256, budget=128, sink=4, recent=32, bits=4, seed=0):
        self.q_heads, self.kv_heads, self.page, self.bits, self.seed = q_heads, kv_heads, page, bits, seed
        self.high, self.budget, self.sink, self.recent = high, budget, sink, recent
        self.width = -(-high // page) + 1
        self.hidden = q_heads * 128
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.project = torch.randn(self.hidden, (q_heads + 2 * kv_heads) * 128, generator=g, device="cuda").bfloat16() / self.hidden ** 0.5
        pages = 2 * seqs * self.width
        self.cache = hq.hq_kv_cache(pages, kv_heads, page, bits)
        self.free = list(range(pages))
        self.table = torch.full((seqs, self.width), -1, dtype=torch.int32)
        self.lens = [0] * seqs
        self.weights = torch.zeros(seqs, kv_heads, self.width * page, device="cuda")
        self.evictions = 0

    def _grow(self, counts):
        """Pages for `counts` more tokens of each sequence; the new tokens' slots, in order."""
        slots = []
        for b, m in enumerate(counts):
            for t in range(self.lens[b], self.lens[b] + m):
                if t % self.page == 0:
                    self.table[b, t // self.page] = self.free.pop()
                slots.append(int(self.table[b, t // self.page]) * self.page + t % self.page)
            self.lens[b] += m
        return torch.tensor(slots, dtype=torch.int64, device="cuda")

    def forward(self, x, counts):
        """x [sum(counts)][hidden] bf16, counts[b] new tokens of sequence b: their attention outputs."""
        rows = x @ self.project
        q = rows[:, :self.q_heads * 128].unflatten(1, (self.q_heads, 128))
        k, v = rows[:, self.q_heads * 128:].unflatten(1, (2, self.kv_heads, 128)).unbind(1)
        hq.hq_kv_append(self.cache, k, v, self._grow(counts), bits=self.bits, seed=self.seed)
        start = torch.tensor([0, *counts]).cumsum(0).to("cuda", torch.int32)
        out = hq.hq_kv_attend(self.cache, q, self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda"), q_start=start,
                              max_q=max(counts), max_len=max(self.lens), bits=self.bits, seed=self.seed, weights=self.weights)
        if max(self.lens) >= self.high:
            self.evict()
        return out.flatten(1)

    def evict(self):
        """Cut every sequence back to at most `budget` tokens."""
        old = self.table.clone()
        need = -(-self.budget // self.page)
        dst = torch.tensor([[self.free.pop() for _ in range(need)] for _ in self.lens], dtype=torch.int32)
        kept, lens, weights = hq.hq_kv_evict(self.cache, old.cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda"), self.weights,
                                             self.budget, self.sink, self.recent, dst.cuda(), bits=self.bits, max_len=max(self.lens))
        self.weights.zero_()
        self.weights[:, :, :self.budget] = weights
        self.lens = lens.tolist()
        self.table.fill_(-1)
        for b, n in enumerate(self.lens):
            used = -(-n // self.page)
            self.table[b, :used] = dst[b, :used]
            self.free += dst[b, used:].tolist()
        self.free += [int(p) for p in old.flatten() if p >= 0]
        self.evictions += 1
        return kept


def generate(steps=200, bits=4, prompts=(100, 37, 1, 64), seed=0, **layer):
    """Runs prompts and `steps` tokens; returns the layer and the outputs of every call."""
    net = PagedLayer(len(prompts), bits=bits, seed=seed, **layer)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    x = torch.randn(sum(prompts), net.hidden, generator=g, device="cuda").bfloat16()
    outs = [net.forward(x, list(prompts))]
    last = torch.tensor(prompts).cumsum(0) - 1
    h = outs[0][last.cuda()]
    for _ in range(steps):
        # the next token's hidden state: the last output, renormalised, and a little noise in place of an embedding
        noise = torch.randn(h.shape, generator=g, device="cuda")
        h = h.float()
        x = (h / h.norm(dim=-1, keepdim=True) * h.shape[-1] ** 0.5 + noise).bfloat16()
        outs.append(net.forward(x, [1] * len(prompts)))
        h = outs[-1]
    return net, outs


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--bits", type=int, default=4, choices=[4, 8])
    args = ap.parse_args()
    net, outs = generate(args.steps, args.bits)
    print(f"{len(outs)} calls, {net.evictions} evictions, lengths {net.lens}, {hq.hq_kv_token_bytes(args.bits)} bytes a token and head "
          f"(bf16: 512), finite: {all(bool(torch.isfinite(o).all()) for o in outs)}")


if __name__ == "__main__":
    main()
