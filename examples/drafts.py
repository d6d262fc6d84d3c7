"""One attention layer that decodes with drafted tokens over the paged SRFT cache.

Prompts of different lengths are attended among themselves (hq_attend_prompt) and appended.  Then every step drafts a small tree
behind each sequence's last token, attends all of it in one call (hq_kv_attend with `parents`), accepts what the model
would have chosen (hq_kv_accept moves it up in the cache) and gives the other drafts' places back.  Pages, block
tables and slots stay on the GPU throughout (hq_kv_reserve); a sequence for which there is no room waits.  The layer's weights are random; drafts are guesses over a small
vocabulary, so some of them are right.

    python examples/drafts.py [--steps N] [--bits 4|8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kv_quantization_tile_amd as hq  # noqa: E402

TREE = [-1, 0, 0, 0, 1, 1, 2, 3]  # a token, three guesses of the next one, four of the one after


class DraftedLayer:
    def __init__(self, seqs, q_heads=8, kv_heads=2, page=16, pages=256, width=64, vocabulary=3, bits=4, seed=0):
        self.q_heads, self.kv_heads, self.page, self.bits, self.seed, self.vocabulary = q_heads, kv_heads, page, bits, seed, vocabulary
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        hidden = q_heads * 128
        draw = lambda *s: torch.randn(*s, generator=self.g, device="cuda").bfloat16()  # noqa: E731
        self.embed = draw(vocabulary, hidden)
        self.project = draw(hidden, (q_heads + 2 * kv_heads) * 128) / hidden ** 0.5
        self.head = draw(hidden, vocabulary)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cache = hq.hq_kv_cache(pages, kv_heads, page, bits)
        self.table, self.lens = torch.full_like(i32(seqs, width), -1), i32(seqs)
        self.free, self.free_count = torch.arange(pages, dtype=torch.int32, device="cuda"), i32(1).fill_(pages)

    def _reserve(self, counts, tokens):
        return hq.hq_kv_reserve(self.table, self.lens, counts, self.free, self.free_count, self.page, tokens)

    def _rows(self, tokens):
        rows = self.embed[tokens.long()] @ self.project
        q = rows[:, :self.q_heads * 128].unflatten(1, (self.q_heads, 128))
        k, v = rows[:, self.q_heads * 128:].unflatten(1, (2, self.kv_heads, 128)).unbind(1)
        return q, k, v

    def _choose(self, out):
        return (out.flatten(1) @ self.head).argmax(-1).to(torch.int32)

    def prompt(self, tokens, counts):
        """tokens [sum(counts)]: the token chosen behind each prompt."""
        q, k, v = self._rows(tokens)
        slots, _, start, granted = self._reserve(torch.tensor(counts, dtype=torch.int32, device="cuda"), len(tokens))
        if granted.tolist() != list(counts):
            raise RuntimeError("the prompts need more pages, or wider tables")
        hq.hq_kv_append(self.cache, k, v, slots, bits=self.bits, seed=self.seed)
        out = hq.hq_attend_prompt(q, k, v, start)
        return self._choose(out[(start[1:] - 1).long()])

    def step(self, last):
        """last [seqs]: the tokens chosen before, not cached yet.  Returns (accepted drafts [seqs][len(TREE)], -1 past the end and
        throughout for a sequence without room; their tokens; the tokens chosen behind them)."""
        seqs, m = len(last), len(TREE)
        tokens = torch.randint(0, self.vocabulary, (seqs, m), generator=self.g, device="cuda", dtype=torch.int32)
        tokens[:, 0] = last
        parents = torch.tensor(TREE, dtype=torch.int32, device="cuda").repeat(seqs)
        q, k, v = self._rows(tokens.flatten())
        slots, _, start, granted = self._reserve(torch.full_like(last, m), seqs * m)
        hq.hq_kv_append(self.cache, k, v, slots, bits=self.bits, seed=self.seed)
        # a sequence that got no places has no drafts in the cache: with a length of 0 none of its tokens are taken for some
        here = granted > 0
        held = torch.where(here, self.lens, 0)
        out = hq.hq_kv_attend(self.cache, q, self.table, held, q_start=start, max_q=m, parents=parents, bits=self.bits, seed=self.seed)
        path, accepted, nxt, change = hq.hq_kv_accept(self.cache, self.table, held, tokens.flatten(), self._choose(out), parents, q_start=start,
                                                       max_q=m, bits=self.bits)
        self._reserve(torch.where(here, change, 0), 0)
        path = torch.where(here[:, None], path, -1)
        taken = torch.where(path >= 0, tokens.gather(1, path.clamp(min=0).long()), path)
        return path, taken, torch.where(here, nxt, last)


def generate(steps=20, bits=4, prompts=(100, 37, 1, 64), seed=0, **layer):
    """Runs prompts and `steps` steps of drafts; returns the layer and each sequence's tokens."""
    net = DraftedLayer(len(prompts), bits=bits, seed=seed, **layer)
    tokens = torch.randint(0, net.vocabulary, (sum(prompts),), generator=net.g, device="cuda", dtype=torch.int32)
    texts = [t.tolist() for t in tokens.split(list(prompts))]
    last = net.prompt(tokens, prompts)
    for _ in range(steps):
        _, taken, last = net.step(last)
        for text, row in zip(texts, taken.tolist()):
            text += [t for t in row if t >= 0]
    return net, texts


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--bits", type=int, default=4, choices=[4, 8])
    args = ap.parse_args()
    net, texts = generate(args.steps, args.bits)
    print(f"{args.steps} steps, tokens cached {net.lens.tolist()}, pages free {int(net.free_count)} of {len(net.free)}")


if __name__ == "__main__":
    main()
