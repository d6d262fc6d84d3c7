"""GPU: places, prompts, drafts and their acceptance together, as a serving loop runs them: every attention against its
definition in binary64, the cache's contents against what was appended, pages accounted for; and the example."""
import importlib.util
import os

import numpy as np
import pytest

import steps_reference as ref
from test_gpu_kv_tree import SEED, dev, host, some_tree

torch = pytest.importorskip("torch")
hq = pytest.importorskip("kv_quantization_tile_amd")

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "drafts.py")


def bf16(g, *shape):
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).cuda().to(torch.bfloat16)


@pytest.mark.parametrize("bits,page,group", [(4, 16, 2), (8, 32, 4)])
def test_prompts_and_drafted_steps(orc, bits, page, group):
    print(f"case: serving steps, {bits} bits, page {page}, group {group}", flush=True)
    g = np.random.default_rng(bits)
    heads, prompts, pages, width = 2, [70, 5, 33], 60, 12
    cache = hq.hq_kv_cache(pages, heads, page, bits)
    table, lens = dev(np.full((3, width), -1, np.int32)), dev(np.zeros(3, np.int32))
    free, count = dev(g.permutation(pages).astype(np.int32)), dev(np.array([pages], np.int32))
    reserve = lambda c, n: hq.hq_kv_reserve(table, lens, dev(np.array(c, np.int32)), free, count, page, n)  # noqa: E731
    fmt = dict(bits=bits, seed=SEED)
    held = [[] for _ in prompts]  # what each sequence's tokens decode to

    def read(slots):
        return [x.float() for x in hq.hq_kv_read(cache, slots, **fmt, out_dtype=torch.float32)]

    # prompts
    q, k, v = (bf16(g, sum(prompts), n, 128) for n in (heads * group, heads, heads))
    slots, positions, start, granted = reserve(prompts, sum(prompts))
    assert granted.tolist() == prompts and positions.tolist() == sum((list(range(n)) for n in prompts), [])
    hq.hq_kv_append(cache, k, v, slots, **fmt)
    got = hq.hq_attend_prompt(q, k, v, start, out=torch.empty(q.shape, device="cuda"))
    want, tol = ref.prompt(*(host(x.float()) for x in (q, k, v)), start.tolist())
    assert (np.linalg.norm(host(got) - want, axis=-1) <= tol + 2.0 ** -23 * np.linalg.norm(want, axis=-1)).all()
    kk, vv = read(slots)
    for b in range(3):
        for i in range(start[b], start[b + 1]):
            held[b].append((kk[i], vv[i]))

    for step in range(4):
        q_lens = [int(n) for n in g.integers(1, 12, 3)]
        trees = [some_tree(g, m) for m in q_lens]
        total = sum(q_lens)
        q, k, v = (bf16(g, total, n, 128) for n in (heads * group, heads, heads))
        slots, _, start, granted = reserve(q_lens, total + 2)
        assert granted.tolist() == q_lens and slots[total:].tolist() == [-1, -1]
        hq.hq_kv_append(cache, k, v, slots[:total], **fmt)
        parents = dev(np.array(sum(trees, []), np.int32))
        out = hq.hq_kv_attend(cache, q, table, lens, q_start=start, max_q=max(q_lens), parents=parents, out=torch.empty(q.shape, device="cuda"), **fmt)
        n = lens.tolist()
        assert n == [len(h) + m for h, m in zip(held, q_lens)]
        want, tol = ref.attend(orc, host(cache), host(q.float()), host(table), n, [ref.tree_sees(t, x, m) for t, x, m in zip(trees, n, q_lens)], bits, SEED)
        assert (np.linalg.norm(host(out) - want, axis=-1) <= tol + 2.0 ** -20 * np.linalg.norm(want, axis=-1)).all()
        kk, vv = read(slots[:total])
        tokens, target = (g.integers(0, 2, total).astype(np.int32) for _ in range(2))
        path, accepted, nxt, change = hq.hq_kv_accept(cache, table, lens, dev(tokens), dev(target), parents, q_start=start, bits=bits)
        for b in range(3):
            part = slice(int(start[b]), int(start[b + 1]))
            p = ref.accept_path(tokens[part], target[part], trees[b])
            assert path[b, :len(p)].tolist() == p and int(accepted[b]) == len(p)
            held[b] += [(kk[part][i], vv[part][i]) for i in p]
        assert hq.hq_kv_reserve(table, lens, change, free, count, page, 0)[3].equal(change)
        assert lens.tolist() == [len(h) for h in held]
        used = []
        for b, h in enumerate(held):
            t = torch.arange(len(h), device="cuda")
            kk2, vv2 = read(table[b, t // page].long() * page + t % page)
            assert torch.equal(kk2, torch.stack([x for x, _ in h])) and torch.equal(vv2, torch.stack([x for _, x in h]))
            used += [int(x) for x in table[b] if x >= 0]
            assert sum(int(x) >= 0 for x in table[b]) == -(-len(h) // page)
        assert sorted(used + free[:int(count)].tolist()) == list(range(pages))
    # sequences end: every page returns
    reserve([-1000] * 3, 0)
    assert int(count) == pages and not lens.any() and (table == -1).all()


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("drafts", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("bits", [4, 8])
def test_example(example, bits):
    print(f"case: the drafts' example, {bits} bits", flush=True)
    net, texts = example.generate(12, bits=bits)
    assert net.lens.tolist() == [len(t) for t in texts]
    used = [int(p) for p in net.table.flatten() if p >= 0]
    assert len(set(used)) == len(used) == sum(-(-len(t) // net.page) for t in texts)
    assert sorted(used + net.free[:int(net.free_count)].tolist()) == list(range(len(net.free)))
    assert all(0 <= t < net.vocabulary for text in texts for t in text) and sum(map(len, texts)) > sum((100, 37, 1, 64)) + 4 * 12
