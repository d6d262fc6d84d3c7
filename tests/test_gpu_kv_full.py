"""GPU: drafted steps where places run out: a sequence that got none waits, and loses nothing that it held."""
import importlib.util
import os

import numpy as np
import pytest

import steps_reference as ref

torch = pytest.importorskip("torch")
hq = pytest.importorskip("kv_quantization_tile_amd")

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "drafts.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("drafts", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("kw", [dict(pages=20), dict(width=8), dict(pages=15), dict(pages=24, width=7)])
def test_example_with_little_room(example, kw):
    """The pool or a table is full after a few steps: the tokens cached are the texts', and their contents stay."""
    print(f"case: the drafts' example, {kw}", flush=True)
    net, texts = example.generate(6, **kw)
    assert net.lens.tolist() == [len(t) for t in texts]

    def held():
        out = []
        for b, n in enumerate(net.lens.tolist()):
            t = torch.arange(n, device="cuda")
            out += hq.hq_kv_read(net.cache, net.table[b, t // net.page].long() * net.page + t % net.page, bits=net.bits, seed=net.seed)
        return out

    last = torch.zeros(len(texts), dtype=torch.int32, device="cuda")
    for _ in range(60):
        before, lens = held(), net.lens.tolist()
        path, taken, nxt = net.step(last)
        grown = [(row >= 0).sum().item() for row in taken]
        assert net.lens.tolist() == [n + g for n, g in zip(lens, grown)]
        assert all(torch.equal(nxt[b], last[b]) for b, g in enumerate(grown) if g == 0)
        for b, (x, y) in enumerate(zip(before, held())):
            assert torch.equal(x, y[:len(x)])
        last = nxt
    used = [int(p) for p in net.table.flatten() if p >= 0]
    assert len(set(used)) == len(used) == sum(-(-n // net.page) for n in net.lens.tolist())
    assert sorted(used + net.free[:int(net.free_count)].tolist()) == list(range(len(net.free)))


def test_example_refuses_prompts_without_room(example):
    print("case: the drafts' example, prompts without room", flush=True)
    with pytest.raises(RuntimeError):
        example.generate(1, pages=14)


def test_a_length_of_zero_leaves_a_sequence_alone():
    """What the documentation has a caller pass for a sequence without places: its drafts see nothing, and nothing of it moves."""
    print("case: drafts of sequences without places", flush=True)
    g = np.random.default_rng(4)
    heads, page, m = 2, 16, 6
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = hq.hq_kv_cache(8, heads, page)
    k, v = (torch.randn(8 * page, heads, 128, device="cuda") for _ in range(2))
    hq.hq_kv_append(cache, k, v, torch.arange(8 * page, device="cuda"))
    table, lens = i32([[0, 1, -1], [2, 3, -1], [4, 5, -1]]), i32([20, 27, 18])
    free, count = i32([-1] * 8), i32([0])
    slots, _, start, granted = hq.hq_kv_reserve(table, lens, i32([m, m, m]), free, count, page, 3 * m)
    # pages run out at the second: the third, which needed none, gets nothing either
    assert granted.tolist() == [m, 0, 0] and lens.tolist() == [26, 27, 18] and (slots[m:] == -1).all()
    here = granted > 0
    held = torch.where(here, lens, 0)
    q = torch.randn(3 * m, 4, 128, device="cuda").to(torch.bfloat16)
    tree = [-1, 0, 0, 1, 1, 3]
    tokens, target = (g.integers(0, 2, 3 * m).astype(np.int32) for _ in range(2))
    parents, before = i32(tree * 3), cache.cpu().numpy()
    out = hq.hq_kv_attend(cache, q, table, held, q_start=start, max_q=m, parents=parents)
    assert not out[m:].any() and out[:m].any()
    path, accepted, nxt, change = hq.hq_kv_accept(cache, table, held, i32(tokens.tolist()), i32(target.tolist()), parents, q_start=start, max_q=m)
    want = before.copy()
    p = ref.accept_path(tokens[:m], target[:m], tree)
    ref.move(want, 4, table[0].tolist(), 26, m, p, page)
    assert path[0, :len(p)].tolist() == p and np.array_equal(cache.cpu().numpy(), want)
    hq.hq_kv_reserve(table, lens, torch.where(here, change, 0), free, count, page, 0)
    assert lens.tolist() == [20 + len(p), 27, 18] and table[1:].tolist() == [[2, 3, -1], [4, 5, -1]]
