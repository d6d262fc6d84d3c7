"""GPU: places in the paged cache (block tables, slots, the page stack) against the definition, value for value."""
import numpy as np
import pytest

import steps_reference as ref

torch = pytest.importorskip("torch")
hq = pytest.importorskip("kv_quantization_tile_amd")

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class World:
    """Sequences with pages of their own, and a stack of the others."""

    def __init__(self, lens, width, page, spare, seed=0, room=0):
        g = np.random.default_rng(seed)
        used = [-(-n // page) for n in lens]
        ids = g.permutation(sum(used) + spare + room).astype(np.int32)
        self.page, self.count = page, spare
        self.lens = np.array(lens, np.int32)
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = ids[at:at + u]
            at += u
        self.free = np.full(len(ids), -1, np.int32)
        self.free[:spare] = ids[at:at + spare]

    def step(self, counts, tokens):
        """One call on the GPU and in the definition; every output and the state compared."""
        d = [dev(x) for x in (self.table, self.lens, np.array(counts, np.int32), self.free, np.array([self.count], np.int32))]
        slots, positions, start, granted = (x.cpu().numpy() for x in hq.hq_kv_reserve(*d, self.page, tokens))
        want = ref.reserve(self.table, self.lens, counts, self.free, self.count, self.page, tokens)
        self.count = want[4]
        for name, got, w in zip(("slots", "positions", "q_start", "granted"), (slots, positions, start, granted), want):
            assert got.dtype == w.dtype and np.array_equal(got, w), name
        for name, got, w in zip(("table", "lens"), (d[0], d[1]), (self.table, self.lens)):
            assert np.array_equal(got.cpu().numpy(), w), name
        assert int(d[4]) == self.count and np.array_equal(d[3].cpu().numpy()[:self.count], self.free[:self.count])
        self.free = d[3].cpu().numpy()  # what lies above the stack's top is nobody's
        return granted


CASES = {
    "one_token": (dict(lens=[5], width=2, page=16, spare=3), [1], 1),
    "page_full": (dict(lens=[16, 32, 15], width=4, page=16, spare=9), [1, 1, 1], 3),
    "nothing": (dict(lens=[5, 0], width=2, page=16, spare=3), [0, 0], 2),
    "prompts": (dict(lens=[0, 0, 7], width=8, page=64, spare=30), [100, 511, 1], 612),
    "padded": (dict(lens=[0, 3], width=8, page=16, spare=30), [20, 5], 77),
    "fewer_places_than_tokens": (dict(lens=[0, 3], width=8, page=16, spare=30), [20, 50], 33),
    "many_tokens": (dict(lens=[0, 100, 9], width=300, page=32, spare=600), [4000, 1, 5000], 9010),
    "ends": (dict(lens=[100, 64, 1, 0, 77], width=8, page=16, spare=0), [-100, -1, -1, -5, -60], 0),
    "ends_and_grows": (dict(lens=[100, 64, 1, 0, 77], width=8, page=16, spare=1), [-100, 33, -1, 60, -60], 93),
    "takes_what_returns": (dict(lens=[64, 0], width=4, page=16, spare=0), [-64, 64], 64),
    "more_than_there_are": (dict(lens=[10, 20], width=4, page=16, spare=0), [-11, -(2 ** 31)], 3),
    "stack_runs_out": (dict(lens=[10, 16, 10, 10, 16], width=9, page=16, spare=3), [1, 32, 40, 1, 1], 75),
    "stack_empty": (dict(lens=[10, 16, 10], width=9, page=16, spare=0), [6, 1, 1], 8),
    "table_too_narrow": (dict(lens=[30, 30, 30], width=2, page=16, spare=9), [3, 2, 40], 45),
    "no_table": (dict(lens=[0, 0], width=0, page=16, spare=4), [1, 0], 1),
    "huge_counts": (dict(lens=[1, 1, 1], width=4, page=16, spare=9), [2 ** 31 - 1, 2 ** 31 - 1, 5], 100),
    "large_pages": (dict(lens=[4096, 4095], width=3, page=4096, spare=9), [1, 2], 3),
}


@pytest.mark.parametrize("name", CASES)
def test_against_definition(name):
    print(f"case: reserve {name}", flush=True)
    kw, counts, tokens = CASES[name]
    World(**kw).step(counts, tokens)


@pytest.mark.parametrize("seqs,most", [(3, 40), (200, 30), (1025, 9), (2500, 3)])
def test_many_steps(seqs, most):
    """Steps of all kinds on one state: more sequences than a workgroup has threads, too."""
    print(f"case: reserve steps of {seqs} sequences", flush=True)
    g = np.random.default_rng(seqs)
    w = World([int(n) for n in g.integers(0, 100, seqs)], 12, 16, seqs, seed=seqs)
    for i in range(6):
        counts = g.integers(-most, most + 1, seqs)
        counts[g.random(seqs) < 0.05] = -1000
        tokens = int(np.maximum(counts, 0).sum())
        w.step(counts.tolist(), max(0, tokens + int(g.integers(-3, 4))))
    used = w.table[w.table >= 0].tolist()
    assert sorted(used + w.free[:w.count].tolist()) == list(range(len(w.free)))


def test_the_negated_call_undoes():
    print("case: reserve undone", flush=True)
    w = World([100, 64, 1, 0, 77, 31], 20, 16, 12, seed=5)
    before = (w.table.copy(), w.lens.copy(), w.count, w.free[:w.count].copy())
    granted = w.step([33, -64, 70, 5, -60, 200], 308)
    assert (granted != 0).any() and (granted == 0).any()
    w.step((-granted).tolist(), 200)
    for a, b in zip(before, (w.table, w.lens, w.count, w.free[:w.count])):
        assert np.array_equal(a, b)


def test_bad_state_is_cut():
    """Lengths and counts outside their ranges, entries and pages that name no page: nothing outside the buffers."""
    print("case: reserve on bad state", flush=True)
    w = World([10, 20, 30], 4, 16, 6, seed=2)
    w.lens[:] = [-7, 1 << 30, 30]
    w.step([5, -3, 3], 8)
    w = World([40, 40, 40], 4, 16, 6, seed=2)
    w.table[0, 1], w.table[1, 2], w.table[2, 2], w.table[2, 0] = -5, 1 << 30, len(w.free), -(1 << 31)
    w.step([-40, -1, 3], 9)
    w.step([0, 0, -43], 0)
    for count in (-4, 1 << 30):
        w = World([40, 40], 4, 16, 6, seed=3, room=2)
        w.count = count
        w.free[:] = np.arange(len(w.free))
        w.step([8, 20], 28)
    # more pages than the stack holds return
    w = World([64, 64], 4, 16, 3, seed=4)
    w.free, w.count = w.free[:5].copy(), 3
    w.table[:] = [[0, 1, 2, 3], [4, 0, 1, 2]]
    w.step([-64, -20], 0)
    # a stack that holds what is no page
    w = World([0, 3], 4, 16, 4, seed=6)
    w.free[1], w.free[2] = -9, 1 << 29
    w.step([40, 20], 60)


def test_caller_buffers_streams_and_graphs():
    """Outputs that are passed in, another stream, and a captured call replayed on other counts."""
    print("case: reserve graph", flush=True)
    w = World([100, 64, 1, 0], 40, 16, 100, seed=1)
    state = [dev(x) for x in (w.table, w.lens, np.zeros(4, np.int32), w.free, np.array([w.count], np.int32))]
    outs = dict(slots=torch.empty(300, dtype=torch.int64, device="cuda"), positions=torch.empty(300, dtype=torch.int32, device="cuda"),
                q_start=torch.empty(5, dtype=torch.int32, device="cuda"), granted=torch.empty(4, dtype=torch.int32, device="cuda"))
    got = hq.hq_kv_reserve(*state, 16, 300, **outs)
    assert all(a is b for a, b in zip(got, outs.values()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hq.hq_kv_reserve(*state, 16, 300, **outs)
    for counts in ([1, 2, 3, 200], [-50, 17, 0, -9], [5, 5, 5, 5]):
        state[2].copy_(torch.tensor(counts, dtype=torch.int32))
        graph.replay()
        want = ref.reserve(w.table, w.lens, counts, w.free, w.count, 16, 300)
        w.count = want[4]
        for a, b in zip(outs.values(), want):
            assert np.array_equal(a.cpu().numpy(), b)
        assert np.array_equal(state[0].cpu().numpy(), w.table) and int(state[4]) == w.count
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hq.hq_kv_reserve(*state, 16, 20, stream=side)
    side.synchronize()
    for a, b in zip(got, ref.reserve(w.table, w.lens, [5, 5, 5, 5], w.free, w.count, 16, 20)):
        assert np.array_equal(a.cpu().numpy(), b)


def test_no_sequences():
    print("case: reserve without sequences", flush=True)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    for tokens in (3, 5000):
        slots, positions, start, granted = hq.hq_kv_reserve(i32(0, 4), i32(0), i32(0), i32(5), i32(1), 16, tokens)
        assert (slots == -1).all() and not positions.any() and start.tolist() == [0] and granted.numel() == 0
