"""GPU: eviction from the paged SRFT cache at the edges of what a call may ask."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
hq = pytest.importorskip("kv_quantization_tile_amd")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,most", [([100, 70, 30], 64), ([9000, 8193], 8192), ([33000, 5], 32768)])
def test_longer_lengths_count_as_max_len(lens, most):
    """With max_len below a length the call keeps what it keeps of the cut sequence, by default too where the weights end there."""
    print(f"case: evict {lens} with max_len {most}", flush=True)
    seqs, heads, page, budget = len(lens), 2, 64, 40
    width = -(-max(lens) // page)
    g = torch.Generator(device="cuda")
    g.manual_seed(most)
    before = torch.randint(0, 256, (seqs * (width + 1), heads, page * hq.hq_kv_token_bytes(4)), dtype=torch.uint8, generator=g, device="cuda")
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    table, dst = i32(np.arange(seqs * width).reshape(seqs, width)), i32(np.arange(seqs * width, seqs * (width + 1)).reshape(seqs, 1))
    weights = torch.rand(seqs, heads, width * page, generator=g, device="cuda")
    results = []
    for n, w, max_len in ((np.minimum(lens, most), weights, None), (lens, weights, most), (lens, weights[..., :most].contiguous(), None)):
        cache = before.clone()
        results.append((*hq.hq_kv_evict(cache, table, i32(n), w, budget, 3, 10, dst, max_len=max_len), cache))
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))
