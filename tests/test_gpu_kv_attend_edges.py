"""GPU: attention over the paged SRFT cache at the edges of what a call may ask: fewer queries computed than a sequence has.

Bounds are kv_reference.attend's; cases are those of test_gpu_kv_attend."""
import numpy as np
import pytest

import kv_reference as ref

torch = pytest.importorskip("torch")
hq = pytest.importorskip("kv_quantization_tile_amd")

from test_gpu_kv_attend import SEED, Case, dev, host, say  # noqa: E402

pytestmark = pytest.mark.gpu


def within(got, want, tol):
    """Rows of outputs against the definition, with the transform back's 12 binary32 roundings."""
    err = np.linalg.norm(got.astype(np.float64) - want, axis=-1)
    bound = tol + 2.0 ** -20 * np.linalg.norm(want, axis=-1)
    assert np.isfinite(got).all() and (err <= bound).all(), np.max(err / np.maximum(bound, 1e-30))


@pytest.mark.parametrize("lens,q_lens,group,max_q,kw", [
    ([120, 90], [2, 2], 2, 1, {}),
    ([120, 90, 4], [6, 5, 9], 2, 5, dict(window=33)),
    ([300, 260], [40, 33], 2, 5, dict(page=64)),                # few rows of sequences with many
    ([300, 260], [40, 33], 2, 20, dict(bits=8)),
    ([700, 400], [150, 1], 2, 140, dict(window=77, lam=True)),  # single tokens beside cut chunks
    ([300, 260], [30, 30], 3, 7, dict(causal=False)),
    ([300, 260], [30, 30], 3, 2, dict(causal=False, window=20)),
])
def test_fewer_queries_than_a_sequence_has(orc, lens, q_lens, group, max_q, kw):
    """The first max_q queries of a sequence stand where they stand among all of them; the others are not written, and
    add no weight."""
    say(f"case: attend {q_lens} queries on {lens} tokens, max_q {max_q}, {kw}")
    c = Case(orc, lens, q_lens, heads=2, group=group, **kw)
    for precise in (False, True):
        want, tol, _, _ = c.want(precise)
        w = torch.zeros(len(lens), 2, max(lens), device="cuda") if precise else None
        forms = [c.run(weights=w, max_q=max_q)]
        if len(set(q_lens)) == 1 and not precise:
            forms.append(c.run(q_start=None, max_q=max_q))
        first = np.concatenate([np.arange(m) < max_q for m in q_lens])
        for out in map(host, forms):
            within(out[first], want[first], tol[first])
            assert np.isnan(out[~first]).all()
    if not c.kw["causal"]:
        return
    # causal, the computed queries are all the queries of a sequence that ends with them
    cut = [max(m - max_q, 0) for m in q_lens]
    _, _, ww, wtol = ref.attend(orc, host(c.cache), c.q[first], c.table, [max(n - x, 0) for n, x in zip(lens, cut)],
                                [m - x for m, x in zip(q_lens, cut)], c.bits, SEED, *c.lam, precise=True, **c.kw)
    got = host(w).astype(np.float64)
    top = ww.shape[2]
    assert (np.abs(got[..., :top] - ww) <= wtol + 2.0 ** -23 * ww).all() and not got[..., top:].any()
