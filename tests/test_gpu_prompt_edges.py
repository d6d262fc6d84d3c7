"""GPU: attention within packed prompts at the edges of what a call may ask: thousands of sequences, rows past 2^32 bytes, caps at
both ends of their range and where the capping changes form, capped scores of keys that are not finite.

Bounds and inputs are those of test_gpu_prompt."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
hq = pytest.importorskip("kv_quantization_tile_amd")

from test_gpu_prompt import check, inputs, say  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,most,long", [(1024, 5, [0, 1023]), (3000, 2, [5, 64, 2999]), (4096, 1, [])])
def test_thousands_of_sequences(seqs, most, long):
    say(f"case: prompt {seqs} sequences of up to {most} tokens, {len(long)} long ones")
    g = np.random.default_rng(seqs)
    lens = g.integers(0, most + 1, seqs)
    lens[long] = 200 + np.arange(len(long))
    check(inputs([int(n) for n in lens], heads=2, group=3), {})


def test_more_sequences_than_a_launch_has_places():
    """2^24 / heads sequences and more, of which few have tokens."""
    say("case: prompt 270000 sequences, 64 heads")
    lens = np.zeros(270000, int)
    lens[[0, 1, 63, 64, 5000, 140000, 269998, 269999]] = [3, 1, 130, 2, 40, 65, 1, 7]
    check(inputs([int(n) for n in lens], heads=64, group=1), {})


@pytest.mark.parametrize("seqs", [64, 65, 300])
def test_offsets_of_many_sequences(seqs):
    """Rows before the first offset, behind the last and of no sequence stay as they were; offsets are cut to the rows there are; empty
    sequences at either end."""
    say(f"case: prompt offsets of {seqs} sequences")
    g = np.random.default_rng(seqs)
    lens = g.integers(0, 9, seqs)
    lens[[0, 1, seqs - 1]], lens[seqs // 2] = 0, 200
    q, k, v, _ = inputs([int(lens.sum()) + 50], heads=2, group=2)
    for first, clamp in ((0, False), (13, False), (50, False), (0, True)):
        start = (first + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
        if clamp:  # what lies outside the rows is none
            start[:2], start[-2:] = (-1 << 31, -7), (q.shape[0], (1 << 31) - 1)
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        hq.hq_attend_prompt(q, k, v, torch.from_numpy(start).cuda(), out=out)
        lo, hi = np.clip(start[[0, -1]], 0, q.shape[0])
        assert torch.isnan(out[:lo]).all() and torch.isnan(out[hi:]).all()
        for a, b in zip(start.clip(0, q.shape[0])[:-1], start.clip(0, q.shape[0])[1:]):
            if a < b:
                one = hq.hq_attend_prompt(q[a:b], k[a:b], v[a:b], torch.tensor([0, b - a], dtype=torch.int32, device="cuda"))
                assert torch.equal(out[a:b], one)


def test_time_grows_with_the_sequences():
    """16 times as many prompts of one token take about 16 times as long, not 256 times: 64 lies between."""
    say("case: prompt, time of 1024 and 16384 sequences")

    def time_of(seqs):
        x = torch.randn(seqs, 48, 128, device="cuda").to(torch.bfloat16)
        q, k, v = x[:, :32], x[:, 32:40], x[:, 40:]
        start = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
        out = hq.hq_attend_prompt(q, k, v, start)
        # a row that sees itself alone
        assert torch.equal(out, v.repeat_interleave(4, 1))
        times = []
        for _ in range(3):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(4):
                hq.hq_attend_prompt(q, k, v, start, out=out)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    assert time_of(16384) < 64 * time_of(1024)


def test_rows_past_32_bits():
    """Rows 8 MiB apart, 4.6 GB of each operand from first to last: what rows side by side give."""
    say("case: prompt, rows far apart")
    q, k, v, start = inputs([130, 300, 120], heads=1, group=2)
    want = hq.hq_attend_prompt(q, k, v, start)
    step = (1 << 23) - 8  # the longest stride there may be, in values
    rows = q.shape[0]
    room = torch.empty(step * (rows - 1) + 512, dtype=torch.bfloat16, device="cuda")
    views, at = [], 0
    for x in (q, k, v):
        view = torch.as_strided(room, x.shape, (step, 128, 1), at)
        view.copy_(x)
        views.append(view)
        at += x.shape[1] * 128
    assert room.numel() * 2 > 1 << 32
    assert torch.equal(hq.hq_attend_prompt(*views, start), want)


@pytest.mark.parametrize("softcap", [2.0 ** -125, 1e-3, 255.5, 256.0, 256.5, 5000.0])
def test_caps(softcap):
    """Up to 256 the cap is in one form, above in another."""
    say(f"case: prompt, cap {softcap}")
    for scale in (128 ** -0.5, 1.0, -0.3):
        check(inputs([150, 40], heads=2, group=2), dict(softcap=softcap, scale=scale))
    check(inputs([150, 40], heads=1, group=2, window=33), dict(softcap=softcap, window=33))


@pytest.mark.parametrize("softcap", [30.0, 1000.0])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_capped_scores_of_keys_that_are_not_finite(what, softcap):
    """A capped score of an infinite key is plus or minus the cap, as large finite ones are; of a NaN, NaN.  Neither reaches
    rows that do not see the key."""
    say(f"case: prompt, key of {what}, cap {softcap}")
    lens, n = [70, 100, 65], 100
    q, k, v, start = inputs(lens, heads=2, group=2)
    q[..., 7] = torch.where(q[..., 7] < 0, -1.0, 1.0).to(q.dtype)  # its product with a large value is large
    clean = hq.hq_attend_prompt(q, k, v, start, softcap=softcap)
    for t in (0, 33, 64, 99):
        bad, large = k.clone(), k.clone()
        bad[70 + t, 1, 7] = what
        large[70 + t, 1, 7] = 1e30 if what > 0 else -1e30
        got, like = (hq.hq_attend_prompt(q, x, v, start, softcap=softcap) for x in (bad, large))
        seen = torch.zeros_like(clean, dtype=torch.bool)
        seen[70 + t:70 + n, 2:] = True
        assert torch.equal(got[~seen], clean[~seen])
        assert torch.isnan(got[seen]).all() if what != what else torch.equal(got[seen], like[seen])
