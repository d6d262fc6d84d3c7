"""GPU: attention within packed prompts against its definition in binary64.

steps_reference.prompt gives, with each output row, the error that the kernel's roundings may make.  Every query looks for the
tokens just inside and just outside what it may see, so one token too many or too few moves its row by far more than that."""
import numpy as np
import pytest

import steps_reference as ref

torch = pytest.importorskip("torch")
hq = pytest.importorskip("kv_quantization_tile_amd")

pytestmark = pytest.mark.gpu


def say(msg):
    print(msg, flush=True)


def inputs(lens, heads=1, group=1, window=0, seed=0, **_):
    g = np.random.default_rng(seed + sum(lens))
    total, start = sum(lens), np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v = (g.standard_normal((total, heads, 128)).astype(np.float32) for _ in range(2))
    q = g.standard_normal((total, heads * group, 128)).astype(np.float32)
    for b, n in enumerate(lens):
        for i in range(n):
            for t in (i, i + 1, i - window, i - window + 1) if window else (i, i + 1, n - 1, n):
                if 0 <= start[b] + t < total:  # the next sequence's first token too
                    q[start[b] + i] += 0.4 * np.repeat(k[start[b] + t], group, 0)
    return [torch.from_numpy(x).cuda().to(torch.bfloat16) for x in (q, k, v)] + [torch.from_numpy(start).cuda()]


def check(args, want_kw, out_dtype=torch.float32, **kw):
    q, k, v, start = args
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    got = hq.hq_attend_prompt(q, k, v, start, out=out, **want_kw, **kw).double().cpu().numpy()
    want, tol = ref.prompt(*(x.float().cpu().numpy() for x in (q, k, v)), start.tolist(), **want_kw)
    half = 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -23
    err, bound = np.linalg.norm(got - want, axis=-1), tol + half * np.linalg.norm(want, axis=-1)
    assert np.isfinite(got).all()
    assert (err <= bound).all(), np.max(err / np.maximum(bound, 1e-30))
    return out


CASES = {
    "one_token": dict(lens=[1]),
    "short": dict(lens=[1, 2, 3, 0, 31, 32, 33, 63, 64, 65]),
    "group_3": dict(lens=[100, 7, 85], heads=2, group=3),
    "group_7": dict(lens=[37, 200, 1], heads=1, group=7),
    "tiles": dict(lens=[255, 256, 257, 513], heads=1, group=1),
    "tiles_8_heads": dict(lens=[129, 300], heads=8, group=4),
    "long": dict(lens=[1500], heads=1, group=2),
    "window_1": dict(lens=[70, 130], window=1),
    "window": dict(lens=[300, 90, 5], heads=2, group=2, window=37),
    "window_64": dict(lens=[400], heads=1, group=1, window=64),
    "window_longer_than_all": dict(lens=[100, 60], heads=1, group=2, window=1000),
    "everything": dict(lens=[100, 65, 300], heads=1, group=2, causal=False),
    "window_without_causal": dict(lens=[100, 300], heads=1, group=2, causal=False, window=50),
    "cap": dict(lens=[150, 40], heads=2, group=2, softcap=20.0),
    "small_cap": dict(lens=[150, 40], heads=1, group=2, softcap=0.5, window=64),
    "large_cap": dict(lens=[150], heads=1, group=2, softcap=1e6),
    "cap_everything": dict(lens=[90], heads=1, group=4, softcap=30.0, causal=False),
    "negative_scale": dict(lens=[70, 200], heads=1, group=2, scale=-0.11),
    "zero_scale": dict(lens=[70, 200], heads=1, group=2, scale=0.0),
    "large_scale": dict(lens=[70, 200], heads=1, group=2, scale=1.0),
}


def keywords(case):
    return {x: case[x] for x in ("causal", "window", "softcap", "scale") if x in case}


@pytest.mark.parametrize("name", CASES)
def test_against_definition(name):
    say(f"case: prompt {name} {CASES[name]}")
    args, kw = inputs(**CASES[name]), keywords(CASES[name])
    wide = check(args, kw)
    narrow = check(args, kw, torch.bfloat16)
    assert torch.equal(wide.to(torch.bfloat16), narrow)


@pytest.mark.parametrize("seqs", [63, 64, 65, 200, 700])
def test_many_sequences(seqs):
    """More sequences than a wavefront has lanes, some of them empty: each is found, and only rows of its own are seen."""
    say(f"case: prompt {seqs} sequences")
    g = np.random.default_rng(seqs)
    lens = [int(n) for n in g.integers(0, 12, seqs)]
    lens[seqs // 2] = 300
    check(inputs(lens, heads=1, group=2), {})


@pytest.mark.parametrize("name", ["group_3", "tiles_8_heads", "window"])
def test_strides_and_repeats(name):
    """Views of a fused projection's rows, heads first, and values shared by all heads; equal calls give equal bits."""
    say(f"case: prompt strides {name}")
    case = CASES[name]
    q, k, v, start = inputs(**case)
    kw = keywords(case)
    first = hq.hq_attend_prompt(q, k, v, start, **kw)
    row = torch.full((q.shape[0], (q.shape[1] + 2 * k.shape[1]) * 128 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    views, at = [], 8
    for x in (q, k, v):
        view = row[:, at:at + x.shape[1] * 128].unflatten(1, (x.shape[1], 128))
        view.copy_(x)
        views.append(view)
        at += x.shape[1] * 128
    assert torch.equal(hq.hq_attend_prompt(*views, start, **kw), first)
    assert torch.equal(hq.hq_attend_prompt(*(x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)), start, **kw), first)
    one = v[:, :1].contiguous()
    assert torch.equal(hq.hq_attend_prompt(q, k, one.expand(-1, k.shape[1], -1), start, **kw),
                       hq.hq_attend_prompt(q, k, one.repeat(1, k.shape[1], 1), start, **kw))
    back = torch.flip(q, [0]).flip([0])
    assert torch.equal(hq.hq_attend_prompt(back, k, v, start, **kw), first)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 20), (False, 30)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_seen_does_not_reach(what, causal, window):
    """A key or value that is not finite reaches the rows that see it and no other, of its own sequence or another's; a value's only
    its own column."""
    say(f"case: prompt {what} in masked places, causal {causal}, window {window}")
    lens, n = [70, 100, 65], 100
    q, k, v, start = inputs(lens, heads=2, group=2, window=window)
    kw = dict(causal=causal, window=window)
    clean = hq.hq_attend_prompt(q, k, v, start, **kw)
    i = torch.arange(n, device="cuda")
    for t in (0, 33, 63, 64, 99):
        sees = ((i >= t) if causal else (i >= 0)) & ((t > i - window) if window else (i >= 0))
        sees = torch.cat([sees.new_zeros(70), sees, sees.new_zeros(65)])
        vv = v.clone()
        vv[70 + t, 1, 5] = what
        got = hq.hq_attend_prompt(q, k, vv, start, **kw)
        hit = torch.zeros_like(clean, dtype=torch.bool)
        hit[:, 2:, 5] = sees[:, None]
        assert torch.equal(got[~hit], clean[~hit])
        assert torch.isnan(got[hit]).all() if what != what else not torch.isfinite(got[hit]).any()
        kk = k.clone()
        kk[70 + t, 1] = float("nan")
        got = hq.hq_attend_prompt(q, kk, v, start, **kw)
        assert torch.equal(got[:, :2], clean[:, :2]) and torch.equal(got[:, 2:][~sees], clean[:, 2:][~sees])
        assert torch.isnan(got[:, 2:][sees]).all()
    # infinities of both signs, and an infinity that its rows weigh
    vv = v.clone()
    vv[70 + 64, 0, 9], vv[70 + 65, 0, 9] = float("inf"), -float("inf")
    got = hq.hq_attend_prompt(q, k, vv, start, causal=True)
    rest = hq.hq_attend_prompt(q, k, v, start, causal=True)
    assert torch.equal(got[70 + 64, :2, 9], torch.full((2,), float("inf"), device="cuda", dtype=torch.bfloat16))
    assert torch.isnan(got[70 + 65:170, :2, 9]).all()
    got[70 + 64:170, :2, 9] = rest[70 + 64:170, :2, 9]
    assert torch.equal(got, rest)
    qq = q.clone()
    qq[75, 1] = what
    got = hq.hq_attend_prompt(qq, k, v, start, **kw)
    assert not torch.isfinite(got[75, 1]).any()
    got[75, 1] = clean[75, 1]
    assert torch.equal(got, clean)


def test_strides_that_lead_nowhere():
    """Of one row, or one head, any stride will do."""
    say("case: prompt strides of one row and one head")
    q, k, v, start = inputs([1], heads=2, group=2)
    odd = lambda x: torch.as_strided(x, x.shape, ((1 << 24) + 1, 128, 1))  # noqa: E731
    assert torch.equal(hq.hq_attend_prompt(odd(q), odd(k), odd(v), start), hq.hq_attend_prompt(q, k, v, start))
    q, k, v, start = inputs([33], heads=1, group=1)
    odd = lambda x: torch.as_strided(x, x.shape, (128, 3, 1))  # noqa: E731
    assert torch.equal(hq.hq_attend_prompt(odd(q), odd(k), odd(v), start), hq.hq_attend_prompt(q, k, v, start))


def test_offsets():
    """Rows that no sequence names stay as they were; offsets are cut to the rows there are."""
    say("case: prompt offsets")
    q, k, v, start = inputs([40, 60, 30], heads=1, group=2)
    full = hq.hq_attend_prompt(q, k, v, start)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for offsets, rows in ((i32(40, 100), slice(40, 100)), (i32(40, 40, 100), slice(40, 100))):
        out = torch.full_like(full, float("nan"))
        hq.hq_attend_prompt(q, k, v, offsets, out=out)
        assert torch.equal(out[rows], full[rows])
        out[rows] = float("nan")
        assert torch.isnan(out).all()
    assert torch.equal(hq.hq_attend_prompt(q, k, v, i32(-5, 40, 100, 999)), full)
    out = torch.full_like(full, float("nan"))
    hq.hq_attend_prompt(q, k, v, i32(0, 40, 40, 40), out=out)
    assert torch.equal(out[:40], full[:40]) and torch.isnan(out[40:]).all()
    assert hq.hq_attend_prompt(q[:0], k[:0], v[:0], i32(0, 0)).shape == (0, 2, 128)
    out = torch.full_like(full, float("nan"))
    assert torch.isnan(hq.hq_attend_prompt(q, k, v, i32(0), out=out)).all()


def test_streams_and_graphs():
    say("case: prompt graph")
    args = inputs([100, 33], heads=2, group=2)
    eager = hq.hq_attend_prompt(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hq.hq_attend_prompt(*args, stream=side)
    side.synchronize()
    assert torch.equal(got, eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = hq.hq_attend_prompt(*args)
    for i in range(3):
        for x in args[:3]:
            x.copy_(torch.randn_like(x))
        args[3].copy_(torch.tensor([[0, 100, 133], [0, 1, 133], [0, 60, 120]][i]))
        graph.replay()
        want = hq.hq_attend_prompt(*args)
        rows = int(args[3][-1])
        assert torch.equal(held[:rows], want[:rows])


def test_refusals():
    say("case: prompt refuses")
    q, k, v, start = inputs([20], heads=2, group=2)
    good = dict(q=q, k=k, v=v, start=start)
    for bad in (dict(q=q[:, :3]), dict(q=q[..., :64]), dict(k=k[:10]), dict(v=v[:, :1]), dict(start=start.long()), dict(start=start[:0]), dict(window=-1),
                dict(out=torch.zeros(20, 4, 64, device="cuda")), dict(start=start.cpu()), dict(q=q.cpu()), dict(k=k[0])):
        with pytest.raises((ValueError, TypeError)):
            hq.hq_attend_prompt(**good | bad)
    for bad in (dict(q=q.float()), dict(v=v.half()), dict(out=torch.zeros(20, 4, 128, device="cuda", dtype=torch.float16))):
        with pytest.raises(TypeError):
            hq.hq_attend_prompt(**good | bad)
    row = torch.zeros(20, 4 * 128 + 1, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(softcap=-1.0), dict(scale=float("nan")), dict(q=row[:, 1:].unflatten(1, (4, 128))), dict(q=row[:, :-1].unflatten(1, (4, 128)))):
        with pytest.raises(hq.HqError):
            hq.hq_attend_prompt(**good | bad)
