"""beam_select on the GPU against its definition in 64 bits: rows, tokens and scores; types, strides, ties, masks, beams at
their end; its refusals and faults."""
import numpy as np
import pytest
import torch

import paged_split_kv_decode_gb300 as psd
from oracle import beams as BM
from _gpu_util import ctx

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _run(logits, scores, beams, k, *, finished=None, pad=0, workspace=None):
    rows = logits.shape[0]
    out = [torch.full((rows // beams, k), -7, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    if workspace is None:
        workspace = psd.beam_workspace(ctx(), rows, beams, k, "cuda")
        workspace.fill_(255)
    done = None if finished is None else torch.tensor(finished, dtype=torch.uint8, device="cuda")
    fault = psd.beam_select(ctx(), logits, torch.as_tensor(np.asarray(scores, dtype=np.float32)).cuda(), *out, workspace,
                            beams=beams, finished=done, pad_token=pad)
    torch.cuda.synchronize()
    return out, int(fault)


def _check(logits, scores, beams, k, *, finished=None, pad=0, faults=0, twins=False):
    """twins: rows hold the same logits in another order.  Their sums are equal, but for what rounding them in another
    order moves (2^-21, see below): which of two equal values in different rows comes first is open."""
    out, fault = _run(logits, scores, beams, k, finished=finished, pad=pad)
    want = BM.select(logits.double().cpu().numpy(), np.asarray(scores, dtype=np.float32), beams, k, finished, pad)
    assert fault == faults
    if twins:
        x = logits.double().cpu().numpy()
        low = np.log(np.exp(x - x.max(-1, keepdims=True)).sum(-1)) + x.max(-1)
        r, t = out[1].cpu().numpy(), out[2].cpu().numpy()
        assert np.all(np.abs(np.asarray(scores)[r] + x[r, t] - low[r] - want[0]) <= 2 * 2.0 ** -21)
        for b in range(len(r)):
            assert len({*zip(r[b], t[b])}) == k and {*r[b]} <= set(range(b * beams, (b + 1) * beams))
            for row in {*r[b]}:                                       # in a row: its largest, in order
                assert list(t[b][r[b] == row]) == list(np.argsort(-x[row], kind="stable")[: int((r[b] == row).sum())])
        return
    assert np.array_equal(out[1].cpu().numpy(), want[1]), (out[1].cpu().numpy() - want[1])
    assert np.array_equal(out[2].cpu().numpy(), want[2])
    got, none = out[0].double().cpu().numpy(), np.isneginf(want[0])
    assert np.array_equal(np.isneginf(got), none)
    # rounded once to f32 (2^-24 of it); the sum of exponentials, whose terms are off by 2^-21 each at most
    # (exp2 2 ulp, its argument rounded), moves the logarithm by no more than that
    d = np.abs(np.where(none, 0, got) - np.where(none, 0, want[0]))
    assert np.all(d <= 2.0 ** -24 * np.abs(np.where(none, 0, want[0])) + 2.0 ** -21)


def _logits(rows, vocab, kind="f32", seed=0, spread=2.5):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((spread * rng.standard_normal((rows, vocab))).astype(np.float32)).to(TYPES[kind]).cuda()


def _scores(rows, seed=0):
    return -5.0 - 3.0 * np.random.default_rng(seed + 99).random(rows)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 31, 256, 1000, 4095, 4096, 4097, 8193, 32000, 50257])
def test_vocabularies(vocab, kind):
    _check(_logits(6, vocab, kind, vocab), _scores(6, vocab), 3, 6)


@pytest.mark.parametrize("beams,k", [(1, 1), (1, 64), (2, 3), (5, 10), (8, 8), (16, 32), (64, 64), (33, 7), (64, 1)])
def test_beams_and_counts(beams, k):
    _check(_logits(2 * beams, 5003, seed=k), _scores(2 * beams, k), beams, k)


def test_more_rows_than_a_grid_is_high():
    rows = 33000
    logits, scores = _logits(rows, 40, seed=5), _scores(rows, 5)
    _check(logits, scores, 10, 4)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_rows_apart_and_off_their_alignment(kind):
    wide = _logits(8, 9001, kind, 3)
    _check(wide[:, :9000], _scores(8), 4, 8)
    _check(wide[:, 1:8200], _scores(8), 4, 8)                       # neither rows nor the first are aligned
    _check(wide[::2, 3:], _scores(4), 2, 5)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_equal_logits_go_to_lower_tokens(kind):
    x = torch.zeros((4, 20000), dtype=TYPES[kind], device="cuda")
    x[:, 15000:15100] = 3.0
    x[:, 15050] = 4.0
    _check(x, [-1.0] * 4, 2, 64)
    _check(torch.full((2, 9999), -2.5, dtype=TYPES[kind], device="cuda"), [-1.0, -1.0], 1, 20)   # all equal


@pytest.mark.parametrize("vocab", [20000, 20001])
def test_equal_rows_go_to_lower_rows(vocab):
    """The same logits and scores in several rows, which lie differently in memory where the vocabulary is odd."""
    x = _logits(1, vocab, seed=8).repeat(6, 1).contiguous()
    _check(x, [-2.0] * 6, 3, 12)
    _check(x, [-2.0, -2.0, -3.0, -2.0, -3.0, -2.0], 6, 30)


@pytest.mark.parametrize("rows,beams,vocab,seed", [(128, 8, 98305, 0), (120, 5, 60001, 1), (300, 4, 9000, 2), (7, 7, 30000, 3), (96, 3, 40000, 4)])
def test_equal_rows_tie_however_rows_are_split(rows, beams, vocab, seed):
    """Rows of a request alike, some of them at their end: the values of its rows are equal, and lower rows come first."""
    rng = np.random.default_rng(seed)
    x = _logits(rows // beams, vocab, seed=seed).repeat_interleave(beams, 0).contiguous()
    done = [bool(b) for b in rng.random(rows) < 0.2]
    s = np.repeat(_scores(rows // beams, seed), beams)
    s[rng.random(rows) < 0.1] = -np.inf
    _check(x, s, beams, 12, finished=done, pad=1)


def test_signed_zeros_are_equal():
    x = torch.full((1, 300), -1.0, device="cuda")
    x[0, 40], x[0, 20], x[0, 30] = 0.0, -0.0, 0.0
    _check(x, [0.0], 1, 4)


def test_masked_logits():
    inf = float("inf")
    x = _logits(6, 9000, seed=12)
    x[0] = -inf                                                       # nothing left
    x[1, 5:] = -inf                                                   # five tokens
    x[2, :] = -inf
    x[2, 8999] = 1.0                                                  # one
    x[3, ::2] = float("nan")
    x[4, :] = float("nan")
    x[5, 100] = -3.4e38
    _check(x, [-1.0] * 6, 3, 7)
    _check(x, [-1.0] * 6, 1, 12)
    _check(x[:2], [-1.0, -inf], 2, 8)                                 # a beam that was never filled
    _check(x[:2], [-inf, -inf], 2, 8)


MASKS = [-1e8, -1e9, -1e10, -1e20, -1e30, -1e38, -2.5e38, torch.finfo(torch.float32).min]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("mask", MASKS)
def test_parts_of_a_row_at_a_large_negative_value(mask, kind):
    """Masks that are finite: the tokens that are left have the values that they have without the others."""
    x, mask = _logits(8, 30000, kind, 13), max(mask, torch.finfo(TYPES[kind]).min)
    x[0, :20000] = mask
    x[1, 5:] = mask
    x[2, ::2] = mask
    x[3, :29000] = mask
    x[4, 4096:] = mask
    x[5, 100] = mask
    x[6, :15000], x[6, 15000:] = -float("inf"), torch.where(x[6, 15000:] > 0, mask, x[6, 15000:])
    _check(x, _scores(8, 13), 4, 5)
    _check(x, _scores(8, 13), 1, 4, finished=[0, 0, 0, 0, 0, 0, 0, 1])
    _check(x[:, :4096], _scores(8, 13), 8, 8)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("value", MASKS + [1e7, -1e7, 3e7, 1e10, 1e30, 3e38, torch.finfo(torch.float32).max])
def test_rows_at_one_value_however_large(value, kind):
    """Rows that are one value, or nearly so: tokens share the row evenly, wherever it lies."""
    value = float(torch.tensor(value).clamp(torch.finfo(TYPES[kind]).min, torch.finfo(TYPES[kind]).max).to(TYPES[kind]))
    for V in (1, 700, 9001):
        x = torch.full((6, V), value, dtype=TYPES[kind], device="cuda")
        x[1] = _logits(1, V, kind, 14)[0]
        if V > 1:
            x[2, V // 2:] = -float("inf")
            x[3, ::3] = float("nan")
            x[4, V - 1] = torch.nextafter(x[4, 0], torch.tensor(0.0, dtype=TYPES[kind], device="cuda"))
        _check(x, [-1.0, -1.5, -2.0, -2.5, -3.0, -9.0], 3, 8)
        _check(x, [-1.0, -1.5, -2.0, -2.5, -3.0, -9.0], 2, 64, finished=[0, 1, 0, 0, 0, 0])


def test_many_rows_at_a_large_value():
    """More rows than CTAs run at once (a CTA a row), some of them of the lowest finite value; the others are not disturbed."""
    x = _logits(700, 3000, seed=16)
    x[::50] = torch.finfo(torch.float32).min
    x[1::50] = -1e10
    _check(x, _scores(700, 16), 7, 10, finished=[r % 9 == 0 for r in range(700)])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_finished_beams(kind):
    x = _logits(8, 7000, kind, 4)
    x[1] = float("nan")                                               # not read
    s = _scores(8)
    _check(x, s, 4, 8, finished=[0, 1, 0, 1, 0, 0, 0, 0], pad=2)
    _check(x, s, 4, 8, finished=[1] * 8, pad=6999)
    s[3] = -np.inf
    _check(x, s, 4, 8, finished=[0, 1, 0, 1, 0, 0, 0, 0], pad=0)


def test_what_has_no_value_is_reported():
    inf = float("inf")
    x = _logits(4, 5000, seed=6)
    x[1, 77] = inf
    _check(x, [-1.0] * 4, 2, 6, faults=4)
    x = _logits(4, 5000, seed=6)
    for bad in (float("nan"), inf):
        _check(x, [-1.0, bad, -1.0, -1.0], 2, 6, faults=4)
        _check(x, [-1.0, bad, -1.0, -1.0], 2, 6, finished=[0, 1, 0, 0], faults=4)


@pytest.mark.parametrize("spread,shift", [(0.0, 0.0), (1e-4, 0.0), (40.0, 0.0), (3.0, 500.0), (3.0, -20000.0), (1e4, 0.0)])
def test_ranges_of_the_logits(spread, shift):
    """Flat, peaked and far from zero.  (Where logits are large their own spacing decides, not the sums.)"""
    rng = np.random.default_rng(1)
    x = (spread * rng.standard_normal((4, 30000)) + shift).astype(np.float32)
    _check(torch.from_numpy(x).cuda(), [-1.0, -1.25, -1.5, -4.0], 2, 16)


def test_rising_and_falling_logits():
    """Each tile's largest above (below) all before: candidates are taken over and thinned out again."""
    x = torch.linspace(-30, 30, 70001, device="cuda")
    _check(torch.stack([x, x.flip(0), x * 0.001, x.flip(0) * 0.001]), [-1.0] * 4, 2, 64, twins=True)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("k", [1, 10, 64])
@pytest.mark.parametrize("pattern", ["half", "steps", "levels", "last"])
def test_many_logits_at_the_top(pattern, k, kind):
    """More logits than the candidates' room are no smaller than the bound: they are thinned out on the way."""
    V, rng = 30011, np.random.default_rng(50)
    x = rng.standard_normal((2, V))
    if pattern == "half":                                             # equal ones, scattered
        x[:, rng.random(V) < 0.5] = 6.0
    elif pattern == "steps":                                          # rising, each value 1500 times
        x[:] = np.arange(V) // 1500 * 0.25
    elif pattern == "levels":                                         # few values in any order
        x = np.floor(x)
    else:                                                             # all equal but the last ones
        x[:], x[:, -5:] = 1.0, 2.0
    _check(torch.from_numpy(x.astype(np.float32)).to(TYPES[kind]).cuda(), [0.0, -0.5], 2, k)


@pytest.mark.parametrize("fill", [0, 127, 255])
@pytest.mark.parametrize("rows,beams,vocab", [(6, 3, 500), (700, 7, 3000), (12, 4, 9000)])
def test_rows_that_are_not_read_leave_nothing(rows, beams, vocab, fill):
    """Whatever the workspace held: rows at their end and empty ones have no part of it."""
    x, s, done = _logits(rows, vocab, seed=51), _scores(rows), [r % 3 == 1 for r in range(rows)]
    s[::5] = -np.inf
    ws = psd.beam_workspace(ctx(), rows, beams, 6, "cuda")
    ws.fill_(fill)
    out, fault = _run(x, s, beams, 6, finished=done, workspace=ws)
    want = BM.select(x.double().cpu().numpy(), np.asarray(s, dtype=np.float32), beams, 6, done, 0)
    assert fault == 0 and np.array_equal(out[1].cpu().numpy(), want[1]) and np.array_equal(out[2].cpu().numpy(), want[2])


@pytest.mark.parametrize("live", [0, 1, 7])
def test_few_rows_are_read(live):
    """All but some rows are at their end: those share the CTAs."""
    rows, x = 64, _logits(64, 40013, seed=52)
    done = np.ones(rows, dtype=bool)
    done[np.random.default_rng(53).permutation(rows)[:live]] = False
    _check(x, _scores(rows), 8, 16, finished=[bool(d) for d in done], pad=3)


def test_near_values_across_rows():
    """Two rows whose best values differ by some 1e-6 either way."""
    x = _logits(2, 100003, seed=15, spread=2.0)
    gap = BM.select(x.double().cpu().numpy(), np.float32([0, 0]), 1, 1)[0][:, 0]
    for d in (-2e-6, 2e-6):
        _check(x, np.float32([-3.0, -3.0 + gap[0] - gap[1] + d]), 2, 6)


def test_workspace_is_used_again_and_results_repeat():
    ws = psd.beam_workspace(ctx(), 64, 8, 16, "cuda")
    x, s = _logits(64, 33001, seed=2), _scores(64)
    first, _ = _run(x, s, 8, 16, workspace=ws)
    _run(_logits(32, 700, "bf16"), _scores(32), 8, 16, workspace=ws)
    again, _ = _run(x, s, 8, 16, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_captured_and_replayed_on_another_stream():
    x, s = _logits(8, 20001, seed=30), torch.as_tensor(_scores(8).astype(np.float32)).cuda()
    out = [torch.zeros((2, 8), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    ws, fault = psd.beam_workspace(ctx(), 8, 4, 8, "cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        psd.beam_select(ctx(), x, s, *out, ws, beams=4, fault=fault)
    for seed in (31, 32):
        x.copy_(_logits(8, 20001, seed=seed))
        g.replay()
        torch.cuda.synchronize()
        want, _ = _run(x, s.cpu().numpy(), 4, 8)
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and int(fault) == 0


def test_the_longest_rows():
    """5 rows of 2^30 logits: offsets beyond 2^32 elements, and a row that many CTAs share."""
    V, low = 1 << 30, -4.0
    x = torch.full((5, V), low, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, 2047, 2048, V // 2, V - 2, V - 1]
    for i, t in enumerate(at):
        x[:, t] = 5.0 + i
    out, fault = _run(x, [0.0, -1.0, -2.0, -3.0, -4.0], 5, 7)
    assert fault == 0
    lse = np.log((V - 7) * np.exp(low) + np.exp(5.0 + np.arange(7)).sum())
    best = sorted(((5.0 + i - r - lse, -r, -t) for r in range(5) for i, t in enumerate(at)), reverse=True)
    got = out[0][0].double().cpu().numpy()
    for n in range(7):                                                # values of several rows are equal but for the sums' rounding
        r, t = int(out[1][0, n]), int(out[2][0, n])
        assert abs(got[n] - best[n][0]) <= 2.0 ** -24 * abs(best[n][0]) + 2.0 ** -21
        assert abs(5.0 + at.index(t) - r - lse - best[n][0]) < 1e-5
    assert len({*zip(out[1][0].tolist(), out[2][0].tolist())}) == 7


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its workspace, are as they are alone."""
    xs, s = [_logits(16, 50001, kind, seed=40) for kind in ("f32", "bf16")], _scores(16)
    alone = [_run(x, s, 8, 16)[0] for x in xs]
    dev = torch.as_tensor(s.astype(np.float32)).cuda()
    outs = [[torch.zeros_like(t) for t in a] for a in alone]
    spaces = [psd.beam_workspace(ctx(), 16, 8, 16, "cuda") for _ in xs]
    faults = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                psd.beam_select(ctx(), xs[i], dev, *outs[i], spaces[i], beams=8, fault=faults[i])
    torch.cuda.synchronize()
    for out, a, fault in zip(outs, alone, faults):
        assert int(fault) == 0 and all(torch.equal(p, q) for p, q in zip(out, a))


@pytest.mark.parametrize("rows,beams,vocab", [(256, 4, 9000), (1200, 4, 500), (8, 8, 50001)])
def test_scores_in_place(rows, beams, vocab):
    """The new scores written over the old ones: all requests are chosen from the old."""
    x, s, done = _logits(rows, vocab, seed=70), _scores(rows), [bool(r % 5 == 2) for r in range(rows)]
    s[::7] = -np.inf
    want, _ = _run(x, s, beams, beams, finished=done)
    flags, ws = torch.tensor(done, device="cuda"), psd.beam_workspace(ctx(), rows, beams, beams, "cuda")
    for _ in range(20):
        scores = torch.as_tensor(s.astype(np.float32)).cuda()
        out = [scores.view(-1, beams)] + [torch.zeros((rows // beams, beams), dtype=torch.int32, device="cuda") for _ in range(2)]
        psd.beam_select(ctx(), x, scores, *out, ws, beams=beams, finished=flags)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_no_rows():
    out = [torch.zeros((0, 4), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    psd.beam_select(ctx(), torch.zeros((0, 10), device="cuda"), torch.zeros(0, device="cuda"), *out,
                    psd.beam_workspace(ctx(), 0, 2, 4, "cuda"), beams=2)
    torch.cuda.synchronize()


def test_argument_errors():
    x, s = _logits(4, 100), torch.zeros(4, device="cuda")
    out = lambda b=2, k=4: [torch.zeros((b, k), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]  # noqa: E731
    ws = psd.beam_workspace(ctx(), 4, 2, 4, "cuda")
    call = lambda *a, **kw: psd.beam_select(ctx(), *a, **{"beams": 2, **kw})  # noqa: E731
    for a, kw in (((x, s, *out(3), ws), {}), ((x, s, *out(), ws), dict(beams=3)), ((x, s[:3], *out(), ws), {}),
                  ((x, s, *out(), ws), dict(finished=torch.zeros(3, dtype=torch.uint8, device="cuda"))),
                  ((x.t().contiguous().t(), s, *out(), ws), {}), ((x.cpu(), s, *out(), ws), {}), ((x, s.cpu(), *out(), ws), {})):
        with pytest.raises((ValueError, TypeError)):
            call(*a, **kw)
    for a, kw in (((x.double(), s, *out(), ws), {}), ((x, s.double(), *out(), ws), {}),
                  ((x, s, *out(), ws), dict(finished=torch.zeros(4, device="cuda")))):
        with pytest.raises(TypeError):
            call(*a, **kw)
    for a, kw, status in (((x, s, *out(2, 65), ws), {}, 2), ((x, s, *out(), ws[:64]), {}, 5),
                          ((_logits(65, 9), torch.zeros(65, device="cuda"), *out(1), ws), dict(beams=65), 2)):
        with pytest.raises(psd.PsdError) as e:
            call(*a, **kw)
        assert e.value.status == status
