"""verify_drafts on the GPU against exact rational arithmetic: accepted counts and tokens
are equal, whatever the sizes."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_split_kv_decode_gb300 as psd
from oracle import tokens as TK
from _gpu_util import ctx

pytestmark = pytest.mark.gpu


def _soft(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def _make(K, V, seed=0, sampled=True, near=0.5):
    rng = np.random.default_rng(seed)
    K = np.array(K)
    indptr = np.concatenate([[0], np.cumsum(K)])
    D, B = int(indptr[-1]), len(K)
    logits = 2 * rng.standard_normal((D + B, V))
    rows = np.arange(D) + np.repeat(np.arange(B), K)
    target, draft = _soft(logits), _soft(logits[rows] + near * rng.standard_normal((D, V)))
    tokens = np.array([rng.choice(V, p=p.astype(np.float64) / p.astype(np.float64).sum()) for p in draft], dtype=np.int64)
    return dict(target=target, draft=draft if sampled else None, tokens=tokens, indptr=indptr,
                uniforms=rng.random(D + B, dtype=np.float32))


def _run(s, pad=0):
    """The call, with rows `pad` elements further apart than vocab."""
    def rows(a):
        if a is None:
            return None
        wide = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), device="cuda")
        wide[:, : a.shape[1]] = torch.from_numpy(a).cuda()
        return wide[:, : a.shape[1]]
    i32 = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).cuda()  # noqa: E731
    B, D = len(s["indptr"]) - 1, len(s["tokens"])
    accepted = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    out = torch.full((D + B,), -9, dtype=torch.int32, device="cuda")
    fault = psd.verify_drafts(ctx(), rows(s["target"]), rows(s["draft"]), i32(s["tokens"]), i32(s["indptr"]),
                              torch.from_numpy(s["uniforms"]).cuda(), accepted, out)
    return accepted.tolist(), out.tolist(), int(fault.item())


def _check(s, pad=0, fault=0):
    accepted, out, f = _run(s, pad)
    want = TK.verify(s["target"], s["draft"], s["tokens"], s["indptr"], s["uniforms"])
    assert accepted == want[0] and out == want[1] and f == fault


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 1024, 1025, 8192, 20011])
@pytest.mark.parametrize("pad", [0, 3])
def test_vocabularies(V, sampled, pad):
    _check(_make([3, 0, 5, 1], V, seed=V, sampled=sampled), pad)


@pytest.mark.parametrize("K", [[0], [1], [0, 0, 0], [70], [33, 1, 0, 2], [2] * 50])
def test_draft_counts(K):
    _check(_make(K, 300, seed=len(K), near=0.05))


def test_many_seeds():
    for seed in range(40):
        _check(_make([4, 4, 4], 257, seed=100 + seed, near=1.0))


def test_numbers_at_the_borders():
    """Sums that meet u * total exactly, and u = 0: the least token whose running sum exceeds
    it, never one without weight."""
    p = np.zeros((1, 64), dtype=np.float32)
    p[0, 8::8] = 1 / 8
    for k in range(7):
        _check(dict(target=p, draft=None, tokens=np.zeros(0), indptr=[0, 0], uniforms=np.array([k / 7], dtype=np.float32)))
        _check(dict(target=p, draft=None, tokens=np.zeros(0), indptr=[0, 0], uniforms=np.array([k / 8], dtype=np.float32)))
    _check(dict(target=p, draft=None, tokens=np.zeros(0), indptr=[0, 0],
                uniforms=np.array([1 - 2.0 ** -24], dtype=np.float32)))


def test_acceptance_borders():
    """u q == p refuses; the next number below accepts; q = p always accepts; q = 0 accepts where p > 0."""
    V = 16
    p = np.full((2, V), 1 / 16, dtype=np.float32)
    q = np.zeros((1, V), dtype=np.float32)
    q[0, 3], q[0, 4] = 0.25, 0.75
    for u in (0.25, np.nextafter(np.float32(0.25), np.float32(0)), 0.0, 0.9999999):
        for tok in (3, 4, 5):
            _check(dict(target=p, draft=q, tokens=np.array([tok]), indptr=[0, 1],
                        uniforms=np.array([u, 0.5], dtype=np.float32)))
    _check(dict(target=p, draft=p[:1], tokens=np.array([7]), indptr=[0, 1],
                uniforms=np.array([0.9999999, 0.5], dtype=np.float32)))


def test_no_residual_falls_back_to_the_target():
    p = np.full((2, 8), 0.125, dtype=np.float32)
    p[0, 2] = 0
    q = np.ones((1, 8), dtype=np.float32)
    _check(dict(target=p, draft=q, tokens=np.array([2]), indptr=[0, 1], uniforms=np.array([0.5, 0.9], dtype=np.float32)))


def test_tiny_probabilities_count():
    p = np.full((1, 5000), 2.0 ** -40, dtype=np.float32)
    p[0, 4321] = 2.0 ** -39
    for u in (0.1, 0.5, 0.99):
        _check(dict(target=p, draft=None, tokens=np.zeros(0), indptr=[0, 0], uniforms=np.array([u], dtype=np.float32)))


def test_faults():
    s = _make([2, 2], 50, seed=3)
    s["tokens"][1] = 50                                # outside the vocabulary
    s["uniforms"][0] = 0.0                             # draft 0 is accepted
    _check(s, fault=4)
    s = _make([1, 0], 50, seed=4)
    s["target"][2] = 0.0                               # nothing to draw from
    _check(s, fault=4)
    s["target"][2] = np.nan
    accepted, out, f = _run(s)
    assert out[2] == -1 and f == 4
    s = _make([1, 1], 50, seed=4)
    s["indptr"] = np.array([0, 1, 5])                  # past the drafts: that request is skipped
    accepted, out, f = _run(s)
    assert f == 4 and accepted[1] == -9 and out[2:] == [-9, -9]


def test_refusals():
    s = _make([1], 8)
    t = torch.from_numpy(s["target"]).cuda()
    d = torch.from_numpy(s["draft"]).cuda()
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    u = torch.zeros(2, device="cuda")
    ok = [t, d, i(1), i(0, 1), u, i(0), i(0, 0)]
    psd.verify_drafts(ctx(), *ok)
    for at, bad, kind in [(0, t[:1], ValueError), (0, t.double(), TypeError), (0, t.t(), ValueError),
                          (1, d[:, :4], ValueError), (2, torch.tensor([1], device="cuda"), TypeError),
                          (3, i(0), ValueError), (4, u[:1], ValueError), (6, i(0), ValueError),
                          (5, torch.zeros(1, dtype=torch.int32), ValueError)]:
        args = list(ok)
        args[at] = bad
        with pytest.raises(kind):
            psd.verify_drafts(ctx(), *args)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    psd.verify_drafts(ctx(), t[:0], None, none, i(0), u[:0], none, none)  # an empty batch


def test_repeats_agree_and_replay():
    s = _make([5] * 20, 30011, seed=8)
    first = _run(s)
    assert all(_run(s) == first for _ in range(3))
    i32 = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).cuda()  # noqa: E731
    args = [torch.from_numpy(s["target"]).cuda(), torch.from_numpy(s["draft"]).cuda(), i32(s["tokens"]), i32(s["indptr"]),
            torch.from_numpy(s["uniforms"]).cuda(), i32(np.zeros(20)), i32(np.zeros(120))]
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        psd.verify_drafts(ctx(), *args, fault=fault)
    args[4].zero_()
    g.replay()
    s["uniforms"][:] = 0
    want = TK.verify(s["target"], s["draft"], s["tokens"], s["indptr"], s["uniforms"])
    assert args[5].tolist() == want[0] and args[6].tolist() == want[1]


@pytest.mark.parametrize("V", [131072, 200001, 262143])
def test_rows_that_sum_far_past_one(V):
    """Weights of 1 everywhere: sums of V, in units of 2^-46 up to 64 bits."""
    s = dict(target=np.ones((1, V), dtype=np.float32), draft=None, tokens=np.zeros(0), indptr=[0, 0])
    for u in (0.0, 0.37, 1 - 2.0 ** -24):
        s["uniforms"] = np.array([u], dtype=np.float32)
        # the least v with v + 1 > u V
        want = int(Fraction(float(s["uniforms"][0])) * V)
        assert _run(s) == ([0], [want], 0)


@pytest.mark.parametrize("V,ones", [(262144, 262144), (300000, 300000), (1100003, 1100003), (1100003, 262144), (1100003, 262145),
                                    (2200003, 300000), (2200003, 2200003)])
def test_sums_that_64_bits_do_not_hold(V, ones):
    """A sum of 2^18 or more is no token's: -1 and a fault, in a batch whose other rows are drawn."""
    target = np.zeros((3, V), dtype=np.float32)
    target[0, 17], target[2, V - 1] = 0.5, 0.25
    target[1, V - ones:] = 1.0
    s = dict(target=target, draft=None, tokens=np.zeros(0), indptr=[0, 0, 0, 0],
             uniforms=np.array([0.3, 0.3, 0.9], dtype=np.float32))
    assert _run(s) == ([0, 0, 0], [17, -1, V - 1], 4)


def test_a_new_fault_word_on_the_stream_of_the_call():
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    p = torch.full((2, 16), 1 / 16, device="cuda")
    args = [p, None, i32(99), i32(0, 1), torch.zeros(2, device="cuda"), i32(0), i32(0, 0)]   # a token outside
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                       # the current stream, some 50 ms
    f = psd.verify_drafts(ctx(), *args, stream=side)
    torch.cuda.synchronize()
    assert int(f) == 4


def _check_in_64_bits(s):
    """Against 64-bit arithmetic, for rows too many or too long for fractions.  The acceptance is exact in
    it.  A weight in units of 2^-46 may differ by one from the kernel's, so a running sum, and the share
    of the total it is compared with, by V each: where the borders that leave are further apart than that
    the token is known, and that has to be nearly always."""
    accepted, out, fault = _run(s)
    assert fault == 0
    V, B, sure = s["target"].shape[1], len(s["indptr"]) - 1, 0
    f64 = lambda a: a.astype(np.float64)  # noqa: E731
    for b in range(B):
        d0, K = int(s["indptr"][b]), int(s["indptr"][b + 1] - s["indptr"][b])
        R, a = d0 + b, 0
        while a < K:
            d = int(s["tokens"][d0 + a])
            q = 1.0 if s["draft"] is None else float(s["draft"][d0 + a, d])
            if not float(s["uniforms"][R + a]) * q < float(s["target"][R + a, d]):
                break
            a += 1
        w = f64(s["target"][R + a])
        if a < K and s["draft"] is not None:
            w = np.maximum(w - f64(s["draft"][d0 + a]), 0)
        elif a < K:
            w[int(s["tokens"][d0 + a])] = 0
        w = w if w.any() else f64(s["target"][R + a])
        sums = np.cumsum(np.rint(w * 2.0 ** 46).astype(np.int64))
        want = int(Fraction(float(s["uniforms"][R + K])) * int(sums[-1]))
        lo, hi = (min(int(np.searchsorted(sums, x, side="right")), V - 1) for x in (want - 2 * V - 2, want + 2 * V + 2))
        assert accepted[b] == a and lo <= out[R + a] <= hi
        assert out[R: R + a] == s["tokens"][d0: d0 + a].tolist() and out[R + a + 1: R + K + 1] == [-1] * (K - a)
        sure += lo == hi
    assert sure >= B - B // 8


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("B,K,V", [(100, 4, 8200), (90, 1, 98305), (200, 2, 4097), (700, 1, 300)])
def test_batches_of_more_ctas_than_the_sms_hold(B, K, V, sampled):
    """More than four CTAs an SM: one block of a warp on its way at a time."""
    rng = np.random.default_rng(B)
    _check_in_64_bits(_make(rng.integers(0, K + 1, B), V, seed=B, sampled=sampled))


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("K,V", [([3, 0, 2], 98305), ([1, 2], 131072), ([5] * 20, 30011), ([1], 1100003), ([1], 2200003)])
def test_long_rows(K, V, sampled):
    """Blocks for every warp of a CTA, two at a time, and from 2.1 million words on blocks of more than
    256 entries."""
    for near in (0.2, 2.0):
        _check_in_64_bits(_make(K, V, seed=V, sampled=sampled, near=near))
