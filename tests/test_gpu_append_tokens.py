"""append_tokens on the GPU against the float64 rotation and append, row by row, and its
refusals and faults."""
import numpy as np
import pytest
import torch

import paged_split_kv_decode_gb300 as psd
from oracle import attention as A
from oracle import tokens as TK
from _gpu_util import ctx

pytestmark = pytest.mark.gpu


def _make(new, before, *, Hq=8, Hkv=2, D=64, Dv=None, page=16, kv="bf16", seed=0, pad_rows=2, fused=True):
    """Inputs on the device; q, k, v as views of one projection's output when fused."""
    rng = np.random.default_rng(seed)
    Dv = D if Dv is None else Dv
    new, total = np.array(new), np.array(new) + np.array(before)
    q_indptr = np.concatenate([[0], np.cumsum(new)])
    pages = -(-total // page)
    page_indptr = np.concatenate([[0], np.cumsum(pages)])
    num_pages = int(page_indptr[-1]) + 2
    page_indices = rng.permutation(num_pages)[: page_indptr[-1]]
    T = int(q_indptr[-1]) + pad_rows
    x = rng.standard_normal((T, Hq * D + Hkv * (D + Dv) + (8 if fused else 0))).astype(np.float32)
    x = torch.from_numpy(x).to(torch.bfloat16).cuda()
    cut = [Hq * D, Hq * D + Hkv * D, Hq * D + Hkv * (D + Dv)]
    views = [x[:, : cut[0]].view(T, Hq, D), x[:, cut[0]: cut[1]].view(T, Hkv, D), x[:, cut[1]: cut[2]].view(T, Hkv, Dv)]
    if not fused:
        views = [v.contiguous() for v in views]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()  # noqa: E731

    def pool(width):
        if kv == "fp8":
            return torch.from_numpy(rng.integers(0, 126, (num_pages, page, Hkv, width)).astype(np.uint8)).cuda()
        return torch.from_numpy(rng.standard_normal((num_pages, page, Hkv, width)).astype(np.float32)).to(torch.bfloat16).cuda()

    return dict(q=views[0], k=views[1], v=views[2], q_indptr=dev(q_indptr), kv_len=dev(total),
                page_indptr=dev(page_indptr), page_indices=dev(page_indices), k_pool=pool(D), v_pool=pool(Dv),
                host=dict(q_indptr=q_indptr, total=total, page_indptr=page_indptr, page_indices=page_indices, page=page))


def _values(t):
    t = t.cpu()
    return A.e4m3_to_f64(t.numpy()).reshape(tuple(t.shape)) if t.dtype == torch.uint8 else t.double().numpy()


def _call(s, rope, **kw):
    q_out = torch.full(s["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    f = psd.append_tokens(ctx(), s["q"], s["k"], s["v"], q_out, q_indptr=s["q_indptr"], kv_len=s["kv_len"],
                          page_indptr=s["page_indptr"], page_indices=s["page_indices"], k_pool=s["k_pool"],
                          v_pool=s["v_pool"], rope=rope, **kw)
    torch.cuda.synchronize()
    return q_out, int(f.item())


def _close(got, want, size, scale, fp8):
    """One rounding to the stored type, after an f32 rotation: sincospi is good to 2 ulp of 1,
    its argument to 2^-24 of a half turn (pi 2^-24 rad), the magnitude and the two products and
    the sum to a rounding each: under 2^-20 of |x| + |y|; the quotient by the scale one more."""
    f32 = size * 2.0 ** -20 + np.abs(want) * 2.0 ** -23
    if fp8:
        bound = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + f32 / scale * 1.0625
    else:
        bound = 2.0 ** -8 * np.abs(want) + f32 * (1 + 2.0 ** -8) + 1e-38
    worst = float(np.max(np.abs(got - want) / bound, initial=0.0))
    assert worst <= 1, worst


def _check(s, rope, *, neox=True, rope_col=0, positions=None, k_scale=1.0, v_scale=1.0, **kw):
    fp8 = s["k_pool"].dtype == torch.uint8
    h, before_k, before_v = s["host"], _values(s["k_pool"]), _values(s["v_pool"])
    pos = None if positions is None else torch.tensor(positions, dtype=torch.int32, device="cuda")
    q_out, fault = _call(s, rope, neox=neox, rope_col=rope_col, positions=pos, k_scale=k_scale, v_scale=v_scale, **kw)
    assert fault == 0
    where = TK.positions_of(h["q_indptr"], h["total"])
    n = len(where)
    at = np.array([p for _, p in where]) if positions is None else np.array(positions[:n])
    rot = lambda x: TK.rotate(x[:n].double().cpu().numpy(), at[:, None], rope.inv_freq, rope.magnitude, rope_col, neox)  # noqa: E731
    want, size = rot(s["q"])
    _close(_values(q_out)[:n], want, size, 1.0, False)
    assert torch.all(q_out[n:] == 7.0)          # rows behind the last request stay
    want, size = rot(s["k"])
    rows = [int(h["page_indices"][h["page_indptr"][b] + p // h["page"]]) * h["page"] + p % h["page"] for b, p in where]
    limit = 448.0 if fp8 else np.inf
    flat = lambda a: a.reshape((-1,) + a.shape[2:])  # noqa: E731
    k, v = flat(_values(s["k_pool"])), flat(_values(s["v_pool"]))
    ks, vs = (k_scale, v_scale) if fp8 else (1.0, 1.0)
    _close(k[rows], np.clip(want / ks, -limit, limit), size, ks, fp8)
    vals = s["v"][:n].double().cpu().numpy()
    _close(v[rows], np.clip(vals / vs, -limit, limit), 0 * vals, vs, fp8)
    rest = np.setdiff1d(np.arange(k.shape[0]), rows)
    assert np.array_equal(k[rest], flat(before_k)[rest]) and np.array_equal(v[rest], flat(before_v)[rest])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("D,rot,col", [(64, 64, 0), (128, 32, 0), (128, 64, 64), (192, 64, 128), (40, 10, 7), (256, 256, 0)])
def test_layouts_and_types(kv, neox, D, rot, col):
    s = _make([3, 1, 0, 17], [0, 40, 9, 15], D=D, kv=kv, seed=D + rot)
    scales = dict(k_scale=0.03, v_scale=0.017) if kv == "fp8" else {}
    _check(s, psd.rope_frequencies(rot), neox=neox, rope_col=col, **scales)


@pytest.mark.parametrize("kind", ["plain", "linear", "ntk", "yarn", "bands"])
def test_far_positions(kind):
    """A million positions out, f32 angles would be off by 2^-4 rad."""
    s = _make([4, 2], [20, 0], D=128, seed=5)
    pos = [0, 1, 65537, 1000003, 2 ** 31 - 1, 123456789, 0, 0]
    _check(s, psd.rope_frequencies(128, base=500000.0, scaling=kind, factor=8.0, original_max_position=8192),
           positions=pos)


@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("fused", [True, False])
def test_pages(page, fused):
    _check(_make([7, 30, 1, 64], [100, 3, 0, 0], page=page, seed=page, fused=fused), psd.rope_frequencies(64))


@pytest.mark.parametrize("B", [1, 31, 32, 33, 200, 1100])
def test_many_requests(B):
    rng = np.random.default_rng(B)
    new = rng.integers(0, 4, B)
    new[rng.integers(B)] = 5
    _check(_make(new, rng.integers(1, 20, B), Hq=2, Hkv=1, seed=B), psd.rope_frequencies(64))


def test_long_prompt():
    _check(_make([700, 1, 1400], [3, 500, 0], Hq=4, Hkv=2, D=128, seed=9), psd.rope_frequencies(128))


@pytest.mark.parametrize("T", [0, 1])
def test_fewest_tokens(T):
    s = _make([T], [4], pad_rows=0)
    _check(s, psd.rope_frequencies(64))


def test_in_place_queries_and_kv_only():
    s = _make([5, 2], [3, 30], fused=False, pad_rows=0)
    want = torch.empty_like(s["q"])
    rope = psd.rope_frequencies(32)
    kw = dict(q_indptr=s["q_indptr"], kv_len=s["kv_len"], page_indptr=s["page_indptr"], page_indices=s["page_indices"],
              k_pool=s["k_pool"], v_pool=s["v_pool"], rope=rope, neox=True)
    psd.append_tokens(ctx(), s["q"], s["k"], s["v"], want, **kw)
    kp, vp = s["k_pool"].clone(), s["v_pool"].clone()
    psd.append_tokens(ctx(), s["q"], s["k"], s["v"], s["q"], **kw)
    assert torch.equal(s["q"], want) and torch.equal(kp, s["k_pool"]) and torch.equal(vp, s["v_pool"])
    s["k_pool"].zero_()
    psd.append_tokens(ctx(), None, s["k"], s["v"], None, **kw)
    rows = s["k_pool"].view(-1, 2, 64).abs().sum((1, 2)) != 0
    assert int(rows.sum()) == 7 and torch.equal(s["k_pool"].view(-1, 2, 64)[rows], kp.view(-1, 2, 64)[rows])


def test_values_that_are_not_finite_and_saturation():
    s = _make([2], [0], kv="fp8", pad_rows=0, fused=False)
    s["v"][0, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e30], dtype=torch.bfloat16)
    _call(s, psd.rope_frequencies(64), neox=True)
    page = int(s["page_indices"][0])
    assert [int(x) for x in s["v_pool"][page, 0, 0, :4]] in ([0x7F, 0x7E, 0xFE, 0x7E], [0xFF, 0x7E, 0xFE, 0x7E])


def test_faults_skip_and_are_flagged():
    rope = psd.rope_frequencies(64)
    s = _make([2, 2], [3, 16], fused=False, pad_rows=0)
    before = s["k_pool"].clone()
    s["page_indices"][0] = 10 ** 6               # the first request's page
    q_out, fault = _call(s, rope, neox=True)
    assert fault == 1 and not torch.any(q_out == 7.0)
    assert torch.equal(s["k_pool"].view(-1, 2, 64).ne(before.view(-1, 2, 64)).any(-1).any(-1).sum(),
                       torch.tensor(2, device="cuda"))
    s = _make([2, 2], [3, 16], fused=False, pad_rows=0)
    s["kv_len"][1] = 60                          # past its page list
    assert _call(s, rope, neox=True)[1] == 1
    s = _make([2, 2], [3, 16], fused=False, pad_rows=0)
    s["kv_len"][0] = 1                           # index -1: no position of its own
    q_out, fault = _call(s, rope, neox=True)
    assert fault == 4 and torch.all(q_out[0] == 7.0) and not torch.any(q_out[1] == 7.0)
    pos = torch.tensor([5, -2, 1, 1], dtype=torch.int32, device="cuda")
    s = _make([2, 2], [3, 16], fused=False, pad_rows=0)
    q_out, fault = _call(s, rope, neox=True, positions=pos)
    assert fault == 4 and torch.all(q_out[1] == 7.0)


def test_refusals():
    s = _make([2], [3], pad_rows=0)
    q_out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    base = dict(q_indptr=s["q_indptr"], kv_len=s["kv_len"], page_indptr=s["page_indptr"],
                page_indices=s["page_indices"], k_pool=s["k_pool"], v_pool=s["v_pool"], rope=psd.rope_frequencies(64),
                neox=True)

    def refused(kind, q=s["q"], k=s["k"], v=s["v"], out=q_out, **kw):
        with pytest.raises(kind):
            psd.append_tokens(ctx(), q, k, v, out, **{**base, **kw})

    refused(psd.PsdError, rope_col=2)
    refused(psd.PsdError, rope=psd.RopeFrequencies([-1.0]))
    refused(psd.PsdError, rope=psd.RopeFrequencies([float("inf")]))
    refused(psd.PsdError, rope=psd.RopeFrequencies([0.5], float("nan")))
    refused(ValueError, out=s["q"])                                  # in place needs contiguous queries
    refused(TypeError, q_indptr=s["q_indptr"].long())
    refused(ValueError, q_indptr=s["q_indptr"][:1])
    refused(ValueError, v=None)
    refused(ValueError, k_pool=s["k_pool"][..., :32])
    refused(TypeError, k=s["k"].float())
    refused(ValueError, k=s["k"].transpose(1, 2))
    fp8 = _make([2], [3], pad_rows=0, kv="fp8")
    refused(psd.PsdError, k_pool=fp8["k_pool"], v_pool=fp8["v_pool"], k_scale=0.0)


def test_graph_replay_on_another_stream():
    """Captured on a side stream, the call reads its tables anew at each replay."""
    s = _make([1, 3], [8, 20], seed=2)
    rope = psd.rope_frequencies(64)
    q_out = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda out: psd.append_tokens(  # noqa: E731
        ctx(), s["q"], s["k"], s["v"], out, q_indptr=s["q_indptr"], kv_len=s["kv_len"], page_indptr=s["page_indptr"],
        page_indices=s["page_indices"], k_pool=s["k_pool"], v_pool=s["v_pool"], rope=rope, neox=False, fault=fault)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(q_out)
    s["kv_len"] -= 1
    g.replay()
    want = torch.zeros_like(q_out)
    torch.cuda.synchronize()
    pools = s["k_pool"].clone(), s["v_pool"].clone()
    call(want)
    assert torch.equal(q_out[:4], want[:4])
    assert torch.equal(pools[0], s["k_pool"]) and torch.equal(pools[1], s["v_pool"]) and int(fault) == 0


def test_a_new_fault_word_on_the_stream_of_the_call():
    """The word that a call makes for itself starts at 0 in the call's stream, whatever the current
    stream is busy with."""
    s = _make([2, 2], [3, 16], fused=False, pad_rows=0)
    s["page_indices"][0] = 10 ** 6                       # skipped by the kernel's own check
    rope, q_out = psd.rope_frequencies(64), torch.empty_like(s["q"])
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)                   # the current stream, some 50 ms
        f = psd.append_tokens(ctx(), s["q"], s["k"], s["v"], q_out, q_indptr=s["q_indptr"], kv_len=s["kv_len"],
                              page_indptr=s["page_indptr"], page_indices=s["page_indices"], k_pool=s["k_pool"],
                              v_pool=s["v_pool"], rope=rope, neox=True, stream=stream)
        torch.cuda.synchronize()
        assert int(f) == 1


def test_a_magnitude_that_f32_does_not_hold():
    s = _make([2], [3], pad_rows=0)
    before = s["k_pool"].clone()
    for magnitude in (1e39, -1e39):
        with pytest.raises(psd.PsdError) as e:
            _call(s, psd.RopeFrequencies([0.5, 0.25], magnitude), neox=True)
        assert e.value.status == 1
    assert torch.equal(s["k_pool"], before)
    _check(s, psd.RopeFrequencies([0.5, 0.25], -3.0))


MANY = dict(new=[300, 1, 0, 450, 76, 2, 113], before=[3, 500, 20, 0, 61, 16, 15])   # two tokens a CTA, the last alone


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("D,rot,col", [(64, 64, 0), (128, 64, 64), (128, 32, 16), (256, 128, 0)])
def test_many_tokens_of_every_layout(kv, neox, D, rot, col):
    s = _make(**MANY, Hq=4, Hkv=2, D=D, kv=kv, seed=D + rot, pad_rows=3)
    rng = np.random.default_rng(D)
    scales = dict(k_scale=0.03, v_scale=0.017) if kv == "fp8" else {}
    _check(s, psd.rope_frequencies(rot), neox=neox, rope_col=col, **scales)
    far = [int(x) for x in rng.integers(0, 2 ** 31, s["q"].shape[0])]
    _check(s, psd.rope_frequencies(rot, scaling="yarn", factor=8.0, original_max_position=4096), neox=neox,
           rope_col=col, positions=far, **scales)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("Dv", [128, 40, 20])
def test_values_of_another_width(Dv, many, kv):
    shape = MANY if many else dict(new=[3, 1, 0, 17], before=[0, 40, 9, 15])
    scales = dict(k_scale=0.03, v_scale=0.017) if kv == "fp8" else {}
    _check(_make(**shape, Hq=4, Hkv=2, D=64, Dv=Dv, kv=kv, seed=Dv), psd.rope_frequencies(32), **scales)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("D,rot,col", [(192, 64, 128), (40, 10, 7)])
def test_keys_alone(D, rot, col, many, kv):
    """No values (they lie in the key rows): queries and keys as with values, bit for bit."""
    shape = MANY if many else dict(new=[3, 1, 0, 17], before=[0, 40, 9, 15])
    s = _make(**shape, Hq=8, Hkv=1, D=D, kv=kv, seed=D)
    rope, start = psd.rope_frequencies(rot), s["k_pool"].clone()
    kw = dict(neox=False, rope_col=col, k_scale=0.03)
    want, fault = _call(s, rope, **kw)
    keys = s["k_pool"].clone()
    s["k_pool"].copy_(start)
    s["v"] = s["v_pool"] = None
    got, fault2 = _call(s, rope, **kw)
    assert fault == fault2 == 0
    assert torch.equal(want, got) and torch.equal(keys, s["k_pool"]) and not torch.equal(keys, start)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_faults_among_many_tokens(kv):
    """Two tokens a CTA, one of them or both at fault: theirs is left out, the others are what they were."""
    rope = psd.rope_frequencies(32)
    make = lambda: _make(**MANY, Hq=4, Hkv=2, D=64, kv=kv, seed=6, pad_rows=0)  # noqa: E731
    s = make()
    start = s["k_pool"].clone(), s["v_pool"].clone()
    T, h = s["q"].shape[0], s["host"]
    where = TK.positions_of(h["q_indptr"], h["total"])
    pos = [p for _, p in where]
    want, fault = _call(s, rope, neox=True)
    assert fault == 0
    rows = [int(h["page_indices"][h["page_indptr"][b] + p // h["page"]]) * h["page"] + p % h["page"] for b, p in where]
    untouched, unwritten = [0, 7, 100, 101, T - 1], [t for t in range(T) if where[t] in {(3, p) for p in range(16, 32)}]
    for t in untouched:
        pos[t] = -1 - t
    bad = make()
    bad["page_indices"][int(h["page_indptr"][3]) + 1] = 2 ** 31 - 1     # a page of request 3
    out, fault = _call(bad, rope, neox=True, positions=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    assert fault == 5 and len(unwritten) == 16
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[untouched] = False
    assert torch.equal(out[keep], want[keep]) and bool((out[~keep] == 7.0).all())
    left = [rows[t] for t in untouched + unwritten]
    for got, good, before in ((bad["k_pool"], s["k_pool"], start[0]), (bad["v_pool"], s["v_pool"], start[1])):
        expect = good.clone().flatten(0, 1)
        expect[left] = before.flatten(0, 1)[left]
        assert torch.equal(got.flatten(0, 1), expect)
