"""multi_token_decode over a cache of 8-bit blocks with a scale each, on the GPU against float64 softmax attention over the
values the codes and scales stand for: blocks, pages, head layouts, lengths, masks, scales far apart; refusals and faults."""
import numpy as np
import pytest
import torch

import paged_split_kv_decode_gb300 as psd
from _gpu_util import ctx
from _scaled_util import Scaled
from _tokens_util import bounds

pytestmark = pytest.mark.gpu


def _check(s, *, out_f32=False, sm_scale=None, got=None):
    o, lse = s.run(out_f32=out_f32, sm_scale=sm_scale) if got is None else got
    n = int(s.q_indptr[-1])
    assert torch.all(o[n:] == 5.0) and torch.all(lse[n:] == 5.0)   # rows behind the last request stay
    want = s.oracle(sm_scale)
    # P meets V as f16: one term for bf16 outputs (2^-11, counted as that), two for f32 outputs (2^-22); a scale is exact
    e_o, e_l = bounds(want, s.D, int(s.total.max()), out_f32, 2 if out_f32 else 1)
    if not out_f32:
        e_o = e_o - (2.0 ** -8 - 2.0 ** -11) * want[2] * (1 + 2.0 ** -8)
    # f16 ends at 2^-24: a weight is off by half of that at least.  In the units of P the row's largest is 2^7 or more, so
    # that is 2^-32 of the largest weight, which is at most 1 after the division by the sum; it meets a code of at most 448
    # in units of the largest scale (V's scales of other blocks are a factor <= 1 in P), once a key.  It shows where the
    # heavy keys have no V: the bound above is relative to sum p |v|.
    ve = s.ve[s.ve != 255]
    e_o = e_o + 2.0 ** -32 * int(s.total.max()) * 448 * 2.0 ** (int(ve.max()) - 127)
    o, lse = o[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()
    empty = np.isneginf(want[1])
    assert np.array_equal(np.isneginf(lse), empty) and not o[empty].any()
    d = np.abs(o - want[0])
    worst = float(np.max(d / e_o))
    assert worst <= 1, (worst, [int(x[0]) for x in np.nonzero(~(d <= e_o))])
    d = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, want[1]))
    worst = float(np.max(d / np.maximum(e_l, 1e-30)))
    assert worst <= 1, (worst, [int(x[0]) for x in np.nonzero(~(d <= e_l))])


RAGGED = dict(new=[1, 5, 0, 3, 40, 2], before=[0, 200, 33, 127, 90, 128])


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (32, 16), (64, 16), (32, 32), (64, 64), (48, 16), (192, 64)])
def test_ragged(page, block, D, out_f32):
    _check(Scaled(**RAGGED, D=D, page=page, block=block, seed=page + D), out_f32=out_f32)


@pytest.mark.parametrize("n", [1, 2, 5])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (3, 1), (10, 2), (7, 1), (8, 1), (9, 1), (16, 1), (28, 4), (33, 1), (40, 8), (128, 1)])
def test_head_layouts(Hq, Hkv, n):
    _check(Scaled([n, 1, n], [60, 200, 3], Hq=Hq, Hkv=Hkv, seed=Hq))


@pytest.mark.parametrize("D,page,block,G", [(8, 16, 16, 2), (40, 16, 16, 2), (80, 32, 32, 4), (256, 16, 16, 2), (64, 16, 16, 130)])
def test_shapes_of_the_general_kernel(D, page, block, G):
    _check(Scaled([2, 0, 33, 1], [50, 7, 0, 300], Hq=2 * G if G < 100 else G, Hkv=2 if G < 100 else 1, D=D, page=page,
                  block=block, seed=D + page))


@pytest.mark.parametrize("n,before", [(1, 0), (1, 15), (1, 16), (1, 17), (1, 63), (1, 64), (1, 127), (1, 128), (2, 15), (16, 0),
                                      (17, 0), (127, 0), (128, 0), (129, 0), (31, 97), (33, 95), (65, 0), (200, 57), (300, 0)])
@pytest.mark.parametrize("G", [1, 4])
def test_lengths_around_the_tiles(n, before, G):
    _check(Scaled([n], [before], Hq=2 * G, Hkv=2, seed=n + before))


@pytest.mark.parametrize("out_f32", [False, True])
def test_long_cache_is_split(out_f32):
    _check(Scaled([2], [9001], Hq=4, Hkv=1, D=128, seed=1), out_f32=out_f32)
    _check(Scaled([1, 1, 3], [5000, 3, 2500], Hq=4, Hkv=2, page=64, block=32, seed=2), out_f32=out_f32)
    _check(Scaled([1], [20000], Hq=2, Hkv=2, D=64, page=64, block=64, seed=3), out_f32=out_f32)


@pytest.mark.parametrize("out_f32", [False, True])
def test_many_requests(out_f32):
    """More requests than a launch carries, most of one token, some of none."""
    rng = np.random.default_rng(4)
    new = [int(x) for x in rng.integers(0, 3, 300)]
    _check(Scaled(new, [int(x) for x in rng.integers(1, 80, 300)], Hq=4, Hkv=2, seed=4), out_f32=out_f32)


@pytest.mark.parametrize("B,keys", [(1, 30), (1, 160), (1, 200), (60, 100), (20, 700), (200, 260), (256, 33), (3, 900)])
@pytest.mark.parametrize("D", [64, 128])
def test_requests_that_are_cut_or_not(D, B, keys):
    """Equal and nearly equal requests: short ones and many of them are not cut, long ones are."""
    rng = np.random.default_rng(B)
    _check(Scaled([1] * B, [keys - int(x) for x in rng.integers(0, 20, B)], Hq=8, Hkv=2, D=D, seed=B), out_f32=bool(B % 2))


def test_prompt_and_single_tokens():
    _check(Scaled([1, 500, 1, 2], [700, 150, 33, 0], Hq=4, Hkv=1, D=128, seed=7))
    _check(Scaled([1, 500, 1, 2], [700, 150, 33, 0], Hq=4, Hkv=1, D=128, seed=7), out_f32=True)


@pytest.mark.parametrize("page,block", [(16, 16), (64, 32)])
@pytest.mark.parametrize("out_f32", [False, True])
def test_trees(page, block, out_f32):
    _check(Scaled([64, 1, 10, 33, 0, 24], [0, 50, 121, 100, 5, 4000], page=page, block=block, tree="random", seed=page),
           out_f32=out_f32)
    _check(Scaled([3, 1, 2, 1], [40, 50, 121, 900], page=page, block=block, tree="random", seed=page), out_f32=out_f32)


def test_tree_rows_that_see_nothing():
    _check(Scaled([5, 3], [0, 0], tree=[0, 1, 0, 0b1000, 0b1111] + [0, 1 << 63, (1 << 64) - 1]))
    _check(Scaled([1, 1], [0, 0], tree=[0, 1]))
    _check(Scaled([2, 3], [9, 0], tree=[(1 << 64) - 1] * 5))


@pytest.mark.parametrize("spread", [0.0, 30.0])
@pytest.mark.parametrize("n", [1, 20])
def test_flat_and_peaked_scores(n, spread):
    _check(Scaled([n, 3], [300, 900], Hq=4, Hkv=1, spread=spread, seed=11), out_f32=True)


def _grow(s, e, step):
    """The scales of a request's blocks, one after another, by 2^step each."""
    for b in range(len(s.total)):
        for j in range(0, int(s.total[b]), s.block):
            page = int(s.page_indices[s.page_indptr[b] + j // s.page])
            e[page, j % s.page // s.block] = int(np.clip(127 - 3 + step * (j // s.block), 95, 170))


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("n", [1, 3, 50])
@pytest.mark.parametrize("step", [-1, 1, 2])
def test_scales_that_rise_and_fall_along_the_cache(step, n, out_f32):
    """V's scales change by a power of two from block to block: what O is kept in units of has to follow.  K's scales are
    the same everywhere, so that every block counts."""
    s = Scaled([n, 1], [250, 100], Hq=4, Hkv=1, D=128, seed=13 + n)
    _grow(s, s.ve, step)
    s.ke[s.ke != 255] = 121
    _check(s, out_f32=out_f32)


@pytest.mark.parametrize("n", [1, 30])
def test_keys_whose_scales_grow(n):
    """Scores that keep growing along the cache: the running maximum moves."""
    s = Scaled([n, 1], [150, 80], Hq=4, Hkv=1, D=64, seed=14)
    _grow(s, s.ke, 1)
    _check(s, out_f32=True)


@pytest.mark.parametrize("n", [1, 30])
def test_blocks_of_zeros(n):
    """A block of zeros has the least scale: its weight in the sum is what the scores say."""
    s = Scaled([n], [130], Hq=4, Hkv=1, D=64, seed=15)
    for j in (0, 3, 4):
        page = int(s.page_indices[j])
        s.v[page] = torch.where(s.v[page] == 0x7F, s.v[page], torch.zeros_like(s.v[page]))
        s.ve[page] = 95
    page = int(s.page_indices[1])
    s.k[page], s.ke[page] = 0, 95
    _check(s, out_f32=True)


@pytest.mark.parametrize("n", [1, 30])
def test_scale_bytes_of_zero(n):
    """Byte 0 stands for 2^-127: scores and values of those blocks are 0 beside the others'."""
    s = Scaled([n], [130], Hq=4, Hkv=1, D=64, seed=16)
    s.ve[int(s.page_indices[2])] = 0
    s.ke[int(s.page_indices[5])] = 0
    _check(s)


@pytest.mark.parametrize("n", [1, 30])
def test_a_scale_of_nan_is_seen(n):
    """Rows that see a block whose scale is NaN are NaN."""
    s = Scaled([n], [130], Hq=4, Hkv=1, D=64, seed=17)
    s.ve[int(s.page_indices[2])] = 255
    o, _ = s.run(out_f32=True)
    assert bool(o[:n].isnan().all())
    s = Scaled([n], [130], Hq=4, Hkv=1, D=64, seed=17)
    s.ke[int(s.page_indices[2])] = 255
    o, lse = s.run(out_f32=True)
    assert bool(o[:n].isnan().all()) and bool(lse[:n].isnan().all())


@pytest.mark.parametrize("sm_scale", [-0.1, 0.0, 1e-30, 3.0])
@pytest.mark.parametrize("n", [1, 30])
def test_softmax_scales(n, sm_scale):
    _check(Scaled([n, 2], [90, 10], seed=18), sm_scale=sm_scale)


def test_query_views_and_output_without_lse():
    s = Scaled([1, 4], [70, 20], D=128, seed=19)
    wide = torch.full((s.T, s.Hq * s.D + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = wide[:, 32: 32 + s.Hq * s.D].view(s.T, s.Hq, s.D)
    q.copy_(s.q)
    _check(s, got=s.run(q=q))
    plan, o = s.plan(), torch.full((s.T, s.Hq, s.D), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = psd.multi_token_workspace(ctx(), plan, s.D, "cuda")
    psd.multi_token_decode(ctx(), s.args(), plan, o, None, ws)
    assert torch.equal(o[: s.T - 3], s.run()[0][: s.T - 3])


@pytest.mark.parametrize("n", [1, 70])
def test_results_repeat(n):
    s = Scaled([n, n, 1], [1000, 30, 3000], Hq=16, Hkv=4, D=128, seed=20)
    a, b = s.run(out_f32=True), s.run(out_f32=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n", [1, 40])
def test_captured_and_replayed(n):
    """A replay reads queries, pools and scales anew."""
    s = Scaled([n, 1], [500, 900], Hq=8, Hkv=2, D=128, seed=21)
    plan = s.plan()
    ws = psd.multi_token_workspace(ctx(), plan, s.D, "cuda")
    args = s.args()
    o = torch.full((s.T, s.Hq, s.D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s.T, s.Hq), 5.0, device="cuda")
    psd.multi_token_decode(ctx(), args, plan, o, lse, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        psd.multi_token_decode(ctx(), args, plan, o, lse, ws)
    t = Scaled([n, 1], [500, 900], Hq=8, Hkv=2, D=128, seed=22)
    for dst, src in zip(args.tensors[:3], (t.q, t.k, t.v)):
        dst.copy_(src)
    args.tensors[3].copy_(torch.from_numpy(t.page_indices))
    args.scales.k.copy_(t.ke)
    args.scales.v.copy_(t.ve)
    g.replay()
    torch.cuda.synchronize()
    assert psd.check_device_error(ctx(), ws) == 0
    _check(t, got=(o, lse))


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D", [64, 128, 80])
def test_bad_page_ids_are_reported(n, D):
    """Page ids outside the pool are not read; the call reports them and others' rows stay right."""
    s = Scaled([n, 1], [200, 100], Hq=4, Hkv=1, D=D, seed=23)
    bad = s.page_indices.copy()
    bad[2], bad[3] = -1, 2 ** 31 - 1
    plan = s.plan()
    ws = psd.multi_token_workspace(ctx(), plan, s.D, "cuda")
    o = torch.full((s.T, s.Hq, s.D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s.T, s.Hq), 5.0, device="cuda")
    psd.multi_token_decode(ctx(), s.args(indices=torch.from_numpy(bad).cuda()), plan, o, lse, ws)
    with pytest.raises(psd.PsdError) as e:
        psd.check_device_error(ctx(), ws)
    assert e.value.fault_bits == 1
    good = s.run()
    assert torch.equal(o[n: n + 1], good[0][n: n + 1]) and torch.equal(lse[n: n + 1], good[1][n: n + 1])


@pytest.mark.parametrize("D,out_f32", [(64, True), (128, False)])
def test_bounded_wait_runs_out_and_is_reported(D, out_f32):
    """Loads of the tcgen05 kernel are withheld from a unit's second key tile on: the waits for them run out (about 1 ms), the
    call completes and reports it, and the next call is right."""
    s = Scaled([40, 70, 9], [1500, 300, 900], D=D, seed=25)
    ctx().test_withhold_loads(1, 2_000_000)
    try:
        with pytest.raises(psd.PsdError) as e:
            s.run(out_f32=out_f32)
    finally:
        ctx().test_withhold_loads(-1)
    assert e.value.status == 4 and e.value.fault_bits == 2
    _check(s, out_f32=out_f32)


@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("Hkv", [1, 2, 3])
@pytest.mark.parametrize("off", [1, 2])
def test_scales_at_any_address(off, Hkv, n):
    """Scale arrays are bytes: they need no alignment."""
    s = Scaled([n, 2], [333, 70], Hq=4 * Hkv, Hkv=Hkv, D=64, page=48, seed=26)
    views = []
    for e in (s.ke, s.ve):
        wide = torch.full((e.numel() + 8,), 255, dtype=torch.uint8, device="cuda")
        views.append(wide[off: off + e.numel()].view(e.shape))
        views[-1].copy_(e)
    s.scales = lambda: psd.BlockScales(*views, 16)
    _check(s, out_f32=True)


@pytest.mark.parametrize("n", [1, 40])
def test_two_streams_at_once(n):
    """Calls that overlap on two streams, each with its workspace, are as they are alone."""
    cases = [Scaled([n, 1, n], [4000, 300, 900 + i], Hq=8, Hkv=2, D=128, seed=27 + i) for i in range(2)]
    alone = [s.run(out_f32=True) for s in cases]
    plans, streams = [s.plan() for s in cases], [torch.cuda.Stream() for _ in cases]
    args = [s.args() for s in cases]
    spaces = [psd.multi_token_workspace(ctx(), p, 128, "cuda") for p in plans]
    outs = [[torch.full_like(t, 5.0) for t in a] for a in alone]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                psd.multi_token_decode(ctx(), args[i], plans[i], *outs[i], spaces[i])
    torch.cuda.synchronize()
    for i, stream in enumerate(streams):
        assert psd.check_device_error(ctx(), spaces[i]) == 0
        assert all(torch.equal(a, b) for a, b in zip(outs[i], alone[i]))


def test_one_workspace_for_call_after_call():
    """Calls of all three kernels behind each other on one stream use one workspace."""
    cases = [Scaled([n, 2], [900, 30], Hq=8, Hkv=2, D=D, seed=30 + n) for n, D in ((1, 128), (40, 128), (3, 80), (2, 64))]
    alone = [s.run() for s in cases]
    plans, args = [s.plan() for s in cases], [s.args() for s in cases]
    size = max(psd.multi_token_workspace(ctx(), p, s.D, "cuda").numel() for s, p in zip(cases, plans))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    outs = [[torch.full_like(t, 5.0) for t in a] for a in alone]
    for _ in range(5):
        for i in range(len(cases)):
            psd.multi_token_decode(ctx(), args[i], plans[i], *outs[i], ws)
    assert psd.check_device_error(ctx(), ws) == 0
    for out, a in zip(outs, alone):
        assert all(torch.equal(x, y) for x, y in zip(out, a))


def test_pools_past_32_bits():
    """Pools of over 2^32 bytes, whose requests lie at both ends."""
    pages, page, Hkv, D = 20000, 64, 16, 256
    for D in (128, 256):
        pages = 2 ** 33 // (page * Hkv * D) + 40
        k = torch.zeros((pages, page, Hkv, D), dtype=torch.uint8, device="cuda")
        v = torch.zeros_like(k)
        ke = torch.full((pages, 1, Hkv), 127, dtype=torch.uint8, device="cuda")
        ve = ke.clone()
        for p, c in ((0, 0x38), (pages - 1, 0x40)):                  # 1.0 and 2.0
            v[p] = c
            ve[p] = 128
        idx = torch.tensor([0, pages - 1], dtype=torch.int32, device="cuda")
        plan = psd.plan_multi_token(psd.HostTable([0, 1, 2], [0, pages - 1], [64, 64], 64), [0, 1, 2])
        q = torch.zeros((2, Hkv, D), dtype=torch.bfloat16, device="cuda")
        args = psd.multi_token_args(q, k, v, idx, sm_scale=1.0, scales=psd.BlockScales(ke, ve, 64))
        o = torch.empty((2, Hkv, D), device="cuda")
        ws = psd.multi_token_workspace(ctx(), plan, D, "cuda")
        psd.multi_token_decode(ctx(), args, plan, o, None, ws)
        assert psd.check_device_error(ctx(), ws) == 0
        assert bool((o[0] == 2.0).all()) and bool((o[1] == 4.0).all())
        del k, v


def test_argument_errors():
    s = Scaled([1, 2], [20, 3], seed=24)
    k, v, idx = s.k.cuda(), s.v.cuda(), torch.from_numpy(s.page_indices).cuda()
    q = s.q.cuda()
    sc = s.scales()
    with pytest.raises(ValueError):
        psd.BlockScales(sc.k, sc.v[:1], 16)
    with pytest.raises(TypeError):
        psd.BlockScales(sc.k.int(), sc.v.int(), 16)
    with pytest.raises(ValueError):                                   # of another pool
        psd.multi_token_args(q, k, v, idx, sm_scale=1.0, scales=psd.BlockScales(sc.k[:2], sc.v[:2], 16))
    with pytest.raises(ValueError):
        psd.multi_token_args(q, k, v, idx, sm_scale=1.0, scales=psd.BlockScales(sc.k, sc.v, 8))
    plan, o = s.plan(), torch.empty((s.T, s.Hq, s.D), device="cuda")
    ws = psd.multi_token_workspace(ctx(), plan, s.D, "cuda")

    def refused(status, **kw):
        with pytest.raises(psd.PsdError) as e:
            psd.multi_token_decode(ctx(), psd.multi_token_args(q, **{**dict(k_pool=k, v_pool=v, page_indices_dev=idx, sm_scale=1.0, scales=sc), **kw}), plan, o, None, ws)
        assert e.value.status == status

    refused(1, k_scale=0.5)
    refused(1, v_scale=2.0)
    refused(1, k_pool=k.to(torch.bfloat16), v_pool=v.to(torch.bfloat16))
    half = psd.BlockScales(sc.k.repeat(1, 2, 1), sc.v.repeat(1, 2, 1), 8)
    refused(1, scales=half)
