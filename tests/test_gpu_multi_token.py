"""multi_token_decode on the GPU against float64 softmax attention, row by row: types, head
layouts, page sizes, lengths, masks, splits along the cache; its refusals and faults."""
import numpy as np
import pytest
import torch

import paged_split_kv_decode_gb300 as psd
from oracle import tokens as TK
from _gpu_util import ctx
from _tokens_util import Step, bounds

pytestmark = pytest.mark.gpu


def _tensor_cores(s, sm_scale):
    return s.D in (64, 128) and s.page % 8 == 0 and s.Hq // s.Hkv <= 128 and sm_scale > 0


def _run(s, *, out_f32=False, sm_scale=None, q=None, workspace=None, plan=None, o=None, lse=None, indices=None):
    sm_scale = s.sm_scale if sm_scale is None else sm_scale
    q = s.q.cuda() if q is None else q
    idx = torch.from_numpy(s.page_indices).cuda() if indices is None else indices
    args = psd.multi_token_args(q, s.k.cuda(), s.v.cuda(), idx, sm_scale=sm_scale, k_scale=s.scales[0],
                                v_scale=s.scales[1], tree_mask=s.tree_dev())
    if plan is None:
        table = psd.HostTable(s.page_indptr, s.page_indices, s.last, s.page)
        plan = psd.plan_multi_token(table, s.q_indptr, s.Hq, s.Hkv)
    if workspace is None:
        workspace = psd.multi_token_workspace(ctx(), plan, s.D, "cuda")
        workspace.fill_(255)
    if o is None:
        o = torch.full((s.T, s.Hq, s.D), 5.0, dtype=torch.float32 if out_f32 else torch.bfloat16, device="cuda")
        lse = torch.full((s.T, s.Hq), 5.0, device="cuda")
    psd.multi_token_decode(ctx(), args, plan, o, lse, workspace)
    assert psd.check_device_error(ctx(), workspace) == 0
    return o, lse


def _check(s, *, out_f32=False, sm_scale=None, got=None):
    o, lse = _run(s, out_f32=out_f32, sm_scale=sm_scale) if got is None else got
    n = int(s.q_indptr[-1])
    assert torch.all(o[n:] == 5.0) and torch.all(lse[n:] == 5.0)   # rows behind the last request stay
    want = s.oracle(sm_scale)
    terms = (1 if not out_f32 else 2 if s.kv == "fp8" else 3) if _tensor_cores(s, s.sm_scale if sm_scale is None else sm_scale) else 0
    e_o, e_l = bounds(want, s.D, int(s.total.max()), out_f32, terms)
    o, lse = o[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()
    empty = np.isneginf(want[1])
    same = np.array_equal(np.isneginf(lse), empty) and not o[empty].any()
    assert same
    d = np.abs(o - want[0])
    worst = float(np.max(d / e_o))
    assert worst <= 1, (worst, [int(x[0]) for x in np.nonzero(~(d <= e_o))])
    d = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, want[1]))
    worst = float(np.max(d / np.maximum(e_l, 1e-30)))
    assert worst <= 1, (worst, [int(x[0]) for x in np.nonzero(~(d <= e_l))])


RAGGED = dict(new=[1, 5, 0, 3, 40, 2], before=[0, 200, 33, 127, 90, 128])


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 24, 64])
def test_ragged(page, D, kv, out_f32):
    _check(Step(**RAGGED, Hq=8, Hkv=2, D=D, page=page, kv=kv, seed=page + D), out_f32=out_f32)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (3, 1), (10, 2), (7, 1), (16, 1), (28, 4), (33, 1), (128, 1)])
def test_head_layouts(Hq, Hkv):
    _check(Step([1, 6, 14], [60, 200, 3], Hq=Hq, Hkv=Hkv, seed=Hq))


@pytest.mark.parametrize("D,page,G", [(8, 16, 2), (40, 16, 2), (80, 8, 4), (256, 16, 2), (64, 1, 4), (64, 5, 4), (128, 12, 1), (64, 16, 130)])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_shapes_of_the_general_kernel(D, page, G, kv):
    _check(Step([2, 0, 33, 1], [50, 7, 0, 300], Hq=2 * G if G < 100 else G, Hkv=2 if G < 100 else 1, D=D, page=page, kv=kv, seed=D + page))


@pytest.mark.parametrize("n,before", [(1, 0), (1, 127), (1, 128), (2, 127), (127, 0), (128, 0), (129, 0), (31, 97),
                                      (32, 96), (33, 95), (64, 0), (65, 0), (200, 57), (300, 0)])
@pytest.mark.parametrize("G", [1, 4])
def test_lengths_around_the_tiles(n, before, G):
    _check(Step([n], [before], Hq=2 * G, Hkv=2, seed=n + before))


@pytest.mark.parametrize("out_f32", [False, True])
def test_long_cache_is_split(out_f32):
    _check(Step([2], [9001], Hq=4, Hkv=1, D=128, seed=1), out_f32=out_f32)
    _check(Step([1, 1, 3], [5000, 3, 2500], Hq=4, Hkv=2, page=64, seed=2), out_f32=out_f32)


@pytest.mark.parametrize("D,page,G,kv,out_f32", [(256, 16, 4, "bf16", False), (96, 7, 1, "fp8", True), (64, 1, 2, "bf16", True),
                                                 (8, 3, 9, "fp8", False), (128, 12, 130, "bf16", False)])
def test_long_cache_of_the_general_kernel(D, page, G, kv, out_f32):
    """Few rows over many keys: the keys are split over CTAs and joined; some rows see far fewer."""
    s = Step([1, 3, 2], [5000, 900, 0], Hq=2 * G, Hkv=2, D=D, page=page, kv=kv, seed=60)
    _check(s, out_f32=out_f32)
    first, again = _run(s, out_f32=out_f32), _run(s, out_f32=out_f32)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("D,page", [(80, 4), (200, 16)])
def test_trees_of_the_general_kernel(D, page):
    s = Step([1, 40, 64, 0, 7], [3000, 70, 1, 20, 129], D=D, page=page, seed=61, tree="random")
    _check(s)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prompt_and_single_tokens(kv):
    _check(Step([1, 500, 1, 2], [700, 150, 33, 0], Hq=4, Hkv=1, kv=kv, D=128, seed=7))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("page", [8, 16, 5])
@pytest.mark.parametrize("out_f32", [False, True])
def test_trees(page, kv, out_f32):
    _check(Step([64, 1, 10, 33, 0, 24], [0, 50, 121, 100, 5, 4000], kv=kv, page=page, tree="random", seed=page),
           out_f32=out_f32)


def test_tree_rows_that_see_nothing():
    """No prefix and no bit set: zeros and -inf, beside rows that see one key or all."""
    masks = [0, 1, 0, 0b1000, 0b1111] + [0, 1 << 63, (1 << 64) - 1]
    _check(Step([5, 3], [0, 0], tree=masks))
    masks = [0] * 8
    _check(Step([5, 3], [0, 130], tree=masks))


def test_tree_bits_past_the_new_tokens_are_ignored():
    _check(Step([2, 3], [9, 0], tree=[(1 << 64) - 1] * 5))


@pytest.mark.parametrize("spread", [0.0, 30.0])
def test_flat_and_peaked_scores(spread):
    _check(Step([20, 3], [300, 900], Hq=4, Hkv=1, spread=spread, seed=11), out_f32=True)


def test_rising_scores_rescale():
    """Keys whose scores keep growing along the cache: the running maximum moves in every tile."""
    s = Step([3], [1500], Hq=4, Hkv=1, seed=12)
    q = torch.zeros_like(s.q)
    q[:, :, 0] = 4.0
    s.q = q
    flat = s.k.view(-1, 1, 64)
    for j in range(1503):
        slot = int(s.page_indices[j // 16]) * 16 + j % 16
        flat[slot, 0, 0] = j * 0.25
    _check(s, out_f32=True)


def test_negative_and_zero_scale():
    s = Step(**RAGGED, seed=13)
    _check(s, sm_scale=-0.2)
    _check(s, sm_scale=0.0)


def test_strided_queries_and_no_lse():
    s = Step(**RAGGED, seed=14)
    wide = torch.full((s.T, s.Hq * s.D + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = wide[:, 8: 8 + s.Hq * s.D].view(s.T, s.Hq, s.D)
    view.copy_(s.q)
    _check(s, got=_run(s, q=view))
    o, _ = _run(s)
    alone = torch.full_like(o, 5.0)
    _run(s, o=alone, lse=None)
    assert torch.equal(o, alone)


@pytest.mark.parametrize("B", [800, 1700])
def test_batches_of_several_launches(B):
    rng = np.random.default_rng(B)
    _check(Step(rng.integers(0, 3, B), rng.integers(1, 40, B), Hq=2, Hkv=1, seed=B))


@pytest.mark.parametrize("kv,D,out_f32", [("bf16", 128, False), ("bf16", 128, True), ("fp8", 128, False), ("bf16", 64, False),
                                          ("fp8", 64, True)])
def test_many_long_units_a_cta(kv, D, out_f32):
    """Several units share a CTA, with odd and even numbers of tiles, and one-tile pieces and units
    of two row tiles between them: every ring and buffer passes from one to the next."""
    new = [2, 1, 3, 5, 1, 2, 70, 1, 4, 2, 3, 1, 1, 2]
    before = [3000, 130, 900, 1500, 2500, 60, 2000, 5, 800, 3900, 257, 1100, 640, 2049]
    s = Step(new, before, Hq=16, Hkv=8, D=D, page=16, kv=kv, seed=31)
    first = _run(s, out_f32=out_f32)
    _check(s, out_f32=out_f32, got=first)
    for _ in range(5):
        again = _run(s, out_f32=out_f32)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("D,kv,out_f32", [(64, "bf16", False), (128, "bf16", False), (64, "fp8", False), (128, "bf16", True)])
def test_many_short_prompts(D, kv, out_f32):
    """Units of two row tiles and one key tile, many to a CTA, with others between them."""
    rng = np.random.default_rng(D)
    new = [int(x) for x in rng.integers(33, 65, 60)]
    before = [int(x) for x in rng.integers(0, 40, 60)]
    new[10], before[10], new[40], before[40] = 2, 70, 1, 300
    s = Step(new, before, Hq=32, Hkv=8, D=D, page=8, kv=kv, seed=33)
    first = _run(s, out_f32=out_f32)
    for _ in range(30):
        again = _run(s, out_f32=out_f32)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    keep = [0, 9, 10, 11, 39, 40, 41, 59]                 # the oracle looks at some of the requests
    o, lse = (x.double().cpu().numpy() for x in first)
    for b in keep:
        lo, hi = int(s.q_indptr[b]), int(s.q_indptr[b + 1])
        pages = s.page_indices[s.page_indptr[b]: s.page_indptr[b + 1]]
        want = TK.attend(s.q[lo:hi].double().numpy(), s.values(s.k, s.scales[0]), s.values(s.v, s.scales[1]), [0, hi - lo],
                         [s.total[b]], [0, len(pages)], pages, s.page, s.sm_scale)
        e_o, e_l = bounds(want, D, int(s.total[b]), out_f32, 3 if out_f32 else 1)
        assert bool((np.abs(o[lo:hi] - want[0]) <= e_o).all()) and bool((np.abs(lse[lo:hi] - want[1]) <= e_l).all())


def test_more_keys_pages_repeat():
    """A page listed twice holds its tokens twice."""
    s = Step([2], [78], Hq=2, Hkv=1, seed=15)
    s.page_indices[2] = s.page_indices[0]
    _check(s)


def test_repeats_are_bit_equal():
    s = Step([1, 300, 5], [4000, 100, 900], Hq=8, Hkv=2, seed=16)
    first = _run(s)
    for _ in range(3):
        again = _run(s)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_agrees_with_single_token_decode():
    """One new token a request is the flat decode of the framework."""
    s = Step([1] * 6, [5, 100, 700, 1, 1300, 64], seed=17, pad_rows=0)
    o, lse = _run(s, out_f32=True)
    table = psd.HostTable(s.page_indptr, s.page_indices, s.last, s.page)
    plan = psd.plan_decode(table, 64, 0)
    args = psd.decode_args(s.q.cuda(), s.k.cuda(), s.v.cuda(), torch.from_numpy(s.page_indices).cuda(),
                           num_pages=s.num_pages, page_size=s.page, Hkv=s.Hkv, Dv=s.D, sm_scale=s.sm_scale)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    psd.cascade_decode(ctx(), args, plan, o2, lse2, psd.workspace_for(plan, s.Hq, s.D, "cuda"))
    # each side is within 2e-5 of the exact result on such pools
    assert float((o - o2).abs().max()) <= 4e-5 and float((lse - lse2).abs().max()) <= 4e-5


def test_states_merge_with_merge_states():
    """(o, lse) of two halves of a cache merge to the whole: lse is in merge_states' units."""
    s = Step([1], [127], Hq=4, Hkv=1, seed=18, pad_rows=0)
    whole = _run(s, out_f32=True)
    parts = []
    for lo, hi in ((0, 4), (4, 8)):
        table = psd.HostTable([0, 4], s.page_indices[lo:hi], [16], 16)
        plan = psd.plan_multi_token(table, [0, 1])
        idx = torch.from_numpy(s.page_indices[lo:hi].copy()).cuda()
        o, lse = torch.empty_like(whole[0]), torch.empty_like(whole[1])
        parts.append(_run(s, plan=plan, indices=idx, o=o, lse=lse))
    v, l = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    o, lse = torch.empty_like(whole[0]), torch.empty_like(whole[1])
    psd.merge_states(ctx(), v, l, torch.tensor([0, 2], dtype=torch.int32, device="cuda"), o, lse)
    assert float((o - whole[0]).abs().max()) <= 4e-5 and float((lse - whole[1]).abs().max()) <= 4e-5


def test_graph_replay_reads_the_inputs_anew():
    s = Step([4, 1, 150], [60, 2000, 10], seed=19)
    q, k, v, idx = s.q.cuda(), s.k.cuda(), s.v.cuda(), torch.from_numpy(s.page_indices).cuda()
    args = psd.multi_token_args(q, k, v, idx, sm_scale=s.sm_scale)
    plan = psd.plan_multi_token(psd.HostTable(s.page_indptr, s.page_indices, s.last, s.page), s.q_indptr)
    ws = psd.multi_token_workspace(ctx(), plan, s.D, "cuda")
    o = torch.full((s.T, s.Hq, s.D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s.T, s.Hq), 5.0, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        psd.multi_token_decode(ctx(), args, plan, o, lse, ws)
    del plan                                            # the lists are in the graph
    for _ in range(2):
        q.copy_(s.q)
        g.replay()
        torch.cuda.synchronize()
        _check(s, got=(o, lse))
        s.q = (s.q.float() * 0.5).to(torch.bfloat16)


def test_two_streams_with_their_own_workspaces():
    steps = [Step([3, 60], [800 + 100 * i, 40], seed=20 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in steps]
    want = [_run(s) for s in steps]
    torch.cuda.synchronize()
    got = []
    for s, st in zip(steps, streams):
        with torch.cuda.stream(st):
            got.append(_run(s))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_graphs_with_their_own_workspaces():
    """Replayed on two streams at a time, over split units in both."""
    steps = [Step([4, 1], [3000, 2500 + i], seed=40 + i) for i in range(2)]
    graphs, outs = [], []
    for s in steps:
        args = psd.multi_token_args(s.q.cuda(), s.k.cuda(), s.v.cuda(), torch.from_numpy(s.page_indices).cuda(),
                                    sm_scale=s.sm_scale)
        plan = psd.plan_multi_token(psd.HostTable(s.page_indptr, s.page_indices, s.last, s.page), s.q_indptr)
        ws = psd.multi_token_workspace(ctx(), plan, s.D, "cuda")
        o = torch.full((s.T, s.Hq, s.D), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((s.T, s.Hq), 5.0, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            psd.multi_token_decode(ctx(), args, plan, o, lse, ws)
        graphs.append((g, args, ws))
        outs.append((o, lse))
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(20):
        for (g, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for s, got in zip(steps, outs):
        _check(s, got=got)


@pytest.mark.parametrize("kv,out_f32", [("bf16", False), ("fp8", False), ("fp8", True)])
@pytest.mark.parametrize("D", [64, 128])
def test_powers_of_two_in_the_queries(kv, out_f32, D):
    """Queries times 2^e and a scale of 2^-e change nothing; a row with one element 2^9 above the
    rest stays within the bounds."""
    s = Step([5, 40], [100, 300], D=D, kv=kv, seed=50)
    want = _run(s, out_f32=out_f32)
    q = s.q.clone()
    for e in (-60, 40):
        s.q = (q.float() * 2.0 ** e).to(torch.bfloat16)
        got = _run(s, out_f32=out_f32, sm_scale=s.sm_scale * 2.0 ** -e)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    s.q = q
    s.q[:, :, 3] *= 512
    _check(s, out_f32=out_f32, sm_scale=s.sm_scale / 64)


@pytest.mark.parametrize("kv,D,out_f32", [("bf16", 128, False), ("fp8", 128, False), ("fp8", 64, True), ("bf16", 64, True), ("bf16", 40, False)])
def test_rows_that_are_not_finite_stay_alone(kv, D, out_f32):
    """NaN or infinite query rows give NaN in their own rows; the others are what they were."""
    s = Step([5, 40], [100, 300], D=D, kv=kv, seed=70)
    o, lse = _run(s, out_f32=out_f32)
    s.q[2, 1] = float("nan")
    s.q[30, 0] = float("inf")
    s.q[31, 5, 7] = -float("inf")
    got_o, got_lse = _run(s, out_f32=out_f32)
    at = torch.zeros((s.T, s.Hq), dtype=torch.bool, device="cuda")
    at[2, 1] = at[30, 0] = at[31, 5] = True
    assert bool(torch.isnan(got_o[at]).all()) and bool(torch.isnan(got_lse[at]).all())
    assert torch.equal(got_o[~at], o[~at]) and torch.equal(got_lse[~at], lse[~at])


def test_nothing_to_attend():
    """No request, and requests without new tokens: the outputs stay as they were."""
    s = Step([0, 0], [20, 33], seed=51)
    o, lse = _run(s)
    assert bool((o == 5.0).all()) and bool((lse == 5.0).all())


@pytest.mark.parametrize("kv,D,out_f32", [("bf16", 64, False), ("bf16", 128, True), ("fp8", 64, True), ("fp8", 128, False)])
def test_bounded_wait_runs_out_and_is_reported(kv, D, out_f32):
    """The loads of each unit's key tiles from index 1 on are withheld: the waits for them run out
    (about 1 ms), every role stops, the call completes and reports it, and the next call is
    clean."""
    s = Step([4, 70, 1], [1500, 300, 900], D=D, kv=kv, seed=52)
    ctx().test_withhold_loads(1, 2_000_000)
    try:
        with pytest.raises(psd.PsdError) as e:
            _run(s, out_f32=out_f32)
    finally:
        ctx().test_withhold_loads(-1)
    assert e.value.status == 4 and e.value.fault_bits == 2
    _check(s, out_f32=out_f32)


@pytest.mark.parametrize("D", [64, 40])
def test_bad_page_id_is_flagged(D):
    s = Step([2, 3], [100, 40], D=D, seed=21)
    bad = torch.from_numpy(s.page_indices).cuda()
    bad[1] = s.num_pages + 9
    with pytest.raises(psd.PsdError) as e:
        _run(s, indices=bad)
    assert e.value.status == 4 and e.value.fault_bits == 1
    _check(s)


def test_refusals():
    s = Step([2, 70], [3, 4], seed=22)
    table = psd.HostTable(s.page_indptr, s.page_indices, s.last, s.page)
    plan = psd.plan_multi_token(table, s.q_indptr)
    q, k, v, idx = s.q.cuda(), s.k.cuda(), s.v.cuda(), torch.from_numpy(s.page_indices).cuda()
    o, lse = torch.empty((s.T, s.Hq, s.D), device="cuda"), torch.empty((s.T, s.Hq), device="cuda")
    ws = psd.multi_token_workspace(ctx(), plan, s.D, "cuda")
    fresh = lambda **kw: psd.multi_token_args(q, k, v, idx, **{"sm_scale": 0.1, **kw})  # noqa: E731

    def refused(status, args, o=o, ws=ws, plan=plan):
        with pytest.raises(psd.PsdError) as e:
            psd.multi_token_decode(ctx(), args, plan, o, lse, ws)
        assert e.value.status == status

    refused(1, fresh(sm_scale=float("nan")))
    refused(1, fresh(tree_mask=torch.zeros(s.T, dtype=torch.int64, device="cuda")))  # 70 new tokens
    refused(5, fresh(), ws=ws[:128])
    refused(1, fresh(), ws=torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")[4: 4 + ws.numel()])
    for field, value in (("Hkv", 3), ("page_size", 8), ("num_tokens", 70), ("num_page_indices", 1), ("q_stride", 1),
                         ("q_stride", s.Hq * s.D + 4), ("kv_dtype", 7), ("num_pages", 0), ("D", 60)):
        a = fresh()
        setattr(a, field, value)
        if field in ("num_tokens", "D"):
            refused(1, a, o=torch.empty((a.num_tokens, a.Hq, a.D), device="cuda")) if field == "D" else None
            continue
        refused(1, a)
    wide = Step([1], [3], D=264, seed=23)
    a = psd.multi_token_args(wide.q.cuda(), wide.k.cuda(), wide.v.cuda(), torch.from_numpy(wide.page_indices).cuda(),
                             sm_scale=0.1)
    p = psd.plan_multi_token(psd.HostTable(wide.page_indptr, wide.page_indices, wide.last, 16), wide.q_indptr)
    with pytest.raises(psd.PsdError) as e:
        psd.multi_token_decode(ctx(), a, p, torch.empty(wide.q.shape, device="cuda"), None, ws)
    assert e.value.status == 2
    with pytest.raises(TypeError):
        psd.multi_token_decode(ctx(), fresh(), plan, o.half(), lse, ws)
    with pytest.raises(ValueError):
        psd.multi_token_decode(ctx(), fresh(), plan, o[:, :1], lse, ws)
    with pytest.raises(ValueError):
        fresh(tree_mask=torch.zeros(3, dtype=torch.int64, device="cuda"))
    broken = psd.plan_multi_token(table, s.q_indptr)
    broken.requests_a[1].token0 = 1
    refused(1, fresh(), plan=broken)
    empty = psd.plan_multi_token(psd.HostTable([0], [], [], 16), [0])
    psd.multi_token_decode(ctx(), fresh(), empty, o, lse, ws)   # nothing to do


@pytest.mark.parametrize("D", [64, 40])
def test_faults_of_replays_and_of_calls_on_one_workspace(D):
    """A bad page id (skipped by the kernel's own check) of a replay is reported whatever calls came
    after the capture, and a replay leaves an unread fault of a call."""
    s = Step([2, 3], [100, 40], D=D, seed=80)
    q, k, v, idx = s.q.cuda(), s.k.cuda(), s.v.cuda(), torch.from_numpy(s.page_indices).cuda()
    good, bad = idx.clone(), idx.clone()
    bad[1] = s.num_pages + 9
    args = psd.multi_token_args(q, k, v, idx, sm_scale=s.sm_scale)
    plan = psd.plan_multi_token(psd.HostTable(s.page_indptr, s.page_indices, s.last, s.page), s.q_indptr)
    ws = psd.multi_token_workspace(ctx(), plan, s.D, "cuda")
    ws.fill_(255)
    o, lse = torch.empty((s.T, s.Hq, D), device="cuda"), torch.empty((s.T, s.Hq), device="cuda")
    call = lambda: psd.multi_token_decode(ctx(), args, plan, o, lse, ws)  # noqa: E731
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g.replay)

    def check(*runs):
        for ids, run in runs:
            idx.copy_(ids)
            run()
        return psd.check_device_error(ctx(), ws)

    def flagged(*runs):
        with pytest.raises(psd.PsdError) as e:
            check(*runs)
        assert e.value.status == 4 and e.value.fault_bits == 1
        assert psd.check_device_error(ctx(), ws) == 0     # a reported fault is cleared

    first, second = graphs
    assert check((good, first)) == 0
    flagged((bad, first))
    flagged((good, call), (bad, first))                   # the context's latest call is another
    flagged((bad, first), (good, call))                   # the call does not take the replay's fault
    flagged((bad, first), (good, second))
    flagged((bad, call), (good, first))                   # nor the replay the call's
    flagged((bad, call), (bad, second))
    assert check((bad, call), (good, call)) == 0          # a call's faults are the latest call's
    assert check((good, first), (good, call), (good, second)) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("sm_scale", [2.0 ** -60, 2.0 ** -120])
def test_small_scales_beside_rows_of_zeros(kv, sm_scale):
    """Scores of almost 0: every visible key weighs the same, hidden ones nothing."""
    s = Step([5, 40], [100, 300], kv=kv, seed=81)
    s.q[[0, 2, 30]] = 0.0
    s.q[3] = 2.0 ** -100
    _check(s, sm_scale=sm_scale, out_f32=True)


@pytest.mark.parametrize("D", [64, 40])
def test_a_plan_of_ones_own_past_the_planners_lengths(D):
    """psd_plan_multi_token takes up to 2^31 - 256 tokens a request, and so does the call."""
    s = Step([1], [3], D=D, seed=82)
    plan = psd.plan_multi_token(psd.HostTable(s.page_indptr, s.page_indices, s.last, s.page), s.q_indptr)
    args = psd.multi_token_args(s.q.cuda(), s.k.cuda(), s.v.cuda(), torch.from_numpy(s.page_indices).cuda(),
                                sm_scale=s.sm_scale)
    args.page_size, args.num_pages, args.num_page_indices, plan.c.page_size = 1 << 30, 1, 2, 1 << 30
    o, ws = torch.empty((s.T, s.Hq, D), device="cuda"), psd.multi_token_workspace(ctx(), plan, D, "cuda")
    for length in (2 ** 31 - 1, 2 ** 31 - 255):      # nothing is launched
        plan.requests_a[0].kv_len = length
        with pytest.raises(psd.PsdError) as e:
            psd.multi_token_decode(ctx(), args, plan, o, None, ws)
        assert e.value.status == 1


@pytest.mark.parametrize("kv,sm_scale,k_scale", [("bf16", 3e38, 1.0), ("fp8", 1e20, 1e20), ("fp8", -1e20, 1e20)])
def test_scales_whose_product_f32_does_not_hold(kv, sm_scale, k_scale):
    s = Step([2], [30], kv=kv, seed=83)
    s.scales, s.sm_scale = (k_scale, 1.0), sm_scale
    with pytest.raises(psd.PsdError) as e:
        _run(s)
    assert e.value.status == 1


@pytest.mark.parametrize("B,D,page,kv,out_f32", [(600, 40, 16, "bf16", False), (300, 64, 5, "fp8", True), (258, 256, 16, "bf16", True)])
def test_batches_of_several_launches_of_the_general_kernel(B, D, page, kv, out_f32):
    """More than 256 requests that have new tokens: the launches share the workspace."""
    rng = np.random.default_rng(B)
    new, before = rng.integers(0 if B == 600 else 1, 3, B), rng.integers(1, 40, B)
    before[[1, B - 1]], new[[1, B - 1]] = 700, 2            # keys split where a launch has few rows
    assert int((new > 0).sum()) > 256
    _check(Step(new, before, Hq=2, Hkv=1, D=D, page=page, kv=kv, seed=B), out_f32=out_f32)


@pytest.mark.parametrize("D,kv", [(64, "bf16"), (128, "fp8"), (40, "bf16")])
def test_calls_that_overlap_on_two_streams(D, kv):
    """Many calls a stream in flight at once, each stream with a workspace of its own."""
    steps = [Step([3, 60], [800 + 100 * i, 40], D=D, kv=kv, seed=90 + i) for i in range(2)]
    want, calls = [_run(s) for s in steps], []
    for s in steps:
        args = psd.multi_token_args(s.q.cuda(), s.k.cuda(), s.v.cuda(), torch.from_numpy(s.page_indices).cuda(),
                                    sm_scale=s.sm_scale, k_scale=s.scales[0], v_scale=s.scales[1])
        plan = psd.plan_multi_token(psd.HostTable(s.page_indptr, s.page_indices, s.last, s.page), s.q_indptr)
        outs = [(torch.full_like(want[0][0], 5.0), torch.full_like(want[0][1], 5.0)) for _ in range(20)]
        calls.append((args, plan, psd.multi_token_workspace(ctx(), plan, D, "cuda"), outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    torch.cuda._sleep(2_000_000)
    for *_, stream in calls:
        stream.wait_stream(torch.cuda.current_stream())     # both begin together
    for i in range(20):
        for args, plan, ws, outs, stream in calls:
            psd.multi_token_decode(ctx(), args, plan, *outs[i], ws, stream=stream)
    torch.cuda.synchronize()
    for (args, plan, ws, outs, stream), w in zip(calls, want):
        assert psd.check_device_error(ctx(), ws) == 0
        assert all(torch.equal(o, w[0]) and torch.equal(lse, w[1]) for o, lse in outs)


def test_fewer_rows_than_the_plan_are_refused():
    s = Step([2, 70], [3, 4], seed=22, pad_rows=0)
    plan = psd.plan_multi_token(psd.HostTable(s.page_indptr, s.page_indices, s.last, s.page), s.q_indptr)
    args = psd.multi_token_args(s.q.cuda()[:71], s.k.cuda(), s.v.cuda(), torch.from_numpy(s.page_indices).cuda(), sm_scale=0.1)
    ws = psd.multi_token_workspace(ctx(), plan, s.D, "cuda")
    with pytest.raises(psd.PsdError) as e:
        psd.multi_token_decode(ctx(), args, plan, torch.empty((71, s.Hq, s.D), device="cuda"), None, ws)
    assert e.value.status == 1


@pytest.mark.parametrize("D", [64, 128])
def test_weights_over_fp8_pools_are_good_to_11_bits(D):
    """Two keys with values 1 and -1: the output is the difference of two nearly equal weights, where a
    weight's rounding shows beside the output's.  Weights of 8 bits would not pass, which is checked on
    the host."""
    s = Step([1] * 20, [1] * 20, Hq=64, Hkv=1, D=D, kv="fp8", spread=0.2, seed=91)
    for b in range(20):
        page = s.v[int(s.page_indices[s.page_indptr[b]])]
        page[0], page[1] = 0x38, 0xB8
    s.scales = (s.scales[0], 1.0)
    o, lse = _run(s)
    want = s.oracle()
    # `bounds` without a rounding of the weights, and 2^-11 of them (2^-32 of the largest where f16 ends)
    e_o, e_l = bounds(want, D, 2, False, 0)
    e_o = e_o + (2.0 ** -11 + 2 * 2.0 ** -32) * want[2] * (1 + 2.0 ** -8)
    n = int(s.q_indptr[-1])
    assert bool((np.abs(o[:n].double().cpu().numpy() - want[0]) <= e_o).all())
    assert bool((np.abs(lse[:n].double().cpu().numpy() - want[1]) <= e_l).all())
    ratio = (1 - np.abs(want[0])) / (1 + np.abs(want[0]))       # of the smaller weight to the larger
    coarse = torch.from_numpy(ratio).to(torch.bfloat16).double().numpy()
    assert bool((np.abs((1 - coarse) / (1 + ratio) - np.abs(want[0])) > e_o).any())
