"""append_tokens into a cache of 8-bit blocks with a scale each, on the GPU against the float64 rotation, the least powers of
two that hold each block, and the nearest codes; what is refused, and what faults leave as it was."""
import numpy as np
import pytest
import torch

import paged_split_kv_decode_gb300 as psd
from oracle import attention as A
from oracle import beams as BM
from oracle import tokens as TK
from _gpu_util import ctx

pytestmark = pytest.mark.gpu


def _make(new, before, *, Hq=8, Hkv=2, D=64, Dv=None, page=16, block=16, seed=0, pad_rows=2, fused=True, swing=4, spread=None):
    rng = np.random.default_rng(seed)
    Dv = D if Dv is None else Dv
    new, total = np.array(new), np.array(new) + np.array(before)
    q_indptr = np.concatenate([[0], np.cumsum(new)])
    pages = -(-total // page)
    page_indptr = np.concatenate([[0], np.cumsum(pages)])
    num_pages = int(page_indptr[-1]) + 2
    page_indices = rng.permutation(num_pages)[: page_indptr[-1]]
    T = int(q_indptr[-1]) + pad_rows
    width = Hq * D + Hkv * (D + Dv) + (8 if fused else 0)
    x = rng.standard_normal((T, width)) * (np.exp(1.5 * rng.standard_normal((T, 1))) if spread is None else spread)
    x = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()
    cut = [Hq * D, Hq * D + Hkv * D, Hq * D + Hkv * (D + Dv)]
    views = [x[:, : cut[0]].view(T, Hq, D), x[:, cut[0]: cut[1]].view(T, Hkv, D), x[:, cut[1]: cut[2]].view(T, Hkv, Dv)]
    if not fused:
        views = [v.contiguous() for v in views]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()  # noqa: E731
    pool = lambda w: torch.from_numpy(rng.integers(0, 126, (num_pages, page, Hkv, w)).astype(np.uint8)).cuda()  # noqa: E731
    scale = lambda: torch.from_numpy((117 + rng.integers(-swing, swing + 1, (num_pages, page // block, Hkv))).astype(np.uint8)).cuda()  # noqa: E731
    return dict(q=views[0], k=views[1], v=views[2], q_indptr=dev(q_indptr), kv_len=dev(total), page_indptr=dev(page_indptr),
                page_indices=dev(page_indices), k_pool=pool(D), v_pool=pool(Dv), ke=scale(), ve=scale(),
                host=dict(q_indptr=q_indptr, total=total, page_indptr=page_indptr, page_indices=page_indices, page=page,
                          block=block))


def _call(s, rope, *, neox=True, **kw):
    q_out = torch.full(s["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda") if s["q"] is not None else None
    kw = {**dict(scales=psd.BlockScales(s["ke"], s["ve"], s["host"]["block"])), **kw}
    f = psd.append_tokens(ctx(), s["q"], s["k"], s["v"], q_out, q_indptr=s["q_indptr"], kv_len=s["kv_len"],
                          page_indptr=s["page_indptr"], page_indices=s["page_indices"], k_pool=s["k_pool"],
                          v_pool=s["v_pool"], rope=rope, neox=neox, **kw)
    torch.cuda.synchronize()
    return q_out, int(f.item())


def _values(codes):
    return A.e4m3_to_f64(codes).reshape(codes.shape)


def _check(s, rope, *, neox=True, rope_col=0, positions=None, left_out=(), faults=0, **kw):
    """left_out: token rows that are not appended."""
    h, N = s["host"], s["host"]["block"]
    before = [t.cpu().numpy().copy() for t in (s["k_pool"], s["v_pool"], s["ke"], s["ve"])]
    pos = None if positions is None else torch.tensor(positions, dtype=torch.int32, device="cuda")
    q_out, fault = _call(s, rope, neox=neox, rope_col=rope_col, positions=pos, **kw)
    assert fault == faults
    after = [t.cpu().numpy() for t in (s["k_pool"], s["v_pool"], s["ke"], s["ve"])]
    where = TK.positions_of(h["q_indptr"], h["total"])
    n = len(where)
    at = np.array([p for _, p in where]) if positions is None else np.array(positions[:n])
    rot = lambda x: TK.rotate(x[:n].double().cpu().numpy(), at[:, None], rope.inv_freq, rope.magnitude, rope_col, neox)  # noqa: E731
    # an f32 rotation: sincospi good to 2 ulp of 1, its argument to 2^-24 of a half turn, two products and a sum:
    # under 2^-20 of |x| + |y|, and a rounding of the result
    slack = lambda turned: 2.0 ** -20 * turned[1] + 2.0 ** -23 * np.abs(turned[0])  # noqa: E731
    if q_out is not None:
        turned = rot(s["q"])
        want, near = turned[0], slack(turned)
        keep = [t for t in range(n) if t not in left_out or faults == 1]
        d = np.abs(q_out[:n].double().cpu().numpy() - want)[keep]
        assert np.all(d <= 2.0 ** -8 * np.abs(want[keep]) + near[keep] * 1.01 + 1e-38)
        assert bool((q_out[n:] == 7.0).all())
    new_v = s["v"][:n].double().cpu().numpy()
    groups = {}                                                        # (page, block) -> [(slot, token)], older tokens
    for t, (b, p) in enumerate(where):
        page = int(h["page_indices"][h["page_indptr"][b] + p // h["page"]])
        start = int(h["total"][b] - (h["q_indptr"][b + 1] - h["q_indptr"][b]))
        key = (page, p % h["page"] // N)
        groups.setdefault(key, ([], max(0, start - p // N * N)))[0].append((p % N, t))
    turned = rot(s["k"])
    for x, near, i in ((turned[0], slack(turned), 0), (new_v, np.zeros_like(new_v), 1)):
        codes, scale, was, had = after[i], after[i + 2], before[i], before[i + 2]
        untouched = np.ones(scale.shape[:2], dtype=bool)
        for (page, j), (tokens, older) in groups.items():
            tokens = [(slot, t) for slot, t in tokens if t not in left_out]
            if not tokens:
                continue
            untouched[page, j] = False
            rows = np.stack([x[t] for _, t in tokens])                 # [m, Hkv, W]
            off = np.stack([near[t] for _, t in tokens])
            tops = np.where(np.isfinite(rows), np.abs(rows), 0.0)
            for head in range(x.shape[1]):
                top, e = tops[:, head].max(), int(scale[page, j, head])
                low = BM.scale_exponent(max(top - off[:, head].max(), 0.0))
                high = BM.scale_exponent(top + off[:, head].max())
                if older:
                    low, high = max(low, int(had[page, j, head])), max(high, int(had[page, j, head]))
                assert low <= e <= high, (page, j, head, low, e, high)
                old = _values(was[page, j * N: (j + 1) * N, head])
                got = _values(codes[page, j * N: (j + 1) * N, head])
                taken = [slot for slot, _ in tokens]
                for slot in range(N):
                    if slot in taken:
                        y = rows[taken.index(slot), head] * 2.0 ** (127 - e)
                        o = off[taken.index(slot), head] * 2.0 ** (127 - e)
                        fine = np.isfinite(y)
                        d = np.abs(got[slot] - np.clip(y, -448, 448))[fine]
                        assert np.all(d <= np.maximum(2.0 ** -4 * np.abs(y[fine]), 2.0 ** -10) + 1.0625 * o[fine])
                        assert np.array_equal(np.isnan(got[slot]), np.isnan(y))
                        assert np.array_equal(got[slot][np.isinf(y)], np.sign(y[np.isinf(y)]) * 448)
                    elif slot < older and older:
                        want = old[slot] if e == had[page, j, head] else BM.e4m3_nearest(old[slot] * 2.0 ** (int(had[page, j, head]) - e))
                        assert np.array_equal(got[slot], want, equal_nan=True)
                    else:
                        assert np.array_equal(codes[page, j * N + slot, head], was[page, j * N + slot, head])
        page_codes = codes.reshape(codes.shape[0], -1, N, *codes.shape[2:])
        assert np.array_equal(scale[untouched], had[untouched])
        assert np.array_equal(page_codes[untouched], was.reshape(page_codes.shape)[untouched])


RAGGED = dict(new=[1, 5, 0, 3, 40, 2, 1], before=[0, 200, 33, 127, 90, 15, 16])
MANY = dict(new=[300, 1, 0, 450, 76, 2, 113], before=[3, 500, 20, 0, 61, 16, 15])   # 16 tokens a CTA


@pytest.mark.parametrize("shape", [RAGGED, MANY])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 16), (32, 32), (64, 64), (96, 32)])
def test_ragged(page, block, D, shape):
    _check(_make(**shape, D=D, page=page, block=block, seed=page + D), psd.rope_frequencies(D))


@pytest.mark.parametrize("shape", [RAGGED, MANY])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("D,rot,col", [(64, 64, 0), (128, 64, 64), (128, 32, 16), (256, 128, 0), (96, 48, 8), (16, 16, 0), (128, 16, 40), (256, 256, 0)])
def test_layouts(D, rot, col, neox, shape):
    s = _make(**shape, Hq=4, Hkv=2, D=D, seed=D + rot)
    _check(s, psd.rope_frequencies(rot), neox=neox, rope_col=col)
    far = [int(x) for x in np.random.default_rng(D).integers(0, 2 ** 31, s["q"].shape[0])]
    _check(s, psd.rope_frequencies(rot, scaling="yarn", factor=8.0, original_max_position=4096), neox=neox, rope_col=col,
           positions=far)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (40, 8), (5, 5)])
@pytest.mark.parametrize("Dv", [8, 40, 64, 200])
def test_heads_and_widths(Dv, Hq, Hkv):
    _check(_make(**RAGGED, Hq=Hq, Hkv=Hkv, Dv=Dv, seed=Dv + Hq), psd.rope_frequencies(64))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 64, 65])
@pytest.mark.parametrize("before", [0, 1, 15, 16, 17, 63])
def test_lengths_around_the_blocks(n, before):
    _check(_make([n], [before], seed=n + before, fused=False), psd.rope_frequencies(32))
    _check(_make([n], [before], page=64, block=64, seed=n + before, pad_rows=0), psd.rope_frequencies(32))


def test_many_single_tokens():
    rng = np.random.default_rng(1)
    before = [int(x) for x in rng.integers(0, 60, 900)]
    _check(_make([1] * 900, before, Hq=2, Hkv=1, seed=1), psd.rope_frequencies(64))


def test_many_requests_without_tokens():
    """Runs of requests without new tokens, longer than what a warp looks at at once."""
    new, before = [], []
    for n, gap in ((130, 40), (1, 33), (2, 70), (90, 31), (1, 32), (1, 0), (1, 100), (120, 64)):
        new += [n] + [0] * gap
        before += [7 * n % 50] + [5] * gap
    _check(_make(new, before, Hq=2, Hkv=1, D=64, seed=61), psd.rope_frequencies(64))


def test_keys_and_values_alone():
    s = _make(**RAGGED, seed=2)
    s["q"] = None
    _check(s, psd.rope_frequencies(64))


@pytest.mark.parametrize("grow", [-6, 0, 1, 3, 9, 40])
def test_blocks_that_are_scaled_anew(grow):
    """A token 2^grow times the largest that its block holds."""
    s = _make([1, 3, 2], [5, 22, 15], seed=3, spread=2.0 ** (grow - 2))
    _check(s, psd.rope_frequencies(64))


def test_token_by_token_is_one_call_per_token():
    """Blocks filled one token at a time: each step against its definition; scales never fall while a block fills."""
    rope = psd.rope_frequencies(64)
    s = _make([1, 1], [0, 7], Hq=2, Hkv=2, page=16, seed=4, pad_rows=0)
    pages = 3
    s["page_indptr"] = torch.tensor([0, pages, 2 * pages], dtype=torch.int32, device="cuda")
    s["page_indices"] = torch.tensor([5, 0, 3, 1, 4, 2], dtype=torch.int32, device="cuda")
    for name, fill in (("k_pool", 0x30), ("v_pool", 0x30), ("ke", 117), ("ve", 117)):
        s[name] = torch.full((6,) + s[name].shape[1:], fill, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(4)
    for step in range(24):
        x = torch.from_numpy((rng.standard_normal((2, 6, 64)) * np.exp(2 * rng.standard_normal())).astype(np.float32)).to(torch.bfloat16).cuda()
        s["q"], s["k"], s["v"] = x[:, :2], x[:, 2:4], x[:, 4:]
        total = np.array([1 + step, 8 + step])
        s["kv_len"] = torch.tensor(total, dtype=torch.int32, device="cuda")
        s["host"].update(q_indptr=np.array([0, 1, 2]), total=total, page_indptr=np.array([0, 3, 6]),
                         page_indices=np.array([5, 0, 3, 1, 4, 2]))
        _check(s, rope)


def test_zeros_and_values_that_are_not_finite():
    s = _make([20, 3], [4, 0], Hq=2, seed=5, fused=False, pad_rows=0)
    s["v"][0], s["v"][3] = 0.0, 0.0
    s["k"][20:], s["v"][20:] = 0.0, 0.0                                 # a request of zeros
    s["v"][5, 0, 3], s["v"][6, 1, 0], s["v"][7, 0, 1] = float("nan"), float("inf"), -float("inf")
    _check(s, psd.rope_frequencies(64))
    s = _make([4], [0], Hq=2, seed=6, fused=False, pad_rows=0)
    s["v"][:] = float("inf")                                           # no finite value: the least scale
    _check(s, psd.rope_frequencies(64))
    assert bool((s["ve"][int(s["page_indices"][0]), 0] == 95).all())


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -34, 2.0 ** 20, 2.0 ** 120])
def test_small_and_large_values(size):
    _check(_make([18, 1], [3, 20], seed=7, spread=size), psd.rope_frequencies(64))


def test_borders_of_the_scales():
    """Largest values at 448 times a power of two and one step above."""
    s = _make([1] * 6, [0, 0, 0, 3, 3, 3], Hq=2, Hkv=1, seed=8, fused=False, pad_rows=0)
    for i, x in enumerate((448.0, 450.0, 1.75, 224.0, 226.0, 0.21875)):
        s["v"][i] = torch.where(s["v"][i] > 0, x, -0.5 * x).to(torch.bfloat16)
    _check(s, psd.rope_frequencies(64))


@pytest.mark.parametrize("shape", [RAGGED, MANY])
@pytest.mark.parametrize("had", [252, 253, 254])
def test_the_largest_scales(had, shape):
    """Blocks that a caller gave scales of 2^125 to 2^127: new codes are in units of these where older tokens are there."""
    s = _make(**shape, seed=14, spread=2.0 ** 123)
    s["ke"][:], s["ve"][:] = had, had
    _check(s, psd.rope_frequencies(64))


def test_older_codes_at_any_new_scale():
    """All 256 codes in a block that a new token scales anew by 2^1 to 2^40: each goes to the nearest code, ties to even."""
    n = 40
    s = _make([1] * n, [15] * n, Hq=1, Hkv=1, D=64, seed=15, fused=False, pad_rows=0)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(4)
    for b in range(n):
        page = int(s["host"]["page_indices"][b])
        s["v_pool"][page].view(-1)[:960], s["ve"][page] = codes[:960], 110
        s["v"][b] = 448.0 * 2.0 ** (110 - 127 + b + 1)
    was = s["v_pool"].clone()
    _, fault = _call(s, psd.rope_frequencies(32))
    assert fault == 0
    for b in range(n):
        page = int(s["host"]["page_indices"][b])
        assert int(s["ve"][page, 0, 0]) == 110 + b + 1
        want = BM.e4m3_nearest(_values(was[page, :15].cpu().numpy()) * 2.0 ** -(b + 1))
        assert np.array_equal(_values(s["v_pool"][page, :15].cpu().numpy()), want, equal_nan=True), b
        assert bool((s["v_pool"][page, 15] == 0x7E).all())


def test_in_place_queries():
    a = _make(**RAGGED, seed=9, fused=False, pad_rows=0)
    want, _ = _call(a, psd.rope_frequencies(64))
    b = _make(**RAGGED, seed=9, fused=False, pad_rows=0)
    psd.append_tokens(ctx(), b["q"], b["k"], b["v"], b["q"], q_indptr=b["q_indptr"], kv_len=b["kv_len"],
                      page_indptr=b["page_indptr"], page_indices=b["page_indices"], k_pool=b["k_pool"], v_pool=b["v_pool"],
                      rope=psd.rope_frequencies(64), neox=True, scales=psd.BlockScales(b["ke"], b["ve"], 16))
    assert torch.equal(want, b["q"]) and torch.equal(a["k_pool"], b["k_pool"]) and torch.equal(a["ke"], b["ke"])


@pytest.mark.parametrize("shape", [RAGGED, MANY])
def test_a_second_call_changes_nothing(shape):
    s = _make(**shape, seed=10)
    _call(s, psd.rope_frequencies(64))
    first = [s[n].clone() for n in ("k_pool", "v_pool", "ke", "ve")]
    _call(s, psd.rope_frequencies(64))
    assert all(torch.equal(a, s[n]) for a, n in zip(first, ("k_pool", "v_pool", "ke", "ve")))


@pytest.mark.parametrize("shape", [RAGGED, MANY])
def test_faults_leave_their_tokens_out(shape):
    s = _make(**shape, seed=11, pad_rows=0)
    h = s["host"]
    where = TK.positions_of(h["q_indptr"], h["total"])
    gone = [t for t, (b, p) in enumerate(where) if b == 3 and 128 <= p < 144] if shape is RAGGED else \
        [t for t, (b, p) in enumerate(where) if b == 3 and 16 <= p < 32]
    at = int(h["page_indptr"][3]) + (8 if shape is RAGGED else 1)
    s["page_indices"][at] = 2 ** 31 - 1
    _check(s, psd.rope_frequencies(64), left_out=gone, faults=1)
    s = _make(**shape, seed=12, pad_rows=0)
    pos = [p for _, p in where]
    gone = [0, 3, len(pos) - 1]                                        # a block's first, one inside, the last
    for t in gone:
        pos[t] = -1
    _check(s, psd.rope_frequencies(64), positions=pos, left_out=gone, faults=4)


@pytest.mark.parametrize("T", [3, 40])
def test_offsets_that_go_past_the_rows_there_are(T):
    """q_indptr counts more tokens than the call has rows: those that are there are appended, and nothing else moves the scale."""
    s = _make([T + 9], [5], Hq=1, Hkv=2, D=64, seed=60, pad_rows=0, spread=1.0, fused=False)
    s["v"][T:] = 1000.0
    h, was, had = s["host"], s["v_pool"].cpu().clone(), s["ve"].cpu().clone()
    cut = {**s, "q": None, "k": s["k"][:T], "v": s["v"][:T]}
    _, fault = _call(cut, psd.rope_frequencies(32))
    assert fault == 0
    for j in range((5 + T + 9 + 15) // 16):                          # blocks of a page each
        page, first = int(h["page_indices"][j]), 16 * j - 5           # the token of the block's first slot
        rows = [t for t in range(max(first, 0), min(first + 16, T))]
        got, e = _values(s["v_pool"][page].cpu().numpy()), s["ve"][page, 0].cpu().numpy()
        if not rows:
            assert torch.equal(s["v_pool"][page].cpu(), was[page]) and torch.equal(s["ve"][page].cpu(), had[page])
            continue
        x = s["v"][rows].double().cpu().numpy()
        for head in range(2):
            least = BM.scale_exponent(np.abs(x[:, head]).max())
            assert e[head] == (max(least, int(had[page, 0, head])) if first < 0 else least)
            slots = [t - first for t in rows]
            y = x[:, head] * 2.0 ** (127 - int(e[head]))
            assert np.all(np.abs(got[slots, head] - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10))
        behind = [i for i in range(16) if first + i >= T]
        assert torch.equal(s["v_pool"][page].cpu()[behind], was[page][behind])


def test_pools_past_32_bits():
    """Pools of over 2^32 bytes: tokens at both ends."""
    page, Hkv, D = 64, 16, 128
    pages = 2 ** 32 // (page * Hkv * D) + 40
    k = torch.zeros((pages, page, Hkv, D), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    ke = torch.full((pages, page // 16, Hkv), 130, dtype=torch.uint8, device="cuda")
    ve = ke.clone()
    x = torch.full((2, Hkv, D), 3.5, dtype=torch.bfloat16, device="cuda")          # 448 * 2^-7: the scale's byte is 120
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    f = psd.append_tokens(ctx(), None, x, x, None, q_indptr=i32([0, 1, 2]), kv_len=i32([17, 64]), page_indptr=i32([0, 1, 2]),
                          page_indices=i32([0, pages - 1]), k_pool=k, v_pool=v, rope=psd.rope_frequencies(32), neox=True,
                          positions=i32([0, 0]), scales=psd.BlockScales(ke, ve, 16))
    assert int(f) == 0
    for pool, e in ((k, ke), (v, ve)):
        for g, slot, block, scale in ((0, 16, 1, 120), (pages - 1, 63, 3, 130)):   # the second's block has older tokens
            code = 0x7E if scale == 120 else 5 << 3 | 6                              # 3.5 * 2^-3 = 1.75 * 2^-2
            assert bool((pool[g, slot] == code).all()) and bool((e[g, block] == scale).all())
            pool[g, slot], e[g, block] = 0, 130
        assert not pool[0].any() and not pool[-1].any() and not pool[pages // 2:].any() and bool((e == 130).all())


def test_captured_and_replayed():
    s = _make(**RAGGED, seed=13)
    rope, sc = psd.rope_frequencies(64), psd.BlockScales(s["ke"], s["ve"], 16)
    q_out, fault = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda out: psd.append_tokens(  # noqa: E731
        ctx(), s["q"], s["k"], s["v"], out, q_indptr=s["q_indptr"], kv_len=s["kv_len"], page_indptr=s["page_indptr"],
        page_indices=s["page_indices"], k_pool=s["k_pool"], v_pool=s["v_pool"], rope=rope, neox=True, scales=sc, fault=fault)
    start = [s[n].clone() for n in ("k_pool", "v_pool", "ke", "ve")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(q_out)
    g.replay()
    torch.cuda.synchronize()
    got = [s[n].clone() for n in ("k_pool", "v_pool", "ke", "ve")]
    for n, t in zip(("k_pool", "v_pool", "ke", "ve"), start):
        s[n].copy_(t)
    want = torch.zeros_like(q_out)
    call(want)
    n = int(s["host"]["q_indptr"][-1])
    assert torch.equal(q_out[:n], want[:n]) and int(fault) == 0
    assert all(torch.equal(a, s[n]) for a, n in zip(got, ("k_pool", "v_pool", "ke", "ve")))


def test_refusals():
    s = _make([2], [3], pad_rows=0, fused=False)
    rope = psd.rope_frequencies(64)

    def refused(what, status=None, rope=rope, **kw):
        t = {**s, **{k: v for k, v in kw.items() if k in s}}
        with pytest.raises(what) as e:
            _call(t, rope, **{k: v for k, v in kw.items() if k not in s})
        if status:
            assert e.value.status == status

    refused(psd.PsdError, 1, k_scale=0.5)
    refused(psd.PsdError, 1, k_pool=s["k_pool"].to(torch.bfloat16), v_pool=s["v_pool"].to(torch.bfloat16))
    refused(psd.PsdError, 2, rope=psd.rope_frequencies(8))
    refused(psd.PsdError, 2, rope=psd.rope_frequencies(16), rope_col=4)
    refused(ValueError, scales=psd.BlockScales(s["ke"], s["ve"], 32))
    refused(ValueError, scales=psd.BlockScales(s["ke"][:1], s["ve"][:1], 16))
    refused(psd.PsdError, 1, scales=psd.BlockScales(s["ke"].repeat(1, 2, 1), s["ve"].repeat(1, 2, 1), 8))
    refused(ValueError, v=None)
    wide = torch.zeros((2, 2, 65), dtype=torch.bfloat16, device="cuda")
    refused(ValueError, k=wide[..., 1:])
    off = torch.zeros(2 * 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(2, 2, 64)
    refused(psd.PsdError, 2, k=off)
    before = s["k_pool"].clone()
    _check(s, rope)
    assert not torch.equal(before, s["k_pool"])
