"""fork_pages, free_pages, compact_pages and copy_pages on the GPU against their definitions in plain Python: every
table entry, count and byte; what is refused, and what a fault leaves as it was."""
import numpy as np
import pytest
import torch

import paged_split_kv_decode_gb300 as psd
from oracle import beams as BM
from _gpu_util import ctx

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int64).astype(np.int32)).cuda()


class Cache:
    """Requests over a pool: `shared` pages common to all, then pages of their own, in random order; a few pages more
    than they need, and pools of odd and even page sizes."""

    def __init__(self, lengths, page, *, shared=0, spare_pages=0, extra=8, widths=((4, 8), (3,), (16,)), seed=0, others=()):
        rng = np.random.default_rng(seed)
        held = [-(-n // page) + spare_pages for n in lengths]
        total = shared + sum(max(h - shared, 0) for h in held) + extra
        ids = list(rng.permutation(total))
        common = [ids.pop() for _ in range(shared)]
        rows = [common[:h] + [ids.pop() for _ in range(max(h - shared, 0))] for h in held]
        self.num_pages, self.page, self.kv_len = total, page, list(lengths)
        self.indptr = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(int)
        self.indices = np.array([g for r in rows for g in r], dtype=int)
        self.ref = np.bincount(self.indices, minlength=total)
        for g in others:                                 # references from outside the table
            self.ref[self.indices[g]] += 1
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.pools = [torch.randint(0, 256, (total, page) + w, generator=gen, device="cuda", dtype=torch.uint8) for w in widths]
        self.pages = psd.PagePools(self.pools)


def run_fork(c, parents, room, *, keep_old=False, capacity=None, in_place=False, call=None):
    N = len(parents)
    most = sum(-(-(c.kv_len[p] + room) // c.page) for p in parents if 0 <= p < len(c.kv_len)) if capacity is None else capacity
    out = dict(new_indptr=torch.full((N + 1,), -7, dtype=torch.int32, device="cuda"),
               new_indices=torch.full((most + 3,) if capacity is None else (capacity,), -7, dtype=torch.int32, device="cuda"),
               new_len=torch.full((N,), -7, dtype=torch.int32, device="cuda"))
    ref = i32(c.ref)
    new_ref = ref if in_place else torch.full_like(ref, -7)
    ws = psd.pages_workspace(c.pages, N, "cuda")
    ws.fill_(255)
    args = dict(page_indptr=i32(c.indptr), page_indices=i32(c.indices), kv_len=i32(c.kv_len), page_size=c.page, room=room,
                ref_count=ref, new_ref_count=None if in_place else new_ref, workspace=ws, keep_old=keep_old, **out)
    if call:
        args.update(call)
    fault = psd.fork_pages(ctx(), c.pages, i32(parents), **args)
    torch.cuda.synchronize()
    return int(fault), out, new_ref


def check_fork(c, parents, room, **kw):
    before = [p.clone() for p in c.pools]
    want = BM.fork(parents, c.indptr, c.indices, c.kv_len, c.page, room, c.ref, kw.get("keep_old", False))
    fault, out, ref = run_fork(c, parents, room, **kw)
    if want is None:                                                  # the pages run out: nothing is written
        assert fault == 8 and all(bool((t == -7).all()) for t in out.values()) and all(map(torch.equal, before, c.pools))
        return
    assert fault == 0
    rows, lengths, counts, copies = want
    flat = [g for r in rows for g in r]
    assert out["new_indptr"].tolist() == list(np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(int))
    assert out["new_indices"][: len(flat)].tolist() == flat
    assert bool((out["new_indices"][len(flat):] == -7).all())      # entries behind the table stay
    assert out["new_len"].tolist() == lengths and ref.tolist() == counts
    for old, pool in zip(before, c.pools):
        for a, b in copies:
            old[b] = old[a]
        assert torch.equal(old, pool)


BOTH = pytest.mark.parametrize("extra", [60, 50000])   # one CTA, or a cluster for many pages


@pytest.mark.parametrize("extra", [300, 50000])
@pytest.mark.parametrize("room", [0, 1, 5, 40])
@pytest.mark.parametrize("page", [1, 5, 16, 64])
def test_lengths_and_rooms(page, room, extra):
    lengths = [0, 1, page - 1, page, page + 1, 3 * page, 7 * page - 1]
    c = Cache(lengths, page, extra=extra, widths=((2,), (3,)), seed=page + room)
    check_fork(c, [0, 1, 1, 1, 2, 3, 3, 4, 4, 6, 6, -1, 5, 6], room)


@pytest.mark.parametrize("keep_old", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@BOTH
def test_shared_prompts_and_references_from_outside(keep_old, in_place, extra):
    c = Cache([50, 50, 50, 33, 48], 16, shared=3, extra=extra, seed=3, others=(3, 11))
    check_fork(c, [0, 0, 1, 2, 2, 2, 3, 4, 4], 1, keep_old=keep_old, in_place=in_place)
    c = Cache([40, 40], 16, shared=3, extra=extra, seed=4)                # both hold the same part-full page
    check_fork(c, [1, 0, 0], 1, keep_old=keep_old, in_place=in_place)


@BOTH
def test_pages_behind_the_tokens_are_let_go(extra):
    c = Cache([20, 33], 16, spare_pages=2, extra=extra, seed=5)
    check_fork(c, [1, 0], 3)


@pytest.mark.parametrize("parents", [[0, 1], [1, 0], [1], [1, 1], [1, 2, 0], [2, 1, 1, 0, 2]])
@pytest.mark.parametrize("room", [0, 1, 20])
@BOTH
def test_pages_full_for_one_and_part_full_for_another(room, parents, extra):
    """Requests that went back (their last tokens dropped) share a page that is full for another: its holder's tokens stay."""
    check_fork(Cache([32, 20, 25], 16, shared=2, extra=extra, seed=50), parents, room)
    c = Cache([32, 20, 25], 16, shared=2, extra=extra, seed=51)
    if 0 in parents and 1 in parents and room:                        # no page of one child is written to by another
        _, out, _ = run_fork(c, parents, room)
        table, indptr, lens = out["new_indices"].tolist(), out["new_indptr"].tolist(), out["new_len"].tolist()
        for i, p in enumerate(parents):
            write = {table[indptr[i] + t // 16] for t in range(lens[i] - room, lens[i])}
            for j in range(len(parents)):
                assert j == i or not write & set(table[indptr[j]: indptr[j + 1]])


@pytest.mark.parametrize("keep_old", [False, True])
@pytest.mark.parametrize("seed", range(4))
@BOTH
def test_requests_that_went_back(seed, keep_old, extra):
    rng = np.random.default_rng(seed)
    lengths = [int(n) for n in rng.integers(1, 120, 40)]
    c = Cache(lengths, 16, shared=5, spare_pages=int(rng.integers(2)), extra=extra + 300, seed=60 + seed)
    check_fork(c, [int(p) for p in rng.integers(-1, 40, 60)], int(rng.integers(0, 30)), keep_old=keep_old)


@pytest.mark.parametrize("parents", [[], [-1, -1], [0]])
@BOTH
def test_few_and_none(parents, extra):
    c = Cache([70, 20, 0], 16, extra=extra, seed=6)
    if parents:
        check_fork(c, parents, 1)
    else:
        ref = i32(c.ref)
        ws = psd.pages_workspace(c.pages, 0, "cuda")
        fault = psd.free_pages(ctx(), i32(c.indptr), i32(c.indices), ref, ws)
        assert int(fault) == 0 and not ref.any()


@BOTH
def test_no_old_requests(extra):
    c = Cache([20], 16, extra=extra, seed=7)
    c.kv_len, c.indptr, c.indices, c.ref = [], np.array([0]), np.zeros(0, int), np.zeros_like(c.ref)
    check_fork(c, [-1, -1], 4)


def test_many_requests_and_pages():
    """More children and pages than threads."""
    rng = np.random.default_rng(8)
    lengths = [int(x) for x in rng.integers(0, 40, 3000)]
    c = Cache(lengths, 4, extra=40000, widths=((2,),), seed=8)
    parents = [int(x) for x in rng.integers(-1, 3000, 9001)]
    check_fork(c, parents, 1)


def test_one_request_with_a_long_cache():
    c = Cache([100003], 16, extra=20000, widths=((1,),), seed=9)
    check_fork(c, [0, 0, 0], 1)


def test_a_large_pool_that_is_full():
    """The cluster runs out of pages as the one CTA does."""
    c = Cache([31, 31], 16, extra=50000, widths=((1,),), seed=10)
    c.ref[c.ref == 0] = 1                                           # all of them somebody's
    check_fork(c, [0, 0], 1)                                        # one copy, in a page that the other request left
    check_fork(c, [0, 0, 0, 0, 1], 2)


def test_every_free_page_is_used():
    c = Cache([31, 31], 16, extra=3, seed=10)
    check_fork(c, [0, 0, 0, 1], 2)                                  # four tails of which two stay, then fresh pages
    c = Cache([31, 31], 16, extra=1, seed=10)
    fault, out, ref = run_fork(c, [0, 0, 0, 0, 1], 2)               # 1 + 2 let go, more needed
    assert BM.fork([0, 0, 0, 0, 1], c.indptr, c.indices, c.kv_len, 16, 2, c.ref) is None
    assert fault == 8
    for t in list(out.values()) + [ref]:
        assert bool((t == -7).all())


def test_many_pools():
    """More pools than one launch carries, of pages down to one byte."""
    c = Cache([40, 17], 16, extra=10, widths=tuple((1 + i % 5,) for i in range(300)), seed=11)
    check_fork(c, [0, 0, 1, 1, 1], 1)


@pytest.mark.parametrize("what,bits", [
    (dict(parents=[0, 2]), 4), (dict(parents=[0, -2]), 4), (dict(kv_len=[-1, 20]), 4), (dict(kv_len=[81, 20]), 4),
    (dict(kv_len=[2 ** 31 - 1, 20]), 4), (dict(indptr=[0, 5, 9]), 4), (dict(indptr=[-1, 5, 7]), 4), (dict(indptr=[0, 5, 4]), 4),
    (dict(indices={2: -1}), 1), (dict(indices={6: 10 ** 9}), 1), (dict(ref={3: -1}), 4), (dict(ref="less"), 4),
    (dict(capacity=2), 4)])
@BOTH
def test_faults_write_nothing(what, bits, extra):
    c = Cache([70, 20], 16, extra=extra, seed=12)
    before = [p.clone() for p in c.pools]
    parents, capacity = what.get("parents", [0, 0, 1]), what.get("capacity")
    c.kv_len = what.get("kv_len", c.kv_len)
    capacity = 32 if capacity is None else capacity
    c.indptr = np.array(what.get("indptr", c.indptr))
    for i, g in what.get("indices", {}).items():
        c.indices[i] = g
    if what.get("ref") == "less":
        c.ref[c.indices[0]] = 0
    elif "ref" in what:
        for g, r in what["ref"].items():
            c.ref[g] = r
    fault, out, ref = run_fork(c, parents, 1, capacity=capacity)
    assert fault & bits and not fault & ~(bits | 4)
    for t in list(out.values()) + [ref]:
        assert bool((t == -7).all())
    assert all(torch.equal(a, b) for a, b in zip(before, c.pools))


# ------------------------------------------------------------------------------------------- compact
@pytest.mark.parametrize("n,live", [(1, 0.0), (1, 1.0), (2, 0.5), (40, 0.3), (1000, 0.66), (1000, 0.0), (1000, 1.0), (20011, 0.4)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(n, live, in_place):
    rng = np.random.default_rng(n)
    ref = np.where(rng.random(n) < live, rng.integers(1, 5, n), 0)
    alive = np.flatnonzero(ref)
    table = rng.choice(alive, 3 * n) if len(alive) else np.zeros(0, int)
    pools = [torch.randint(0, 256, (n,) + w, device="cuda", dtype=torch.uint8) for w in ((32,), (7,))]
    pages, before = psd.PagePools(pools), [p.clone() for p in pools]
    count, to, counts, moves = BM.compact(ref)
    a, r = i32(table), i32(ref)
    out = {} if in_place else dict(new_indices=torch.full_like(a, -7), new_ref_count=torch.full_like(r, -7))
    num_live, page_map = torch.full((1,), -7, dtype=torch.int32, device="cuda"), torch.full_like(r, -7)
    ws = psd.pages_workspace(pages, 0, "cuda")
    ws.fill_(255)
    fault = psd.compact_pages(ctx(), pages, a, r, num_live=num_live, workspace=ws, page_map=page_map, **out)
    assert int(fault) == 0 and int(num_live) == count and page_map.tolist() == to
    assert out.get("new_indices", a).tolist() == [to[g] for g in table]
    assert out.get("new_ref_count", r).tolist() == counts
    for old, pool in zip(before, pools):
        for x, y in moves:
            old[y] = old[x]
        assert torch.equal(old, pool)


@pytest.mark.parametrize("table,ref,bits", [([0, 5], [1, 0, 1, 1], 1), ([-1], [1, 0, 1, 1], 1), ([1], [1, 0, 1, 1], 1),
                                            ([0], [1, -1, 1, 1], 4)])
def test_compact_faults_write_nothing(table, ref, bits):
    pools = [torch.arange(4, device="cuda", dtype=torch.uint8).repeat_interleave(8).view(4, 8)]
    pages, before = psd.PagePools(pools), pools[0].clone()
    a, r = i32(table), i32(ref)
    num_live, page_map = torch.full((1,), -7, dtype=torch.int32, device="cuda"), torch.full_like(r, -7)
    fault = psd.compact_pages(ctx(), pages, a, r, num_live=num_live, page_map=page_map,
                              workspace=psd.pages_workspace(pages, 0, "cuda"))
    assert int(fault) == bits and int(num_live) == -7 and bool((page_map == -7).all())
    assert a.tolist() == table and r.tolist() == ref and torch.equal(before, pools[0])


# --------------------------------------------------------------------------------------------- copies
@pytest.mark.parametrize("width", [1, 16, 48, 1000, 4096, 16400])
def test_copies(width):
    pools = [torch.randint(0, 256, (12, width), device="cuda", dtype=torch.uint8), torch.randn(12, 3, 2, device="cuda")]
    # a pool that starts off a 16-byte boundary
    flat = torch.randint(0, 256, (12 * width + 1,), device="cuda", dtype=torch.uint8)
    pools.append(flat[1:].view(12, width))
    before = [p.clone() for p in pools]
    fault = psd.copy_pages(ctx(), psd.PagePools(pools), i32([3, 3, 7, 5, -1, 2, 12]), i32([0, 11, 1, 5, 4, -1, 6]))
    assert int(fault) == 1                                            # the pairs that name no page are left out
    for old, pool in zip(before, pools):
        old[[0, 11, 1]] = old[[3, 3, 7]]
        assert torch.equal(old, pool)


@pytest.mark.parametrize("widths", [(40001, 16, 131072), (16384, 16383, 16400), (2 ** 25 + 16, 7, 2 ** 25 + 1)])
def test_copies_of_large_pages(widths):
    """Pages of several parts beside small ones, on and off their alignment."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    pools = [torch.randint(0, 256, (6, w), dtype=torch.uint8, device="cuda", generator=gen) for w in widths]
    before = [p.clone() for p in pools]
    fault = psd.copy_pages(ctx(), psd.PagePools(pools), i32([5, 1, 3]), i32([0, 2, 3]))
    assert int(fault) == 0
    for old, pool in zip(before, pools):
        old[[0, 2]] = old[[5, 1]]
        assert torch.equal(old, pool)


@pytest.mark.parametrize("off", [0, 1, 2, 3])
def test_tables_off_their_alignment(off):
    """Tables and counts that begin anywhere in a larger tensor, and an old table that begins behind other entries."""
    c = Cache([40, 70, 20, 33], 16, shared=1, extra=30, seed=40)
    parents, N = [0, 2, 2, 1], 4
    wide = lambda a: torch.cat([i32([7] * off), i32(a)])[off:]  # noqa: E731
    lead = 3
    indptr, indices = [x + lead for x in c.indptr], [0] * lead + list(c.indices)
    out = dict(new_indptr=wide([0] * (N + 1)), new_indices=wide([0] * 40), new_len=wide([0] * N))
    new_ref, ws = wide(c.ref), psd.pages_workspace(c.pages, N, "cuda")
    before = [p.clone() for p in c.pools]
    fault = psd.fork_pages(ctx(), c.pages, i32(parents), page_indptr=wide(indptr), page_indices=wide(indices),
                           kv_len=wide(c.kv_len), page_size=16, room=1, ref_count=wide(c.ref), new_ref_count=new_ref,
                           workspace=ws, **out)
    rows, lengths, counts, copies = BM.fork(parents, c.indptr, c.indices, c.kv_len, 16, 1, c.ref)
    flat = [x for r in rows for x in r]
    assert int(fault) == 0 and out["new_indices"][: len(flat)].tolist() == flat
    assert new_ref.tolist() == counts and out["new_len"].tolist() == lengths
    for old, pool in zip(before, c.pools):
        for a, b in copies:
            old[b] = old[a]
        assert torch.equal(old, pool)


def test_pools_past_32_bits():
    """5 GB of pages: offsets beyond 2^32 bytes."""
    pool = torch.zeros((40000, 131072), dtype=torch.uint8, device="cuda")
    pool[39990], pool[20000] = 7, 9
    fault = psd.copy_pages(ctx(), psd.PagePools([pool]), i32([39990, 20000]), i32([5, 39999]))
    assert int(fault) == 0 and bool((pool[5] == 7).all()) and bool((pool[39999] == 9).all()) and not pool[39998].any()


# ---------------------------------------------------------------------------------- use and refusals
def test_captured_and_replayed():
    """A graph reads its tables, counts and parents anew at each replay."""
    c = Cache([40, 50, 20], 16, shared=1, extra=30, seed=20)
    parents = i32([0, 1, 2])
    N = 3
    out = dict(new_indptr=i32([0] * 4), new_indices=i32([0] * 16), new_len=i32([0] * N))
    ref, new_ref, ws = i32(c.ref), i32(c.ref), psd.pages_workspace(c.pages, N, "cuda")
    kv_len, fault = i32(c.kv_len), i32([0])
    args = dict(page_indptr=i32(c.indptr), page_indices=i32(c.indices), kv_len=kv_len, page_size=16, room=1, ref_count=ref,
                new_ref_count=new_ref, workspace=ws, fault=fault, **out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        psd.fork_pages(ctx(), c.pages, parents, **args)
    for now, lens in (([2, 2, 0], [33, 50, 19]), ([1, -1, 1], [40, 47, 20])):
        parents.copy_(i32(now))
        kv_len.copy_(i32(lens))
        before = [p.clone() for p in c.pools]
        g.replay()
        torch.cuda.synchronize()
        rows, lengths, counts, copies = BM.fork(now, c.indptr, c.indices, lens, 16, 1, c.ref)
        flat = [x for r in rows for x in r]
        assert out["new_indices"][: len(flat)].tolist() == flat and new_ref.tolist() == counts and int(fault) == 0
        assert out["new_len"].tolist() == lengths
        for old, pool in zip(before, c.pools):
            for a, b in copies:
                old[b] = old[a]
            assert torch.equal(old, pool)


def test_argument_errors():
    c = Cache([40, 50], 16, extra=9, seed=21)
    fork = lambda **kw: run_fork(c, [0, 1], 1, call=kw)  # noqa: E731
    for kw in (dict(page_indptr=i32([0, 3])), dict(new_len=i32([0])), dict(ref_count=i32([1])), dict(new_ref_count=i32([1])),
               dict(kv_len=torch.zeros(2, dtype=torch.int32)), dict(new_indices=i32([0] * 40)[::2])):
        with pytest.raises(ValueError):
            fork(**kw)
    for kw in (dict(kv_len=i32([1, 1]).long()), dict(workspace=i32([0]))):
        with pytest.raises(TypeError):
            fork(**kw)
    table = i32(c.indices)
    for kw, status in ((dict(page_size=0), 1), (dict(room=-1), 1), (dict(page_indices=table, new_indices=table), 1),
                       (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), 5)):
        with pytest.raises(psd.PsdError) as e:
            fork(**kw)
        assert e.value.status == status
    with pytest.raises(ValueError):
        psd.PagePools([])
    with pytest.raises(ValueError):
        psd.PagePools([torch.zeros(3, 4, device="cuda"), torch.zeros(4, 4, device="cuda")])
    with pytest.raises(ValueError):
        psd.PagePools([torch.zeros(3, 4, device="cuda").t()])
