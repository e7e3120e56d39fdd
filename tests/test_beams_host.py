"""CPU tests of beam search over a cache of 8-bit blocks: what the library refuses before it launches anything, what the
binding passes on, and pins of the oracle's definitions."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import beams as BM


@pytest.fixture(scope="module")
def lib():
    from paged_split_kv_decode_gb300 import _lib
    return _lib.load()


@pytest.fixture(scope="module")
def blank():
    """Zeroes in a context's place: calls that are refused read no more of it."""
    return C.create_string_buffer(65536)


def _ptr(n=16):
    """An address that is aligned and never read."""
    return 1 << 20 | n * 4096


def _message(lib):
    return lib.psd_last_error().decode()


def _append_args(L, **kw):
    f = (C.c_double * 32)(*([0.5] * 32))
    a = L.AppendArgs(_ptr(1), _ptr(2), _ptr(3), 512, 128, 128, _ptr(4), 4, 2, 8, 2, 64, 64, 0, 64, 1, f, 1.0, _ptr(5), _ptr(6),
                     None, _ptr(7), _ptr(8), 4, _ptr(9), _ptr(10), 8, 16, 1, 1.0, 1.0, _ptr(11))
    a.keep = f
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("args,scales,status,word", [
    (dict(), None, 1, "NULL scales"), (dict(), dict(k=None), 1, "NULL scales"), (dict(), dict(block=8), 1, "blocks of 16"),
    (dict(), dict(block=0), 1, "blocks of 16"), (dict(), dict(block=32), 1, "multiple of the block"),
    (dict(kv_dtype=0), dict(), 1, "e4m3"), (dict(k_scale=2.0), dict(), 1, "must be 1"), (dict(v_scale=0.5), dict(), 1, "must be 1"),
    (dict(D=68, q_stride=600, k_stride=136), dict(), 2, "multiples of 8"), (dict(Dv=0, v=None, v_pool=None), dict(), 2, "Dv 0"),
    (dict(Dv=264, v_stride=528), dict(), 2, "264"), (dict(rot_dim=8), dict(), 2, "rot_dim 8"), (dict(rot_dim=16, rot_col=4), dict(), 2, "rot_col 4"),
    (dict(k=_ptr(2) + 8), dict(), 2, "aligned"), (dict(k_stride=132), dict(), 2, "multiples of 8"), (dict(v_pool=_ptr(10) + 4), dict(), 2, "aligned"),
    (dict(k_stride=100), dict(), 1, "token stride"), (dict(num_tokens=-1), dict(), 1, "bad sizes"), (dict(fault_dev=None), dict(), 1, "NULL pointer")])
def test_append_refusals(lib, blank, args, scales, status, word):
    from paged_split_kv_decode_gb300 import _lib as L
    s = None if scales is None else L.BlockScales(**{**dict(k=_ptr(20), v=_ptr(21), block=16), **scales})
    a = _append_args(L, **args)
    assert lib.append_tokens_scaled(blank, C.byref(a), s, None) == status
    assert word in _message(lib) and "append_tokens_scaled" in _message(lib)


def test_append_of_nothing(lib, blank):
    from paged_split_kv_decode_gb300 import _lib as L
    s = L.BlockScales(_ptr(20), _ptr(21), 16)
    assert lib.append_tokens_scaled(blank, C.byref(_append_args(L, num_tokens=0, k=None)), s, None) == 0
    assert lib.append_tokens_scaled(None, C.byref(_append_args(L)), s, None) == 1


def _decode(L, lib, blank, scales, **kw):
    r = (L.TokenRequest * 1)(L.TokenRequest(0, 1, 0, 5))
    plan = L.MultiTokenPlan(1, r, 1, 16, 1, 1)
    a = L.MultiTokenArgs(_ptr(1), 512, _ptr(2), _ptr(3), _ptr(4), 1, 4, 1, 8, 2, 64, 16, 1, 1.0, 1.0, 0.125, None, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.multi_token_decode_scaled(blank, C.byref(a), scales, C.byref(plan), _ptr(5), None, _ptr(6), 1 << 40, None)


@pytest.mark.parametrize("args,scales,status,word", [
    (dict(), None, 1, "NULL scales"), (dict(), dict(v=None), 1, "NULL pointer"), (dict(), dict(block=24), 1, "blocks of 16"),
    (dict(), dict(block=64), 1, "multiple of the block"), (dict(kv_dtype=0), dict(), 1, "e4m3"), (dict(k_scale=0.5), dict(), 1, "must be 1"),
    (dict(Hq=7), dict(), 1, "Hq"), (dict(sm_scale=math.inf), dict(), 1, "finite"), (dict(page_size=32), dict(block=32), 1, "page_size"),
    (dict(num_tokens=0), dict(), 1, "token rows"), (dict(D=264), dict(), 2, "head dim")])
def test_attention_refusals(lib, blank, args, scales, status, word):
    from paged_split_kv_decode_gb300 import _lib as L
    s = None if scales is None else L.BlockScales(**{**dict(k=_ptr(20), v=_ptr(21), block=16), **scales})
    assert _decode(L, lib, blank, s, **args) == status
    assert word in _message(lib) and "multi_token_decode_scaled" in _message(lib)


def _beam(L, **kw):
    a = L.BeamArgs(_ptr(1), 100, 0, _ptr(2), None, 8, 4, 100, 8, 0, _ptr(3), _ptr(4), _ptr(5), _ptr(6))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("args,status", [
    (dict(rows=9), 1), (dict(rows=-4), 1), (dict(beams=0), 1), (dict(k=0), 1), (dict(vocab=0), 1), (dict(k=65), 2),
    (dict(beams=65, rows=65), 2), (dict(logits_type=3), 1), (dict(logits_type=-1), 1), (dict(logits_stride=99), 1),
    (dict(logits=None), 1), (dict(scores=None), 1), (dict(out_rows=None), 1), (dict(fault_dev=None), 1), (dict(logits=_ptr(1) + 2), 1),
    (dict(logits=_ptr(1) + 1, logits_type=1), 1), (dict(vocab=(1 << 30) + 1, logits_stride=1 << 31), 2),
    (dict(out_scores=_ptr(2)), 1), (dict(out_scores=_ptr(2) + 4, beams=8), 1), (dict(out_rows=_ptr(2) + 28), 1), (dict(out_tokens=_ptr(2)), 1)])
def test_selection_refusals(lib, blank, args, status):
    from paged_split_kv_decode_gb300 import _lib as L
    assert lib.beam_select(blank, C.byref(_beam(L, **args)), _ptr(7), 1 << 40, None) == status
    assert "beam_select" in _message(lib)


def test_selection_workspace_and_nothing(lib, blank):
    from paged_split_kv_decode_gb300 import _lib as L
    need = lib.psd_beam_workspace_bytes(blank, 8, 4, 8)
    assert need > 0
    assert lib.beam_select(blank, C.byref(_beam(L)), _ptr(7), need - 1, None) == 5
    assert lib.beam_select(blank, C.byref(_beam(L)), None, need, None) == 1
    assert lib.beam_select(blank, C.byref(_beam(L)), _ptr(7) + 8, need, None) == 1
    assert lib.beam_select(blank, C.byref(_beam(L, rows=0, logits=None)), None, 0, None) == 0
    assert lib.beam_select(None, C.byref(_beam(L)), _ptr(7), need, None) == 1
    for bad in ((-1, 4, 8), (8, 0, 8), (8, 4, 0), (8, 65, 8), (8, 4, 65)):
        assert lib.psd_beam_workspace_bytes(blank, *bad) == 0


def _fork(L, to, **kw):
    a = L.ForkArgs(_ptr(1), 4, 1, _ptr(2), _ptr(3), 10, _ptr(4), 3, 16, 0, _ptr(5), _ptr(6), 50, _ptr(7), _ptr(8), 20, _ptr(9),
                   C.cast(to, C.c_void_p), len(to), _ptr(11))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("args,status", [
    (dict(num_new=-1), 1), (dict(batch=-1), 1), (dict(page_size=0), 1), (dict(room=-1), 1), (dict(new_capacity=-1), 1),
    (dict(num_pages=0), 1), (dict(num_pages=1 << 31), 1), (dict(num_new=(1 << 24) + 1), 2), (dict(num_page_indices=1 << 31), 2),
    (dict(parents=None), 1), (dict(kv_len=None), 1), (dict(page_indices=None), 1), (dict(ref_count=None), 1), (dict(new_len=None), 1),
    (dict(fault_dev=None), 1), (dict(new_indices=_ptr(3) + 16), 1), (dict(new_indptr=_ptr(2)), 1), (dict(new_len=_ptr(4)), 1),
    (dict(new_len=_ptr(1)), 1), (dict(new_ref_count=_ptr(5) + 64), 1), (dict(pools=None), 1), (dict(num_pools=-1), 1)])
def test_fork_refusals(lib, blank, args, status):
    from paged_split_kv_decode_gb300 import _lib as L
    pools = (L.PagePool * 1)(L.PagePool(_ptr(10), 64))
    assert lib.fork_pages(blank, C.byref(_fork(L, pools, **args)), _ptr(12), 1 << 40, None) == status
    assert "fork_pages" in _message(lib)


def test_page_calls_refusals(lib, blank):
    from paged_split_kv_decode_gb300 import _lib as L
    good = (L.PagePool * 1)(L.PagePool(_ptr(10), 64))
    need = lib.psd_pages_workspace_bytes(50, 4)
    assert lib.fork_pages(blank, C.byref(_fork(L, good)), _ptr(12), need - 1, None) == 5
    assert lib.fork_pages(blank, C.byref(_fork(L, good)), _ptr(12) + 4, need, None) == 1
    assert lib.fork_pages(None, C.byref(_fork(L, good)), _ptr(12), need, None) == 1
    for bad in (L.PagePool(None, 64), L.PagePool(_ptr(10), 0), L.PagePool(_ptr(10), 1 << 41)):
        assert lib.fork_pages(blank, C.byref(_fork(L, (L.PagePool * 1)(bad))), _ptr(12), need, None) == 1
    assert lib.psd_pages_workspace_bytes(0, 4) == 0 and lib.psd_pages_workspace_bytes(50, -1) == 0

    def compact(**kw):
        a = L.CompactArgs(_ptr(1), 10, _ptr(2), 50, _ptr(3), _ptr(4), _ptr(5), None, C.cast(good, C.c_void_p), 1, _ptr(6))
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.compact_pages(blank, C.byref(a), _ptr(12), lib.psd_pages_workspace_bytes(50, 0) - (1 if kw.get("num_pools") == 0 else 0), None)

    for kw, status in ((dict(num_page_indices=-1), 1), (dict(ref_count=None), 1), (dict(num_live=None), 1), (dict(new_indices=_ptr(1) + 4), 1),
                       (dict(new_ref_count=_ptr(2) + 4), 1), (dict(page_map=_ptr(2)), 1), (dict(page_map=_ptr(1)), 1),
                       (dict(num_pages=-3), 1), (dict(num_pools=0), 5)):
        assert compact(**kw) == status, kw
    p = C.cast(good, C.c_void_p)
    assert lib.copy_pages(blank, p, 1, 50, _ptr(1), _ptr(2), -1, _ptr(3), None) == 1
    assert lib.copy_pages(blank, p, 1, 50, None, _ptr(2), 4, _ptr(3), None) == 1
    assert lib.copy_pages(blank, p, 1, 0, _ptr(1), _ptr(2), 4, _ptr(3), None) == 1
    assert lib.copy_pages(blank, p, 1, 50, None, None, 0, None, None) == 0
    assert lib.free_pages(blank, None, None, 0, 1, _ptr(1), 50, _ptr(3), _ptr(4), need, None) == 1


def test_binding_passes_on_what_it_is_given(monkeypatch):
    """On CPU tensors, whose device number is -1, against a library that only records."""
    import paged_split_kv_decode_gb300 as psd
    from paged_split_kv_decode_gb300 import api
    seen = {}

    class Library:
        def __getattr__(self, name):
            def call(*a):
                seen[name] = a
                return 0
            return call

    class Fake:
        device, handle, _h = -1, None, None

    monkeypatch.setattr(api.L, "load", lambda: Library())
    monkeypatch.setattr(api, "_ctx_stream", lambda ctx, stream: 5)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    x, ws, fault = torch.zeros((6, 11))[:, :9], torch.zeros(300, dtype=torch.uint8), i32(1)
    out = [torch.zeros((2, 4), dtype=t) for t in (torch.float32, torch.int32, torch.int32)]
    s, done = torch.zeros(6), torch.zeros(6, dtype=torch.bool)
    psd.beam_select(Fake, x, s, *out, ws, beams=3, finished=done, pad_token=7, fault=fault)
    a = api.L.BeamArgs.from_buffer_copy(seen["beam_select"][1])
    assert (a.logits, a.logits_stride, a.logits_type, a.scores, a.finished) == (x.data_ptr(), 11, 0, s.data_ptr(), done.data_ptr())
    assert (a.rows, a.beams, a.vocab, a.k, a.pad_token) == (6, 3, 9, 4, 7)
    assert (a.out_scores, a.out_rows, a.out_tokens, a.fault_dev) == tuple(t.data_ptr() for t in out + [fault])
    assert seen["beam_select"][2:] == (ws.data_ptr(), 300, 5)

    class Pools:
        num_pages, device, count, address = 40, -1, 3, 12345
        fit = psd.PagePools.fit

    t = dict(page_indptr=i32(4), page_indices=i32(20), kv_len=i32(3), new_indptr=i32(6), new_indices=i32(30), new_len=i32(5))
    parents, ref, new = i32(5), i32(40), i32(40)
    psd.fork_pages(Fake, Pools(), parents, page_size=16, room=2, ref_count=ref, new_ref_count=new, workspace=ws, fault=fault,
                   keep_old=True, **t)
    a = api.L.ForkArgs.from_buffer_copy(seen["fork_pages"][1])
    assert (a.parents, a.num_new, a.room, a.batch, a.page_size, a.keep_old) == (parents.data_ptr(), 5, 2, 3, 16, 1)
    assert (a.num_page_indices, a.num_pages, a.new_capacity, a.pools, a.num_pools) == (20, 40, 30, 12345, 3)
    assert (a.page_indptr, a.page_indices, a.kv_len, a.new_indptr, a.new_indices, a.new_len) == tuple(x.data_ptr() for x in t.values())
    assert (a.ref_count, a.new_ref_count, a.fault_dev) == (ref.data_ptr(), new.data_ptr(), fault.data_ptr())
    table, live, to = i32(20), i32(1), i32(40)
    psd.compact_pages(Fake, Pools(), table, ref, num_live=live, workspace=ws, page_map=to, fault=fault)
    a = api.L.CompactArgs.from_buffer_copy(seen["compact_pages"][1])
    assert (a.page_indices, a.num_page_indices, a.ref_count, a.num_pages) == (table.data_ptr(), 20, ref.data_ptr(), 40)
    assert (a.new_indices, a.new_ref_count, a.num_live, a.page_map) == (table.data_ptr(), ref.data_ptr(), live.data_ptr(), to.data_ptr())
    assert (a.pools, a.num_pools, a.fault_dev) == (12345, 3, fault.data_ptr())
    sc = psd.BlockScales(torch.zeros((4, 2, 2), dtype=torch.uint8), torch.ones((4, 2, 2), dtype=torch.uint8), 16)
    sc.fit((4, 32, 2, 64), -1)
    for shape, dev in (((4, 16, 2, 64), -1), ((5, 32, 2, 64), -1), ((4, 32, 2, 64), 0)):
        with pytest.raises(ValueError):
            sc.fit(shape, dev)


@pytest.mark.parametrize("args", [dict(out_rows=_ptr(8) + 4), dict(out_tokens=_ptr(8)), dict(out_scores=_ptr(8) - 60), dict(out_scores=_ptr(2), k=4, finished=_ptr(2) + 31)])
def test_selection_refuses_outputs_over_flags(lib, blank, args):
    """Flags that another request's part of the call may still read."""
    from paged_split_kv_decode_gb300 import _lib as L
    assert lib.beam_select(blank, C.byref(_beam(L, **{**dict(finished=_ptr(8)), **args})), _ptr(7), 1 << 40, None) == 1
    assert "overlap finished" in _message(lib)


@pytest.mark.parametrize("args", [dict(page_map=_ptr(4)), dict(page_map=_ptr(3)), dict(num_live=_ptr(2) + 40), dict(num_live=_ptr(1)),
                                  dict(num_live=_ptr(4) + 196), dict(new_indices=_ptr(2)), dict(new_ref_count=_ptr(1)),
                                  dict(new_ref_count=_ptr(3) + 36), dict(page_map=_ptr(9), num_live=_ptr(9) + 4)])
def test_compaction_refuses_outputs_over_each_other(lib, blank, args):
    from paged_split_kv_decode_gb300 import _lib as L
    good = (L.PagePool * 1)(L.PagePool(_ptr(20), 64))
    a = L.CompactArgs(_ptr(1), 10, _ptr(2), 50, _ptr(3), _ptr(4), _ptr(5), None, C.cast(good, C.c_void_p), 1, _ptr(6))
    for k, v in args.items():
        setattr(a, k, v)
    assert lib.compact_pages(blank, C.byref(a), _ptr(12), 1 << 40, None) == 1
    assert "apart" in _message(lib)


# ------------------------------------------------------------- pins of the oracle
def test_oracle_codes_are_torchs():
    x = np.random.default_rng(0).standard_normal(20000) * np.exp(4 * np.random.default_rng(1).standard_normal(20000))
    x = np.concatenate([x, A.e4m3_to_f64(np.arange(127, dtype=np.uint8)), [2.0 ** -10, 2.0 ** -11, 3 * 2.0 ** -11, 464.0, 1e9, 17.0, 19.0, 0.0]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(BM.e4m3_nearest(x.astype(np.float64)), want)


def test_oracle_scales_hold_their_blocks():
    for top in (448.0, np.nextafter(448.0, 500), 1.0, 1.75, 1.76, 3e38, 2.0 ** -33, 0.0):
        e = BM.scale_exponent(top)
        assert top <= 448 * 2.0 ** (e - 127) and (e == 95 or top > 448 * 2.0 ** (e - 128))
    assert list(BM.scale_values([0, 127, 130])) == [2.0 ** -127, 1.0, 8.0] and np.isnan(BM.scale_values([255])[0])
    v = np.arange(8.0).reshape(1, 4, 1, 2)
    assert np.array_equal(BM.dequantise(v, np.array([[[127], [128]]]), 2)[0, :, 0], [[0, 1], [2, 3], [8, 10], [12, 14]])


def test_oracle_selection_is_the_sorted_log_softmax():
    rng = np.random.default_rng(2)
    x, s = rng.standard_normal((4, 9)), rng.standard_normal(4)
    got = BM.select(x, s, 2, 5)
    for b in range(2):
        v = torch.log_softmax(torch.from_numpy(x[2 * b: 2 * b + 2]), -1).numpy() + s[2 * b: 2 * b + 2, None]
        order = np.argsort(-v.ravel(), kind="stable")[:5]
        assert np.allclose(got[0][b], v.ravel()[order], atol=1e-12)
        assert list(got[1][b]) == list(2 * b + order // 9) and list(got[2][b]) == list(order % 9)
    got = BM.select(np.zeros((1, 3)), [0.0], 1, 5)
    assert list(got[2][0]) == [0, 1, 2, -1, -1] and list(got[1][0]) == [0, 0, 0, -1, -1]
    assert np.allclose(got[0][0, :3], -math.log(3)) and np.isneginf(got[0][0, 3:]).all()
    got = BM.select(np.full((2, 3), np.nan), [-1.0, -2.0], 2, 2, finished=[0, 1], pad=9)
    assert (got[0][0, 0], got[1][0, 0], got[2][0, 0]) == (-2.0, 1, 9) and got[1][0, 1] == -1


def test_oracle_pages_by_hand():
    # one request of 5 tokens on pages of 2: pages 4, 0, 6 (the last part full); two children and one more token each
    rows, lengths, ref, copies = BM.fork([0, 0], [0, 3], [4, 0, 6], [5], 2, 1, [1, 0, 0, 0, 1, 0, 1])
    assert rows == [[4, 0, 6], [4, 0, 1]] and lengths == [6, 6] and ref == [2, 1, 0, 0, 2, 0, 1] and copies == [(6, 1)]
    rows, _, ref, copies = BM.fork([0, 0], [0, 3], [4, 0, 6], [5], 2, 1, [1, 0, 0, 0, 1, 0, 1], keep_old=True)
    assert rows == [[4, 0, 1], [4, 0, 2]] and ref == [3, 1, 1, 0, 3, 0, 1] and copies == [(6, 1), (6, 2)]
    rows, _, ref, _ = BM.fork([0, -1], [0, 3], [4, 0, 6], [5], 2, 0, [1, 0, 0, 0, 1, 0, 2])
    assert rows == [[4, 0, 6], []] and ref == [1, 0, 0, 0, 1, 0, 2]
    assert BM.fork([0, 0], [0, 1], [0], [1], 2, 1, [1]) is None
    assert BM.compact([0, 2, 0, 1, 5]) == (3, [-1, 1, -1, 0, 2], [1, 2, 5, 0, 0], [(3, 0), (4, 2)])


@pytest.mark.parametrize("seed", range(6))
def test_oracle_forks_keep_every_count(seed):
    """Whatever goes on: the counts are the new tables' entries and those outside, and no two requests write to one page."""
    rng = np.random.default_rng(seed)
    page, ref = int(rng.integers(1, 6)), [0] * 400
    rows, lengths = [[]], [0]
    for step in range(12):
        parents = [int(x) for x in rng.integers(-1, len(rows), int(rng.integers(1, 7)))]
        indptr = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
        room = int(rng.integers(1, 5))
        new, lengths, ref, copies = BM.fork(parents, indptr, [g for r in rows for g in r], lengths, page, room, ref)
        assert list(np.bincount(np.array([g for r in new for g in r], dtype=int), minlength=400)) == ref
        for r, L in zip(new, lengths):
            for j in range((L - room) // page, len(r)) if r else []:
                assert ref[r[j]] == 1                                  # what gets the new tokens is nobody else's
        assert not {b for _, b in copies} & {a for a, _ in copies}
        rows = new


@pytest.mark.parametrize("x", [0.0, -1e10, -3.4e38, 3.4e38])
def test_oracle_rows_of_one_value(x):
    """Tokens share such a row evenly, wherever it lies."""
    got = BM.select(np.full((1, 4), x), [-1.0], 1, 4)
    assert np.allclose(got[0], -1 - math.log(4)) and list(got[2][0]) == [0, 1, 2, 3]
