"""CPU tests of a step with several new tokens: rotary frequencies and plans of the library
against the oracle, the refusals of its host calls, and pins of the oracle itself."""
import math

import numpy as np
import pytest

from oracle import tokens as TK


@pytest.fixture(scope="module")
def psd():
    import paged_split_kv_decode_gb300 as psd
    psd.load()
    return psd


@pytest.mark.parametrize("kind", ["plain", "linear", "ntk", "yarn", "bands"])
@pytest.mark.parametrize("r,base,factor", [(64, 10000.0, 4.0), (128, 500000.0, 8.0), (4, 10000.0, 1.0), (16, 1e6, 0.5)])
def test_frequencies_against_the_oracle(psd, kind, r, base, factor):
    kw = dict(low=1.0, high=4.0) if kind == "bands" else {}
    got = psd.rope_frequencies(r, base=base, scaling=kind, factor=factor, original_max_position=4096)
    f, m = TK.rope_frequencies(kind, r, base, factor, 4096, **kw)
    # pow and log of two libraries: a few ulp of 64 bits each
    assert np.allclose(got.inv_freq, f, rtol=1e-13, atol=0) and abs(got.magnitude - m) < 1e-14
    assert got.rot_dim == r


def test_scalings_keep_the_fast_and_divide_the_slow(psd):
    plain = psd.rope_frequencies(128).inv_freq
    for kind in ("yarn", "bands"):
        f = psd.rope_frequencies(128, scaling=kind, factor=16.0, original_max_position=4096).inv_freq
        assert f[0] == plain[0] and math.isclose(f[-1], plain[-1] / 16, rel_tol=1e-12)
        assert np.all(np.diff(f) < 0)
    assert math.isclose(psd.rope_frequencies(128, scaling="ntk", factor=8.0).inv_freq[-1], plain[-1] / 8, rel_tol=1e-12)


@pytest.mark.parametrize("kw", [dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=514), dict(rot_dim=64, base=1.0),
                                dict(rot_dim=64, base=float("nan")), dict(rot_dim=64, scaling="linear", factor=0.0),
                                dict(rot_dim=64, scaling="yarn", factor=2.0), dict(rot_dim=2, scaling="ntk", factor=2.0),
                                dict(rot_dim=64, scaling="bands", factor=2.0, original_max_position=10, low=4.0, high=4.0),
                                dict(rot_dim=64, scaling="yarn", factor=2.0, original_max_position=10, low=0.0)])
def test_frequency_refusals(psd, kw):
    with pytest.raises(psd.PsdError) as e:
        psd.rope_frequencies(**kw)
    assert e.value.status == 1
    with pytest.raises(ValueError):
        psd.rope_frequencies(64, scaling="other")


def test_plan(psd):
    table = psd.HostTable([0, 2, 3, 7], [4, 1, 0, 9, 8, 7, 6], [3, 16, 1], 16)
    plan = psd.plan_multi_token(table, [0, 5, 5, 30], 8, 2)
    assert plan.requests == [(0, 5, 0, 19), (5, 0, 2, 16), (5, 25, 3, 49)]
    assert (plan.batch, plan.page_size, plan.num_tokens, plan.max_new) == (3, 16, 30, 25)
    empty = psd.plan_multi_token(psd.HostTable([0], [], [], 16), [0])
    assert (empty.batch, empty.num_tokens, empty.max_new) == (0, 0, 0)


@pytest.mark.parametrize("q_indptr", [[1, 2, 3], [0, 20, 21], [0, 2, 1], [0, 0, 33]])
def test_plan_refusals(psd, q_indptr):
    table = psd.HostTable([0, 2, 4], [4, 1, 0, 9], [3, 16], 16)  # 19 and 32 tokens
    with pytest.raises(psd.PsdError) as e:
        psd.plan_multi_token(table, q_indptr)
    assert e.value.status == 1


def test_plan_argument_errors(psd):
    table = psd.HostTable([0, 2, 4], [4, 1, 0, 9], [3, 16], 16)
    with pytest.raises(ValueError):
        psd.plan_multi_token(table, [0, 1])
    with pytest.raises(ValueError):
        psd.plan_multi_token(table, [0, 1, 2], 8, 3)
    with pytest.raises(psd.PsdError):  # a request with no page
        psd.plan_multi_token(psd.HostTable([0, 0], [], [0], 16), [0, 0])


# ------------------------------------------------------------- pins of the oracle
def test_oracle_attention_is_causal_softmax():
    rng = np.random.default_rng(3)
    n, D = 5, 8
    q, K, V = rng.standard_normal((n, 1, D)), rng.standard_normal((3, 2, 1, D)), rng.standard_normal((3, 2, 1, D))
    args = (q, K, V, [0, n], [n], [0, 3], [2, 0, 1], 2, 0.5)
    o, lse, _, _ = TK.attend(*args)
    keys = np.concatenate([K[2], K[0], K[1]])[:n, 0]
    vals = np.concatenate([V[2], V[0], V[1]])[:n, 0]
    for i in range(n):
        w = np.exp(0.5 * keys[: i + 1] @ q[i, 0])
        assert np.allclose(o[i, 0], w @ vals[: i + 1] / w.sum()) and math.isclose(lse[i, 0], math.log2(w.sum()))
    chain = [(1 << (i + 1)) - 1 for i in range(n)]   # every token's ancestors are all before it
    assert np.allclose(TK.attend(*args, tree=chain)[0], o)
    o, lse, _, _ = TK.attend(*args, tree=[0] * n)
    assert np.all(o == 0) and np.all(np.isneginf(lse))


def test_oracle_verification_keeps_the_target_distribution():
    """Over a grid of drafts and numbers, the first token out is distributed as p."""
    p, q = np.array([0.5, 0.25, 0.125, 0.125]), np.array([0.125, 0.125, 0.25, 0.5])
    N, mass = 16, np.zeros(4)
    for d in range(4):
        for i in range(N):
            for j in range(N):
                u = np.array([(i + 0.5) / N, (j + 0.5) / N], dtype=np.float32)
                _, out = TK.verify(np.stack([p, p]).astype(np.float32), q[None].astype(np.float32), [d], [0, 1], u)
                mass[out[0]] += q[d] / N / N
    assert np.allclose(mass, p, atol=1 / N)


def test_replaced_frequencies_are_the_ones_in_use(psd):
    """The address and width a call passes on are those of the array that is there."""
    import ctypes

    def in_use(r):
        return list((ctypes.c_double * (r.rot_dim // 2)).from_address(r.address))

    r = psd.rope_frequencies(64)
    assert in_use(r) == list(r.inv_freq) and r.rot_dim == 64
    r.inv_freq = [1.0, 0.5, 0.25]
    assert r.rot_dim == 6 and in_use(r) == [1.0, 0.5, 0.25]
    own = np.array([0.5, 0.125])
    r.inv_freq = own
    own[0] = 7.0                                     # the caller's array stays the caller's
    assert in_use(r) == [0.5, 0.125] == list(r.inv_freq)
    r.inv_freq[1] = 2.0
    assert in_use(r) == [0.5, 2.0]
    for name in ("rot_dim", "address"):
        with pytest.raises(AttributeError):
            setattr(r, name, 2)


def test_faults_are_read_on_the_stream_of_the_contexts_device(psd, monkeypatch):
    """multi_token_decode runs on the current stream of its context's device, which need not be the
    current device; its faults are read behind it on the same stream."""
    from paged_split_kv_decode_gb300 import api
    seen = []

    class Library:
        def psd_check_device_error(self, handle, workspace, stream, bits):
            seen.append(getattr(stream, "value", stream))
            return 0

    class Fake:
        device, handle, _h = 1, None, None

    monkeypatch.setattr(api, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(api.torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(api, "_dev_ptr", lambda t, name: 0)
    monkeypatch.setattr(api.L, "load", lambda: Library())
    assert api._ctx_stream(Fake, None) == 1001
    assert api.check_device_error(Fake, None) == 0 and seen == [1001]
    api.check_device_error(Fake, None, stream=77)
    assert seen[1] == 77
