"""A step of several new tokens as it is used: append, attention over what was appended,
verification, and the next step over the tokens that stayed."""
import numpy as np
import pytest
import torch

import paged_split_kv_decode_gb300 as psd
from oracle import attention as A
from oracle import tokens as TK
from _gpu_util import ctx
from _tokens_util import bounds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 8), (40, 5)])
def test_three_steps(D, page, kv):
    """A prompt, then two verified steps whose cache drops the refused drafts; the attention is
    checked against the rows the pools really hold, the verification against exact
    arithmetic."""
    rng = np.random.default_rng(D + page)
    B, Hq, Hkv, V, num_pages = 3, 4, 2, 97, 64
    rope = psd.rope_frequencies(2 * (D // 4), scaling="yarn", factor=4.0, original_max_position=64)
    shape = (num_pages, page, Hkv, D)
    pools = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") if kv == "fp8" else
             torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    scales = (0.02, 0.015) if kv == "fp8" else (1.0, 1.0)
    free = list(rng.permutation(num_pages))
    lists, length = [[] for _ in range(B)], [0] * B
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).cuda()  # noqa: E731
    for new in ([7, 30, 1], [4, 1, 3], [2, 5, 5]):
        for b in range(B):
            length[b] += new[b]
            while len(lists[b]) * page < length[b]:
                lists[b].append(int(free.pop()))
            # pages the refused drafts needed may now be behind the end
        pages = [ls[: -(-n // page)] for ls, n in zip(lists, length)]
        page_indptr = np.concatenate([[0], np.cumsum([len(p) for p in pages])])
        indices = np.concatenate(pages).astype(np.int32)
        q_indptr = np.concatenate([[0], np.cumsum(new)])
        T = int(q_indptr[-1])
        qkv = torch.from_numpy(rng.standard_normal((T, (Hq + 2 * Hkv) * D)).astype(np.float32)).to(torch.bfloat16).cuda()
        q = qkv[:, : Hq * D].view(T, Hq, D)
        k = qkv[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
        v = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        q_rot = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        dev = i32(indices)
        psd.append_tokens(ctx(), q, k, v, q_rot, q_indptr=i32(q_indptr), kv_len=i32(length), page_indptr=i32(page_indptr),
                          page_indices=dev, k_pool=pools[0], v_pool=pools[1], rope=rope, neox=False,
                          k_scale=scales[0], v_scale=scales[1], fault=fault)
        last = [n - (len(p) - 1) * page for n, p in zip(length, pages)]
        plan = psd.plan_multi_token(psd.HostTable(page_indptr, indices, last, page), q_indptr, Hq, Hkv)
        ws = psd.multi_token_workspace(ctx(), plan, D, "cuda")
        o, lse = torch.empty((T, Hq, D), device="cuda"), torch.empty((T, Hq), device="cuda")
        args = psd.multi_token_args(q_rot, pools[0], pools[1], dev, sm_scale=D ** -0.5, k_scale=scales[0],
                                    v_scale=scales[1])
        psd.multi_token_decode(ctx(), args, plan, o, lse, ws)
        assert psd.check_device_error(ctx(), ws) == 0
        values = [A.e4m3_to_f64(p.cpu().numpy()).reshape(shape) * c if kv == "fp8" else p.double().cpu().numpy()
                  for p, c in zip(pools, scales)]
        want = TK.attend(q_rot.double().cpu().numpy(), *values, q_indptr, length, page_indptr, indices, page, D ** -0.5)
        e_o, e_l = bounds(want, D, max(length), True, 3)
        assert bool(np.all(np.abs(o.double().cpu().numpy() - want[0]) <= e_o))
        assert bool(np.all(np.abs(lse.double().cpu().numpy() - want[1]) <= e_l))
        # the outputs stand for the target's logits; every new token but the first is a draft
        drafts = np.array(new) - 1
        d_indptr = np.concatenate([[0], np.cumsum(drafts)])
        head = torch.from_numpy(rng.standard_normal((Hq * D, V)).astype(np.float32)).cuda()
        target = torch.softmax(o.reshape(T, -1) @ head, -1)
        rows = np.concatenate([np.arange(d_indptr[b], d_indptr[b + 1]) + b for b in range(B)]).astype(np.int64)
        draft = torch.softmax(torch.log(target[torch.from_numpy(rows).cuda()] + 1e-9) * 0.7, -1)
        tokens = torch.argmax(draft, -1).to(torch.int32) if len(rows) else torch.zeros(0, dtype=torch.int32, device="cuda")
        u = torch.from_numpy(rng.random(T, dtype=np.float32)).cuda()
        accepted, out = i32(np.zeros(B)), i32(np.zeros(T))
        psd.verify_drafts(ctx(), target, draft, tokens, i32(d_indptr), u, accepted, out, fault=fault)
        a, said = TK.verify(target.cpu().numpy(), draft.cpu().numpy(), tokens.cpu().numpy(), d_indptr, u.cpu().numpy())
        assert accepted.tolist() == a and out.tolist() == said
        length = [n - int(d) + x for n, d, x in zip(length, drafts, a)]  # refused drafts leave the cache
    assert int(fault) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_captured_step(kv):
    """Append, attention and verification in one graph, replayed over other queries: as the calls
    one by one."""
    B, new, before, Hq, Hkv, D, page, V = 3, [5, 1, 4], [300, 900, 40], 8, 2, 64, 16, 50
    length = [n + x for n, x in zip(new, before)]
    pages = [-(-n // page) for n in length]
    rng = np.random.default_rng(7)
    indptr = np.concatenate([[0], np.cumsum(pages)])
    indices = rng.permutation(int(indptr[-1])).astype(np.int32)
    q_indptr = np.concatenate([[0], np.cumsum(new)])
    d_indptr = q_indptr - np.arange(B + 1)
    T = int(q_indptr[-1])
    i32 = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).cuda()  # noqa: E731
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *n: torch.randn(*n, device="cuda", generator=gen).to(torch.bfloat16)  # noqa: E731
    shape = (len(indices), page, Hkv, D)
    start = [torch.randint(0, 96, shape, dtype=torch.uint8, device="cuda", generator=gen) if kv == "fp8" else rand(*shape)
             for _ in range(2)]
    pools = [p.clone() for p in start]
    q, k, v = rand(T, Hq, D), rand(T, Hkv, D), rand(T, Hkv, D)
    q_rot, o, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((T, Hq), device="cuda")
    rope = psd.rope_frequencies(D)
    idx, q_ind, kv_len, p_ind = i32(indices), i32(q_indptr), i32(length), i32(indptr)
    plan = psd.plan_multi_token(psd.HostTable(indptr, indices, [n - (c - 1) * page for n, c in zip(length, pages)], page),
                                q_indptr, Hq, Hkv)
    ws = psd.multi_token_workspace(ctx(), plan, D, "cuda")
    args = psd.multi_token_args(q_rot, *pools, idx, sm_scale=D ** -0.5, k_scale=0.02, v_scale=0.015)
    probs = torch.softmax(torch.randn(T, V, device="cuda", generator=gen), -1)
    tokens, u = i32(rng.integers(0, V, T - B)), torch.rand(T, device="cuda", generator=gen)
    accepted, out, fault = i32(np.zeros(B)), i32(np.zeros(T)), i32(np.zeros(1))
    d_ind = i32(d_indptr)

    def step():
        psd.append_tokens(ctx(), q, k, v, q_rot, q_indptr=q_ind, kv_len=kv_len, page_indptr=p_ind, page_indices=idx,
                          k_pool=pools[0], v_pool=pools[1], rope=rope, neox=True, k_scale=0.02, v_scale=0.015, fault=fault)
        psd.multi_token_decode(ctx(), args, plan, o, lse, ws)
        psd.verify_drafts(ctx(), probs, None, tokens, d_ind, u, accepted, out, fault=fault)

    def outputs():
        torch.cuda.synchronize()
        assert int(fault) == 0 and psd.check_device_error(ctx(), ws) == 0
        return [x.clone() for x in (q_rot, o, lse, accepted, out, *pools)]

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        q.copy_(rand(T, Hq, D))
        u.copy_(torch.rand(T, device="cuda", generator=gen))
        results = []
        for run in (step, g.replay):
            for p, at in zip(pools, start):
                p.copy_(at)
            for x in (q_rot, o, lse, accepted, out):
                x.zero_()
            run()
            results.append(outputs())
        assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("kv,page", [("bf16", 16), ("fp8", 16), ("bf16", 12)])
def test_pools_past_32_bits(kv, page):
    """The same step in a small pool and at the end of one with more than 2^31 elements (bf16: more
    than 2^32 bytes) agrees bit for bit."""
    new, before, Hq, Hkv, D = [5, 40], [300, 20], 16, 8, 128
    length = [n + x for n, x in zip(new, before)]
    pages = [-(-n // page) for n in length]
    indptr = np.concatenate([[0], np.cumsum(pages)])
    used = int(indptr[-1])
    many = (1 << 31) // (page * Hkv * D) + 100
    order = np.random.default_rng(11).permutation(used).astype(np.int32)
    q_indptr = np.concatenate([[0], np.cumsum(new)])
    T = int(q_indptr[-1])
    i32 = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).cuda()  # noqa: E731
    gen = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *n: torch.randn(*n, device="cuda", generator=gen).to(torch.bfloat16)  # noqa: E731
    shape = (used, page, Hkv, D)
    start = [torch.randint(0, 96, shape, dtype=torch.uint8, device="cuda", generator=gen) if kv == "fp8" else rand(*shape)
             for _ in range(2)]
    q, k, v = rand(T, Hq, D), rand(T, Hkv, D), rand(T, Hkv, D)
    rope, results = psd.rope_frequencies(D), []
    for pool_pages in (used, many):
        pools = [torch.empty((pool_pages, page, Hkv, D), dtype=x.dtype, device="cuda") for x in start]
        for pool, x in zip(pools, start):
            pool[pool_pages - used:] = x
        indices = order + (pool_pages - used)
        idx, q_rot = i32(indices), torch.empty_like(q)
        fault = psd.append_tokens(ctx(), q, k, v, q_rot, q_indptr=i32(q_indptr), kv_len=i32(length), page_indptr=i32(indptr),
                                  page_indices=idx, k_pool=pools[0], v_pool=pools[1], rope=rope, neox=True,
                                  k_scale=0.02, v_scale=0.015)
        plan = psd.plan_multi_token(psd.HostTable(indptr, indices, [n - (c - 1) * page for n, c in zip(length, pages)], page),
                                    q_indptr, Hq, Hkv)
        ws = psd.multi_token_workspace(ctx(), plan, D, "cuda")
        o, lse = torch.empty_like(q), torch.empty((T, Hq), device="cuda")
        psd.multi_token_decode(ctx(), psd.multi_token_args(q_rot, *pools, idx, sm_scale=D ** -0.5, k_scale=0.02,
                                                           v_scale=0.015), plan, o, lse, ws)
        assert int(fault) == 0 and psd.check_device_error(ctx(), ws) == 0
        results.append([q_rot, o, lse] + [pool[pool_pages - used:].clone() for pool in pools])
        del pools
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert not torch.equal(results[0][3], start[0])
