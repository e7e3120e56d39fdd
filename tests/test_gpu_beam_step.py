"""A beam search as it is used: prompts into a cache of 8-bit blocks, then steps of append, attention, selection and fork,
the pool compacted on the way; each step's parts against their definitions, and the cache at the end against one that a
request of its own would have."""
import numpy as np
import pytest
import torch

import paged_split_kv_decode_gb300 as psd
from oracle import attention as A
from oracle import beams as BM
from oracle import tokens as TK
from _gpu_util import ctx
from _tokens_util import bounds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,page,block", [(64, 16, 16), (128, 32, 16), (80, 64, 64)])
def test_beams_over_scaled_blocks(D, page, block):
    rng = np.random.default_rng(D + page)
    B, W, Hq, Hkv, V, num_pages, steps = 2, 3, 4, 2, 500, 90, 9
    rope = psd.rope_frequencies(16 * (D // 32))
    i32 = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).cuda()  # noqa: E731
    k_pool = torch.full((num_pages, page, Hkv, D), 0x7F, dtype=torch.uint8, device="cuda")
    v_pool = k_pool.clone()
    ke = torch.full((num_pages, page // block, Hkv), 255, dtype=torch.uint8, device="cuda")
    ve = ke.clone()
    cache = psd.PagePools([k_pool, v_pool, ke, ve])
    scales = psd.BlockScales(ke, ve, block)
    ref, fault = i32([0] * num_pages), i32([0])
    ws_pages = psd.pages_workspace(cache, B * W, "cuda")
    ws_beam = psd.beam_workspace(ctx(), B * W, W, W, "cuda")
    embed = torch.from_numpy(rng.standard_normal((V, (Hq + 2 * Hkv) * D)).astype(np.float32)).to(torch.bfloat16).cuda()
    head = torch.from_numpy((rng.standard_normal((Hq * D, V)) * 0.05).astype(np.float32)).cuda()
    prompts = [list(map(int, rng.integers(0, V, n))) for n in (21, 37)]

    def step(tokens, lens, new, table_dev, table_host):
        """Appends the tokens and attends; checks the attention against what the pools hold."""
        q_indptr = np.concatenate([[0], np.cumsum(new)])
        qkv = embed[torch.tensor(tokens, device="cuda")]
        T = len(tokens)
        q, k, v = qkv[:, : Hq * D].view(T, Hq, D), qkv[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D), qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        q_rot = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        psd.append_tokens(ctx(), q, k, v, q_rot, q_indptr=i32(q_indptr), kv_len=table_dev[2], page_indptr=table_dev[0],
                          page_indices=table_dev[1], k_pool=k_pool, v_pool=v_pool, rope=rope, neox=True, scales=scales, fault=fault)
        last = [n - (-(-n // page) - 1) * page for n in lens]
        plan = psd.plan_multi_token(psd.HostTable(table_host[0], table_host[1], last, page), q_indptr, Hq, Hkv)
        ws = psd.multi_token_workspace(ctx(), plan, D, "cuda")
        o, lse = torch.empty((T, Hq, D), device="cuda"), torch.empty((T, Hq), device="cuda")
        psd.multi_token_decode(ctx(), psd.multi_token_args(q_rot, k_pool, v_pool, table_dev[1], sm_scale=D ** -0.5, scales=scales),
                               plan, o, lse, ws)
        assert psd.check_device_error(ctx(), ws) == 0
        values = lambda c, e: BM.dequantise(A.e4m3_to_f64(c.cpu().numpy()).reshape(tuple(c.shape)), e.cpu().numpy(), block)  # noqa: E731
        want = TK.attend(q_rot.double().cpu().numpy(), values(k_pool, ke), values(v_pool, ve), q_indptr, lens, table_host[0],
                         table_host[1], page, D ** -0.5)
        e_o, e_l = bounds(want, D, max(lens), True, 2)
        assert np.all(np.abs(o.double().cpu().numpy() - want[0]) <= e_o)
        assert np.all(np.abs(lse.double().cpu().numpy() - want[1]) <= e_l)
        return o[torch.tensor(q_indptr[1:] - 1, device="cuda")].flatten(1) @ head

    def fork(parents, old, room, keep_old=False):
        out = (i32([0] * (len(parents) + 1)), i32([0] * 60), i32([0] * len(parents)))
        host = [t.cpu().numpy() for t in old] + [ref.cpu().numpy()]
        psd.fork_pages(ctx(), cache, parents, page_indptr=old[0], page_indices=old[1], kv_len=old[2], page_size=page, room=room,
                       ref_count=ref, new_indptr=out[0], new_indices=out[1], new_len=out[2], workspace=ws_pages,
                       keep_old=keep_old, fault=fault)
        rows, lengths, counts, _ = BM.fork(parents.tolist(), host[0], host[1], host[2], page, room, host[3], keep_old)
        flat = [g for r in rows for g in r]
        assert out[2].tolist() == lengths and ref.tolist() == counts and out[1][: len(flat)].tolist() == flat
        return out, (np.concatenate([[0], np.cumsum([len(r) for r in rows])]), np.array(flat))

    # the prompts: a table of empty requests makes room, one append takes them in
    empty = (i32([0] * (B + 1)), i32([0]), i32([0] * B))
    lens = [len(p) for p in prompts]
    pages = [-(-n // page) for n in lens]
    indptr, indices = np.concatenate([[0], np.cumsum(pages)]), rng.permutation(num_pages)[: sum(pages)]
    ref.copy_(i32(np.bincount(indices, minlength=num_pages)))
    table = (i32(indptr), i32(indices), i32(lens))
    logits = step(sum(prompts, []), lens, lens, table, (indptr, indices))
    # the first selection: each prompt's row stands for all its beams, of which one is alive
    scores = torch.full((B * W,), -np.inf, device="cuda")
    scores[::W] = 0.0
    out = [torch.empty((B, W), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    chains = {}
    logits, first = logits.repeat_interleave(W, 0).contiguous(), True
    history = [list(p) for p in prompts for _ in range(W)]
    for n in range(steps):
        psd.beam_select(ctx(), logits, scores, *out, ws_beam, beams=W, fault=fault)
        want = BM.select(logits.double().cpu().numpy(), scores.cpu().numpy(), W, W)
        assert np.array_equal(out[1].cpu().numpy(), want[1]) and np.array_equal(out[2].cpu().numpy(), want[2])
        assert np.allclose(out[0].cpu().numpy(), want[0], rtol=1e-6, atol=1e-6)
        scores = out[0].flatten().clone()
        parents = out[1].flatten()
        tokens = out[2].flatten().tolist()
        history = [history[p] + [t] for p, t in zip(parents.tolist(), tokens)]
        if first:
            parents, first = torch.div(parents, W, rounding_mode="floor").int(), False   # rows of the prompts' table
        table, host = fork(parents, table, 1)
        if n == 4:
            live = i32([0])
            psd.compact_pages(ctx(), cache, table[1][: len(host[1])], ref, num_live=live, workspace=ws_pages, fault=fault)
            m = int(live)
            assert bool((ref[:m] > 0).all()) and not bool(ref[m:].any())
            host = (host[0], table[1][: len(host[1])].cpu().numpy())
        lens = [len(h) for h in history]
        logits = step(tokens, lens, [1] * (B * W), table, host)
    assert int(fault) == 0
    # what each beam attends to now: its own history, as if it had been written alone, but for what scaling blocks anew rounds
    for b, h in enumerate(history):
        qkv = embed[torch.tensor(h, device="cuda")].double().cpu().numpy()
        k = TK.rotate(qkv[:, Hq * D: (Hq + Hkv) * D].reshape(-1, Hkv, D), np.arange(len(h))[:, None], rope.inv_freq, 1.0, 0, True)[0]
        v = qkv[:, (Hq + Hkv) * D:].reshape(-1, Hkv, D)
        row = host[1][host[0][b]: host[0][b + 1]]
        for x, pool, e in ((k, k_pool, ke), (v, v_pool, ve)):
            s = BM.scale_values(np.repeat(e[torch.tensor(row, device="cuda").long()].cpu().numpy(), block, 1).reshape(-1, Hkv))[: len(h), :, None]
            got = A.e4m3_to_f64(pool[torch.tensor(row, device="cuda").long()].cpu().numpy()).reshape(-1, Hkv, D)[: len(h)] * s
            # half a step, relative, or half of the least step of the block; as much again where it was scaled anew
            assert np.all(np.abs(got - x) <= 1.07 * 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * s + 1e-5)
    psd.free_pages(ctx(), table[0], table[1], ref, ws_pages, fault=fault)
    assert not ref.any() and int(fault) == 0


@pytest.mark.parametrize("D,n_beams", [(64, 3), (128, 8)])
def test_a_step_as_one_graph(D, n_beams):
    """Selection, fork, append and attention captured together: a replay is the step anew, from the logits on."""
    rng = np.random.default_rng(D)
    B, W, Hq, Hkv, V, page, L0 = 2, n_beams, 8, 2, 3000, 16, 37
    N, held, rope = B * W, 3, psd.rope_frequencies(D)
    i32 = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).cuda()  # noqa: E731
    num_pages = N * held + N + 5
    rows = [[2 * b, 2 * b + 1, 2 * B + r] for b in range(B) for r in range(b * W, (b + 1) * W)]   # two pages shared, one each
    start = dict(k=torch.from_numpy(rng.integers(0, 120, (num_pages, page, Hkv, D)).astype(np.uint8)).cuda(),
                 v=torch.from_numpy(rng.integers(0, 120, (num_pages, page, Hkv, D)).astype(np.uint8)).cuda(),
                 ke=torch.full((num_pages, 1, Hkv), 118, dtype=torch.uint8, device="cuda"),
                 ve=torch.full((num_pages, 1, Hkv), 119, dtype=torch.uint8, device="cuda"),
                 ref=i32(np.bincount(np.array(rows).ravel(), minlength=num_pages)),
                 scores=torch.from_numpy(rng.standard_normal(N).astype(np.float32)).cuda())
    now = {k: t.clone() for k, t in start.items()}
    logits = torch.zeros((N, V), device="cuda")
    qkv = torch.from_numpy(rng.standard_normal((N, (Hq + 2 * Hkv) * D)).astype(np.float32)).to(torch.bfloat16).cuda()
    q, k, v = (qkv[:, a * D: b * D].unflatten(1, (b - a, D)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    out = [now["scores"].view(B, W)] + [torch.zeros((B, W), dtype=torch.int32, device="cuda") for _ in range(2)]
    old = (i32(np.arange(N + 1) * held), i32(np.array(rows).ravel()), i32([L0] * N))
    new = (i32([0] * (N + 1)), i32([0] * (N * held)), i32([0] * N))
    cache, scales = psd.PagePools([now[x] for x in ("k", "v", "ke", "ve")]), psd.BlockScales(now["ke"], now["ve"], page)
    ws_pages, ws_beam = psd.pages_workspace(cache, N, "cuda"), psd.beam_workspace(ctx(), N, W, W, "cuda")
    plan = psd.plan_multi_token(psd.HostTable(np.arange(N + 1) * held, np.arange(N * held), [L0 + 1 - 32] * N, page), np.arange(N + 1), Hq, Hkv)
    ws = psd.multi_token_workspace(ctx(), plan, D, "cuda")
    q_rot, o, lse = torch.empty((N, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.empty((N, Hq, D), device="cuda"), torch.empty((N, Hq), device="cuda")
    q_indptr, fault = i32(np.arange(N + 1)), i32([0])

    def step():
        psd.beam_select(ctx(), logits, now["scores"], *out, ws_beam, beams=W, fault=fault)
        psd.fork_pages(ctx(), cache, out[1].view(-1), page_indptr=old[0], page_indices=old[1], kv_len=old[2], page_size=page, room=1,
                       ref_count=now["ref"], new_indptr=new[0], new_indices=new[1], new_len=new[2], workspace=ws_pages, fault=fault)
        psd.append_tokens(ctx(), q, k, v, q_rot, q_indptr=q_indptr, kv_len=new[2], page_indptr=new[0], page_indices=new[1],
                          k_pool=now["k"], v_pool=now["v"], rope=rope, neox=True, scales=scales, fault=fault)
        psd.multi_token_decode(ctx(), psd.multi_token_args(q_rot, now["k"], now["v"], new[1], sm_scale=D ** -0.5, scales=scales), plan,
                               o, lse, ws)

    def again(seed):
        for x, t in start.items():
            now[x].copy_(t)
        logits.copy_(torch.from_numpy(np.random.default_rng(seed).standard_normal((N, V)).astype(np.float32)))

    def result():
        torch.cuda.synchronize()
        assert int(fault) == 0 and psd.check_device_error(ctx(), ws) == 0
        return [t.clone() for t in (*out, *new, *now.values(), q_rot, o, lse)]

    want = []
    for seed in (1, 2, 3):
        again(seed)
        step()
        want.append(result())
    assert not torch.equal(want[0][1], want[1][1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for seed in (3, 1, 2):
        again(seed)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(result(), want[seed - 1]))
