"""The operators of beam search over a cache of 8-bit blocks, as measured cases: plain torch forms and the calls a
user makes.

A step of beam search over a paged cache whose e4m3 blocks (some tokens of one KV head) each have a power of two as
their scale: ``append_tokens`` with ``scales`` rotates the new tokens and writes them into their blocks, which may
have to be scaled anew; ``multi_token_decode`` with ``scales`` attends over the cache; ``beam_select`` takes the best
continuations over a request's beams and the vocabulary; ``fork_pages`` gives each its parent's pages, copying what
two would write to, and ``compact_pages`` moves the live pages of a pool to its front.  A case's "op" says which of
them it runs.
"""
import math
import zlib

import numpy as np
import torch

own = False

LN2 = math.log(2.0)
_CTX = []


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of a batch: each token joins a block that is part full, or opens one.
        {"name": "append_step", "op": "append", "batch": 32, "new_lo": 1, "new_hi": 1, "ctx_lo": 100, "ctx_hi": 1024,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "block": 16, "rot": 128, "neox": True},
        # Ragged prompts entering the cache together.
        {"name": "append_prompts", "op": "append", "batch": 7, "new_lo": 500, "new_hi": 2100, "ctx_lo": 0,
         "ctx_hi": 700, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "block": 16, "rot": 128, "neox": True},
        # The smallest attention: four beams of a toy model.
        {"name": "attend_small", "op": "attend", "batch": 4, "new_lo": 1, "new_hi": 1, "ctx_lo": 60, "ctx_hi": 400,
         "Hq": 8, "Hkv": 2, "D": 64, "page": 16, "block": 16, "tree": False, "out": "bf16"},
        # A decode step over the flat decode configuration's contexts.
        {"name": "attend_step", "op": "attend", "batch": 32, "new_lo": 1, "new_hi": 1, "ctx_lo": 512, "ctx_hi": 4096,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "block": 16, "tree": False, "out": "bf16"},
        # Few requests over long caches, f32 outputs: the work has to be split along the cache.
        {"name": "attend_long", "op": "attend", "batch": 3, "new_lo": 1, "new_hi": 1, "ctx_lo": 20000, "ctx_hi": 65536,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "block": 64, "tree": False, "out": "f32"},
        # A chunk of a prompt over what earlier chunks left: the compute-bound end.
        {"name": "attend_chunk", "op": "attend", "batch": 1, "new_lo": 2048, "new_hi": 2048, "ctx_lo": 4096,
         "ctx_hi": 4096, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "block": 16, "tree": False, "out": "bf16"},
        # One request's beams, twice as many continuations as beams.
        {"name": "select_small", "op": "select", "batch": 1, "beams": 4, "vocab": 32000, "k": 8, "type": "f32",
         "finished": 0.0},
        # A batch of requests on a vocabulary whose rows are not aligned, some beams at their end.
        {"name": "select_batch", "op": "select", "batch": 16, "beams": 8, "vocab": 98305, "k": 16, "type": "f32",
         "finished": 0.2},
        # 16-bit logits, as a projection leaves them: many are equal.
        {"name": "select_half", "op": "select", "batch": 48, "beams": 5, "vocab": 131072, "k": 10, "type": "bf16",
         "finished": 0.1},
        # One request's beams go on: four layers' K and V.
        {"name": "fork_small", "op": "fork", "batch": 1, "beams": 4, "ctx_lo": 300, "ctx_hi": 900, "Hkv": 8, "D": 128,
         "page": 16, "layers": 4, "room": 1, "none": 0.0},
        # A batch of requests with eight beams each: sixteen layers' K and V.
        {"name": "fork_batch", "op": "fork", "batch": 16, "beams": 8, "ctx_lo": 512, "ctx_hi": 4096, "Hkv": 8,
         "D": 128, "page": 16, "layers": 16, "room": 1, "none": 0.05},
        # A pool of which two thirds are live.
        {"name": "compact_pool", "op": "compact", "pages": 8192, "live": 0.66, "Hkv": 8, "D": 128, "page": 16,
         "layers": 4, "requests": 48},
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "select", "select", "fork", "fork", "compact"])
    if op == "select":
        kind = rng.choice(["f32", "f32", "bf16", "f16"])
        beams = _spread(rng, 1, 16)
        vocab = _spread(rng, 500, 131072)
        return {"op": op, "batch": _spread(rng, 1, max(1, min(64, 12000000 // (beams * vocab)))), "beams": beams,
                "vocab": vocab, "k": rng.choice([beams, 2 * beams, rng.randint(1, 2 * beams)]), "type": kind,
                "finished": rng.choice([0.0, 0.2, 0.6])}
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64])
    if op == "compact":
        layers = rng.randint(1, 4)
        return {"op": op, "pages": _spread(rng, 20, 8192 * 16 // page), "live": rng.uniform(0.1, 1.0), "Hkv": Hkv,
                "D": D, "page": page, "layers": layers, "requests": _spread(rng, 1, 64)}
    if op == "fork":
        beams = _spread(rng, 1, 12)
        hi = _spread(rng, 20, 3000)
        return {"op": op, "batch": _spread(rng, 1, max(1, 100 // beams)), "beams": beams, "ctx_lo": hi // 5,
                "ctx_hi": hi, "Hkv": Hkv, "D": D, "page": page, "layers": rng.randint(1, 16),
                "room": rng.choice([0, 1, 1, 1, 5, 40]), "none": rng.choice([0.0, 0.1, 0.5])}
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    block = rng.choice([16, 32, 64])
    page = max(page, block)
    if op == "append":
        new = _spread(rng, 1, 2000)
        return {"op": op, "batch": _spread(rng, 1, max(1, 8000 // new)), "new_lo": max(1, new // 3), "new_hi": new,
                "ctx_lo": 0, "ctx_hi": _spread(rng, 1, 600), "Hq": Hkv * G, "Hkv": Hkv, "D": D, "page": page,
                "block": block, "rot": rng.choice([16, 32, D // 2, D]), "neox": rng.random() < 0.5}
    kind = rng.choice(["single", "single", "drafts", "tree", "prompt"])
    out = rng.choice(["bf16", "bf16", "f32"])
    if kind == "prompt":
        new = _spread(rng, 100, 1500)
        return {"op": op, "batch": _spread(rng, 1, max(1, 1500 // new)), "new_lo": max(1, new // 2), "new_hi": new,
                "ctx_lo": 0, "ctx_hi": _spread(rng, 1, 4096), "Hq": Hkv * G, "Hkv": Hkv, "D": D, "page": page,
                "block": block, "tree": False, "out": out}
    hi = {"single": 1, "drafts": rng.randint(2, 16), "tree": rng.randint(4, 64)}[kind]
    batch = _spread(rng, 1, 64)
    ctx = _spread(rng, 50, min(65536, 200000 // batch))
    return {"op": op, "batch": batch, "new_lo": 1, "new_hi": hi, "ctx_lo": rng.choice([0, ctx // 4, ctx // 2]),
            "ctx_hi": ctx, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "page": page, "block": block, "tree": kind == "tree",
            "out": out}


# --------------------------------------------------------------------------------------------------- inputs
def _shapes(case):
    """The generator of a case's ragged lengths: they are the case's own, whatever the seed."""
    return np.random.default_rng(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))


def _lengths(case):
    rng = _shapes(case)
    n = rng.integers(case["new_lo"], case["new_hi"] + 1, case["batch"])
    before = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, case["batch"])
    return n.astype(np.int64), (n + before).astype(np.int64)


def _table(case, rng, total):
    """A page table whose pages lie in random order, with a few spare pages in the pool."""
    P = case["page"]
    pages = -(-total // P)
    indptr = np.zeros(len(total) + 1, np.int64)
    np.cumsum(pages, out=indptr[1:])
    num_pages = int(indptr[-1]) + 3
    indices = rng.permutation(num_pages)[: indptr[-1]]
    return indptr, indices, total - (pages - 1) * P, num_pages


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device="cuda", dtype=dtype)


def _select_inputs(case, s, rng, gen):
    B, W, V = case["batch"], case["beams"], case["vocab"]
    kind = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[case["type"]]
    x = 2.5 * torch.randn((B * W, V), generator=gen, device="cuda", dtype=torch.float32)
    # a beam's logits lean on its sibling's; masked tokens are -inf
    x[:, rng.integers(0, V, max(1, V // 50))] = -math.inf
    s["logits"] = x.to(kind)
    scores = -3.0 * torch.rand(B * W, generator=gen, device="cuda", dtype=torch.float32) - 5.0
    scores[_dev(rng.random(B * W) < 0.05, torch.bool)] = -math.inf      # a beam that was never filled
    s["scores"] = scores
    s["finished"] = _dev(rng.random(B * W) < case["finished"], torch.uint8) if case["finished"] else None
    s["pad"] = 2


def _fork_inputs(case, s, rng, gen):
    """Beams that share their prompt's pages and have some of their own; each goes on, or not, or several times."""
    B, W, P = case["batch"], case["beams"], case["page"]
    shape = _shapes(case)
    prompt = shape.integers(case["ctx_lo"], case["ctx_hi"] + 1, B)
    made = shape.integers(0, 3 * P, B)                               # tokens since the prompt
    parents, kv_len = [], np.repeat(prompt + made, W)
    shared = prompt // P                                             # a prompt's full pages
    each = -(-(prompt + made) // P) - shared                         # a beam's own
    room = -(-(prompt + made + case["room"]) // P)
    num_pages = int((shared + W * (each + 3 + case["room"] // P)).sum()) + 16
    ids = rng.permutation(num_pages)
    rows, at = [], 0
    for b in range(B):
        common = ids[at: at + shared[b]]
        at += shared[b]
        for _ in range(W):
            rows.append(np.concatenate([common, ids[at: at + each[b]]]))
            at += each[b]
        pick = b * W + rng.integers(0, W, W)
        parents.append(np.where(shape.random(W) < case["none"], -1, pick))
    indptr = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
    indices = np.concatenate(rows)
    s["parents_host"], s["kv_len_host"], s["indptr_host"], s["indices_host"] = np.concatenate(parents), kv_len, indptr, indices
    s["ref_host"] = np.bincount(indices, minlength=num_pages)
    s["parents"], s["kv_len"] = _dev(s["parents_host"], torch.int32), _dev(kv_len, torch.int32)
    s["indptr"], s["indices"] = _dev(indptr, torch.int32), _dev(indices, torch.int32)
    s["ref"] = _dev(s["ref_host"], torch.int32)
    s["new_ref"] = torch.zeros_like(s["ref"])
    s["new_indptr"] = torch.zeros(B * W + 1, dtype=torch.int32, device="cuda")
    s["new_indices"] = torch.zeros(int((room * W).sum()), dtype=torch.int32, device="cuda")
    s["new_len"] = torch.zeros(B * W, dtype=torch.int32, device="cuda")
    s["pools"] = _pools(case, num_pages, gen)


def _pools(case, num_pages, gen):
    """Codes of K and V, layer by layer: here only bytes to be moved."""
    shape = (num_pages, case["page"], case["Hkv"], case["D"])
    return [torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)
            for _ in range(2 * case["layers"])]


def _compact_inputs(case, s, rng, gen):
    n = case["pages"]
    live = np.flatnonzero(_shapes(case).random(n) < case["live"])
    order = rng.permutation(live)
    cuts = np.sort(rng.integers(0, len(order) + 1, case["requests"] - 1)) if case["requests"] > 1 else []
    rows = [np.concatenate([order[:3], r]) for r in np.split(order, cuts)]   # all share the first pages
    s["indices_host"] = np.concatenate(rows)
    s["ref_host"] = np.bincount(s["indices_host"], minlength=n)
    s["indices"], s["ref"] = _dev(s["indices_host"], torch.int32), _dev(s["ref_host"], torch.int32)
    s["new_indices"], s["new_ref"] = torch.zeros_like(s["indices"]), torch.zeros_like(s["ref"])
    s["num_live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["pools"] = _pools(case, n, gen)


def _cache_inputs(case, s, rng, gen):
    n, total = _lengths(case)
    q_indptr = np.zeros(len(n) + 1, np.int64)
    np.cumsum(n, out=q_indptr[1:])
    page_indptr, page_indices, last, num_pages = _table(case, rng, total)
    T, Hq, Hkv, D, P = int(q_indptr[-1]), case["Hq"], case["Hkv"], case["D"], case["page"]
    s |= {"n": n, "total": total, "q_indptr_host": q_indptr, "page_indptr_host": page_indptr,
          "page_indices_host": page_indices, "last_host": last,
          "q_indptr": _dev(q_indptr, torch.int32), "kv_len": _dev(total, torch.int32),
          "page_indptr": _dev(page_indptr, torch.int32), "page_indices": _dev(page_indices, torch.int32)}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    def pool():
        """Blocks of differing size, quantised with the power of two that just holds each block's largest value."""
        x = normal(num_pages, P // case["block"], case["block"], Hkv, D)
        x = x * torch.exp(0.7 * normal(num_pages, P // case["block"], 1, Hkv, 1))
        top = x.abs().amax((2, 4), keepdim=True)
        e = torch.ceil(torch.log2(top.double() / 448)).float()
        codes = (x / torch.exp2(e)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return codes.view(num_pages, P, Hkv, D), (e[:, :, 0, :, 0] + 127).to(torch.uint8).contiguous()

    (s["k_pool"], s["k_scales"]), (s["v_pool"], s["v_scales"]) = pool(), pool()
    if case["op"] == "append":
        # q, k and v are views of one fused projection's output
        qkv = normal(T, (Hq + 2 * Hkv) * D).to(torch.bfloat16)
        s["q"] = qkv[:, : Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        s["inv_freq"] = 10000.0 ** (-2.0 * np.arange(case["rot"] // 2) / case["rot"])
        return
    s["q"] = normal(T, Hq, D).to(torch.bfloat16)
    s["scale"] = D ** -0.5
    s["tree"] = None
    if case["tree"]:
        masks = []
        for m in n:
            of = []
            for i in range(int(m)):
                of.append((of[int(rng.integers(i))] if i else 0) | (1 << i))
            masks += of
        s["tree"] = _dev(np.array([x - (1 << 64) if x >> 63 else x for x in masks], np.int64), torch.int64)


def _inputs(case, seed):
    """The case's inputs, from the seed alone."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    make = {"select": _select_inputs, "fork": _fork_inputs, "compact": _compact_inputs}.get(case["op"], _cache_inputs)
    make(case, s, rng, gen)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import paged_split_kv_decode_gb300 as psd
        if not _CTX:
            _CTX.append(psd.Context())
        s["psd"], s["ctx"] = psd, _CTX[0]
        s["fault"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] in ("append", "attend"):
            s["scales"] = psd.BlockScales(s["k_scales"], s["v_scales"], case["block"])
        if case["op"] == "append":
            s["rope"] = psd.RopeFrequencies(s["inv_freq"])
        elif case["op"] == "attend":
            table = psd.HostTable(s["page_indptr_host"], s["page_indices_host"], s["last_host"], case["page"])
            s["plan"] = psd.plan_multi_token(table, s["q_indptr_host"], case["Hq"], case["Hkv"])
            s["workspace"] = psd.multi_token_workspace(s["ctx"], s["plan"], case["D"], "cuda")
        elif case["op"] == "select":
            s["workspace"] = psd.beam_workspace(s["ctx"], case["batch"] * case["beams"], case["beams"], case["k"],
                                                "cuda")
        else:
            s["pages"] = psd.PagePools(s["pools"])
            s["workspace"] = psd.pages_workspace(s["pages"], case["batch"] * case["beams"] if case["op"] == "fork" else 0,
                                                 "cuda")
    return s


# ------------------------------------------------------------------------------------------------- plain forms
def _append_plain(s):
    c = s["case"]
    P, r, N, Hkv, D = c["page"], c["rot"], c["block"], c["Hkv"], c["D"]
    q_indptr, kv_len = s["q_indptr"].long(), s["kv_len"].long()
    T = s["q"].shape[0]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(q_indptr, t, right=True) - 1
    at = kv_len[b] - (q_indptr[b + 1] - t)
    before = (kv_len[b] - (q_indptr[b + 1] - q_indptr[b]))
    page = s["page_indices"].long()[s["page_indptr"].long()[b] + at // P]
    angle = at.double()[:, None] * torch.from_numpy(s["inv_freq"]).to("cuda")[None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotate(x):
        x = x.float()
        a, y = (x[..., : r // 2], x[..., r // 2: r]) if c["neox"] else (x[..., 0:r:2], x[..., 1:r:2])
        u, w = a * cos - y * sin, y * cos + a * sin
        turned = torch.cat([u, w], -1) if c["neox"] else torch.stack([u, w], -1).flatten(-2)
        return torch.cat([turned, x[..., r:]], -1)

    # The blocks that get tokens, and how many older ones each holds.
    block = (page * P + at % P) // N                                   # of the pool, a token
    blocks = s["k_scales"].shape[0] * (P // N)
    touched = torch.zeros(blocks, dtype=torch.bool, device="cuda")
    touched[block] = True
    held = torch.zeros(blocks, dtype=torch.int64, device="cuda")
    held[block] = (before - at // N * N).clamp(min=0)
    older = held > 0
    in_use = torch.arange(N, device="cuda")[None] < held[:, None]
    index = block[:, None].expand(T, Hkv)

    def put(pool, scales, x):
        top = torch.zeros((blocks, Hkv), dtype=torch.float32, device="cuda")
        top.scatter_reduce_(0, index, x.abs().amax(-1), "amax")
        # the least power of two that holds it
        m, e = torch.frexp(top / 448)
        e = torch.where(m == 0.5, e - 1, e).clamp(-32, 127)
        e = torch.where(top == 0, -32, e) + 127
        had = scales.view(blocks, Hkv).int()
        e = torch.where(older[:, None], torch.maximum(e, had), e)
        e = torch.where(touched[:, None], e, had)
        codes = pool.view(blocks, N, Hkv, D)
        down = torch.exp2((had - e).float())[:, None, :, None]
        again = in_use[:, :, None, None] & (e > had)[:, None, :, None]
        old = codes.view(torch.float8_e4m3fn).float() * down
        codes.copy_(torch.where(again, old.to(torch.float8_e4m3fn).view(torch.uint8), codes))
        scales.view(blocks, Hkv).copy_(e.to(torch.uint8))
        y = x * torch.exp2((127 - e[block]).float())[..., None]
        pool.view(-1, Hkv, D)[page * P + at % P] = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    put(s["k_pool"], s["k_scales"], rotate(s["k"]))
    put(s["v_pool"], s["v_scales"], s["v"].float())
    return rotate(s["q"]).to(torch.bfloat16)


def _rows(pool, scales, slot, block):
    """Pool rows in 32 bits."""
    x = pool.view(-1, *pool.shape[2:])[slot].view(torch.float8_e4m3fn).float()
    return x * torch.exp2(scales.view(-1, scales.shape[-1])[slot // block].float() - 127)[..., None]


def _attend_group(s, which, o, lse):
    """The requests `which` (host indices) padded to one batch."""
    if not len(which):
        return
    c = s["case"]
    P, Hkv, D = c["page"], c["Hkv"], c["D"]
    G = c["Hq"] // Hkv
    n_most, L_most = int(s["n"][which].max()), int(s["total"][which].max())
    b = _dev(which, torch.int64)
    q_indptr, kv_len = s["q_indptr"].long(), s["kv_len"].long()
    n, L = q_indptr[b + 1] - q_indptr[b], kv_len[b]
    key = torch.minimum(torch.arange(L_most, device="cuda")[None], L[:, None] - 1)
    slot = s["page_indices"].long()[s["page_indptr"].long()[b][:, None] + key // P] * P + key % P
    K, V = _rows(s["k_pool"], s["k_scales"], slot, c["block"]), _rows(s["v_pool"], s["v_scales"], slot, c["block"])
    i = torch.arange(n_most, device="cuda")[None]
    tok = q_indptr[b][:, None] + torch.minimum(i, n[:, None] - 1)
    Q = s["q"][tok].float().view(len(which), n_most, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(len(which), Hkv, -1, D)
    S = Q @ K.permute(0, 2, 3, 1)                                           # [g, Hkv, n G, L]
    j = torch.arange(L_most, device="cuda")[None, None]
    start = (L - n)[:, None, None]
    if s["tree"] is None:
        seen = j <= start + i[..., None]
    else:
        bit = (j - start).clamp(0, 63)
        seen = (j < start) | ((s["tree"][tok][..., None] >> bit) & 1).bool()
    seen = seen & (j < L[:, None, None])
    seen = seen[:, None, :, None].expand(-1, 1, -1, G, -1).reshape(len(which), 1, -1, L_most)
    S = (S * s["scale"]).masked_fill(~seen, -math.inf)
    m = S.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (S - m).exp()
    l = p.sum(-1, keepdim=True)
    out = (p @ V.permute(0, 2, 1, 3)) / l.clamp(min=1e-30)
    low = (m + l.log()) / LN2
    live = i < n[:, None]
    o[tok[live]] = out.view(-1, Hkv, n_most, G, D).permute(0, 2, 1, 3, 4).reshape(-1, n_most, c["Hq"], D)[live].to(o.dtype)
    lse[tok[live]] = low.view(-1, Hkv, n_most, G).permute(0, 2, 1, 3).reshape(-1, n_most, c["Hq"])[live]


def _attend_plain(s, o, lse):
    short = s["n"] <= 64
    _attend_group(s, np.flatnonzero(short), o, lse)
    _attend_group(s, np.flatnonzero(~short), o, lse)


def _select_plain(s, scores, rows, tokens):
    c = s["case"]
    B, W, V, k = c["batch"], c["beams"], c["vocab"], c["k"]
    x = s["logits"].double()
    low = x.amax(-1, keepdim=True)
    v = x - low - (x - low).exp().sum(-1, keepdim=True).log() + s["scores"].double()[:, None]
    if s["finished"] is not None:
        done = s["finished"].bool()[:, None]
        pad = torch.arange(V, device="cuda")[None] == s["pad"]
        v = torch.where(done, torch.where(pad, s["scores"].double()[:, None], -math.inf), v)
    v = v.view(B, W * V)
    most = min(k, W * V)
    least = v.topk(most, -1).values[:, -1:]
    # of those that equal the last one taken, the first in order
    more, same = v > least, v == least
    take = more | (same & (same.cumsum(-1) <= most - more.sum(-1, keepdim=True)))
    order = torch.arange(W * V, 0, -1, device="cuda", dtype=torch.int32)[None].expand(B, -1)
    at = W * V - torch.where(take, order, 0).topk(most, -1).values.long()
    best, by = v.gather(-1, at).sort(dim=-1, descending=True, stable=True)
    at = at.gather(-1, by)
    there = best > -math.inf
    scores.fill_(-math.inf)
    rows.fill_(-1)
    tokens.fill_(-1)
    scores[:, :most] = best.float()
    rows[:, :most] = torch.where(there, at // V + W * torch.arange(B, device="cuda")[:, None], -1).int()
    tokens[:, :most] = torch.where(there, at % V, -1).int()


def _fork_plain(s):
    c = s["case"]
    P, room = c["page"], c["room"]
    parent, indptr, old = s["parents"].long(), s["indptr"].long(), s["indices"].long()
    N, pages, cap = parent.shape[0], s["ref"].shape[0], s["new_indices"].shape[0]
    alive, of = parent >= 0, parent.clamp(min=0)
    length = torch.where(alive, s["kv_len"].long()[of], 0)
    full, tail = length // P, (length % P > 0) & alive
    want = torch.where(alive, (length + room + P - 1) // P, 0)
    new_indptr = torch.cat([want.new_zeros(1), want.cumsum(0)])
    ref = s["ref"].clone()
    ref.index_add_(0, old, torch.full_like(s["indices"], -1))                # the old requests go
    page = old[(indptr[of] + full).clamp(max=old.shape[0] - 1)]              # a child's last page, part full
    i = torch.arange(N, device="cuda")
    if room:
        first = torch.full((pages + 1,), N, device="cuda")
        first.scatter_reduce_(0, torch.where(tail, page, pages), i, "amin")
        kept = tail & (ref[page] == 0) & (first[page] == i)
    else:
        kept = tail
    j = torch.arange(cap, device="cuda")
    of_new = (torch.searchsorted(new_indptr, j, right=True) - 1).clamp(max=N - 1)
    off, valid = j - new_indptr[of_new], j < new_indptr[N]
    stays = valid & ((off < full[of_new]) | ((off == full[of_new]) & kept[of_new]))
    got = old[torch.where(stays, indptr[of[of_new]] + off, 0)]
    ref.index_add_(0, got, stays.int())
    free = ref == 0
    ranked = torch.zeros(pages + 1, dtype=torch.int64, device="cuda")
    ranked.scatter_(0, torch.where(free, free.cumsum(0) - 1, pages), torch.arange(pages, device="cuda"))
    fresh = valid & ~stays
    new = ranked[torch.where(fresh, fresh.cumsum(0) - 1, 0).clamp(max=pages)]
    ref.index_add_(0, torch.where(fresh, new, 0), fresh.int())
    s["new_indices"].copy_(torch.where(valid, torch.where(stays, got, new), s["new_indices"]))
    s["new_indptr"].copy_(new_indptr)
    s["new_len"].copy_(torch.where(alive, length + room, 0))
    s["new_ref"].copy_(ref)
    copied = (tail & ~kept).nonzero()[:, 0]
    src, dst = page[copied], s["new_indices"].long()[new_indptr[copied] + full[copied]]
    [p.index_copy_(0, dst, p[src]) for p in s["pools"]]


def _compact_plain(s):
    live = s["ref"] > 0
    n = live.sum()
    at = torch.arange(live.shape[0], device="cuda")
    holes = (~live & (at < n)).nonzero()[:, 0]
    moved = (live & (at >= n)).nonzero()[:, 0]
    to = at.clone()
    to[moved] = holes
    s["num_live"].copy_(n)
    s["new_indices"].copy_(to[s["indices"].long()])
    s["new_ref"].zero_()
    s["new_ref"][to[live]] = s["ref"][live]
    [p.index_copy_(0, holes, p[moved]) for p in s["pools"]]


def run(s):
    c = s["case"]
    if c["op"] == "append":
        if own:
            q_out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
            s["psd"].append_tokens(s["ctx"], s["q"], s["k"], s["v"], q_out, q_indptr=s["q_indptr"], kv_len=s["kv_len"],
                                   page_indptr=s["page_indptr"], page_indices=s["page_indices"], k_pool=s["k_pool"],
                                   v_pool=s["v_pool"], rope=s["rope"], neox=c["neox"], scales=s["scales"],
                                   fault=s["fault"])
        else:
            q_out = _append_plain(s)
        return (q_out, s["k_pool"].view(torch.float8_e4m3fn), s["v_pool"].view(torch.float8_e4m3fn), s["k_scales"],
                s["v_scales"])
    if c["op"] == "attend":
        o = torch.empty(s["q"].shape, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device="cuda")
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
        if own:
            args = s["psd"].multi_token_args(s["q"], s["k_pool"], s["v_pool"], s["page_indices"],
                                             sm_scale=s["scale"], tree_mask=s["tree"], scales=s["scales"])
            s["psd"].multi_token_decode(s["ctx"], args, s["plan"], o, lse, s["workspace"])
        else:
            _attend_plain(s, o, lse)
        return o, lse
    if c["op"] == "select":
        scores = torch.empty((c["batch"], c["k"]), dtype=torch.float32, device="cuda")
        rows = torch.empty((c["batch"], c["k"]), dtype=torch.int32, device="cuda")
        tokens = torch.empty((c["batch"], c["k"]), dtype=torch.int32, device="cuda")
        if own:
            s["psd"].beam_select(s["ctx"], s["logits"], s["scores"], scores, rows, tokens, s["workspace"],
                                 beams=c["beams"], finished=s["finished"], pad_token=s["pad"], fault=s["fault"])
        else:
            _select_plain(s, scores, rows, tokens)
        return scores, rows, tokens
    if c["op"] == "fork":
        if own:
            s["psd"].fork_pages(s["ctx"], s["pages"], s["parents"], page_indptr=s["indptr"], page_indices=s["indices"],
                                kv_len=s["kv_len"], page_size=c["page"], room=c["room"], ref_count=s["ref"],
                                new_ref_count=s["new_ref"], new_indptr=s["new_indptr"], new_indices=s["new_indices"],
                                new_len=s["new_len"], workspace=s["workspace"], fault=s["fault"])
        else:
            _fork_plain(s)
        return s["new_indptr"], s["new_indices"], s["new_len"], s["new_ref"], s["pools"]
    if own:
        s["psd"].compact_pages(s["ctx"], s["pages"], s["indices"], s["ref"], new_indices=s["new_indices"],
                               new_ref_count=s["new_ref"], num_live=s["num_live"], workspace=s["workspace"],
                               fault=s["fault"])
    else:
        _compact_plain(s)
    return s["num_live"], s["new_indices"], s["new_ref"], s["pools"]


# ------------------------------------------------------------------------------------------------------- work
def work(case):
    """What one pass cannot do without."""
    if case["op"] == "select":
        rows = case["batch"] * case["beams"]
        size = 4 if case["type"] == "f32" else 2
        read = rows * (1 - case["finished"])
        return {"bytes": int(read * case["vocab"] * size + rows * 5 + case["batch"] * case["k"] * 12),
                "flops": int(read * case["vocab"] * 4)}
    if case["op"] in ("fork", "compact"):
        a_page = case["page"] * case["Hkv"] * case["D"] * 2 * case["layers"]
        if case["op"] == "compact":
            n, live = case["pages"], int((_shapes(case).random(case["pages"]) < case["live"]).sum())
            # of the live pages, as many move as there are holes in front
            moves = live - int((_shapes(case).random(case["pages"]) < case["live"])[:live].sum())
            return {"bytes": int(2 * moves * a_page + 8 * n + 8 * live), "flops": int(n + live)}
        shape = _shapes(case)
        prompt = shape.integers(case["ctx_lo"], case["ctx_hi"] + 1, case["batch"])
        made = shape.integers(0, 3 * case["page"], case["batch"])
        W, P = case["beams"], case["page"]
        part = int((((prompt + made) % P) > 0).sum()) if case["room"] else 0
        # of W children that pick W parents alike, W (1 - 1/W)^W find their page taken
        copies = part * W * (1 - case["none"]) * (1 - 1 / W) ** W
        entries = W * int((-(-(prompt + made) // P)).sum())
        return {"bytes": int(2 * copies * a_page + 8 * entries + 8 * (prompt // P).sum()), "flops": int(2 * entries)}
    new, total = _lengths(case)
    n, keys = int(new.sum()), int(total.sum())
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        return {"bytes": n * D * (4 * Hq + 2 * Hkv * 3), "flops": n * (Hq + Hkv) * case["rot"] * 3}
    pairs = int((new * (total - new) + new * (new + 1) // 2).sum())
    return {"bytes": keys * Hkv * (D + 1 / case["block"]) * 2 + n * Hq * (D * (2 + (2 if case["out"] == "bf16" else 4)) + 4),
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The definitions, request by request, in 64 bits."""
    s = _inputs(case, seed)
    return {"append": _append_exact, "attend": _attend_exact, "select": _select_exact, "fork": _fork_exact,
            "compact": _compact_exact}[case["op"]](case, s)


def _e4m3_exact(x):
    """The nearest e4m3 values (ties to even) of numbers in 64 bits, at most 448 in size."""
    x = x.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _append_exact(case, s):
    r, P, N = case["rot"], case["page"], case["block"]
    pools = [s["k_pool"].view(torch.float8_e4m3fn).double(), s["v_pool"].view(torch.float8_e4m3fn).double()]
    scales = [s["k_scales"].clone(), s["v_scales"].clone()]
    q_out = s["q"].double().clone()
    f = torch.from_numpy(s["inv_freq"]).to("cuda")
    pairs = torch.arange(r // 2, device="cuda")
    a, b = (pairs, pairs + r // 2) if case["neox"] else (2 * pairs, 2 * pairs + 1)

    def turn(x, pos):
        z = torch.polar(torch.ones_like(pos * f), pos * f)[:, None]
        w = torch.complex(x[..., a], x[..., b]) * z
        x = x.clone()
        x[..., a], x[..., b] = w.real, w.imag
        return x

    for m in range(case["batch"]):
        lo, hi = int(s["q_indptr_host"][m]), int(s["q_indptr_host"][m + 1])
        L = int(s["total"][m])
        start = L - (hi - lo)
        at = torch.arange(start, L, device="cuda")
        pos = at.double()[:, None]
        pages = s["page_indices_host"][s["page_indptr_host"][m]: s["page_indptr_host"][m + 1]]
        q_out[lo:hi] = turn(s["q"][lo:hi].double(), pos)
        for x, pool, e in ((turn(s["k"][lo:hi].double(), pos), pools[0], scales[0]), (s["v"][lo:hi].double(), pools[1], scales[1])):
            # all blocks of the request that hold new tokens, padded to whole blocks with zeros
            first, last = start // N, (L - 1) // N
            rows = torch.zeros((last - first + 1) * N, *x.shape[1:], dtype=torch.float64, device="cuda")
            rows[start - first * N: L - first * N] = x
            rows = rows.view(last - first + 1, N, *x.shape[1:])
            top = rows.abs().amax((1, 3))
            want = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)), -32.0).clamp(min=-32.0) + 127
            k = np.arange(first, last + 1)
            page, sub = _dev(pages[k * N // P], torch.int64), _dev(k * N % P // N, torch.int64)
            if start % N:
                had = e[page[0], sub[0]].double()
                want[0] = torch.maximum(want[0], had)
                j0 = int(sub[0]) * N
                older = pool[page[0], j0: j0 + start % N] * torch.exp2(had - want[0])[None, :, None]
                pool[page[0], j0: j0 + start % N] = _e4m3_exact(older)
            e[page, sub] = want.to(torch.uint8)
            y = (rows * torch.exp2(127 - want)[:, None, :, None]).clamp(-448.0, 448.0).flatten(0, 1)[start - first * N: L - first * N]
            pool[_dev(pages[np.arange(start, L) // P], torch.int64), at % P] = y
    return q_out, pools[0], pools[1], scales[0], scales[1]


def _attend_exact(case, s):
    Hq, Hkv, D, N = case["Hq"], case["Hkv"], case["D"], case["block"]
    G = Hq // Hkv
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")

    def values(pool, scales, pages, L):
        x = pool[pages].view(torch.float8_e4m3fn).double().flatten(0, 1)
        return (x * torch.pow(2.0, scales[pages].double() - 127).flatten(0, 1).repeat_interleave(N, 0)[..., None])[:L]

    for m in range(case["batch"]):
        lo, hi, L = int(s["q_indptr_host"][m]), int(s["q_indptr_host"][m + 1]), int(s["total"][m])
        n = hi - lo
        pages = _dev(s["page_indices_host"][s["page_indptr_host"][m]: s["page_indptr_host"][m + 1]], torch.int64)
        K, V = values(s["k_pool"], s["k_scales"], pages, L), values(s["v_pool"], s["v_scales"], pages, L)
        hidden = torch.ones((n, L), dtype=torch.bool, device="cuda").triu(L - n + 1)
        if s["tree"] is not None:
            bits = (s["tree"][lo:hi, None] >> torch.arange(n, device="cuda")) & 1
            hidden[:, L - n:] = bits == 0
        for h in range(Hq):
            t = (s["q"][lo:hi, h].double() @ K[:, h // G].T) * s["scale"]
            t.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(t, -1)
            t = torch.where(z.isfinite()[:, None], torch.exp(t - z[:, None]), 0.0)
            o[lo:hi, h], lse[lo:hi, h] = t @ V[:, h // G], z / LN2
    return o, lse


def _select_exact(case, s):
    B, W, V, k = case["batch"], case["beams"], case["vocab"], case["k"]
    scores = torch.full((B, k), -math.inf, dtype=torch.float64, device="cuda")
    rows = torch.full((B, k), -1, dtype=torch.int32, device="cuda")
    tokens = torch.full((B, k), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        found = []
        for r in range(b * W, b * W + W):
            base = float(s["scores"][r])
            if s["finished"] is not None and int(s["finished"][r]):
                found.append((-base, r, s["pad"]))
                continue
            v = torch.log_softmax(s["logits"][r].double(), 0) + base
            top = torch.sort(v, descending=True, stable=True)
            found += [(-x, r, t) for x, t in zip(top.values[:k].tolist(), top.indices[:k].tolist())]
        for i, (x, r, t) in enumerate(sorted(f for f in found if f[0] < math.inf)[:k]):
            scores[b, i], rows[b, i], tokens[b, i] = -x, r, t
    return scores, rows, tokens


def _fork_exact(case, s):
    P, room = case["page"], case["room"]
    indptr, indices, ref = s["indptr_host"], s["indices_host"], s["ref_host"].copy()
    for g in indices:
        ref[g] -= 1
    gone = ref.copy()
    new, blanks, copies, taken = [], [], [], set()
    for p in s["parents_host"]:
        if p < 0:
            new.append(([], 0))
            continue
        L = int(s["kv_len_host"][p])
        row = []
        for j in range(-(-(L + room) // P)):
            g = int(indices[indptr[p] + j]) if j * P < L else -1
            if g >= 0 and room and (j + 1) * P > L:                 # part full: the new tokens go there
                if gone[g] > 0 or g in taken:
                    copies.append((g, len(new), j))
                    g = -1
                else:
                    taken.add(g)
            if g < 0:
                blanks.append((len(new), j))
            else:
                ref[g] += 1
            row.append(g)
        new.append((row, L + room))
    free = np.flatnonzero(ref == 0)
    for (i, j), g in zip(blanks, free):
        new[i][0][j] = int(g)
        ref[g] = 1
    dst = [new[i][0][j] for _, i, j in copies]
    src = [g for g, _, _ in copies]
    flat = np.concatenate([np.array(r, np.int64) for r, _ in new]) if new else np.zeros(0)
    s["new_indices"][: len(flat)] = _dev(flat, torch.int32)
    pools = [p.clone() for p in s["pools"]]
    for old, p in zip(s["pools"], pools):
        if dst:
            p[_dev(dst, torch.int64)] = old[_dev(src, torch.int64)]
    ends = np.concatenate([[0], np.cumsum([len(r) for r, _ in new])])
    return (_dev(ends, torch.int32), s["new_indices"], _dev([L for _, L in new], torch.int32), _dev(ref, torch.int32), pools)


def _compact_exact(case, s):
    ref = s["ref_host"]
    n = int((ref > 0).sum())
    holes = [g for g in range(n) if ref[g] == 0]
    to = {g: g for g in range(n)}
    to.update(zip([g for g in range(n, len(ref)) if ref[g] > 0], holes))
    new = np.zeros_like(ref)
    pools = [p.clone() for p in s["pools"]]
    for g, h in to.items():
        new[h] = max(new[h], ref[g])
    moved = [(g, h) for g, h in to.items() if g != h]
    for old, p in zip(s["pools"], pools):
        if moved:
            p[_dev([h for _, h in moved], torch.int64)] = old[_dev([g for g, _ in moved], torch.int64)]
    return (_dev([n], torch.int32), _dev([to[int(g)] for g in s["indices_host"]], torch.int32), _dev(new, torch.int32), pools)
