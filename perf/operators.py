"""The operators of a step with several new tokens a request, as measured cases: plain torch forms and the calls
a user makes.

A serving step that verifies drafted tokens, or takes a chunk of a prompt, runs three operators over the paged
cache: ``append_tokens`` rotates the new queries and keys and writes the pool rows, ``multi_token_decode`` attends
the new tokens over the cache (causally or with a draft tree's mask), and ``verify_drafts`` decides which drafts stay
and draws the next token.  A case's "op" says which of them it runs.
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
        # The smallest append: a toy model's single decode step, where the launch is all of it.
        {"name": "append_one_token", "op": "append", "batch": 4, "new_lo": 1, "new_hi": 1, "ctx_lo": 96, "ctx_hi": 400,
         "Hq": 8, "Hkv": 2, "D": 64, "page": 16, "kv": "bf16", "rot": 64, "neox": True, "scaling": "none", "shift": 0},
        # Drafted tokens of a batch going into an fp8 cache, interleaved pairs on half of the head, YaRN frequencies.
        {"name": "append_drafts_fp8", "op": "append", "batch": 32, "new_lo": 5, "new_hi": 5, "ctx_lo": 512,
         "ctx_hi": 1024, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "kv": "fp8", "rot": 64, "neox": False,
         "scaling": "yarn", "shift": 60000},
        # Ragged prompts entering the cache together (half layout, frequencies scaled by bands).
        {"name": "append_prompts", "op": "append", "batch": 7, "new_lo": 500, "new_hi": 2100, "ctx_lo": 0, "ctx_hi": 700,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "kv": "bf16", "rot": 128, "neox": True, "scaling": "bands",
         "shift": 0},
        # The smallest attention: two short requests of a toy model.
        {"name": "attend_short", "op": "attend", "batch": 2, "new_lo": 1, "new_hi": 3, "ctx_lo": 20, "ctx_hi": 100,
         "Hq": 8, "Hkv": 2, "D": 64, "page": 16, "kv": "bf16", "tree": False, "out": "bf16", "long": 0},
        # Four drafts and the last accepted token of each request, over the flat decode configuration's contexts.
        {"name": "attend_drafts", "op": "attend", "batch": 32, "new_lo": 5, "new_hi": 5, "ctx_lo": 512, "ctx_hi": 4096,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "kv": "bf16", "tree": False, "out": "bf16", "long": 0},
        # Draft trees of up to 24 nodes over an fp8 cache.
        {"name": "attend_trees_fp8", "op": "attend", "batch": 16, "new_lo": 9, "new_hi": 24, "ctx_lo": 512,
         "ctx_hi": 8192, "Hq": 32, "Hkv": 8, "D": 128, "page": 32, "kv": "fp8", "tree": True, "out": "bf16", "long": 0},
        # Single tokens over long caches, few requests: the work has to be split along the cache.  f32 outputs.
        {"name": "attend_long_single", "op": "attend", "batch": 3, "new_lo": 1, "new_hi": 1, "ctx_lo": 20000,
         "ctx_hi": 65536, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "kv": "bf16", "tree": False, "out": "f32",
         "long": 0},
        # A chunk of a long prompt over what earlier chunks left in the cache: the compute-bound end.
        {"name": "attend_prompt_chunk", "op": "attend", "batch": 1, "new_lo": 4096, "new_hi": 4096, "ctx_lo": 4096,
         "ctx_hi": 4096, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "kv": "bf16", "tree": False, "out": "bf16",
         "long": 0},
        # One prompt among requests that decode, on 64-wide heads and pages of 8 tokens.
        {"name": "attend_mixed", "op": "attend", "batch": 12, "new_lo": 1, "new_hi": 4, "ctx_lo": 100, "ctx_hi": 3000,
         "Hq": 16, "Hkv": 4, "D": 64, "page": 8, "kv": "bf16", "tree": False, "out": "bf16", "long": 1500},
        # The smallest verification.
        {"name": "verify_small", "op": "verify", "batch": 4, "drafts_lo": 1, "drafts_hi": 4, "vocab": 32000,
         "sampled": True},
        # A large batch with sampled drafts, on a vocabulary whose rows are not aligned.
        {"name": "verify_batch", "op": "verify", "batch": 128, "drafts_lo": 5, "drafts_hi": 5, "vocab": 98305,
         "sampled": True},
        # Drafts looked up in the prompt: they have no probabilities of their own.
        {"name": "verify_lookup", "op": "verify", "batch": 48, "drafts_lo": 0, "drafts_hi": 7, "vocab": 131072,
         "sampled": False},
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "verify"])
    if op == "verify":
        hi = rng.randint(1, 8)
        return {"op": op, "batch": _spread(rng, 1, 128), "drafts_lo": rng.randint(0, hi), "drafts_hi": hi,
                "vocab": _spread(rng, 1000, 131072), "sampled": rng.random() < 0.6}
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([8, 16, 24, 32, 64])
    kv = rng.choice(["bf16", "bf16", "fp8"])
    if op == "append":
        new = _spread(rng, 1, 2000)
        return {"op": op, "batch": _spread(rng, 1, max(1, 8000 // new)), "new_lo": max(1, new // 3), "new_hi": new,
                "ctx_lo": 0, "ctx_hi": _spread(rng, 1, 600), "Hq": Hkv * G, "Hkv": Hkv, "D": D, "page": page, "kv": kv,
                "rot": rng.choice([16, 32, D // 2, D]), "neox": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                "shift": rng.choice([0, 0, _spread(rng, 1000, 1000000)])}
    kind = rng.choice(["drafts", "tree", "prompt", "single"])
    out = rng.choice(["bf16", "bf16", "f32"])
    if kind == "prompt":
        new = _spread(rng, 100, 2048)
        ctx = _spread(rng, 1, 4096)
        return {"op": op, "batch": _spread(rng, 1, max(1, 2048 // new)), "new_lo": max(1, new // 2), "new_hi": new,
                "ctx_lo": 0, "ctx_hi": ctx, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "page": page, "kv": kv, "tree": False,
                "out": out, "long": 0}
    hi = {"drafts": rng.randint(2, 16), "tree": rng.randint(4, 64), "single": 1}[kind]
    batch = _spread(rng, 1, 48)
    ctx = _spread(rng, 50, min(65536, 200000 // batch))
    return {"op": op, "batch": batch, "new_lo": 1, "new_hi": hi, "ctx_lo": rng.choice([0, ctx // 4, ctx // 2]),
            "ctx_hi": ctx, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "page": page, "kv": kv, "tree": kind == "tree",
            "out": out, "long": rng.choice([0, 0, 700]) if kind == "drafts" and batch <= 12 else 0}


# --------------------------------------------------------------------------------------------------- inputs
def _rope(case):
    """(inverse frequencies in 64 bits, magnitude): the definition of each scaling."""
    r, base = case["rot"], 10000.0
    factor, original = 8.0, 8192
    i = np.arange(r // 2, dtype=np.float64)
    f = base ** (-2.0 * i / r)
    kind = case["scaling"]
    if kind == "linear":
        return f / factor, 1.0
    if kind == "ntk":
        return (base * factor ** (r / (r - 2.0))) ** (-2.0 * i / r), 1.0
    if kind == "yarn":
        dim = lambda turns: r * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), r - 1)
        keep = 1.0 - np.clip((i - lo) / (hi - lo if hi > lo else 0.001), 0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    if kind == "bands":
        turns = original * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep), 1.0
    return f, 1.0


def _shapes(case):
    """The generator of a case's ragged lengths: they are the case's own, whatever the seed."""
    return np.random.default_rng(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))


def _lengths(case):
    rng = _shapes(case)
    n = rng.integers(case["new_lo"], case["new_hi"] + 1, case["batch"])
    before = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, case["batch"])
    if case.get("long"):
        n[rng.integers(case["batch"])] = case["long"]
    if case.get("tree"):
        n = np.minimum(n, 64)
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


def _inputs(case, seed):
    """The case's inputs, from the seed alone."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": case}
    if case["op"] == "verify":
        V = case["vocab"]
        K = _shapes(case).integers(case["drafts_lo"], case["drafts_hi"] + 1, case["batch"]).astype(np.int64)
        indptr = np.zeros(case["batch"] + 1, np.int64)
        np.cumsum(K, out=indptr[1:])
        D = int(indptr[-1])
        rows = np.arange(D) + np.repeat(np.arange(case["batch"]), K)   # target row of each draft
        logits = 2.5 * normal(D + case["batch"], V)
        s["target"] = torch.softmax(logits, -1)
        near = torch.softmax(logits[_dev(rows, torch.int64)] + 0.6 * normal(D, V), -1)
        if case["sampled"]:
            c = near.double().cumsum(-1)
            u = torch.rand((D, 1), generator=gen, device="cuda", dtype=torch.float64) * c[:, -1:]
            s["tokens"] = (c <= u).sum(-1).clamp(max=V - 1).to(torch.int32)
            s["draft"] = near
        else:
            s["tokens"] = near.argmax(-1).to(torch.int32)
            s["draft"] = None
        s["uniforms"] = torch.rand(D + case["batch"], generator=gen, device="cuda", dtype=torch.float32)
        s["indptr"] = _dev(indptr, torch.int32)
        s["most"] = int(K.max()) if len(K) else 0
        return s
    n, total = _lengths(case)
    q_indptr = np.zeros(len(n) + 1, np.int64)
    np.cumsum(n, out=q_indptr[1:])
    page_indptr, page_indices, last, num_pages = _table(case, rng, total)
    T, Hq, Hkv, D, P = int(q_indptr[-1]), case["Hq"], case["Hkv"], case["D"], case["page"]
    s |= {"n": n, "total": total, "q_indptr_host": q_indptr, "page_indptr_host": page_indptr,
          "page_indices_host": page_indices, "last_host": last, "num_pages": num_pages,
          "q_indptr": _dev(q_indptr, torch.int32), "kv_len": _dev(total, torch.int32),
          "page_indptr": _dev(page_indptr, torch.int32), "page_indices": _dev(page_indices, torch.int32)}
    shape = (num_pages, P, Hkv, D)
    s["k_scale"], s["v_scale"] = (0.0625, 0.03125) if case["kv"] == "fp8" else (1.0, 1.0)

    def pool(scale):
        x = normal(*shape)
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if case["kv"] == "fp8" \
            else x.to(torch.bfloat16)

    s["k_pool"], s["v_pool"] = pool(s["k_scale"]), pool(s["v_scale"])
    if case["op"] == "append":
        # q, k and v are views of one fused projection's output.
        qkv = normal(T, (Hq + 2 * Hkv) * D).to(torch.bfloat16)
        s["q"] = qkv[:, : Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        s["inv_freq"], s["magnitude"] = _rope(case)
        # Positions of the caller's own: a cache whose early pages were given up.
        at = np.concatenate([np.arange(t - m, t) for m, t in zip(n, total)]) if T else np.zeros(0)
        s["positions"] = _dev(at + case["shift"], torch.int32) if case["shift"] else None
        return s
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
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import paged_split_kv_decode_gb300 as psd
        if not _CTX:
            _CTX.append(psd.Context())
        s["psd"], s["ctx"] = psd, _CTX[0]
        s["fault"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] == "append":
            s["rope"] = psd.RopeFrequencies(s["inv_freq"], s["magnitude"])
        elif case["op"] == "attend":
            table = psd.HostTable(s["page_indptr_host"], s["page_indices_host"], s["last_host"], case["page"])
            s["plan"] = psd.plan_multi_token(table, s["q_indptr_host"], case["Hq"], case["Hkv"])
            s["workspace"] = psd.multi_token_workspace(s["ctx"], s["plan"], case["D"], "cuda")
    return s


# ------------------------------------------------------------------------------------------------- plain forms
def _append_plain(s):
    c = s["case"]
    P, r = c["page"], c["rot"]
    q_indptr, kv_len = s["q_indptr"].long(), s["kv_len"].long()
    T = s["q"].shape[0]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(q_indptr, t, right=True) - 1
    at = kv_len[b] - (q_indptr[b + 1] - t)
    slot = s["page_indices"].long()[s["page_indptr"].long()[b] + at // P] * P + at % P
    pos = at if s["positions"] is None else s["positions"].long()
    angle = pos.double()[:, None] * torch.from_numpy(s["inv_freq"]).to("cuda")[None]
    cos = (angle.cos().float() * s["magnitude"])[:, None]
    sin = (angle.sin().float() * s["magnitude"])[:, None]

    def rotate(x):
        x = x.float()
        a, y = (x[..., : r // 2], x[..., r // 2: r]) if c["neox"] else (x[..., 0:r:2], x[..., 1:r:2])
        u, w = a * cos - y * sin, y * cos + a * sin
        turned = torch.cat([u, w], -1) if c["neox"] else torch.stack([u, w], -1).flatten(-2)
        return torch.cat([turned, x[..., r:]], -1)

    def put(pool, x, scale):
        rows = pool.view(-1, c["Hkv"], c["D"])
        if c["kv"] == "fp8":
            rows[slot] = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            rows[slot] = x.to(torch.bfloat16)

    put(s["k_pool"], rotate(s["k"]), s["k_scale"])
    put(s["v_pool"], s["v"].float(), s["v_scale"])
    return rotate(s["q"]).to(torch.bfloat16)


def _rows(pool, slot, scale):
    """Pool rows in 32 bits."""
    x = pool.view(-1, *pool.shape[2:])[slot]
    return x.view(torch.float8_e4m3fn).float() * scale if pool.dtype == torch.uint8 else x.float()


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
    K, V = _rows(s["k_pool"], slot, s["k_scale"]), _rows(s["v_pool"], slot, s["v_scale"])
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


def _verify_plain(s, accepted, tokens):
    V, B = s["case"]["vocab"], s["case"]["batch"]
    first = s["indptr"].long()
    K = first[1:] - first[:-1]
    j = torch.arange(s["most"] + 1, device="cuda")[None]
    b = torch.arange(B, device="cuda")[:, None]
    row = first[:-1, None] + b + torch.minimum(j, K[:, None])
    D = s["tokens"].shape[0]
    draft = (first[:-1, None] + j).clamp(max=max(D - 1, 0))
    tok = s["tokens"].long()[draft] if D else torch.zeros_like(draft)
    p = s["target"].view(-1)[row * V + tok].double()
    q = s["draft"].view(-1)[draft * V + tok].double() if s["draft"] is not None else torch.ones_like(p)
    ok = (s["uniforms"][row].double() * q < p) & (j < K[:, None])
    n = ok.long().cumprod(-1).sum(-1)
    at = first[:-1] + b[:, 0] + n
    w = s["target"][at].double()
    refused = (n < K)[:, None]
    if D and s["draft"] is not None:
        w = torch.where(refused, (w - s["draft"][(first[:-1] + n).clamp(max=D - 1)].double()).clamp(min=0), w)
    elif D:
        w = torch.where(refused & (torch.arange(V, device="cuda")[None] == tok.gather(1, n[:, None])), 0.0, w)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, s["target"][at].double())
    sums = w.cumsum(-1)
    # the draw's number is that of the place after the last draft
    u = s["uniforms"][first[1:] + b[:, 0]].double()[:, None] * sums[:, -1:]
    new = (sums <= u).sum(-1).clamp(max=V - 1)
    accepted.copy_(n)
    said = torch.where(j < n[:, None], tok, torch.where(j == n[:, None], new[:, None], -1))
    live = j <= K[:, None]
    tokens[row[live]] = said[live].to(torch.int32)


def run(s):
    c = s["case"]
    if c["op"] == "append":
        if own:
            q_out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
            s["psd"].append_tokens(s["ctx"], s["q"], s["k"], s["v"], q_out, q_indptr=s["q_indptr"], kv_len=s["kv_len"],
                                   page_indptr=s["page_indptr"], page_indices=s["page_indices"], k_pool=s["k_pool"],
                                   v_pool=s["v_pool"], rope=s["rope"], neox=c["neox"], positions=s["positions"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"], fault=s["fault"])
        else:
            q_out = _append_plain(s)
        if c["kv"] == "fp8":
            return q_out, s["k_pool"].view(torch.float8_e4m3fn), s["v_pool"].view(torch.float8_e4m3fn)
        return q_out, s["k_pool"], s["v_pool"]
    if c["op"] == "attend":
        o = torch.empty(s["q"].shape, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device="cuda")
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
        if own:
            args = s["psd"].multi_token_args(s["q"], s["k_pool"], s["v_pool"], s["page_indices"],
                                             sm_scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                             tree_mask=s["tree"])
            s["psd"].multi_token_decode(s["ctx"], args, s["plan"], o, lse, s["workspace"])
        else:
            _attend_plain(s, o, lse)
        return o, lse
    accepted = torch.empty(c["batch"], dtype=torch.int32, device="cuda")
    tokens = torch.empty(s["uniforms"].shape, dtype=torch.int32, device="cuda")
    if own:
        s["psd"].verify_drafts(s["ctx"], s["target"], s["draft"], s["tokens"], s["indptr"], s["uniforms"], accepted,
                               tokens, fault=s["fault"])
    else:
        _verify_plain(s, accepted, tokens)
    return accepted, tokens


# ------------------------------------------------------------------------------------------------------- work
def work(case):
    """What one pass cannot do without."""
    B = case["batch"]
    if case["op"] == "verify":
        K = (case["drafts_lo"] + case["drafts_hi"]) / 2
        rows = 2 if case["sampled"] and case["drafts_hi"] else 1
        return {"bytes": int(B * case["vocab"] * 4 * rows + B * (K + 1) * 20),
                "flops": int(B * case["vocab"] * (rows + 1))}
    new, total = _lengths(case)
    n, keys = int(new.sum()), int(total.sum())
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    kv = 1 if case["kv"] == "fp8" else 2
    if case["op"] == "append":
        return {"bytes": n * D * (4 * Hq + 2 * Hkv * (2 + kv)), "flops": n * (Hq + Hkv) * case["rot"] * 3}
    pairs = int((new * (total - new) + new * (new + 1) // 2).sum())
    return {"bytes": keys * Hkv * D * 2 * kv + n * Hq * (D * (2 + (2 if case["out"] == "bf16" else 4)) + 4),
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The definitions, request by request, in 64 bits."""
    s = _inputs(case, seed)
    if case["op"] == "append":
        return _append_exact(case, s)
    return _attend_exact(case, s) if case["op"] == "attend" else _verify_exact(case, s)


def _values(pool, scale=1.0):
    return (pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool).double() * scale


def _append_exact(case, s):
    fp8, r, P = case["kv"] == "fp8", case["rot"], case["page"]
    k_pool, v_pool = _values(s["k_pool"]), _values(s["v_pool"])
    q_out = s["q"].double().clone()
    f = torch.from_numpy(s["inv_freq"]).to("cuda")
    pairs = torch.arange(r // 2, device="cuda")
    a, b = (pairs, pairs + r // 2) if case["neox"] else (2 * pairs, 2 * pairs + 1)
    limit = 448.0 if fp8 else math.inf

    def turn(x, pos):
        z = torch.polar(torch.full_like(pos * f, s["magnitude"]), pos * f)[:, None]
        w = torch.complex(x[..., a], x[..., b]) * z
        x = x.clone()
        x[..., a], x[..., b] = w.real, w.imag
        return x

    for m in range(case["batch"]):
        lo, hi = int(s["q_indptr_host"][m]), int(s["q_indptr_host"][m + 1])
        slots = torch.arange(int(s["total"][m]) - (hi - lo), int(s["total"][m]), device="cuda")
        pos = (slots + case["shift"]).double()[:, None]
        page = _dev(s["page_indices_host"][s["page_indptr_host"][m]: s["page_indptr_host"][m + 1]], torch.int64)[slots // P]
        q_out[lo:hi] = turn(s["q"][lo:hi].double(), pos)
        k_pool[page, slots % P] = (turn(s["k"][lo:hi].double(), pos) / s["k_scale"]).clamp(-limit, limit)
        v_pool[page, slots % P] = (s["v"][lo:hi].double() / s["v_scale"]).clamp(-limit, limit)
    return q_out, k_pool, v_pool


def _attend_exact(case, s):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for m in range(case["batch"]):
        lo, hi, L = int(s["q_indptr_host"][m]), int(s["q_indptr_host"][m + 1]), int(s["total"][m])
        n = hi - lo
        pages = _dev(s["page_indices_host"][s["page_indptr_host"][m]: s["page_indptr_host"][m + 1]], torch.int64)
        K = _values(s["k_pool"][pages], s["k_scale"]).flatten(0, 1)[:L]
        V = _values(s["v_pool"][pages], s["v_scale"]).flatten(0, 1)[:L]
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


def _verify_exact(case, s):
    accepted, tokens = [], []
    first, drafts, u = s["indptr"].tolist(), s["tokens"].tolist(), s["uniforms"].tolist()
    for m in range(case["batch"]):
        K, said, n = first[m + 1] - first[m], [], 0
        row = first[m] + m
        q = None
        for j in range(K):
            d = drafts[first[m] + j]
            qd = float(s["draft"][first[m] + j, d]) if s["draft"] is not None else 1.0
            if not u[row + j] * qd < float(s["target"][row + j, d]):
                q = torch.zeros(case["vocab"], dtype=torch.float64, device="cuda")
                if s["draft"] is not None:
                    q = s["draft"][first[m] + j].double()
                else:
                    q[d] = 1.0
                break
            said.append(d)
            n += 1
        p = s["target"][row + n].double()
        w = p if q is None else (p - q).relu()
        w = w if float(w.sum()) > 0 else p
        sums = torch.cumsum(w, 0)
        new = int(torch.searchsorted(sums, sums[-1] * u[row + K], right=True))
        accepted.append(n)
        tokens += said + [min(new, case["vocab"] - 1)] + [-1] * (K - n)
    return (torch.tensor(accepted, dtype=torch.int32, device="cuda"),
            torch.tensor(tokens, dtype=torch.int32, device="cuda"))
