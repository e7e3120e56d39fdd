"""Seeded inputs of a step with several new tokens a request, and error bounds."""
import numpy as np
import torch

import synth
from oracle import attention as A
from oracle import tokens as TK

LOG2E = 1.0 / np.log(2.0)


class Step:
    """Ragged requests over shuffled pages.  Pool rows outside the requests' tokens hold NaN;
    three rows of q behind the last request hold NaN too.  `new` and `before` give each
    request's new tokens and the tokens already in its cache."""

    def __init__(self, new, before, *, Hq=8, Hkv=2, D=64, page=16, kv="bf16", seed=0, tree=None, spread=1.0,
                 pad_rows=3, device="cuda"):
        rng = np.random.default_rng(seed)
        self.new, self.total = np.array(new), np.array(new) + np.array(before)
        self.Hq, self.Hkv, self.D, self.page, self.kv = Hq, Hkv, D, page, kv
        self.q_indptr = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        pages = -(-self.total // page)
        self.page_indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        self.num_pages = int(self.page_indptr[-1]) + 2
        self.page_indices = rng.permutation(self.num_pages)[: self.page_indptr[-1]].astype(np.int32)
        self.last = (self.total - (pages - 1) * page).astype(np.int32)
        self.T = int(self.q_indptr[-1]) + pad_rows
        valid = synth._valid_slots(self.page_indptr, self.page_indices, self.last, self.num_pages, page)
        self.scales = (1.0, 1.0)
        if kv == "bf16":
            self.k = synth.fill_pool_bf16(rng, self.num_pages, page, Hkv, D, valid, True)
            self.v = synth.fill_pool_bf16(rng, self.num_pages, page, Hkv, D, valid, True)
        else:
            self.k, ks = synth.fill_pool_fp8(rng, self.num_pages, page, Hkv, D, valid, True)
            self.v, vs = synth.fill_pool_fp8(rng, self.num_pages, page, Hkv, D, valid, True)
            self.scales = (float(ks), float(vs))
        q = rng.standard_normal((self.T, Hq, D)).astype(np.float32) * spread
        q[int(self.q_indptr[-1]):] = np.nan
        self.q = torch.from_numpy(q).to(torch.bfloat16)
        self.sm_scale = D ** -0.5
        self.tree = None
        if tree == "random":
            masks = []
            for n in self.new:
                of = []
                for i in range(int(n)):
                    of.append((of[int(rng.integers(i))] if i else 0) | (1 << i))
                masks += of
            masks += [0] * pad_rows
            self.tree = masks
        elif tree is not None:
            self.tree = list(tree) + [0] * pad_rows

    def values(self, pool, scale):
        if self.kv == "bf16":
            return pool.double().numpy()
        return A.e4m3_to_f64(pool.numpy()).reshape(tuple(pool.shape)) * scale

    def oracle(self, sm_scale=None):
        n = int(self.q_indptr[-1])
        return TK.attend(self.q[:n].double().numpy(), self.values(self.k, self.scales[0]),
                         self.values(self.v, self.scales[1]), self.q_indptr, self.total, self.page_indptr,
                         self.page_indices, self.page, self.sm_scale if sm_scale is None else sm_scale, self.tree)

    def tree_dev(self):
        if self.tree is None:
            return None
        return torch.tensor([x - (1 << 64) if x >> 63 else x for x in self.tree], dtype=torch.int64, device="cuda")


def bounds(oracle, D, n_keys, out_f32, terms):
    """Error bounds of (o, lse) from the arithmetic the kernels state.

    Scores: an f32 sum of D exact products (each add off by at most 2^-23 of the running
    absolute sum, truncation included), then a scale, an fma and a subtraction in log2
    units.  exp2: 2 ulp.  P meets V as `terms` bf16 terms (0: as f32): off by 2^-8 of it, or
    2^-24 with three; two stands for two f16 terms, 2^-22.  O and l: f32 sums of n_keys terms, in any grouping; a lazy maximum can
    rescale them a few times (each a rounding, counted in the same term).  The output
    is rounded to bf16 (2^-8) or f32.  An error e of every score moves o by at most
    2 e sum p |v|."""
    o, lse, pv, top = oracle
    empty, lse = np.isneginf(lse), np.where(np.isneginf(lse), 0.0, lse)
    score = (D + 8) * 2.0 ** -23 * top + (np.abs(lse) + 40) * 2.0 ** -22 + 2.0 ** -20
    sums = (n_keys + 64) * 2.0 ** -23
    p_round = {0: 0.0, 1: 2.0 ** -8, 2: 2.0 ** -22, 3: 2.0 ** -24}[terms]
    out = 2.0 ** -24 if out_f32 else 2.0 ** -8
    e_o = (2 * score[..., None] + sums * 2 + p_round) * pv * (1 + out) + out * np.abs(o) + 1e-30
    e_l = (score + sums) * LOG2E + 2.0 ** -22 * np.abs(lse) + 1e-30
    return e_o, np.where(empty, 0, e_l)
