"""Seeded caches of 8-bit blocks with a scale each, and the tokens that are attended over or appended to them."""
import numpy as np
import torch

import paged_split_kv_decode_gb300 as psd
from oracle import attention as A
from oracle import beams as BM
from oracle import tokens as TK
from _gpu_util import ctx

NAN_CODE = 0x7F


class Scaled:
    """Ragged requests over shuffled pages.  Slots outside the requests' tokens hold the NaN code, blocks without tokens
    the scale of NaN, rows of q behind the last request NaN.  `swing`: the scales' exponents lie within 127 +- swing."""

    def __init__(self, new, before, *, Hq=8, Hkv=2, D=64, page=16, block=16, seed=0, tree=None, spread=1.0, swing=3,
                 pad_rows=3):
        rng = np.random.default_rng(seed)
        self.new, self.total = np.array(new), np.array(new) + np.array(before)
        self.Hq, self.Hkv, self.D, self.page, self.block = Hq, Hkv, D, page, block
        self.q_indptr = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        pages = -(-self.total // page)
        self.page_indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        self.num_pages = int(self.page_indptr[-1]) + 2
        self.page_indices = rng.permutation(self.num_pages)[: self.page_indptr[-1]].astype(np.int32)
        self.last = (self.total - (pages - 1) * page).astype(np.int32)
        self.T = int(self.q_indptr[-1]) + pad_rows
        used = np.zeros((self.num_pages, page), dtype=bool)
        for b in range(len(self.total)):
            for j in range(int(self.total[b])):
                used[self.page_indices[self.page_indptr[b] + j // page], j % page] = True
        blocks = used.reshape(self.num_pages, page // block, block).any(-1)

        def pool():
            c = rng.integers(0, 127, (self.num_pages, page, Hkv, D)) | (rng.integers(0, 2, (self.num_pages, page, Hkv, D)) << 7)
            # mostly values of ordinary size, some of any
            small = rng.integers(0x20, 0x40, c.shape) | (c & 0x80)
            c = np.where(rng.random(c.shape) < 0.02, c, small)
            c[~used] = NAN_CODE
            e = 127 - 3 + rng.integers(-swing, swing + 1, (self.num_pages, page // block, Hkv))
            e[~blocks] = 255
            return torch.from_numpy(c.astype(np.uint8)), torch.from_numpy(e.astype(np.uint8))

        (self.k, self.ke), (self.v, self.ve) = pool(), pool()
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
            self.tree = masks + [0] * pad_rows
        elif tree is not None:
            self.tree = list(tree) + [0] * pad_rows

    def values(self, codes, e):
        return BM.dequantise(A.e4m3_to_f64(codes.cpu().numpy()).reshape(tuple(codes.shape)), e.cpu().numpy(), self.block)

    def oracle(self, sm_scale=None):
        n = int(self.q_indptr[-1])
        return TK.attend(self.q[:n].double().numpy(), self.values(self.k, self.ke), self.values(self.v, self.ve),
                         self.q_indptr, self.total, self.page_indptr, self.page_indices, self.page,
                         self.sm_scale if sm_scale is None else sm_scale, self.tree)

    def scales(self):
        return psd.BlockScales(self.ke.cuda(), self.ve.cuda(), self.block)

    def tree_dev(self):
        if self.tree is None:
            return None
        return torch.tensor([x - (1 << 64) if x >> 63 else x for x in self.tree], dtype=torch.int64, device="cuda")

    def plan(self):
        table = psd.HostTable(self.page_indptr, self.page_indices, self.last, self.page)
        return psd.plan_multi_token(table, self.q_indptr, self.Hq, self.Hkv)

    def args(self, *, sm_scale=None, q=None, indices=None):
        return psd.multi_token_args(self.q.cuda() if q is None else q, self.k.cuda(), self.v.cuda(),
                                    torch.from_numpy(self.page_indices).cuda() if indices is None else indices,
                                    sm_scale=self.sm_scale if sm_scale is None else sm_scale, tree_mask=self.tree_dev(),
                                    scales=self.scales())

    def run(self, *, out_f32=False, workspace=None, **kw):
        plan = self.plan()
        if workspace is None:
            workspace = psd.multi_token_workspace(ctx(), plan, self.D, "cuda")
            workspace.fill_(255)
        o = torch.full((self.T, self.Hq, self.D), 5.0, dtype=torch.float32 if out_f32 else torch.bfloat16, device="cuda")
        lse = torch.full((self.T, self.Hq), 5.0, device="cuda")
        psd.multi_token_decode(ctx(), self.args(**kw), plan, o, lse, workspace)
        assert psd.check_device_error(ctx(), workspace) == 0
        return o, lse
