"""multi_token_decode over 8-bit blocks whose scales lie far apart or change along the cache, on both tensor-core kernels: what
the outputs are in units of must not show.  Caches are alike for all heads and requests, so that a few rows say it all."""
import numpy as np
import pytest
import torch

from oracle import tokens as TK
from _scaled_util import Scaled
from _tokens_util import bounds

pytestmark = pytest.mark.gpu

PAGE, BLOCK = 64, 16
LOG2E = np.float32(1.4426950408889634)


class Cache(Scaled):
    """B requests of `new` tokens over one cache that they all have: codes k and v [L, D], a scale byte a block.  Queries are
    `q` in column 0."""

    def __init__(self, B, new, k, v, ke, ve, *, G=4, Hkv=2, sm_scale=1.0, q=1.0):
        L, self.D = k.shape
        self.Hq, self.Hkv, self.page, self.block, self.tree, self.sm_scale = G * Hkv, Hkv, PAGE, BLOCK, None, float(sm_scale)
        self.new, self.total = np.full(B, new), np.full(B, L)
        self.q_indptr = (np.arange(B + 1) * new).astype(np.int32)
        self.num_pages = pages = -(-L // PAGE)
        self.page_indptr = (np.arange(B + 1) * pages).astype(np.int32)
        self.page_indices = np.tile(np.arange(pages), B).astype(np.int32)
        self.last = np.full(B, L - (pages - 1) * PAGE).astype(np.int32)
        self.T = B * new

        def pool(c):
            wide = np.full((pages * PAGE, 1, self.D), 0x7F, dtype=np.uint8)
            wide[:L, 0] = c
            return torch.from_numpy(np.repeat(wide, Hkv, 1).reshape(pages, PAGE, Hkv, self.D).copy())

        def scales(e):
            wide = np.full(pages * PAGE // BLOCK, 255, dtype=np.uint8)
            wide[: len(e)] = e
            return torch.from_numpy(np.repeat(wide[:, None], Hkv, 1).reshape(pages, PAGE // BLOCK, Hkv).copy())

        self.k, self.v, self.ke, self.ve = pool(k), pool(v), scales(ke), scales(ve)
        self.q = torch.zeros((self.T, self.Hq, self.D), dtype=torch.bfloat16)
        self.q[..., 0] = q

    def one(self):
        """Of one request, as TK.attend gives it."""
        n, pages = int(self.new[0]), self.num_pages
        return TK.attend(self.q[:n].double().numpy(), self.values(self.k, self.ke), self.values(self.v, self.ve), self.q_indptr[:2],
                         self.total[:1], self.page_indptr[:2], self.page_indices[:pages], PAGE, self.sm_scale)


def _scale_for(low, high, step, rest):
    """An sm_scale whose product with log2 e, in f32, is in [low, high) and rest * 2^-20 beyond a multiple of step * 2^-20."""
    x = np.float32(low) / LOG2E
    while True:
        x = np.nextafter(x, np.float32(np.inf))
        y = x * LOG2E
        if low <= y < high and int(np.float64(y) * 2 ** 20) % step == rest:
            return float(x)


def _codes(rng, shape, low=0x20, high=0x40):
    """Codes of ordinary size: 2^-3 to 2, either sign."""
    return (rng.integers(low, high, shape) | rng.integers(0, 2, shape) << 7).astype(np.uint8)


def _same(a, b):
    """Two calls that differ in powers of two alone: each of up to four exponentials of powers (of two ulp, 2^-22) may show,
    beside nothing else."""
    for x, y in zip(a, b):
        x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
        worst = float(np.max(np.abs(x - y) / np.maximum(np.abs(y), 1e-30)))
        assert worst <= 2.0 ** -20, worst


@pytest.mark.parametrize("jump", [False, True])
@pytest.mark.parametrize("n,G", [(1, 4), (3, 4), (40, 1), (40, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_values_in_other_units(D, n, G, jump):
    """The first half of the values in units of 2^-5, with codes in place of that, or of 2^-3 as the second half, which is
    zeros.  Scores are equal (or grow once, with the units), and their sum with the units' exponent does not fit f32."""
    rng, L = np.random.default_rng(D + n), 2048
    k = np.zeros((L, D), dtype=np.uint8)
    k[:, 0] = 0x38
    if jump:
        k[L // 2:, 0] = 0x40                                         # scores of 12.. and 24..
    v = np.zeros((L, D), dtype=np.uint8)
    v[: L // 2] = 0x38 + rng.integers(0, 8, (L // 2, D))             # 1 .. 1.875
    ke = np.full(L // BLOCK, 127)
    ve = np.full(L // BLOCK, 124)
    sm = _scale_for(12.5, 12.75, 16, 6)
    want = Cache(40, n, k, np.where(v > 0, v - 16, 0).astype(np.uint8), ke, ve, G=G, Hkv=4, sm_scale=sm).run(out_f32=True)
    ve[: len(ve) // 2] = 122
    got = Cache(40, n, k, v, ke, ve, G=G, Hkv=4, sm_scale=sm).run(out_f32=True)
    _same(got, want)


@pytest.mark.parametrize("n,G", [(1, 4), (3, 4), (40, 1), (40, 4)])
@pytest.mark.parametrize("e", [95, 130, 160])
def test_blocks_of_zeros_in_other_units(e, n, G):
    """Tiles of zeros have any scale: their weights do not change."""
    rng, L, D = np.random.default_rng(e + n), 2048, 64
    k = np.zeros((L, D), dtype=np.uint8)
    k[:, 0] = 0x38
    v = np.zeros((L, D), dtype=np.uint8)
    v[:64], v[1024:1088] = _codes(rng, (64, D)), _codes(rng, (64, D))
    ke, ve = np.full(L // BLOCK, 127), np.full(L // BLOCK, 170)
    sm = _scale_for(12.5, 12.75, 8, 4)
    want = Cache(40, n, k, v, ke, ve, G=G, Hkv=4, sm_scale=sm).run(out_f32=True)
    ve[[j for j in range(len(ve)) if not v[16 * j: 16 * j + 16].any()]] = e
    got = Cache(40, n, k, v, ke, ve, G=G, Hkv=4, sm_scale=sm).run(out_f32=True)
    _same(got, want)


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("n,G", [(1, 4), (40, 1), (40, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_and_scores_that_grow_in_one_tile(D, n, G, out_f32):
    """In one tile V's scale rises and scores pass the largest so far by more than 2^8, again and again: O is brought to other
    units twice before the tile's P V is added."""
    rng, L = np.random.default_rng(D + n), 1536
    k, v = np.zeros((L, D), dtype=np.uint8), _codes(rng, (L, D))
    ke, ve, at = np.full(L // BLOCK, 127), np.full(L // BLOCK, 118), 0
    k[:, 0] = 0xC0                                                    # -2, then 12 more a jump
    for j, x in ((70, 0x28), (400, 0x40), (450, 0x44), (1100, 0x48), (1300, 0x4C)):   # 1/4, 2, 3, 4, 6: log2 units times 12.6
        k[j:, 0] = x
        ve[j // BLOCK:] += 2
    s = Cache(40, n, k, v, ke, ve, G=G, Hkv=4, sm_scale=_scale_for(12.5, 12.75, 16, 6))
    o, lse = s.run(out_f32=out_f32)
    want = s.one()
    e_o, e_l = bounds(want, D, L, out_f32, 2 if out_f32 else 1)
    e_o = e_o + 2.0 ** -32 * L * 448 * 2.0 ** (int(ve.max()) - 127)   # what f16 holds of a weight (see the ragged tests)
    o, lse = o.double().cpu().numpy().reshape(40, n, s.Hq, D), lse.double().cpu().numpy().reshape(40, n, s.Hq)
    assert float(np.max(np.abs(o - want[0]) / e_o)) <= 1
    assert float(np.max(np.abs(lse - want[1]) / e_l)) <= 1


@pytest.mark.parametrize("gap", [15, 24, 25, 26, 28, 30, 33])
@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("n", [1, 40])
def test_values_far_below_the_tiles_largest_scale(n, out_f32, gap):
    """The largest scale of a tile is that of keys without weight: the others' values are rounded to 2^-25 of it, no more."""
    rng, L, D = np.random.default_rng(gap), 64, 64
    k, v = np.zeros((L, D), dtype=np.uint8), _codes(rng, (L, D), 0x70, 0x7F)   # 128 to 448
    k[:16, 0] = 0xFE                                                  # -448: a weight of e^-448
    ke, ve = np.full(4, 127), np.array([170, 170 - gap, 170 - gap, 170 - gap])
    s = Cache(2, n, k, v, ke, ve)
    o, lse = s.run(out_f32=out_f32)
    want = s.one()
    e_o, e_l = bounds(want, D, L, out_f32, 2 if out_f32 else 1)
    # a value's rounding, and that of its weight to 2^-32 of the largest
    e_o = e_o + 2.0 ** 43 * (2.0 ** -25 + 2.0 ** -32 * 448)
    o, lse = o.double().cpu().numpy().reshape(2, n, s.Hq, D), lse.double().cpu().numpy().reshape(2, n, s.Hq)
    assert float(np.max(np.abs(o - want[0]) / e_o)) <= 1
    assert float(np.max(np.abs(lse - want[1]) / e_l)) <= 1


@pytest.mark.parametrize("gap", [15, 24, 25, 26, 28])
@pytest.mark.parametrize("n", [1, 40])
def test_keys_far_below_the_tiles_largest_scale(n, gap):
    """The largest K scale of a tile is that of keys whose scores leave them no weight."""
    rng, L, D = np.random.default_rng(gap), 64, 64
    k, v = np.zeros((L, D), dtype=np.uint8), _codes(rng, (L, D))
    k[:16, 0] = 0xFE
    k[16::2, 0] = 0x7E                                                # 448 and 0
    ke, ve = np.array([170, 170 - gap, 170 - gap, 170 - gap]), np.full(4, 127)
    unit = 2.0 ** gap / 448                                           # a score of 1 for 448 at the small scale
    s = Cache(2, n, k, v, ke, ve, sm_scale=unit * 2.0 ** -43)
    o, lse = s.run(out_f32=True)
    want = s.one()
    # a key's rounding is 2^-25 of the largest scale, so 2^-25 unit in its score; twice that of sum p |v| in the output
    score = 2.0 ** -25 * unit
    top = want[3].copy()
    rows = (want[0], want[1], want[2], np.minimum(top, 1.0))          # (the scores that have a weight are 1 at most)
    e_o, e_l = bounds(rows, D, L, True, 2)
    o, lse = o.double().cpu().numpy().reshape(2, n, s.Hq, D), lse.double().cpu().numpy().reshape(2, n, s.Hq)
    assert float(np.max(np.abs(o - want[0]) / (e_o + 2 * score * want[2]))) <= 1
    assert float(np.max(np.abs(lse - want[1]) / (e_l + score * LOG2E))) <= 1


@pytest.mark.parametrize("n", [1, 3, 40])
def test_scales_from_zero_on(n):
    """Blocks of byte 0 and 1 (2^-127 and 2^-126): all of them count."""
    rng, L, D = np.random.default_rng(n), 1800, 64
    k, v = np.zeros((L, D), dtype=np.uint8), _codes(rng, (L, D), 0x70, 0x7F)
    ke, j = np.full(-(-L // BLOCK), 127), np.arange(-(-L // BLOCK))
    for ve in (j // 40, np.array([0, 1, 0, 2])[j // 29], 0 * j):
        s = Cache(40, n, k, v, ke, ve, Hkv=4)
        o, _ = s.run(out_f32=True)
        want = s.one()
        # (results are far from f32's subnormals, 2^-149; weights are equal)
        e_o = bounds(want, D, L, True, 2)[0] - 1e-30 + 2.0 ** -32 * 448 * 2.0 ** (int(ve.max()) - 127) + 2.0 ** -149
        assert float(np.max(np.abs(o.double().cpu().numpy().reshape(40, n, s.Hq, D) - want[0]) / e_o)) <= 1


@pytest.mark.parametrize("n", [1, 40])
def test_keys_of_scale_zero(n):
    """Byte 0 of K's blocks under queries of 2^124: the scores count."""
    rng, L, D = np.random.default_rng(n), 64, 64
    k, v = np.zeros((L, D), dtype=np.uint8), _codes(rng, (L, D))
    k[::2, 0] = 0x38                                                  # scores of 2^-127 2^124 16 = 2, and 0
    s = Cache(2, n, k, v, np.zeros(4, dtype=int), np.full(4, 127), sm_scale=16.0, q=2.0 ** 124)
    o, lse = s.run(out_f32=True)
    want = s.one()
    e_o, e_l = bounds(want, D, L, True, 2)
    o, lse = o.double().cpu().numpy().reshape(2, n, s.Hq, D), lse.double().cpu().numpy().reshape(2, n, s.Hq)
    assert float(np.max(np.abs(o - want[0]) / e_o)) <= 1
    assert float(np.max(np.abs(lse - want[1]) / e_l)) <= 1
