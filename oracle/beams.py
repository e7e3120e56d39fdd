"""Float64 and pure-Python definitions of a beam search step over a cache of 8-bit blocks: the blocks' scales and
codes, the selection over beams and vocabulary, and the operations on pages."""
import math

import numpy as np


# --------------------------------------------------------------------- 8-bit blocks
def scale_exponent(top):
    """The least e >= 95 with top <= 448 * 2^(e - 127)."""
    e = 95
    while top > math.ldexp(448.0, e - 127):
        e += 1
    return e


def scale_values(codes):
    """2^(e - 127) of the bytes, NaN for 255."""
    codes = np.asarray(codes, dtype=np.int64)
    return np.where(codes == 255, np.nan, np.ldexp(1.0, codes - 127))


def dequantise(values, scales, block):
    """Pool values [pages, page, Hkv, W] (of the codes) times their blocks' scales [pages, page / block, Hkv]."""
    return values * np.repeat(scale_values(scales), block, axis=1)[..., None]


def e4m3_nearest(x):
    """The nearest e4m3 values, ties to even, saturating at 448 (infinities too); NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    y = np.clip(x, -448.0, 448.0)
    _, exponent = np.frexp(np.where(np.isfinite(y), y, 1.0))
    step = np.ldexp(1.0, np.maximum(exponent - 1, -6) - 3)
    return np.where(np.isnan(x), np.nan, np.round(y / step) * step)


# ------------------------------------------------------------------------ selection
def select(logits, scores, beams, k, finished=None, pad=0):
    """(scores [B, k], rows, tokens) in 64 bits; -inf, -1, -1 where there are too few."""
    B = len(scores) // beams
    out = np.full((B, k), -np.inf), np.full((B, k), -1), np.full((B, k), -1)
    for b in range(B):
        found = []
        for r in range(b * beams, (b + 1) * beams):
            s = float(scores[r])
            if math.isnan(s) or math.isinf(s):
                continue
            if finished is not None and finished[r]:
                found.append((-s, r, 0.0, pad))
                continue
            x = np.asarray(logits[r], dtype=np.float64)
            x = np.where(np.isnan(x), -np.inf, x)
            top = x.max()
            if math.isinf(top):
                continue
            share = math.log(math.fsum(np.exp(x - top)))              # (beside a far-off top it would be lost)
            order = np.lexsort((np.arange(len(x)), -x))[:k]
            found += [(-(s + ((x[t] - top) - share)), r, -x[t], int(t)) for t in order if x[t] > -np.inf]
        for i, (v, r, _, t) in enumerate(sorted(found)[:k]):
            out[0][b, i], out[1][b, i], out[2][b, i] = -v, r, t
    return out


# ---------------------------------------------------------------------------- pages
def fork(parents, indptr, indices, kv_len, page, room, ref, keep_old=False):
    """(rows of page ids, lengths, counts, copies [(source, destination)]), or None where pages run out."""
    ref = [int(r) for r in ref]
    if not keep_old:
        for g in indices[int(indptr[0]): int(indptr[-1])]:
            ref[int(g)] -= 1
    others, taken = list(ref), set()
    for p in parents:                       # what a child holds as a full page nobody may write to
        for j in range(int(kv_len[p]) // page if p >= 0 else 0):
            others[int(indices[int(indptr[p]) + j])] += 1
    rows, lengths, fresh, copies = [], [], [], []
    for i, p in enumerate(parents):
        if p < 0:
            rows.append([])
            lengths.append(0)
            continue
        L = int(kv_len[p])
        row = []
        for j in range(-(-(L + room) // page)):
            g = int(indices[int(indptr[p]) + j]) if j * page < L else None
            if g is not None and room > 0 and (j + 1) * page > L:
                if others[g] > 0 or g in taken:
                    copies.append((g, i, j))
                    g = None
                else:
                    taken.add(g)
            if g is None:
                fresh.append((i, j))
            else:
                ref[g] += 1
            row.append(g)
        rows.append(row)
        lengths.append(L + room)
    free = [g for g, r in enumerate(ref) if r == 0]
    if len(free) < len(fresh):
        return None
    for (i, j), g in zip(fresh, free):
        rows[i][j] = g
        ref[g] = 1
    return rows, lengths, ref, [(g, rows[i][j]) for g, i, j in copies]


def compact(ref):
    """(live pages, new id of each page or -1, new counts, moves [(source, destination)])."""
    n = sum(r > 0 for r in ref)
    holes = [g for g in range(n) if ref[g] == 0]
    movers = [g for g in range(n, len(ref)) if ref[g] > 0]
    to = [g if g < n and r > 0 else -1 for g, r in enumerate(ref)]
    for a, b in zip(movers, holes):
        to[a] = b
    new = [0] * len(ref)
    for g, r in enumerate(ref):
        if r > 0:
            new[to[g]] = int(r)
    return n, to, new, list(zip(movers, holes))
