"""A step of several new tokens a request (oracle; test infrastructure only): rotation
and append, attention of the new tokens over the cache, verification of drafts, each
written out in float64 from its definition.

The source pages decline multi-token steps (mlxcel PR #1004, Task item 4) and list
speculative acceptance among the neighbouring items (Left out / unsure), so the
definitions are the C header's: include/psd.h, "steps of several new tokens".
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

LOG2E = 1.0 / math.log(2.0)


# ------------------------------------------------------------------- frequencies
def rope_frequencies(kind, r, base=10000.0, factor=1.0, original=0, low=1.0, high=32.0):
    """(inv_freq [r/2], magnitude), one frequency at a time."""
    out, magnitude = [], 1.0
    if kind == "ntk":
        base = base * factor ** (r / (r - 2.0))
    if kind == "yarn" and factor > 1:
        magnitude = 0.1 * math.log(factor) + 1.0
    for i in range(r // 2):
        f = base ** (-2.0 * i / r)
        if kind == "linear":
            f /= factor
        elif kind == "yarn":
            where = lambda t: r * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            lo = max(math.floor(where(high)), 0)
            hi = min(math.ceil(where(low)), r - 1)
            ramp = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * (1 - ramp) + f / factor * ramp
        elif kind == "bands":
            keep = min(max((original * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f = f * keep + f / factor * (1 - keep)
        out.append(f)
    return np.array(out), magnitude


# ------------------------------------------------------------------------ append
def rotate(x, pos, inv_freq, magnitude, col, neox):
    """Rows x [.., D] (float64) rotated at positions pos [..]; also a bound on |x| + |y| of
    each column's pair times the magnitude (what an error of cos or sin is multiplied by)."""
    r2 = len(inv_freq)
    x = np.array(x, dtype=np.float64)
    size = np.zeros_like(x)
    for i in range(r2):
        a, b = (col + i, col + i + r2) if neox else (col + 2 * i, col + 2 * i + 1)
        angle = np.asarray(pos, dtype=np.float64) * inv_freq[i]
        c, s = magnitude * np.cos(angle), magnitude * np.sin(angle)
        u, w = x[..., a].copy(), x[..., b].copy()
        x[..., a], x[..., b] = u * c - w * s, w * c + u * s
        size[..., a] = size[..., b] = (np.abs(u) + np.abs(w)) * magnitude
    return x, size


def positions_of(q_indptr, kv_len):
    """[(request, index in the request)] of every token row."""
    out = []
    for b in range(len(kv_len)):
        n = int(q_indptr[b + 1] - q_indptr[b])
        out += [(b, int(kv_len[b]) - n + i) for i in range(n)]
    return out


# --------------------------------------------------------------------- attention
def attend(q, k_pool, v_pool, q_indptr, kv_len, page_indptr, page_indices, page_size, sm_scale, tree=None):
    """o [T, Hq, D], lse [T, Hq] (log2) and, per row and head, the numbers error bounds are
    made of: sum p |v| per column [T, Hq, D] and the largest sum |q k| sm_scale over seen keys."""
    T, Hq, D = q.shape
    Hkv = k_pool.shape[2]
    G = Hq // Hkv
    o, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    pv, top = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        L, t0, t1 = int(kv_len[b]), int(q_indptr[b]), int(q_indptr[b + 1])
        n = t1 - t0
        slots = [int(page_indices[page_indptr[b] + j // page_size]) * page_size + j % page_size for j in range(L)]
        K = k_pool.reshape(-1, Hkv, D)[slots]
        V = v_pool.reshape(-1, Hkv, D)[slots]
        for i in range(n):
            if tree is None:
                seen = np.arange(L) <= L - n + i
            else:
                mask = int(tree[t0 + i]) & ((1 << 64) - 1)
                seen = np.array([j < L - n or bool((mask >> (j - (L - n))) & 1) for j in range(L)])
            if not seen.any():
                continue
            for h in range(Hq):
                Ks, Vs = K[seen, h // G], V[seen, h // G]
                t = Ks @ q[t0 + i, h] * sm_scale
                m = t.max()
                p = np.exp(t - m)
                l = p.sum()
                o[t0 + i, h] = p @ Vs / l
                lse[t0 + i, h] = (m + math.log(l)) * LOG2E
                pv[t0 + i, h] = p @ np.abs(Vs) / l
                top[t0 + i, h] = (np.abs(Ks) @ np.abs(q[t0 + i, h])).max() * abs(sm_scale)
    return o, lse, pv, top


# ------------------------------------------------------------------ verification
def verify(target, draft, tokens, indptr, uniforms):
    """(accepted, out_tokens), in exact rational arithmetic."""
    accepted, out = [], []
    V = target.shape[1]
    for b in range(len(indptr) - 1):
        d0, K = int(indptr[b]), int(indptr[b + 1] - indptr[b])
        R, a, q = d0 + b, 0, None
        while a < K:
            d = int(tokens[d0 + a])
            inside = 0 <= d < V
            qd = Fraction(1) if draft is None else (Fraction(float(draft[d0 + a, d])) if inside else Fraction(0))
            if inside and Fraction(float(uniforms[R + a])) * qd < Fraction(float(target[R + a, d])):
                a += 1
                continue
            q = [Fraction(0)] * V
            if inside and draft is not None:
                q = [Fraction(float(x)) for x in draft[d0 + a]]
            elif inside:
                q[d] = Fraction(1)
            break
        p = [Fraction(float(x)) for x in target[R + a]]
        w = p if q is None else [max(x - y, Fraction(0)) for x, y in zip(p, q)]
        if sum(w) == 0:
            w = p
        share, run, new = Fraction(float(uniforms[R + K])) * sum(w), Fraction(0), -1
        for v, x in enumerate(w):
            run += x
            if run > share:
                new = v
                break
        accepted.append(a)
        out += [int(t) for t in tokens[d0: d0 + a]] + [new] + [-1] * (K - a)
    return accepted, out
