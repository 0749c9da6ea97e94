"""fp64 NumPy oracle of the calls around the layer: head norm and rotation, paged append, attention with shared
prefixes, draft verification.

Definitions follow include/pw.h; the write-ups describe none of these steps.  Test infrastructure only: it shares no
code with the CUDA path.  Loops are plain on purpose.
"""
from __future__ import annotations

import numpy as np


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """x [T, H, D] -> fp64 [T, H, D]: RMS norm by weight (None: none), then the first cos_sin.shape[1] values turned."""
    x = np.asarray(x, dtype=np.float64).copy()
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    if cos_sin is None:
        return x
    maxpos, rot = cos_sin.shape
    out = x.copy()
    for t, p in enumerate(positions):
        row = np.asarray(cos_sin[min(max(int(p), 0), maxpos - 1)], dtype=np.float64)
        for i in range(rot // 2):
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            a, b, c, s = x[t, :, ia], x[t, :, ib], row[i], row[rot // 2 + i]
            out[t, :, ia] = a * c - b * s
            out[t, :, ib] = b * c + a * s
    return out


def append(cache, rows, slots):
    """cache [pages, H, page, D] with rows [T, H, D] written at the slots inside it (others write nothing)."""
    cache = np.array(cache)
    pages, _, page, _ = cache.shape
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            cache[s // page, :, s % page] = rows[t]
    return cache


def gather(cache, pages, n, h):
    """The first n rows of head h along a list of pages (a page outside the cache reads as zeros)."""
    P, _, page, D = cache.shape
    out = np.zeros((n, D))
    for i in range(n):
        p = int(pages[i // page])
        if 0 <= p < P:
            out[i] = cache[p, h, i % page]
    return out


def attend(q, kc, vc, table, lens, q_len, scale, ptable=None, plens=None, offsets=None):
    """Returns (out, lse, A, ds, n) per query row and head: the attention, its log-sum-exp, the weighted sum of |v|,
    the largest sum of |q||k| * scale over the keys seen, and the number of keys seen (for error bounds)."""
    kc, vc = np.asarray(kc, dtype=np.float64), np.asarray(vc, dtype=np.float64)
    q = np.asarray(q, dtype=np.float64)
    N, H, D = q.shape
    B, hkv, page = N // q_len, kc.shape[1], kc.shape[2]
    G = H // hkv
    out, A = np.zeros((N, H, D)), np.zeros((N, H, D))
    lse, ds, seen = np.full((N, H), -np.inf), np.zeros((N, H)), np.zeros((N, H), dtype=int)
    n_groups = 0 if plens is None else len(plens)
    offsets = [0, B] if offsets is None else list(offsets)
    for b in range(B):
        group = [g for g in range(n_groups) if offsets[g] <= b < offsets[g + 1]]
        ns = min(max(int(lens[b]), 0), table.shape[1] * page)
        for h in range(hkv):
            k, v = gather(kc, table[b], ns, h), gather(vc, table[b], ns, h)
            pk, pv = np.zeros((0, D)), np.zeros((0, D))
            if group:
                g = group[0]
                npre = min(max(int(plens[g]), 0), ptable.shape[1] * page)
                pk, pv = gather(kc, ptable[g], npre, h), gather(vc, ptable[g], npre, h)
            for j in range(q_len):
                vis = max(0, ns - q_len + 1 + j)
                kk, vv = np.concatenate([pk, k[:vis]]), np.concatenate([pv, v[:vis]])
                if not len(kk):
                    continue
                for c in range(G):
                    r, hh = b * q_len + j, h * G + c
                    s = scale * (kk @ q[r, hh])
                    w = np.exp(s - s.max())
                    out[r, hh] = (w @ vv) / w.sum()
                    A[r, hh] = (w @ np.abs(vv)) / w.sum()
                    lse[r, hh] = s.max() + np.log(w.sum())
                    ds[r, hh] = abs(scale) * (np.abs(kk) @ np.abs(q[r, hh])).max()
                    seen[r, hh] = len(kk)
    return out, lse, A, ds, seen


def verify(p, q, tokens, n_draft, u, noise):
    """Accepted counts and tokens, every product, difference and quotient rounded to fp32 once."""
    f = np.float32
    B, K1, V = p.shape
    K = K1 - 1
    out, accepted = np.full((B, K1), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    with np.errstate(all="ignore"):
        for b in range(B):
            n = min(max(int(n_draft[b]), 0), K) if K else 0
            a = 0
            while a < n:
                x = int(tokens[b, a])
                if not 0 <= x < V or not f(u[b, a]) * f(q[b, a, x]) < f(p[b, a, x]):
                    break
                out[b, a] = x
                a += 1
            full = np.fmax(p[b, a].astype(f), f(0))
            r = np.fmax(p[b, a].astype(f) - q[b, a].astype(f), f(0)) if a < n else full
            if not (r > 0).any():
                r = full
            score = r / noise[b].astype(f)
            score[~(score >= 0)] = 0
            out[b, a] = int(np.argmax(score))  # the first of equal ones
            accepted[b] = a
    return out, accepted
