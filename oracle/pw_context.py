"""fp64 NumPy oracle of whole prompts, their scores and a cache that is short of memory: prompt attention, token log
probabilities, the 4-bit cache, weights added up by key and eviction.

Definitions follow include/pw.h; the write-ups describe none of these steps.  Test infrastructure only: it shares no
code with the CUDA path.  Loops are plain on purpose.
"""
from __future__ import annotations

import numpy as np


def prompt(q, k, v, offsets, scale):
    """Returns (out, lse, A, ds, n) per row and head as pw_serve.attend does; rows of no sequence stay NaN in out and lse."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    T, H, D = q.shape
    G = H // k.shape[1]
    out, A = np.full((T, H, D), np.nan), np.zeros((T, H, D))
    lse, ds, seen = np.full((T, H), np.nan), np.zeros((T, H)), np.zeros((T, H), dtype=int)
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        for i in range(lo, hi):
            for h in range(H):
                kk, vv = k[lo:i + 1, h // G], v[lo:i + 1, h // G]
                s = scale * (kk @ q[i, h])
                w = np.exp(s - s.max())
                out[i, h], A[i, h] = (w @ vv) / w.sum(), (w @ np.abs(vv)) / w.sum()
                lse[i, h] = s.max() + np.log(w.sum())
                ds[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
                seen[i, h] = i + 1 - lo
    return out, lse, A, ds, seen


def logprobs(x, tokens, n_top):
    """(logprobs, entropy, top ids, top logprobs) of rows x [T, V]; ids -1 and -inf where no logit is left."""
    x = np.asarray(x, dtype=np.float64)
    T, V = x.shape
    lp, ent = np.zeros(T), np.zeros(T)
    ids, tops = np.full((T, n_top), -1), np.full((T, n_top), -np.inf)
    for t in range(T):
        row = x[t]
        number = ~np.isnan(row)
        m = row[number].max() if number.any() else -np.inf
        if np.isnan(row).any() or m == np.inf:
            logp = np.full(V, np.nan)
            ent[t] = np.nan
        elif m == -np.inf:
            logp = np.full(V, -np.inf)
        else:
            logp = (row - m) - np.log(np.exp(row - m).sum())
            p = np.exp(logp)
            ent[t] = -(p[p > 0] * logp[p > 0]).sum()
        if tokens[t] >= 0:
            lp[t] = logp[tokens[t]] if tokens[t] < V else np.nan
        order = sorted((i for i in range(V) if row[i] > -np.inf), key=lambda i: (-row[i], i))[:n_top]
        ids[t, :len(order)] = order
        tops[t, :len(order)] = logp[order]
    return lp, ent, ids, tops


def quantise(x, to_type):
    """4-bit form of x [..., D] (values of the heads' type): codes, least values, steps; `to_type` rounds fp32 values to it."""
    f = np.float32
    g = np.asarray(x).astype(f).reshape(*np.shape(x)[:-1], -1, 32)
    with np.errstate(all="ignore"):
        least, most = g.min(-1), g.max(-1)
        step = to_type(((most - least).astype(f) / f(15)).astype(f)).astype(f)
        # the next lower step where the top code would stand for no number of the type
        over = np.isfinite(step) & np.isinf(to_type((least.astype(np.float64) + 15 * step.astype(np.float64)).astype(f)).astype(f))
        lower = step
        for j in range(24, 0, -1):  # the first that rounds below it is its neighbour
            lower = np.where(lower < step, lower, to_type((step * f(1 - 2.0 ** -j)).astype(f)).astype(f))
        step = np.where(over, lower, step)
        c = np.rint(((g - least[..., None]).astype(f) / step[..., None]).astype(f))
    c = np.where(step[..., None] > 0, np.clip(c, 0, 15), 0)
    bad = ~np.isfinite(g).all(-1) | ~np.isfinite(step)
    least, step = np.where(bad, np.nan, least), np.where(bad, np.nan, step)
    return np.where(bad[..., None], 0, c).astype(int).reshape(np.shape(x)), least, step


def values(code, least, step):
    g = code.reshape(*code.shape[:-1], -1, 32)
    return (least[..., None].astype(np.float64) + g * step[..., None].astype(np.float64)).reshape(code.shape)


def weigh(q, kc, table, lens, lse, mass, q_len, scale, decay):
    """(out, bound): the weights added up by key, and the sum over rows of weight x (1 + scale |q||k| + |lse|)."""
    q, kc = np.asarray(q, dtype=np.float64), np.asarray(kc, dtype=np.float64)
    out = np.array(mass, dtype=np.float64)
    bound = np.zeros(out.shape)
    P, hkv, page, _ = kc.shape
    G = q.shape[1] // hkv
    for b in range(len(lens)):
        n = min(max(int(lens[b]), 0), table.shape[1] * page, out.shape[1])
        out[b, :n] *= decay
        for i in range(n):
            p = int(table[b][i // page])
            for j in range(q_len):
                if i > n - q_len + j:
                    continue
                for h in range(q.shape[1]):
                    r = b * q_len + j
                    if np.isneginf(lse[r, h]):
                        continue
                    key = kc[p, h // G, i % page] if 0 <= p < P else np.zeros(q.shape[2])
                    w = np.exp(scale * (q[r, h] @ key) - lse[r, h])
                    out[b, i] += w
                    bound[b, i] += w * (1 + abs(scale) * (np.abs(q[r, h]) @ np.abs(key)) + abs(lse[r, h]))
    return out, bound


def stays(mass, n, budget, recent):
    """The positions that stay, in order: the last `recent`, then by mass, the lower position of equal ones."""
    left = min(n, budget)
    recent = min(recent, left)
    older = sorted(range(n - recent), key=lambda i: (-(mass[i] if mass[i] == mass[i] else -np.inf), mass[i] != mass[i], i))
    return sorted(older[:left - recent]) + list(range(n - recent, n))


def evict(kc, vc, table, lens, mass, budget, recent, new_table):
    """(k cache, v cache, new lens, new mass, kept) after an eviction."""
    k0, v0 = np.array(kc), np.array(vc)
    kc, vc, mass = np.array(kc), np.array(vc), np.array(mass)
    P, _, page, _ = kc.shape
    kept, out, new_lens = np.full((len(lens), budget), -1), np.zeros(mass.shape, dtype=mass.dtype), []
    for b in range(len(lens)):
        n = min(max(int(lens[b]), 0), table.shape[1] * page, mass.shape[1])
        who = stays(mass[b], n, budget, recent)
        new_lens.append(len(who))
        kept[b, :len(who)] = who
        out[b, :len(who)] = mass[b][who]
        for j, i in enumerate(who):
            a, z = int(table[b][i // page]), int(new_table[b][j // page])
            if 0 <= z < P:
                kc[z, :, j % page] = k0[a, :, i % page] if 0 <= a < P else 0
                vc[z, :, j % page] = v0[a, :, i % page] if 0 <= a < P else 0
    return kc, vc, np.array(new_lens, dtype=np.int32), out, kept
