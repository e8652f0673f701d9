"""fp64 CPU oracle of the operators on trees of drafted tokens, from the definitions.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares no code with
the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np

from .cache import Cache, e4m3_decode, e4m3_encode


def ancestors(parents) -> np.ndarray:
    """bool [n, n]: node j is i or one of its ancestors."""
    n = len(parents)
    out = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            out[i, j] = True
            j = parents[j]
    return out


def to_bits(masks, words) -> np.ndarray:
    """uint32 [T, words] of the sequences' bool masks, one below the other."""
    out = np.zeros((sum(len(m) for m in masks), words), np.uint32)
    t = 0
    for m in masks:
        for row in m:
            for j in np.flatnonzero(row):
                out[t, j // 32] |= np.uint32(1 << (j % 32))
            t += 1
    return out


def attend(cache: Cache, q, cu, lens, masks, scale=0.0):
    """(O, LSE [H, T]) and, for the error bounds, per sequence terms [H, n, L] = scale
    sum |q k| and spread [n, H, D] = sum p |v|.  masks[b]: bool [n, n]."""
    q = np.asarray(q, np.float64)
    T, H, D = q.shape
    G = H // cache.codes[0].shape[1]
    scale = scale or 1 / math.sqrt(D)
    O, LSE = np.zeros(q.shape), np.zeros((H, T))
    terms, spread = [], np.zeros(q.shape)
    for b, total in enumerate(lens):
        rows = slice(cu[b], cu[b + 1])
        n = cu[b + 1] - cu[b]
        seen = np.ones((n, total), bool)
        seen[:, total - n:] = masks[b]
        K, V = (np.repeat(cache.numbers(s, b, total), G, 0) for s in (0, 1))
        x = q[rows].transpose(1, 0, 2)
        s = np.where(seen, scale * x @ K.transpose(0, 2, 1), -np.inf)
        terms.append(scale * np.abs(x) @ np.abs(K).transpose(0, 2, 1))
        m = s.max(-1, initial=-np.inf, keepdims=True)
        p = np.exp(s - np.where(np.isfinite(m), m, 0))
        l = p.sum(-1, keepdims=True)
        with np.errstate(divide="ignore"):
            LSE[:, rows] = (np.where(np.isfinite(m), m, 0) + np.log(l))[..., 0]
        w = p / np.where(l == 0, 1, l)
        O[rows] = (w @ V).transpose(1, 0, 2)
        spread[rows] = (w @ np.abs(V)).transpose(1, 0, 2)
    return O, LSE, terms, spread


def keep(cache: Cache, paths, cu, lens):
    """Moves each sequence's path together; returns the new lengths."""
    ps = cache.page_size
    for side in (0, 1):
        codes, scale = cache.codes[side], cache.scale[side]
        for b, path in enumerate(paths):
            base = lens[b] - (cu[b + 1] - cu[b])
            was_codes, was_scale = codes.copy(), scale.copy()
            where = {base + j: base + p for j, p in enumerate(path)}  # slot of the result: token it comes from
            for i in sorted({t // ps for t in where}):
                page = cache.table[b, i]
                sources = {t: where.get(t, t) for t in range(i * ps, min((i + 1) * ps, lens[b]))}
                for h in range(codes.shape[1]):
                    top = max([was_scale[page, h]] + [was_scale[cache.table[b, s // ps], h] for t, s in sources.items() if t in where])
                    for t, s in sources.items():
                        from_ = cache.table[b, s // ps]
                        x = was_codes[from_, h, s % ps]
                        if was_scale[from_, h] != top:
                            x = e4m3_encode(e4m3_decode(x) * (was_scale[from_, h] / top))
                        codes[page, h, t % ps] = x
                    scale[page, h] = top
    return np.array([lens[b] - (cu[b + 1] - cu[b]) + len(p) for b, p in enumerate(paths)], np.int32)
