"""fp64 CPU oracle of the rotary and 8-bit cache operators.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares no code with
the CUDA library.  Everything is written from the definitions: e4m3 by its
table of values, rotations as complex products, attention row by row.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def _e4m3_table() -> np.ndarray:
    """The value of each code: sign, 4 exponent bits (bias 7), 3 mantissa bits;
    exponent 0 is subnormal; 0x7F and 0xFF are NaN (there are no infinities)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = -x if c & 128 else x
    out[[0x7F, 0xFF]] = np.nan
    return out


E4M3 = _e4m3_table()


def e4m3_decode(codes) -> np.ndarray:
    return E4M3[np.asarray(codes, np.uint8)]


def e4m3_encode(x) -> np.ndarray:
    """Nearest code, ties to the even mantissa, saturating; NaN stays NaN."""
    x = np.asarray(x, np.float64)
    pos = E4M3[:0x7F]  # ascending
    a = np.minimum(np.abs(x), E4M3_MAX)
    a = np.where(np.isnan(a), 0, a)
    hi = np.clip(np.searchsorted(pos, a), 1, 0x7E)
    lo = hi - 1
    d_lo, d_hi = a - pos[lo], pos[hi] - a
    take = np.where(d_lo < d_hi, lo, np.where(d_hi < d_lo, hi, np.where(lo % 2 == 0, lo, hi)))
    code = take | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def scale_for(values) -> float:
    """The power of two 2^e, -80 <= e <= 120, with the least e for which the
    largest finite magnitude is at most 448 2^e."""
    v = np.abs(np.asarray(values, np.float64))
    v = v[np.isfinite(v)]
    big = float(v.max()) if v.size else 0.0
    e = -80
    while e < 120 and big > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rope_angles(rotary_dim, base, scaling="none", factor=1.0, original_context=0.0, alpha=1.0, beta=32.0):
    """(theta_i, factor on the result) of a rotation's pairs."""
    r = rotary_dim
    if scaling == "ntk":
        base = base * factor ** (r / (r - 2))
    theta = np.array([base ** (-2 * i / r) for i in range(r // 2)])
    if scaling == "linear":
        theta = theta / factor
    m = 1.0
    if scaling == "ramp":
        turns = original_context * theta / (2 * math.pi)
        g = np.clip((turns - alpha) / (beta - alpha), 0, 1)
        theta = theta * (g + (1 - g) / factor)
        m = 0.1 * math.log(factor) + 1
    return theta, m


def rope(x, positions, theta, interleaved=False, result_factor=1.0, inverse=False):
    """x [T, H, D]: pair i of each head as a complex number times
    result_factor e^(+-i p theta_i)."""
    x = np.asarray(x, np.float64)
    n = len(theta)
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    turn = np.exp((-1j if inverse else 1j) * np.outer(np.asarray(positions, np.float64), theta))
    z = (x[..., a] + 1j * x[..., b]) * (result_factor * turn)[:, None, :]
    y = x.copy()
    y[..., a], y[..., b] = z.real, z.imag
    return y


class Cache:
    """A paged cache: code arrays [pages, heads, page_size, dim] and scales
    [pages, heads] for keys and values, and the page table."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale, table):
        self.codes = [np.array(k_codes, np.uint8), np.array(v_codes, np.uint8)]
        self.scale = [np.array(k_scale, np.float64), np.array(v_scale, np.float64)]
        self.table = np.asarray(table)
        self.page_size = self.codes[0].shape[2]

    def append(self, k, v, cu, lens):
        ps = self.page_size
        for side, x in enumerate((k, v)):
            x = np.asarray(x, np.float64)
            for b, total in enumerate(lens):
                n = cu[b + 1] - cu[b]
                held = total - n
                for i in range(held // ps, -(-total // ps)):
                    if n == 0:
                        break
                    lo, hi = max(held, i * ps), min(total, (i + 1) * ps)
                    page = self.table[b, i]
                    for h in range(x.shape[1]):
                        new = x[cu[b] + lo - held:cu[b] + hi - held, h]
                        scale = scale_for(new)
                        first = lo - i * ps
                        if first:
                            was = self.scale[side][page, h]
                            if was >= scale:
                                scale = was
                            else:
                                old = e4m3_decode(self.codes[side][page, h, :first]) * (was / scale)
                                self.codes[side][page, h, :first] = e4m3_encode(old)
                        self.codes[side][page, h, first:hi - i * ps] = e4m3_encode(new / scale)
                        self.scale[side][page, h] = scale

    def numbers(self, side, b, total):
        """[heads, total, dim] of sequence b."""
        ps = self.page_size
        pages = self.table[b, :-(-total // ps)]
        x = e4m3_decode(self.codes[side][pages]) * self.scale[side][pages][..., None, None]
        return x.transpose(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :total]

    def code_sums(self, side, b, total):
        """[heads, dim]: sum over the tokens of |code|, times the sequence's largest scale."""
        x = np.abs(self.numbers(side, b, total))
        if total == 0:
            return x.sum(1)
        scale = self.scale[side][self.table[b, np.arange(total) // self.page_size]].T  # [heads, total]
        return (x / scale[..., None]).sum(1) * scale.max(1)[:, None]

    def _visible(self, total, n, causal):
        j, i = np.arange(total), np.arange(n)
        return (j[None] <= (total - n + i)[:, None]) if causal else np.ones((n, total), bool)

    def attend(self, q, cu, lens, causal=True, scale=0.0):
        """(O, LSE [H, T]) with rows outside the sequences left 0; also, per
        sequence, what the error bounds need: (terms [H, n, L] = scale sum |q k|,
        spread [n, H, D] = sum p |v|)."""
        q = np.asarray(q, np.float64)
        T, H, D = q.shape
        G = H // self.codes[0].shape[1]
        scale = scale or 1 / math.sqrt(D)
        O, LSE = np.zeros(q.shape), np.zeros((H, T))
        terms, spread = [], np.zeros(q.shape)
        for b, total in enumerate(lens):
            n = cu[b + 1] - cu[b]
            K, V = (np.repeat(self.numbers(s, b, total), G, 0) for s in (0, 1))
            x = q[cu[b]:cu[b + 1]].transpose(1, 0, 2)
            s = scale * x @ K.transpose(0, 2, 1)
            terms.append(scale * np.abs(x) @ np.abs(K).transpose(0, 2, 1))
            s = np.where(self._visible(total, n, causal), s, -np.inf)
            m = s.max(-1, initial=-np.inf, keepdims=True)
            m = np.where(np.isfinite(m), m, 0)
            p = np.exp(s - m)
            l = p.sum(-1, keepdims=True)
            with np.errstate(divide="ignore"):
                LSE[:, cu[b]:cu[b + 1]] = (m + np.log(l))[..., 0]
            w = p / np.where(l == 0, 1, l)
            O[cu[b]:cu[b + 1]] = (w @ V).transpose(1, 0, 2)
            spread[cu[b]:cu[b + 1]] = (w @ np.abs(V)).transpose(1, 0, 2)
        return O, LSE, terms, spread

    def weights(self, q, lse, cu, lens, causal=True, scale=0.0):
        """Per sequence [heads, total]: the weights that its tokens receive, and
        the largest scale sum |q k| behind each."""
        q, lse = np.asarray(q, np.float64), np.asarray(lse, np.float64)
        T, H, D = q.shape
        Hk = self.codes[0].shape[1]
        G = H // Hk
        scale = scale or 1 / math.sqrt(D)
        out, terms = [], []
        for b, total in enumerate(lens):
            n = cu[b + 1] - cu[b]
            K = np.repeat(self.numbers(0, b, total), G, 0)
            x = q[cu[b]:cu[b + 1]].transpose(1, 0, 2)
            s = scale * x @ K.transpose(0, 2, 1)
            with np.errstate(invalid="ignore"):
                p = np.where(self._visible(total, n, causal), np.exp(s - lse[:, cu[b]:cu[b + 1], None]), 0)
            out.append(p.reshape(Hk, G * n, total).sum(1))
            terms.append((scale * np.abs(x) @ np.abs(K).transpose(0, 2, 1)).reshape(Hk, G * n, total).max(1, initial=0))
        return out, terms

    def evict(self, weights, lens, budgets, recent, dst: "Cache"):
        """Fills dst's pages; returns per sequence the kept indices [heads, n]."""
        ps, result = self.page_size, []
        heads = self.codes[0].shape[1]
        for b, total in enumerate(lens):
            keep = min(total, budgets[b])
            tail = min(recent, keep)
            rows = []
            for h in range(heads):
                w = np.asarray(weights[b, h, :total - tail], np.float64)
                w = np.where(np.isnan(w), -np.inf, w)
                best = sorted(range(total - tail), key=lambda j: (-w[j], j))[:keep - tail]
                rows.append(sorted(best) + list(range(total - tail, total)))
                for side in (0, 1):
                    for i in range(0, keep, ps):
                        part = rows[h][i:i + ps]
                        pages = [self.table[b, j // ps] for j in part]
                        scale = max(self.scale[side][p, h] for p in pages)
                        to = dst.table[b, i // ps]
                        dst.scale[side][to, h] = scale
                        for slot, (j, p) in enumerate(zip(part, pages)):
                            x = e4m3_decode(self.codes[side][p, h, j % ps]) * (self.scale[side][p, h] / scale)
                            dst.codes[side][to, h, slot] = e4m3_encode(x)
            result.append(np.array(rows, np.int64).reshape(heads, keep))
        return result
