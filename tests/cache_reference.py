"""Plain 64-bit implementations of the cache operators on the CPU, the
references of the GPU tests."""
import math

import numpy as np
import torch

NAN_CODE = 0x7F


def code_values():
    """The 256 e4m3 codes' values."""
    out = np.zeros(256)
    for c in range(256):
        s, e, m = (-1.0 if c & 0x80 else 1.0), (c >> 3) & 15, c & 7
        if (c & 0x7F) == NAN_CODE:
            out[c] = np.nan
        else:
            out[c] = s * (m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
    return out


VALUES = code_values()


def encode(x):
    """e4m3 values of x: nearest, ties to even, saturated at 448, NaN kept."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    with np.errstate(invalid="ignore"):
        e = np.maximum(np.frexp(np.where(a > 0, a, 1.0))[1] - 1, -6)
        step = np.ldexp(1.0, e - 3)
        r = np.minimum(np.round(a / step) * step, 448.0)
    return np.where(np.isnan(x), np.nan, np.copysign(r, x))


def fit_scale(x):
    """The smallest 2^e, e >= -100, that brings the finite values of x within 448."""
    f = np.abs(x[np.isfinite(x)])
    amax = float(f.max()) if f.size else 0.0
    e = -100
    while amax > math.ldexp(448.0, e):
        e += 1
    return math.ldexp(1.0, e)


class Pool:
    """The pools as 64-bit values of the codes (without the scale)."""

    def __init__(self, k, v, k_scale, v_scale):
        self.codes = {"k": VALUES[k], "v": VALUES[v]}       # from uint8 arrays (P, H, ps, D)
        self.scale = {"k": k_scale.astype(np.float64), "v": v_scale.astype(np.float64)}
        self.pages, self.heads, self.ps, self.dim = k.shape

    def page(self, table, b, j):
        p = int(table[b, j // self.ps])
        return p if 0 <= p < self.pages else -1

    def append(self, new_k, new_v, table, start, count=None):
        for name, new in (("k", new_k), ("v", new_v)):
            B, L, H, _ = new.shape
            for b in range(B):
                n = L if count is None else min(max(int(count[b]), 0), L)
                at = {}
                for j in range(n):
                    pos = int(start[b]) + j
                    if 0 <= pos < table.shape[1] * self.ps and self.page(table, b, pos) >= 0:
                        at.setdefault(self.page(table, b, pos), []).append((pos % self.ps, j))
                for page, slots in at.items():
                    first = slots[0][0]
                    for h in range(H):
                        x = np.stack([new[b, j, h] for _, j in slots])
                        s = fit_scale(x)
                        if first > 0:
                            old = self.scale[name][page, h]
                            s = max(s, old)
                            if s != old:
                                self.codes[name][page, h, :first] = encode(self.codes[name][page, h, :first] * old / s)
                        for i, (slot, _) in enumerate(slots):
                            self.codes[name][page, h, slot] = encode(x[i] / s)
                        self.scale[name][page, h] = s

    def tokens(self, name, table, b, h, positions):
        out = np.zeros((len(positions), self.dim))
        for i, j in enumerate(positions):
            p = self.page(table, b, j)
            if p >= 0:
                out[i] = self.codes[name][p, h, j % self.ps] * self.scale[name][p, h]
        return out

    def attend(self, q, table, lens, scale, mask=None):
        """(out, lse, probabilities' sums per token, and the error scales
        sum p |v| and max_j scale max|q| sum |k|) of 64-bit q (B, L, Hq, D)."""
        B, L, Hq, D = q.shape
        H, cap = self.heads, table.shape[1] * self.ps
        G = Hq // H
        out, spread = np.zeros((B, L, Hq, D)), np.zeros((B, L, Hq, D))
        lse, size = np.full((B, L, Hq), -np.inf), np.zeros((B, L, Hq))
        weights = np.zeros((B, H, cap))
        for b in range(B):
            n = min(max(int(lens[b]), 0), cap)
            pos = [j for j in range(n) if self.page(table, b, j) >= 0 and (mask is None or mask[b, j])]
            if not pos:
                continue
            for h in range(H):
                k, v = self.tokens("k", table, b, h, pos), self.tokens("v", table, b, h, pos)
                r = q[b, :, h * G:(h + 1) * G].reshape(L * G, D)
                with np.errstate(invalid="ignore", over="ignore"):
                    x = (r @ k.T) * scale
                    m = x.max(1)
                    p = np.exp(x - m[:, None])
                    z = m + np.log(p.sum(1))
                    p = p / p.sum(1)[:, None]
                    out[b, :, h * G:(h + 1) * G] = (p @ v).reshape(L, G, D)
                    spread[b, :, h * G:(h + 1) * G] = (p @ np.abs(v)).reshape(L, G, D)
                    size[b, :, h * G:(h + 1) * G] = (scale * np.abs(r).max(1) * np.abs(k).sum(1).max()).reshape(L, G)
                lse[b, :, h * G:(h + 1) * G] = z.reshape(L, G)
                ok = np.isfinite(z)
                weights[b, h, pos] = p[ok].sum(0)
        return out, lse, weights, spread, size

    def evict(self, table, lens, weights, budget, first, last, dst):
        B, H, cap = weights.shape
        keep = np.full((B, H, budget), -1, dtype=np.int32)
        moved = np.zeros((B, H, cap), dtype=weights.dtype)
        new_lens = np.zeros(B, dtype=np.int32)
        for b in range(B):
            n = min(max(int(lens[b]), 0), cap)
            m = min(n, budget)
            new_lens[b] = m
            for h in range(H):
                w = np.where(np.isnan(weights[b, h]), -np.inf, weights[b, h].astype(np.float64))
                nan = np.isnan(weights[b, h])
                edge = [j for j in range(n) if j < first or j >= n - last]
                rest = sorted((j for j in range(n) if first <= j < n - last), key=lambda j: (nan[j], -w[j], j))
                ids = sorted(edge + rest[:m - len(edge)]) if m < n else list(range(n))
                keep[b, h, :m] = ids
                moved[b, h, :m] = weights[b, h, ids]
                for name in ("k", "v"):
                    x = self.tokens(name, table, b, h, ids)
                    for col in range(-(-m // self.ps)):
                        to = int(dst[b, col])
                        if not 0 <= to < self.pages:
                            continue
                        y = x[col * self.ps:(col + 1) * self.ps]
                        s = fit_scale(y)
                        self.codes[name][to, h, :len(y)] = encode(y / s)
                        self.scale[name][to, h] = s
        return keep, new_lens, moved


def random_pool(rng, pages, heads, ps, dim, device="cuda", spread=3):
    """uint8 codes without NaN and power-of-two scales, as host arrays."""
    def codes():
        x = torch.from_numpy(rng.standard_normal((pages, heads, ps, dim)) * 100).float().clamp(-448, 448)
        return x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()

    def scales():
        return np.exp2(-rng.integers(6, 6 + spread, (pages, heads))).astype(np.float32)

    return codes(), codes(), scales(), scales()


def same_values(got, want):
    """Whether uint8 codes stand for the 64-bit values `want` (-0 equals 0)."""
    g = VALUES[got]
    return np.array_equal(np.isnan(g), np.isnan(want)) and np.array_equal(g[~np.isnan(g)], want[~np.isnan(want)])
