"""The 4-bit cache in numpy, from the layout that include/softmax_rows.h documents: element by element, for the tests."""
from __future__ import annotations

import numpy as np
import torch


def np_of(t: torch.Tensor) -> np.ndarray:
    """A 16-bit or 32-bit float tensor as float64."""
    return t.detach().double().cpu().numpy()


class Cache:
    """Bytes [pages][heads][blocks][20 d] and where each element of a token lies in them."""

    def __init__(self, data: np.ndarray):
        self.data = data
        self.d = data.shape[3] // 20
        self.page = data.shape[2] * 16
        d, G = self.d, self.d // 32
        self.G = G
        r, e = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
        j, w = e // 32, e % 32
        self.k_nibble = 8 * (r * (d // 8) + G * (w // 8) + j) + w % 8
        f, t, p = r // 8, r % 8 // 2, r % 2
        self.v_nibble = 16 * d + 4 * (2 * (((8 * f + w // 4) * 4 + t) * G + j) + p) + w % 4
        r, j = np.meshgrid(np.arange(16), np.arange(G), indexing="ij")
        self.k_half = 8 * d + r * G + j  # fp16 index of the scale; the zero is 16 G further
        self.v_half = 8 * d + 32 * G + 2 * (r // 2 * G + j) + r % 2

    def block(self, table_row, pos, head):
        return self.data[table_row[pos // self.page], head, pos % self.page // 16]

    def token(self, table_row, pos, head):
        """(key, value) of one token in float64."""
        b, r = self.block(table_row, pos, head), pos % 16
        half = b.view(np.float16).astype(np.float64)
        out = []
        for nib, hf in ((self.k_nibble[r], self.k_half[r]), (self.v_nibble[r], self.v_half[r])):
            c = (b[nib // 2] >> (4 * (nib % 2))) & 15
            out.append(c * np.repeat(half[hf], 32) + np.repeat(half[hf + 16 * self.G], 32))
        return out

    def sequence(self, table_row, n, head):
        """Keys and values [n, d] of a sequence's first n tokens."""
        nb = -(-n // 16)
        pages = np.asarray(table_row)[np.arange(nb) * 16 // self.page]
        b = self.data[pages, head, np.arange(nb) * 16 % self.page // 16]  # [nb, 20 d]
        half = b.view(np.float16).astype(np.float64)
        out = []
        for nib, hf in ((self.k_nibble, self.k_half), (self.v_nibble, self.v_half)):
            c = (b[:, nib // 2] >> (4 * (nib % 2)).astype(np.uint8)) & 15
            x = c * np.repeat(half[:, hf], 32, axis=2) + np.repeat(half[:, hf + 16 * self.G], 32, axis=2)
            out.append(x.reshape(-1, self.d)[:n])
        return out

    def amplitude(self, table_row, n, head):
        """Per token and element, 15 s + |z| of keys and values: what their codes and zeros are at most."""
        nb = -(-n // 16)
        pages = np.asarray(table_row)[np.arange(nb) * 16 // self.page]
        half = np.abs(self.data[pages, head, np.arange(nb) * 16 % self.page // 16].view(np.float16).astype(np.float64))
        return [np.repeat(15 * half[:, hf] + half[:, hf + 16 * self.G], 32, axis=2).reshape(-1, self.d)[:n]
                for hf in (self.k_half, self.v_half)]

    def put(self, table_row, pos, head, key, value):
        """Store one token (float32 arrays) with the documented arithmetic."""
        b, r = self.block(table_row, pos, head), pos % 16
        for x, nib, hf in ((key, self.k_nibble[r], self.k_half[r]), (value, self.v_nibble[r], self.v_half[r])):
            c, s, z = quantise(x)
            lo, hi = nib[nib % 2 == 0], nib[nib % 2 == 1]
            b[lo // 2] = (b[lo // 2] & 0xF0) | c[nib % 2 == 0]
            b[hi // 2] = (b[hi // 2] & 0x0F) | (c[nib % 2 == 1] << 4)
            half = b.view(np.float16)
            half[hf], half[hf + 16 * self.G] = s, z


def quantise(x: np.ndarray):
    """Codes, scales and zeros of a float32 array's groups of 32, every float32 operation rounded by itself."""
    x = np.clip(x.astype(np.float32), np.float32(-65504), np.float32(65504)).reshape(-1, 32)
    lo, hi = x.min(1), x.max(1)
    z, s = lo.astype(np.float16), ((hi - lo) / np.float32(15)).astype(np.float16)
    zf, sf = z.astype(np.float32)[:, None], s.astype(np.float32)[:, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.clip(np.rint((x - zf) / sf), 0, 15)
    return np.where(sf > 0, c, 0).astype(np.uint8).reshape(-1), s, z


def rotate(x: np.ndarray, cs: np.ndarray, neighbours: bool) -> np.ndarray:
    """A head's elements (float32) rotated by cs [rotated] (cosines, then sines)."""
    x, half = x.copy(), len(cs) // 2
    c, s = cs[:half], cs[half:]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if neighbours else (slice(0, half), slice(half, 2 * half))
    u, w = x[a].copy(), x[b].copy()
    x[a], x[b] = u * c - w * s, w * c + u * s
    return x


def attention(cache: Cache, table, lens, cu, q: np.ndarray, scale: float):
    """(o, lse, bound on |delta o|, bound on |delta lse|) of q [T, heads, d] in float64; rows of no sequence are NaN.

    The bounds follow the arithmetic.  A score is a sum of d products of q with 15 s + |z| at most, and some 16 further
    fp32 roundings: each is off by 2^-24 of the sum of magnitudes (``big``).  A weight is off by as much again in
    relative terms, by 2^-21 for the exponential, and by 2^-11 for its rounding to fp16; the product with a scale of V is
    rounded to fp16 once more.  Weights are 2^9 times those relative to the maximum, so fp16's smallest steps add at most
    2^-25 / 2^9 to each, twice.  Sums over n keys are at most n / 16 terms long in one lane (2^-24 each).
    """
    T, heads, d = q.shape
    hkv = cache.data.shape[1]
    o, lse = np.full((T, heads, d), np.nan), np.full((T, heads), np.nan)
    do, dl = np.zeros((T, heads, d)), np.zeros((T, heads))
    for b, n in enumerate(lens):
        new = cu[b + 1] - cu[b]
        for h in range(hkv):
            k, v = cache.sequence(table[b], n, h)
            ka, va = cache.amplitude(table[b], n, h)
            va = va.max(0) if n else 0
            for t in range(new):
                see, i = max(0, n - new + t + 1), cu[b] + t
                for hq in range(h * (heads // hkv), (h + 1) * (heads // hkv)):
                    if see == 0:
                        o[i, hq], lse[i, hq] = 0, -np.inf
                        continue
                    z = k[:see] @ q[i, hq] * scale
                    m = z.max()
                    p = np.exp(z - m)
                    l = p.sum()
                    o[i, hq], lse[i, hq] = p @ v[:see] / l, m + np.log(l)
                    big = (ka[:see] @ np.abs(q[i, hq])).max() * scale
                    ds = (d + 16) * 2.0 ** -24 * big
                    dw = 2 * ds + 2.0 ** -21 + (see / 16 + 64) * 2.0 ** -24
                    do[i, hq] = va * (2 * 2.0 ** -11 + 2 * dw + see * 2.0 ** -33)
                    dl[i, hq] = ds + dw + 2.0 ** -22 * (abs(m) + np.log(see + 1) + 9)
    return o, lse, do, dl
