"""Plain implementation of the block-scaled cache and its attention (numpy, no code
shared with the kernels): the producer in fp32 step by step, attention in fp64."""
from __future__ import annotations

import numpy as np

BS = 16
U16, U24 = 2.0 ** -11, 2.0 ** -24   # half a step of f16 and fp32, relative


def bf16(x):
    """fp32 array rounded to nearest-even bf16, as fp32 values."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32)


def tables(rng, lens, extra=2, max_blocks=None):
    """Block tables [B, max_blocks] over a shuffled pool; unused entries point outside of it."""
    n = [(L + BS - 1) // BS for L in lens]
    nb = sum(n) + extra
    mb = max_blocks or max(1, max(n))
    perm = rng.permutation(nb).astype(np.int32)
    out = np.full((len(lens), mb), nb + 7, np.int32)
    at = 0
    for b, k in enumerate(n):
        out[b, :k] = perm[at:at + k]
        at += k
    return out, nb


class Cache:
    """Codes by (block, head, token, dim) and scales by (block, head)."""

    def __init__(self, NB, Hkv, D):
        self.codes = {"k": np.zeros((NB, Hkv, BS, D), np.int8), "v": np.zeros((NB, Hkv, BS, D), np.int8)}
        self.scale = {"k": np.zeros((NB, Hkv), np.float32), "v": np.zeros((NB, Hkv), np.float32)}

    def random(self, rng, zero_blocks=0.0, spread=1.0):
        for w in "kv":
            NB, Hkv, _, D = self.codes[w].shape
            x = rng.standard_normal((NB, Hkv, BS, D)).astype(np.float32)
            x *= np.exp2(rng.uniform(-spread, spread, (NB, Hkv, 1, 1))).astype(np.float32)
            if w == "v" and zero_blocks:
                x[rng.random((NB, Hkv)) < zero_blocks] = 0
            s = (np.abs(x).max((2, 3)) / np.float32(127)).astype(np.float32)
            with np.errstate(divide="ignore", invalid="ignore"):
                q = np.where(s[..., None, None] > 0, np.rint(x / s[..., None, None]), 0)
            self.codes[w] = np.clip(q, -127, 127).astype(np.int8)
            self.scale[w] = s
        return self

    def write(self, x, lens, news, table):
        """The ragged producer; x = {"k": [T, Hkv, D], "v": ...} fp32 (bf16 values)."""
        for w in "kv":
            codes, scale = self.codes[w], self.scale[w]
            at = 0
            for b, (L, n) in enumerate(zip(lens, news)):
                for lb in range((L - n) // BS, (L + BS - 1) // BS if n else 0):
                    f, e = max(0, L - n - lb * BS), min(BS, L - lb * BS)
                    rows = x[w][at + lb * BS + f - (L - n): at + lb * BS + e - (L - n)]
                    blk = table[b, lb]
                    for h in range(codes.shape[1]):
                        old = scale[blk, h] if f else np.float32(0)
                        s = max(old, np.float32(np.abs(rows[:, h]).max() / np.float32(127)))
                        if f and s != old:
                            r = np.float32(old / s)
                            codes[blk, h, :f] = np.rint((codes[blk, h, :f].astype(np.float32) * r).astype(np.float32)).astype(np.int8)
                        if f == 0 or s != old:
                            scale[blk, h] = s
                        if s > 0:
                            codes[blk, h, f:e] = np.rint((rows[:, h] / s).astype(np.float32)).astype(np.int8)
                        else:
                            codes[blk, h, f:e] = 0
                at += n

    def paged(self, w):
        c = self.codes[w]
        NB, H, _, D = c.shape
        if w == "k":
            return np.ascontiguousarray(c.reshape(NB, H, BS, D // 16, 16).transpose(0, 1, 3, 2, 4))
        return np.ascontiguousarray(c.transpose(0, 1, 3, 2))

    def history(self, table_row, L, w):
        """fp32 products code x scale [L, Hkv, D]."""
        pos = np.arange(L)
        blk = table_row[pos // BS]
        return self.codes[w][blk, :, pos % BS].astype(np.float32) * self.scale[w][blk][..., None]


def attend(q, cache, table_row, n, lo, hi, pos, scale, cap=0.0, slopes=None, bits16=True):
    """fp64 attention of rows q [R, Hq, D] over the first n tokens of a sequence; row r sees keys lo[r] .. hi[r] - 1.

    Returns (out, err): err bounds what a kernel may be off before the output's own rounding.  With u the score in
    log2 units and p the weights, the score's error e_u (log2 units) and the weight's relative rounding r give
      |d out| <= sum_t p_t (|v_t| + |out|) (ln2 e_u + r)
    e_u: the dot product's fp32 accumulation, (D / 16 + 4) roundings of the largest partial sum (<= sum |q k|); five
    roundings of u itself and of terms up to 32 (the block's log2 scale, the running maximum); the cap's 1 - 2/(e + 1),
    four roundings of numbers up to 2 cap.  A hardware 2^x is good to 2^-22.  r: half a step of f16, 2^-11, or for two
    f16 parts 2^-22, and the fp32 sums over n keys (one rounding per 16 of them and a join of 64).
    Weights w = p sV in units of the largest meet the codes; below f16's normal range they keep an absolute 2^-25 of
    that unit, so 2^-25 max(p sV) sum |code| more."""
    R, Hq, D = q.shape
    k, v = cache.history(table_row, n, "k"), cache.history(table_row, n, "v")
    where = table_row[np.arange(n) // BS]
    codes, vs = cache.codes["v"][where, :, np.arange(n) % BS], cache.scale["v"][where]
    Hkv = k.shape[1]
    out = np.zeros((R, Hq, D))
    err = np.zeros((R, Hq, D))
    t = np.arange(n)
    ln2, log2e = np.log(2.0), 1.0 / np.log(2.0)
    for r in range(R):
        a, b = max(0, lo[r]), min(n, hi[r])
        if a >= b:
            continue
        for h in range(Hq):
            kk, vv = k[a:b, h // (Hq // Hkv)].astype(np.float64), v[a:b, h // (Hq // Hkv)].astype(np.float64)
            qq = q[r, h].astype(np.float64)
            s = kk @ qq * scale
            mag = np.abs(kk) @ np.abs(qq) * abs(scale) * log2e
            e_u = U24 * 2 * (D / 16 + 4) * mag
            if cap:
                s = cap * np.tanh(s / cap)
                e_u = e_u + U24 * 8 * cap * log2e
            if slopes is not None:
                s = s - float(slopes[h]) * np.abs(pos[r] - t[a:b])
            e_u = e_u + U24 * 5 * (np.abs(s - s.max()) * log2e + np.abs(s.max()) * log2e + 32)
            p = np.exp(s - s.max())
            p /= p.sum()
            o = p @ vv
            out[r, h] = o
            rel = ln2 * e_u + 2.0 ** -22 + (U16 if bits16 else 2.0 ** -22) + U24 * ((b - a) / 16 + 64)
            err[r, h] = (p * rel) @ (np.abs(vv) + np.abs(o))
            g = h // (Hq // Hkv)
            err[r, h] += 2.0 ** -25 * (p * vs[a:b, g]).max() * np.abs(codes[a:b, g].astype(np.float64)).sum(0)
    return out, err
