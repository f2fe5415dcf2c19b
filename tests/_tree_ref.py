"""Plain 64-bit forms of the tree and cache operators, written from their
definitions in include/dfl2.h, one entry at a time; host memory only."""
import numpy as np
import torch

HALF_ULP = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}  # 8 and 11 significant bits
DENORMAL = {torch.bfloat16: 0.0, torch.float16: 2.0**-25}


def ancestors(parents):
    """bool [T,T]: j is i or an ancestor of i."""
    T = len(parents)
    a = np.zeros((T, T), bool)
    for i in range(T):
        j = i
        while j >= 0:
            a[i, j] = True
            j = parents[j]
    return a


def pack_bits(a):
    """bool [..., T] -> int32 words [..., ceil(T/32)], bit j of word j // 32."""
    T = a.shape[-1]
    W = (T + 31) // 32
    out = np.zeros(a.shape[:-1] + (W,), np.uint32)
    for j in range(T):
        out[..., j // 32] |= a[..., j].astype(np.uint32) << np.uint32(j % 32)
    return out.view(np.int32)


def attention(q, keys, vals, seen, scale):
    """One sequence: q [T,Hq,D], keys, vals [n,Hkv,D], seen bool [T,n].  Returns out,
    lse and, for the error bounds, sum_j p|v|, the largest |score| term sum and
    sum_j |v| / sum_j exp(s_j - max); all float64."""
    T, Hq, D = q.shape
    Hkv = keys.shape[1]
    out = np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    mass = np.zeros((T, Hq, D))
    mag = np.zeros((T, Hq))
    tail = np.zeros((T, Hq, D))
    for i in range(T):
        at = np.nonzero(seen[i])[0]
        if len(at) == 0:
            continue
        for h in range(Hq):
            g = h * Hkv // Hq
            k, v = keys[at, g], vals[at, g]
            s = (k @ q[i, h]) * scale
            mag[i, h] = np.max(np.abs(k) @ np.abs(q[i, h])) * abs(scale)
            m = s.max()
            e = np.exp(s - m)
            z = e.sum()
            lse[i, h] = m + np.log(z)
            with np.errstate(invalid="ignore"):
                out[i, h] = (e / z) @ v
                mass[i, h] = (e / z) @ np.abs(v)
                tail[i, h] = np.abs(v).sum(0) / z
    return out, lse, mass, mag, tail


def attention_bounds(ref, dtype, D, n):
    """How far the kernel may be from attention()'s values.

    Scores: D products summed in float32 (each addition rounds by 2^-24 of at most
    the sum of the terms' sizes), then the scaling and 2^x (its argument rounds by
    2^-24 of its size, 2^x itself by 2 units): the weights are off by a factor of
    1 + e.  They are rounded to the type for the product with V (half a unit
    each), numerator and denominator are sums of n float32 terms, and the result
    is rounded once to the type.  float16 also loses what lies under half its
    smallest number."""
    out, lse, mass, mag, tail = ref
    u = HALF_ULP[dtype]
    e = (D + 8) * 2.0**-24 * mag + 2.0**-21
    sums = n * 2.0**-24
    ob = u * np.abs(out) + (u + (2 * e + 2 * sums)[..., None]) * mass
    ob = ob * 1.01 + DENORMAL[dtype] * (tail + 1) + 1e-30
    lb = e + sums + 2.0**-22 * (np.abs(np.where(np.isfinite(lse), lse, 0)) + 1)
    return ob, lb


class CacheModel:
    """The page bookkeeping of one cache, and every position's row as a number."""

    def __init__(self, rows, cols, pages, ps):
        self.ps, self.cols = ps, cols
        self.table = np.full((rows, cols), -1, np.int32)
        self.refs = np.zeros(pages, np.int32)
        self.val = np.zeros((pages, ps), np.int64)  # stands for the K/V row

    def free_pages(self):
        return np.nonzero(self.refs == 0)[0]

    def bits(self):
        return pack_bits((self.refs == 0)[None])[0]

    def _spans(self, spans):
        """[(row, c0, c1, ok)] in order -> served flags, pages filled in."""
        left = list(self.free_pages())
        have, cum, served = len(left), 0, []
        for row, c0, c1, ok in spans:
            if not ok:
                served.append(0)
                continue
            miss = [c for c in range(c0, c1) if self.table[row, c] < 0]
            cum += len(miss)
            if miss and cum > have:
                served.append(0)
                continue
            for c in miss:
                p = left.pop(0)
                self.table[row, c] = p
                self.refs[p] = 1
            served.append(1)
        return served

    def reserve(self, rows, length, count):
        ps = self.ps
        return self._spans([(r, n // ps, -(-(n + c) // ps), -(-(n + c) // ps) <= self.cols)
                            for r, n, c in zip(rows, length, count)])

    def at(self, row, pos):
        return self.table[row, pos // self.ps], pos % self.ps

    def write(self, rows, length, count, vals):
        for b, (r, n, c) in enumerate(zip(rows, length, count)):
            for t in range(c):
                self.val[self.at(r, n + t)] = vals[b, t]

    def drop(self, row, c0, c1):
        for c in range(c0, min(c1, self.cols)):
            p = self.table[row, c]
            if p >= 0:
                self.refs[p] -= 1
                self.table[row, c] = -1

    def compact(self, rows, length, count, path, n_path):
        for b, (r, n, c) in enumerate(zip(rows, length, count)):
            got = [self.val[self.at(r, n + path[b][i])] for i in range(n_path[b])]
            for i, x in enumerate(got):
                self.val[self.at(r, n + i)] = x
            self.drop(r, -(-(n + n_path[b]) // self.ps), -(-(n + c) // self.ps))
        return [n + k for n, k in zip(length, n_path)]

    def fork(self, src, dst, length):
        ps = self.ps
        spans = []
        for a, z, n in zip(src, dst, length):
            c1 = -(-n // ps)
            ok = c1 <= self.cols and (self.table[z, :c1] < 0).all() and (self.table[a, :c1] >= 0).all()
            spans.append((z, n // ps, c1, ok))
        served = self._spans(spans)
        for a, z, n, ok in zip(src, dst, length, served):
            if not ok:
                continue
            for c in range(n // ps):
                self.table[z, c] = self.table[a, c]
                self.refs[self.table[a, c]] += 1
            for s in range(n % ps):
                self.val[self.table[z, n // ps], s] = self.val[self.table[a, n // ps], s]
        return served

    def free(self, rows):
        for r in rows:
            self.drop(r, 0, self.cols)
