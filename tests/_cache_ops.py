"""Plain 64-bit forms of the 4-bit cache, recorded weights and eviction, and their inputs."""
from __future__ import annotations

import numpy as np
import torch

BLOCK = 32


# ------------------------------------------------------------------ 4-bit codec
def quantize(x):
    """x [..., D] -> (codes int [..., D], scales float16 [..., D/32]) in fp64."""
    x = np.nan_to_num(np.asarray(x, dtype=np.float64), nan=0.0, posinf=np.inf, neginf=-np.inf)
    x = np.clip(x, -7 * 65504.0, 7 * 65504.0)
    blk = x.reshape(*x.shape[:-1], -1, BLOCK)
    s = (np.abs(blk).max(-1) / 7.0).astype(np.float16)
    sd = s.astype(np.float64)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(sd > 0, np.rint(blk / sd), 0.0)
    return np.clip(c, -7, 7).astype(np.int64).reshape(x.shape), s


def pack(codes):
    """Codes [..., D] -> bytes [..., D/2]: word o * (D/32) + j holds elements 32j + 8o + n."""
    D = codes.shape[-1]
    out = np.zeros((*codes.shape[:-1], D // 2), dtype=np.uint8)
    for e in range(D):
        j, o, n = e // 32, e % 32 // 8, e % 8
        at = (o * (D // 32) + j) * 4 + n // 2
        out[..., at] |= ((codes[..., e] + 8) << (4 * (n % 2))).astype(np.uint8)
    return out


def unpack(by):
    D = by.shape[-1] * 2
    out = np.zeros((*by.shape[:-1], D), dtype=np.int64)
    for e in range(D):
        j, o, n = e // 32, e % 32 // 8, e % 8
        at = (o * (D // 32) + j) * 4 + n // 2
        out[..., e] = ((by[..., at] >> (4 * (n % 2))) & 15).astype(np.int64) - 8
    return out


def dequantize(by, scales):
    s = np.repeat(np.asarray(scales, dtype=np.float64), BLOCK, axis=-1)
    return unpack(by) * s


# ------------------------------------------------------------------ cache layouts
class Layout:
    """Where token t of (sequence, head) lives: paged through a shuffled table with
    spare blocks, or contiguous.  `cap` tokens per sequence; `room`: a table with that
    many tokens of capacity, its entries beyond `cap` unmapped."""

    def __init__(self, batch, hkv, cap, paged, page=16, spare=2, seed=0, room=0):
        self.room = room
        self.batch, self.hkv, self.cap, self.page, self.paged = batch, hkv, cap, page, paged
        if paged:
            self.blocks = -(-cap // page)
            self.cap = self.blocks * page
            total = batch * self.blocks + spare
            perm = np.random.RandomState(seed).permutation(total)[:batch * self.blocks]
            self.table = perm.reshape(batch, self.blocks).astype(np.int32)
            self.rows = (total, hkv, page)
        else:
            self.table = None
            self.rows = (batch, hkv, cap)

    def dense(self, x, b):
        """Sequence b's rows [Hkv, cap, ...] of a cache array."""
        if not self.paged:
            return x[b]
        y = x[self.table[b]]                            # [blocks, Hkv, page, ...]
        return np.moveaxis(y, 0, 1).reshape(self.hkv, self.cap, *x.shape[3:])

    def put(self, x, b, rows):
        """Write sequence b's rows [Hkv, cap, ...] back."""
        if not self.paged:
            x[b] = rows
            return
        y = rows.reshape(self.hkv, self.blocks, self.page, *x.shape[3:])
        x[self.table[b]] = np.moveaxis(y, 1, 0)

    def used(self, lens):
        """Which cache rows hold a token, as a bool array of the cache's row shape."""
        m = np.zeros(self.rows, dtype=bool)
        for b, n in enumerate(lens):
            d = np.zeros((self.hkv, self.cap), dtype=bool)
            d[:, :n] = True
            if self.paged:
                y = d.reshape(self.hkv, self.blocks, self.page)
                m[self.table[b]] = np.moveaxis(y, 1, 0)
            else:
                m[b] = d
        return m

    @property
    def capacity(self):
        """Tokens per sequence that the table (or the contiguous cache) has room for."""
        return max(self.cap, -(-self.room // self.page) * self.page if self.paged else 0)

    def table_gpu(self):
        if self.table is None:
            return None
        more = self.capacity // self.page - self.table.shape[1]
        return torch.from_numpy(np.pad(self.table, ((0, 0), (0, more)), constant_values=-1)).cuda()


def ranges(n, tq, window, cap):
    """[(lo, hi)] of the keys that each of the tq queries attends."""
    n = min(max(n, 0), cap)
    got = []
    for i in range(tq):
        hi = max(n - tq + 1 + i, 0)
        got.append((hi - window if 0 < window < hi else 0, hi))
    return got


def attend(q, k, v, lens, lay, scale, window=None):
    """fp64 attention.  q [B, tq, Hq, D]; k(b), v(b) -> [Hkv, cap, D] fp64.
    Returns out, sum p |v|, the largest sum |q||k| scale of any row, and the
    per-key weights [B][Hkv, cap]."""
    B, tq, Hq, D = q.shape
    G = Hq // lay.hkv
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    out = np.zeros(q.shape)
    absum = np.zeros(q.shape)
    weights, size = [], 0.0
    for b in range(B):
        kb = torch.from_numpy(np.nan_to_num(k(b), nan=0.0)).to(dev)
        vb = torch.from_numpy(np.nan_to_num(v(b), nan=0.0)).to(dev)
        qb = torch.from_numpy(q[b].astype(np.float64)).to(dev)
        wt = torch.zeros((lay.hkv, lay.cap), dtype=torch.float64, device=dev)
        for i, (lo, hi) in enumerate(ranges(lens[b], tq, 0 if window is None else window[b],
                                            lay.cap)):
            if hi <= lo:
                continue
            for h in range(lay.hkv):
                qq = qb[i, h * G:(h + 1) * G]
                p = torch.softmax(qq @ kb[h, lo:hi].T * scale, dim=-1)
                size = max(size, float((qq.abs() @ kb[h, lo:hi].abs().T).max()) * abs(scale))
                out[b, i, h * G:(h + 1) * G] = (p @ vb[h, lo:hi]).cpu().numpy()
                absum[b, i, h * G:(h + 1) * G] = (p @ vb[h, lo:hi].abs()).cpu().numpy()
                wt[h, lo:hi] += p.sum(0)
        weights.append(wt.cpu().numpy())
    return out, absum, size, weights


def score_slack(size, D):
    """Relative error of a weight from the fp32 scores: D products summed in any order
    (2^-23 per addition of the tensor cores' truncated sums, of their absolute sum), in
    the score itself and in the normaliser, and ex2's and the sums' own roundings."""
    return 2 * D * 2.0 ** -23 * size + 2.0 ** -18


def out_tolerance(out, absum, size, D, n=0, smax=0.0):
    """P and P * scale are rounded to fp16 (2^-11 each), the result once more.

    Below 2^-14 those two roundings are of fixed steps of 2^-24, so each is off by up to 2^-25
    whatever the value: of P (times a value of at most 7 smax) and of P * scale (times a code of
    at most 7), for each of n keys, over a weight sum of at least 1 (the running maximum never
    passes a row's largest score).  P * scale is carried times 2^-e: e = 0 while the largest scale
    smax lies in [2^-12, 2^7), else 2^e <= max(2 smax, 2^-14)."""
    unit = 1.0 if 2.0 ** -12 <= smax < 2.0 ** 7 else max(2 * smax, 2.0 ** -14)
    fixed = n * 2.0 ** -25 * (7 * smax + 7 * unit) if smax else 0.0
    return ((2 * 2.0 ** -11 + score_slack(size, D)) * absum + 2.0 ** -11 * np.abs(out) +
            2.0 ** -24 + fixed)


def acc_tolerance(before, added, size, D, cols):
    """The weight's own error, `cols` fp32 additions of it and one to the running total."""
    return added * (score_slack(size, D) + cols * 2.0 ** -24) + 2.0 ** -23 * (np.abs(before) + added)


# ------------------------------------------------------------------ eviction
def select(acc, n, budget, sink, recent):
    """Kept token indices of one (sequence, head): acc [cap]."""
    if n <= budget:
        return list(range(n))
    a = np.where(np.isnan(acc), -np.inf, acc.astype(np.float64))
    mid = sorted(range(sink, n - recent), key=lambda t: (-a[t], t))
    return sorted(list(range(sink)) + mid[:budget - sink - recent] + list(range(n - recent, n)))


def evict(arrays, acc, lay, lens, budget, sink, recent):
    """New arrays, acc, kept and lengths (numpy copies)."""
    arrays = [a.copy() for a in arrays]
    acc = acc.copy()
    kept = np.full((lay.batch, lay.hkv, budget), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        n = min(max(n, 0), lay.cap)
        dense = [lay.dense(a, b).copy() for a in arrays]
        total = lay.dense(acc, b).copy()
        for h in range(lay.hkv):
            idx = select(total[h], n, budget, sink, recent)
            kept[b, h, :len(idx)] = idx
            if n <= budget:
                continue
            for d in dense:
                d[h, :budget] = d[h, idx].copy()
            total[h, :budget] = total[h, idx].copy()
            total[h, budget:n] = 0
        for a, d in zip(arrays, dense):
            lay.put(a, b, d)
        lay.put(acc, b, total)
    return arrays, acc, kept, np.minimum(np.clip(lens, 0, lay.cap), budget).astype(np.int32)


# ------------------------------------------------------------------ inputs
class Int4Cache:
    """A 4-bit cache of N(0, 1) * k_mag / v_mag rows; rows behind the lengths hold NaN
    scales and arbitrary codes."""

    def __init__(self, lay, D, lens, seed=0, k_mag=1.0, v_mag=1.0):
        r = np.random.RandomState(seed)
        self.lay, self.D = lay, D
        used = lay.used(lens)
        got = {}
        for name, mag in (("k", k_mag), ("v", v_mag)):
            x = r.standard_normal((*lay.rows, D)) * np.asarray(mag)
            codes, s = quantize(x.astype(np.float32))
            by = pack(codes)
            by[~used] = r.randint(0, 256, by[~used].shape)
            s[~used] = np.nan
            got[name] = (by, s)
        (self.k, self.ks), (self.v, self.vs) = got["k"], got["v"]

    def tolerance(self, out, absum, size):
        return out_tolerance(out, absum, size, self.D, self.lay.cap, float(np.nanmax(self.vs)))

    def gpu(self):
        return [torch.from_numpy(x.copy()).cuda() for x in (self.k, self.ks, self.v, self.vs)]

    def key(self, b):
        return dequantize(self.lay.dense(self.k, b), self.lay.dense(self.ks, b))

    def value(self, b):
        return dequantize(self.lay.dense(self.v, b), self.lay.dense(self.vs, b))


def queries(B, tq, Hq, D, seed, mag=1.0):
    q = np.random.RandomState(seed + 77).standard_normal((B, tq, Hq, D)) * mag
    return q.astype(np.float16)


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def lens_gpu(lens):
    return torch.tensor(list(lens), dtype=torch.int32, device="cuda")
