"""CPU model of the 8-bit block cache: a unit is a list of blocks that hold their tokens' 16-bit rows.

Codes, scales and key bounds are functions of a block's rows alone, taken in float32 as the quantiser fixes them;
attention is float64 over the dequantised rows; block scores are exact integers times float32 scales.
"""
from __future__ import annotations

import numpy as np

SMALLEST = np.float32(2.0 ** -64)


def e4m3_values():
    """The finite values of the codes 0 .. 126 (sign bit clear): 3 mantissa bits, exponent bias 7."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))


E4M3 = e4m3_values()


def round_e4m3(x):
    """Nearest e4m3 code of float32 x (ties to the even code), saturated: uint8."""
    a = np.minimum(np.abs(x.astype(np.float64)), 448.0)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, up = a - E4M3[lo], E4M3[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def decode(codes, kind):
    """float64 values of uint8 codes of `kind` ("e4m3" or "int8")."""
    if kind == "int8":
        return codes.astype(np.uint8).view(np.int8).astype(np.float64)
    c = codes.astype(np.int64)
    return np.where(c & 128, -1.0, 1.0) * E4M3[np.minimum(c & 127, 126)]


def scale_of(x, qmax):
    inv = np.float32(1.0) / np.float32(qmax)
    return max(np.float32(np.abs(x).max().astype(np.float32) * inv), SMALLEST)


def quantise(x, kind):
    """Codes uint8 and scale of the rows x [n, D] (float32 values of 16-bit numbers) of one block."""
    x = x.astype(np.float32)
    if not np.isfinite(x).all():
        return np.zeros(x.shape, np.uint8), np.float32(np.nan)
    s = scale_of(x, 448.0 if kind == "e4m3" else 127.0)
    y = x * (np.float32(1.0) / s)
    if kind == "e4m3":
        return round_e4m3(y), s
    return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8), s


def bounds(x):
    """Key bounds int8 [2, D] (low, high) and their scale."""
    x = x.astype(np.float32)
    if not np.isfinite(x).all():
        return np.zeros((2, x.shape[1]), np.int8), np.float32(np.nan)
    s = scale_of(x, 127.0)
    inv = np.float32(1.0) / s
    lo = np.clip(np.floor(x.min(axis=0) * inv), -127, 127)
    hi = np.clip(np.ceil(x.max(axis=0) * inv), -127, 127)
    return np.stack([lo, hi]).astype(np.int8), s


class Block:
    def __init__(self, pos, D):
        self.pos, self.acc = pos, 0.0
        self.k, self.v = np.zeros((0, D), np.float32), np.zeros((0, D), np.float32)


class Unit:
    """One (sequence, KV head)."""

    def __init__(self, D, block, kind):
        self.D, self.P, self.kind, self.blocks, self.seq_len = D, block, kind, [], 0

    @property
    def count(self):
        return sum(len(b.k) for b in self.blocks)

    def append(self, k, v, weight=None):
        for i in range(len(k)):
            if not self.blocks or len(self.blocks[-1].k) == self.P:
                self.blocks.append(Block(self.seq_len, self.D))
            b = self.blocks[-1]
            b.k, b.v = np.concatenate([b.k, k[i:i + 1]]), np.concatenate([b.v, v[i:i + 1]])
            if weight is not None:
                b.acc += float(weight[i])
            self.seq_len += 1

    def dequantised(self):
        """Keys and values [count, D] as the codes give them, float64."""
        out = []
        for name in ("k", "v"):
            rows = [np.zeros((0, self.D))]
            for b in self.blocks:
                codes, s = quantise(getattr(b, name), self.kind)
                rows.append(decode(codes, self.kind) * np.float64(s))
            out.append(np.concatenate(rows))
        return out

    def seen(self, limit, chosen=None):
        """Which tokens a query sees that is allowed the first `limit`, of the chosen blocks."""
        t = np.arange(self.count)
        m = t < limit
        return m if chosen is None else m & np.isin(t // self.P, chosen)

    def evict(self, keep, n_first, n_last):
        n, keep = len(self.blocks), max(keep, n_first + n_last)
        if n <= keep:
            return 0
        self.blocks = [self.blocks[i] for i in choose([b.acc for b in self.blocks], keep, n_first, n_last)]
        return n - keep


def choose(score, n_sel, n_first, n_last):
    """Indices, ascending: the first, the last and those of the largest scores (ties to the lower; NaN largest)."""
    n = len(score)
    if n <= n_sel:
        return list(range(n))
    fixed = list(range(n_first)) + list(range(n - n_last, n))
    key = lambda i: (0, 0.0) if np.isnan(score[i]) else (1, -float(score[i]))
    best = sorted(range(n_first, n - n_last), key=lambda i: (key(i), i))[:n_sel - n_first - n_last]
    return sorted(fixed + best)


def attend(q, k, v, mask, scale):
    """q [R, D], k / v [n, D], mask [R, n]: softmax(scale q k^T) v in float64; (o, lse, p).  No token: 0, -inf."""
    q = q.astype(np.float64)
    s = np.where(mask, scale * (q @ k.T), -np.inf)
    top = s.max(axis=1, keepdims=True, initial=-np.inf)
    p = np.where(mask, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
    tot = p.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = (np.log(tot) + top)[:, 0]
        p = np.where(tot > 0, p / tot, 0.0)
    return p @ v, np.where(tot[:, 0] > 0, lse, -np.inf), p


def block_scores(q, unit_blocks):
    """float32 score of each block for the group's queries q [g, D]."""
    q = q.astype(np.float32)
    sq, q8 = [], []
    for row in q:
        if not np.isfinite(row).all():
            sq.append(np.float32(np.nan))
            q8.append(np.zeros(len(row), np.int64))
            continue
        s = scale_of(row, 127.0)
        sq.append(s)
        q8.append(np.clip(np.rint(row * (np.float32(1.0) / s)), -127, 127).astype(np.int64))
    out = []
    for b in unit_blocks:
        bd, sb = bounds(b.k)
        per_head = [np.float32(int(np.maximum(x * bd[0].astype(np.int64), x * bd[1].astype(np.int64)).sum())) * s
                    for x, s in zip(q8, sq)]
        out.append(np.float32(np.max(per_head)) * sb)       # np.max keeps NaN
    return out
