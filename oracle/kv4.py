"""Float64 oracle of the 4-bit KV cache: the row format, attention with accumulated
weights, and eviction. Plain numpy, row by row; shares no code with the library."""

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# byte b: five exponent bits, three fraction bits, no sign (the fp16 with bits b << 7)
SCALES = np.array([b * 2.0 ** -17 if b < 8 else (1 + b % 8 / 8) * 2.0 ** (b // 8 - 15)
                   for b in range(227)])
MAX_STORED = 6 * SCALES[226]


def quantise_blocks(x):
    """[n, 16] values -> (values as stored, scale bytes [n]). Of two codes equally near, the
    even one."""
    x = np.clip(np.asarray(x, dtype=np.float64), -MAX_STORED, MAX_STORED)
    byte = np.searchsorted(6 * SCALES, np.abs(x).max(axis=1))  # the first that covers it
    s = SCALES[byte][:, None]
    a = np.divide(np.abs(x), s, out=np.zeros_like(x), where=s > 0)
    best, dist = np.zeros_like(a), np.full_like(a, np.inf)
    for code in (0, 2, 4, 6, 1, 3, 5, 7):  # odd codes only where strictly nearer
        d = np.abs(a - MAGNITUDES[code])
        best = np.where(d < dist, MAGNITUDES[code], best)
        dist = np.minimum(d, dist)
    return np.sign(x) * best * s, byte


def quantise(x):
    """Stored values of x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    return quantise_blocks(x.reshape(-1, 16))[0].reshape(x.shape) if x.size else x


def dequantise(codes, scales):
    """Values of packed codes [..., D / 2] and scale bytes [..., D / 16]."""
    codes = np.asarray(codes)
    nib = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (2 * codes.shape[-1],))
    v = MAGNITUDES[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    return v * np.repeat(SCALES[np.asarray(scales)], 16, axis=-1)


def attend(q, keys, vals, end, scale):
    """(O, lse, P, A) of queries q [R, D]: query r over the first end[r] rows; P [R, n] the
    probabilities, A [R, D] the sum of p |v| (what a rounding of p is relative to)."""
    n = keys.shape[0]
    s = scale * (q @ keys.T)
    s[np.arange(n)[None] >= np.asarray(end)[:, None]] = -np.inf
    m = s.max(axis=1, keepdims=True) if n else np.full((q.shape[0], 1), -np.inf)
    m0 = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(s - m0)
    total = e.sum(axis=1, keepdims=True)
    p = e / np.where(total > 0, total, 1.0)
    with np.errstate(divide="ignore"):
        lse = (m0 + np.log(total))[:, 0]
    return p @ vals, lse, p, p @ np.abs(vals)


def rows_after_eviction(weight, pos, total, keep, first, recent):
    """Source row of each row after an eviction down to `keep` rows."""
    n = len(weight)
    src = list(range(min(n, keep)))
    if n <= keep:
        return src
    safe = [int(p) < first or int(p) >= total - recent for p in pos]

    def rank(j):  # smaller: kept sooner
        w = float(weight[j])
        return (not safe[j], np.isnan(w), 0.0 if safe[j] or np.isnan(w) else -w, j)

    kept = set(sorted(range(n), key=rank)[:keep])
    holes = [j for j in range(keep) if j not in kept]
    movers = [j for j in range(keep, n) if j in kept]
    for to, frm in zip(holes, movers):
        src[to] = frm
    return src


class Kv4Oracle:
    """The cache, a list of rows per (sequence, KV head)."""

    def __init__(self, batch, kv_heads, head_dim, capacity):
        self.B, self.H, self.D, self.N = batch, kv_heads, head_dim, capacity
        self.k = [[np.zeros((0, head_dim)) for _ in range(kv_heads)] for _ in range(batch)]
        self.v = [[np.zeros((0, head_dim)) for _ in range(kv_heads)] for _ in range(batch)]
        self.pos = [[np.zeros(0, dtype=np.int64) for _ in range(kv_heads)] for _ in range(batch)]
        self.weight = [[np.zeros(0) for _ in range(kv_heads)] for _ in range(batch)]
        self.total, self.last = [0] * batch, [0] * batch

    def held(self, b):
        return len(self.pos[b][0])

    def append(self, K, V, counts=None, replace=False):
        """K, V [B, T, H, D]."""
        K, V = quantise(K), quantise(V)
        for b in range(self.B):
            back = self.last[b] if replace else 0
            n0 = self.held(b) - back
            want = K.shape[1] if counts is None else int(counts[b])
            n = min(want, self.N - n0)
            self.total[b] -= back
            for h in range(self.H):
                self.k[b][h] = np.concatenate((self.k[b][h][:n0], K[b, :n, h]))
                self.v[b][h] = np.concatenate((self.v[b][h][:n0], V[b, :n, h]))
                self.pos[b][h] = np.concatenate((self.pos[b][h][:n0],
                                                 self.total[b] + np.arange(n)))
                self.weight[b][h] = np.concatenate((self.weight[b][h][:n0], np.zeros(n)))
            self.total[b] += n
            self.last[b] = n

    def attend(self, Q, counts=None, causal=False, scale=None, add_weight=False):
        """(O [B, T, heads, D], lse [B, heads, T], A, E): A as in attend(), E [B, heads, T] the
        largest sum |q k| scale of a query, which score errors are relative to. NaN where
        nothing is written."""
        B, T, heads, D = Q.shape
        scale = D ** -0.5 if scale is None else scale
        O, A = np.full(Q.shape, np.nan), np.full(Q.shape, np.nan)
        lse, E = np.full((B, heads, T), np.nan), np.full((B, heads, T), np.nan)
        for b in range(B):
            n, t = self.held(b), T if counts is None else int(counts[b])
            end = [n - t + i + 1 if causal else n for i in range(t)]
            for hq in range(heads):
                h = hq // (heads // self.H)
                if t == 0:
                    continue
                q = Q[b, :t, hq]
                o, l, p, a = attend(q, self.k[b][h], self.v[b][h], end, scale)
                O[b, :t, hq], lse[b, hq, :t], A[b, :t, hq] = o, l, a
                E[b, hq, :t] = scale * (np.abs(q) @ np.abs(self.k[b][h]).T).max(axis=1,
                                                                               initial=0.0)
                if add_weight:
                    self.weight[b][h] = self.weight[b][h] + p.sum(axis=0)
        return O, lse, A, E

    def evict(self, keep, first=0, recent=0):
        for b in range(self.B):
            if self.held(b) <= keep:
                continue
            for h in range(self.H):
                src = rows_after_eviction(self.weight[b][h], self.pos[b][h], self.total[b], keep,
                                          first, recent)
                for part in (self.k, self.v, self.pos, self.weight):
                    part[b][h] = part[b][h][src]
            self.last[b] = 0
