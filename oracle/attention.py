"""Plain fp64 definitions of softmax attention with a bias by distance, its gradients, attention over
a paged cache, and the cache's tables (numpy, CPU), for the tests."""
from __future__ import annotations

import numpy as np


def bucket(distance, buckets, reach, causal):
    """Bucket of a distance (query's position less key's), in whole numbers."""
    side = buckets if causal else buckets // 2
    exact = side // 2
    m = side - exact
    n = abs(int(distance))
    if n < exact:
        b = n
    else:
        b = max(j for j in range(m) if n ** m >= exact ** (m - j) * reach ** j)
        b += exact
    return b + (side if distance < 0 and not causal else 0)


def distances(n_q, n_k):
    return (np.arange(n_q)[:, None] + (n_k - n_q)) - np.arange(n_k)[None, :]


class Head:
    """One sequence and query head: q [n_q][Dk], k [n_k][Dk], v [n_k][Dv]."""

    def __init__(self, q, k, v, scale, causal, bias=None, reach=0):
        n_q, n_k = len(q), len(k)
        self.q, self.k, self.v, self.scale = q, k, v, scale
        gap = distances(n_q, n_k)
        with np.errstate(all="ignore"):
            self.s = scale * (q @ k.T)
        self.bucket = None
        if bias is not None:
            lo, hi = int(gap.min(initial=0)), int(gap.max(initial=0))
            of = np.array([bucket(d, len(bias), reach, causal) for d in range(lo, hi + 1)])
            self.bucket = of[gap - lo]
            self.s = self.s + bias[self.bucket]
        self.seen = gap >= 0 if causal else np.ones((n_q, n_k), bool)
        s = np.where(self.seen, self.s, -np.inf)
        with np.errstate(all="ignore"):
            top = s.max(-1, initial=-np.inf)
            e = np.where(self.seen, np.exp(s - np.where(np.isinf(top), 0.0, top)[:, None]), 0.0)
            total = e.sum(-1)
            self.lse = np.where(total == 0, -np.inf, np.where(np.isinf(top), 0.0, top) + np.log(total))
            self.p = np.where((total == 0)[:, None], 0.0, e / np.where(total == 0, 1.0, total)[:, None])
        # a key that a query does not see is no term, whatever its value
        self.o = np.stack([self.p[i, self.seen[i]] @ v[self.seen[i]] for i in range(n_q)]) if n_q else np.zeros((0, v.shape[1]))

    def backward(self, do, n_buckets=0):
        self.do = do
        self.dp = do @ self.v.T
        self.delta = (do * self.o).sum(-1)
        self.ds = self.p * (self.dp - self.delta[:, None])
        self.dq = self.scale * self.ds @ self.k
        self.dk = self.scale * self.ds.T @ self.q
        self.dv = self.p.T @ do
        if self.bucket is not None:
            self.dbias = np.array([self.ds[self.bucket == b].sum() for b in range(n_buckets)])
        return self


def step(q, k_cache, v_cache, table, lengths, scale, bias=None, reach=0):
    """q [B][H][Dk], caches [blocks][block_size][K][D] -> o [B][H][Dv], lse [H][B]."""
    B, H, _ = q.shape
    blocks, bs, K, _ = k_cache.shape
    r = H // K
    o, lse = np.zeros((B, H, v_cache.shape[-1])), np.full((H, B), -np.inf)
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * bs)
        at = np.arange(n)
        ids = table[b][at // bs] if n else np.zeros(0, int)
        there = (ids >= 0) & (ids < blocks)
        at, ids = at[there], ids[there]
        for h in range(H):
            if not len(at):
                continue
            s = scale * (k_cache[ids, at % bs, h // r] @ q[b, h])
            if bias is not None:
                s = s + bias[h][[bucket(n - 1 - j, bias.shape[1], reach, True) for j in at]]
            if s.max() == -np.inf:
                continue
            e = np.exp(s - s.max())
            lse[h, b] = s.max() + np.log(e.sum())
            o[b, h] = e @ v_cache[ids, at % bs, h // r] / e.sum()
    return o, lse


def tables(lengths, added, free_blocks, cursor, table, block_size, T):
    """-> table, lengths, cursor, slots [T], positions [T], offsets [B + 1]."""
    table = table.copy()
    max_blocks = table.shape[1]
    slots, positions, offsets = np.full(T, -1, np.int64), np.zeros(T, np.int32), [0]
    out, t = [], 0
    held_blocks = lambda n: min(-(-n // block_size), max_blocks)  # noqa: E731
    for b, (n, a) in enumerate(zip(lengths, added)):
        n, a = max(int(n), 0), max(int(a), 0)
        a = min(a, T - t)
        for j in range(held_blocks(n), held_blocks(n + a)):
            table[b, j] = free_blocks[cursor] if 0 <= cursor < len(free_blocks) else -1
            cursor += 1
        for p in range(n, n + a):
            j = p // block_size
            if j < max_blocks and table[b, j] >= 0:
                slots[t] = int(table[b, j]) * block_size + p % block_size
            positions[t] = p
            t += 1
        out.append(n + a)
        offsets.append(t)
    return table, np.array(out, np.int32), cursor, slots, positions, np.array(offsets, np.int64)
