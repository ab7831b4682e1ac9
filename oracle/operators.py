"""Plain fp64 definitions of the operators between the layers (numpy, CPU), for the tests.

rotary, linear_attention (with its gradients) and group_norm (with its gradients), each from
its formula.  linear_attention also returns the sums of absolute terms that bound the
rounding errors of any evaluation order.
"""
from __future__ import annotations

import math

import numpy as np

NONE, GELU, SILU = 0, 1, 2


# --- rotary ---------------------------------------------------------------------------

def rotary_frequencies(rot, base=10000.0, scaling="plain", factor=1.0, context=0.0, slow=1.0, fast=32.0):
    """Angle per position of each channel pair."""
    j = np.arange(rot // 2, dtype=np.float64)
    if scaling == "raised" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * j / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "banded":
        w = np.clip((context * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        f = f * w + f / factor * (1 - w)
    return f


def rotary(x, pos, freq, rot, interleaved, magnitude=1.0, inverse=False):
    """x [T][H][d][N] turned by angle pos freq, pair by pair."""
    y = x.copy()
    s = -1.0 if inverse else 1.0
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        c, d = magnitude * np.cos(pos * freq[j]), s * magnitude * np.sin(pos * freq[j])
        c, d = c[:, None, None], d[:, None, None]
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * d, x[:, :, b] * c + x[:, :, a] * d
    return y


# --- linear attention -----------------------------------------------------------------

def _powers(log_decay, n):
    """exp(log_decay n) with 0 to the power 0 = 1; 0 where n < 0."""
    n = np.asarray(n, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        p = np.exp(np.where(n == 0, 0.0, log_decay * np.maximum(n, 0)))
    return np.where(n < 0, 0.0, p)


def _sequence(q, k, v, do, la, scale, S0, dS1, absolute):
    """One sequence and kv head: q, do [r][n][D], k, v [n][D]."""
    r, n = q.shape[:2]
    t = np.arange(n)
    near = _powers(la, t[:, None] - t[None, :])
    grow, fade = _powers(la, t + 1)[:, None], _powers(la, n - 1 - t)[:, None]
    full = _powers(la, np.array(n))
    out = {"S1": full * S0 + (k * fade).T @ v}
    o = []
    for h in range(r):
        P = (q[h] @ k.T) * near * scale
        if absolute:
            P = np.abs(P)
        o.append(P @ v + (q[h] @ S0) * grow * scale)
    out["o"] = np.stack(o) if r else np.zeros((0, n, v.shape[1]))
    if do is None:
        return out
    dq, dk, dv, dS0 = [], fade * (v @ dS1.T), fade * (k @ dS1), full * dS1
    for h in range(r):
        P, dP = (q[h] @ k.T) * near * scale, (do[h] @ v.T) * near * scale
        if absolute:
            P, dP = np.abs(P), np.abs(dP)
        dq.append(dP @ k + (do[h] @ S0.T) * grow * scale)
        dk = dk + dP.T @ q[h]
        dv = dv + P.T @ do[h]
        dS0 = dS0 + scale * (q[h] * grow).T @ do[h]
    return out | {"dq": np.stack(dq), "dk": dk, "dv": dv, "dS0": dS0}


def linear_attention(q, k, v, log_decay, scale, offsets, S0=None, do=None, dS1=None, absolute=None):
    """q [T][H][Dk], k [T][K][Dk], v [T][K][Dv], S0 [B][K][Dk][Dv] -> dict of o [T][H][Dv], S1 and, with do,
    dq, dk, dv, dS0.

    absolute = "scores": the same sums with every decayed score q.k (d_o.v) and every other factor replaced by
    its absolute value; "all": every single number replaced by its absolute value."""
    if absolute:
        inner = absolute == "scores"
        if not inner:
            q, k = np.abs(q), np.abs(k)
            v = np.abs(v)
            do = None if do is None else np.abs(do)
        scale = abs(scale)
        S0 = None if S0 is None else np.abs(S0)
        dS1 = None if dS1 is None else np.abs(dS1)
    T, H, Dk = q.shape
    K, Dv = k.shape[1], v.shape[2]
    B, r = len(offsets) - 1, H // K
    res = {"o": np.zeros((T, H, Dv)), "S1": np.zeros((B, K, Dk, Dv))}
    if do is not None:
        res |= {"dq": np.zeros((T, H, Dk)), "dk": np.zeros((T, K, Dk)), "dv": np.zeros((T, K, Dv)),
                "dS0": np.zeros((B, K, Dk, Dv))}
    for b in range(B):
        s = slice(int(offsets[b]), int(offsets[b + 1]))
        for g in range(K):
            hs = slice(g * r, (g + 1) * r)
            zero = np.zeros((Dk, Dv))
            qq, kk, vv = q[s, hs].transpose(1, 0, 2), k[s, g], v[s, g]
            dd = None if do is None else do[s, hs].transpose(1, 0, 2)
            A0, A1 = (zero if x is None else x[b, g] for x in (S0, dS1))
            if absolute == "scores":
                # the scores keep their own cancellation; what they multiply does not
                one = _sequence_scores(qq, kk, vv, dd, log_decay[g], scale, A0, A1)
            else:
                one = _sequence(qq, kk, vv, dd, log_decay[g], scale, A0, A1, False)
            res["S1"][b, g] = one["S1"]
            res["o"][s, hs] = one["o"].transpose(1, 0, 2)
            if do is not None:
                res["dq"][s, hs] = one["dq"].transpose(1, 0, 2)
                res["dk"][s, g], res["dv"][s, g], res["dS0"][b, g] = one["dk"], one["dv"], one["dS0"]
    return res


def _sequence_scores(q, k, v, do, la, scale, S0, dS1):
    r, n = q.shape[:2]
    t = np.arange(n)
    near = _powers(la, t[:, None] - t[None, :])
    out = {"S1": np.zeros_like(S0), "o": np.stack([np.abs(q[h] @ k.T * near * scale) @ np.abs(v) for h in range(r)])}
    if do is None:
        return out
    dk, dv, dq = np.zeros(k.shape), np.zeros(v.shape), []
    for h in range(r):
        P, dP = np.abs(q[h] @ k.T * near * scale), np.abs(do[h] @ v.T * near * scale)
        dq.append(dP @ np.abs(k))
        dk += dP.T @ np.abs(q[h])
        dv += P.T @ np.abs(do[h])
    return out | {"dq": np.stack(dq), "dk": dk, "dv": dv, "dS0": np.zeros_like(S0)}


# --- group norm -----------------------------------------------------------------------

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(z, act):
    """(value, derivative)."""
    if act == SILU:
        p = 1.0 / (1.0 + np.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    if act == GELU:
        p = 0.5 * (1 + _erf(z / math.sqrt(2.0)))
        return z * p, p + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return z, np.ones_like(z)


def group_norm(x, gamma, beta, groups, eps, act, offsets, dy=None):
    """x [T][C][N] -> y, stats [B][groups][2] and, with dy, dx, dgamma, dbeta."""
    T, C, N = x.shape
    B, cg = len(offsets) - 1, C // groups
    gamma = np.ones(C) if gamma is None else gamma
    beta = np.zeros(C) if beta is None else beta
    y, stats = np.zeros_like(x), np.zeros((B, groups, 2))
    res = {"y": y, "stats": stats}
    if dy is not None:
        res |= {"dx": np.zeros_like(x), "dgamma": np.zeros(C), "dbeta": np.zeros(C)}
    for b in range(B):
        s = slice(int(offsets[b]), int(offsets[b + 1]))
        if s.start == s.stop:
            continue
        for j in range(groups):
            cs = slice(j * cg, (j + 1) * cg)
            p = x[s, cs]
            mean = p.mean()
            rstd = 1.0 / math.sqrt(((p - mean) ** 2).mean() + eps) if ((p - mean) ** 2).mean() + eps > 0 else math.inf
            xh = (p - mean) * rstd
            stats[b, j] = mean, rstd
            y[s, cs], slope = activation(gamma[None, cs, None] * xh + beta[None, cs, None], act)
            if dy is None:
                continue
            dz = dy[s, cs] * slope
            res["dgamma"][cs] += (dz * xh).sum((0, 2))
            res["dbeta"][cs] += dz.sum((0, 2))
            g = dz * gamma[None, cs, None]
            res["dx"][s, cs] = (g - g.mean() - xh * (g * xh).mean()) * rstd
    return res
