"""Problems of softmax attention for the GPU tests, and the bounds that their outputs are held to.

With u the plan type's unit roundoff (2^-24, 2^-8, 2^-11) and e = 2^-24, from the arithmetic:

- A score is a sum of D products in fp32, times the scale, plus the bias, minus a maximum, in
  powers of two: off by at most e ((D + 4) scale sum |q||k| + 8 |s| + 8 |bias|) =: es.  The
  exponential adds 4 e, the maximum (or lse) e times its own size; with it a probability is off by a
  relative ep = 2 (es + e (4 + 2 |lse|)) at most (2: an exponential of a small number).
- Probabilities enter their products rounded once (u); fp16 holds them times 2^12, so those below
  2^-26 of a row's largest lose up to 2^-37 of it.
- A sum of n terms in fp32 is off by at most n e times the sum of their sizes.
- o = sum P v / sum P: numerator off by sum P |v| (u + ep + n e), the sum of P by ep + n e.
- delta = do . o with o rounded: off by sum |do| (bound of o) + D e sum |do||o|; dP by D e sum |do||v|.
  dS = P (dP - delta) is off by |dS| (ep + 4 e) + P (those two), and rounded once (u) where it enters a
  product; fp16 holds a row's (dk: a key's) dS at a power of two whose floor is 2^-37 of the largest.
- Numbers below 2^-126 are held as 0, in every type: a probability loses up to 2^-126, dS up to 2^-126 (|dP|
  + |delta| + 1), a product as much again (steep scores have probabilities of 1e-50, whose gradients fp64 holds).
- An output is rounded once: u |ref|, in fp16 at least 2^-25.
Bounds are of fp64 sums, so they carry a factor 1.01 and terms u * u are left to it.
"""
import numpy as np

import synthetic
from gpu_util import to_f64, torch_dtype
from oracle import attention as att

F32, BF16, F16 = synthetic.F32, synthetic.BF16, synthetic.F16
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
E = 2.0 ** -24
TINY = 2.0 ** -126


def eqdt(eq, dt):
    return {F32: eq.EQL_F32, BF16: eq.EQL_BF16, F16: eq.EQL_F16}[dt]


def head_bounds(h, dt, absbias, backward):
    """Bounds of o, lse and the gradients of one head (att.Head)."""
    u, (n_q, Dk), (n_k, Dv) = U[dt], h.q.shape, h.v.shape
    up = 0.0 if dt == F32 else u  # fp32 probabilities are not rounded again
    sc = abs(h.scale)
    s = np.where(h.seen, np.abs(h.s), 0.0)
    es = E * ((Dk + 4) * sc * (np.abs(h.q) @ np.abs(h.k).T) + 8 * s + 8 * absbias)
    lse = np.where(np.isinf(h.lse), 0.0, np.abs(h.lse))[:, None]
    ep = 2 * (es + E * (4 + 2 * lse))
    worst = np.where(h.seen, ep, 0.0).max(-1, initial=0.0)[:, None]
    pv = h.p @ np.abs(h.v)
    # fp16: probabilities below 2^-26 of the largest
    low = 2.0 ** -37 * h.p.max(-1, initial=0.0)[:, None] if dt == F16 else 0.0
    lost = (low + TINY) * (h.seen @ (np.abs(h.v) + 1))
    raw_o = pv * (up + 2 * worst + 2 * (n_k + 4) * E) + lost
    floor = 2.0 ** -25 if dt == F16 else 0.0
    b = {"o": 1.01 * raw_o + np.maximum(u * np.abs(h.o), floor)}
    b["lse"] = 1.01 * (worst[:, 0] + (n_k + 8) * E) + 4 * E * lse[:, 0]
    if not backward:
        return b
    d = (np.abs(h.do) * b["o"]).sum(-1) + (Dv + 2) * E * (np.abs(h.do) * np.abs(h.o)).sum(-1)
    dp = (Dv + 2) * E * (np.abs(h.do) @ np.abs(h.v).T)
    eds = np.abs(h.ds) * (ep + 4 * E) + h.p * (1 + ep) * (dp + d[:, None])
    eds = eds + TINY * (np.abs(h.dp) + np.abs(h.delta)[:, None] + 1)
    ads = np.abs(h.ds)
    size = ads + eds
    fl_q = 2.0 ** -36 * size.max(-1, initial=0.0)[:, None] if dt == F16 else 0.0
    fl_k = 2.0 ** -36 * size.max(0, initial=0.0)[None, :] if dt == F16 else 0.0
    # (an unseen pair is no term)
    tq, tk = np.where(h.seen, eds + up * size + fl_q, 0.0), np.where(h.seen, eds + up * size + fl_k, 0.0)
    b["dq"] = sc * (tq @ np.abs(h.k) + (n_k + 4) * E * size @ np.abs(h.k)) + n_k * (1 + sc) * TINY
    b["dk"] = sc * (tk.T @ np.abs(h.q) + (n_q + 4) * E * size.T @ np.abs(h.q)) + n_q * (1 + sc) * TINY
    tp = h.p * (up + ep) + ((2.0 ** -37 if dt == F16 else 0.0) + TINY) * h.seen
    b["dv"] = tp.T @ np.abs(h.do) + (n_q + 4) * E * h.p.T @ np.abs(h.do) + n_q * TINY
    if h.bucket is not None:
        t = np.where(h.seen, eds + (n_q + n_k + 8) * E * size, 0.0)
        b["dbias"] = np.array([t[h.bucket == i].sum() for i in range(h.n_buckets)])
    return b


class Problem:
    """Attention over sequences of lens queries and kv_lens keys.  layout: "apart", "fused" (q, k and v slices of
    one buffer's rows; equal lengths only) or "odd" (rows that start at no vector boundary)."""

    def __init__(self, eq, dt, N, H, K, dk, dv, lens, kv_lens=None, causal=False, buckets=0, reach=0, packed=True, seed=0,
                 layout="apart", scale=None, std=1.0, do_std=1.0, behind=0, bias_std=1.0):
        import torch
        self.eq, self.dt, self.lens = eq, dt, list(lens)
        self.kv_lens = self.lens if kv_lens is None else list(kv_lens)
        self.N, self.H, self.K, self.dk, self.dv = N, H, K, dk, dv
        self.causal, self.buckets, self.reach = causal, buckets, reach
        self.B, self.T, self.S = len(self.lens), sum(self.lens) + behind, sum(self.kv_lens) + behind
        self.behind = behind
        self.scale = float(np.float32(1 / np.sqrt(dk * N) if scale is None else scale))
        self.plan = eq.eqlinear_attention_plan(N, H, K, dk, dv, eqdt(eq, dt), causal=causal, buckets=buckets, max_distance=reach)
        g = torch.Generator().manual_seed(seed)
        tdt = torch_dtype(dt)
        rand = lambda *s: (torch.randn(*s, generator=g) * std).to(tdt).cuda()  # noqa: E731
        seven = lambda *s: torch.full(s, 7.0, dtype=tdt, device="cuda")  # noqa: E731

        def views(fill):
            parts = [(self.T, H, dk), (self.S, K, dk), (self.S, K, dv)]
            if layout == "fused":
                assert self.T == self.S
                buf = fill(self.T, sum(h * d for _, h, d in parts), N)
                at, out = 0, []
                for _, h, d in parts:
                    out.append(buf[:, at:at + h * d].unflatten(1, (h, d)))
                    at += h * d
                return out
            if layout == "odd":
                out = []
                for t, h, d in parts:
                    buf = fill(t * (h * (d * N + 1) + 1) + 1)
                    out.append(buf.as_strided((t, h, d, N), (h * (d * N + 1) + 1, d * N + 1, N, 1), 1))
                return out
            return [fill(t, h, d, N) for t, h, d in parts]

        self.q, self.k, self.v = views(rand)
        self.dq, self.dk_, self.dv_ = views(seven)
        self.do = (torch.randn(self.T, H, dv, N, generator=g) * do_std).to(tdt).cuda()
        self.o = seven(self.T, H, dv, N)
        self.lse = torch.full((H, self.T), 7.0, device="cuda")
        self.bias = (torch.randn(H, buckets, generator=g) * bias_std).to(tdt).cuda() if buckets else None
        self.dbias = torch.full((H, buckets), 7.0, device="cuda") if buckets else None
        self.off, self.kv_off = (np.concatenate([[0], np.cumsum(n)]).astype(np.int64) for n in (self.lens, self.kv_lens))
        self.offsets = torch.from_numpy(self.off).cuda() if packed else None
        self.kv_offsets = torch.from_numpy(self.kv_off).cuda() if packed and kv_lens is not None else None

    def workspace(self, backward):
        import torch
        n = self.eq.eqlinear_attention_workspace(self.plan, self.T, self.S, self.B, backward=backward)
        return torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") if n else None  # NaNs to whoever reads them

    def forward(self, stream=None, workspace=None):
        self.eq.eqlinear_attention(self.plan, self.q, self.k, self.v, self.o, scale=self.scale, bias=self.bias, lse=self.lse,
                                   offsets=self.offsets, kv_offsets=self.kv_offsets, batch=self.B,
                                   workspace=workspace if workspace is not None else self.workspace(False), stream=stream)

    def backward(self, stream=None, workspace=None):
        self.eq.eqlinear_attention_backward(
            self.plan, self.q, self.k, self.v, self.o, self.do, self.lse, self.dq, self.dk_, self.dv_, scale=self.scale,
            bias=self.bias, dbias=self.dbias, offsets=self.offsets, kv_offsets=self.kv_offsets, batch=self.B,
            workspace=workspace if workspace is not None else self.workspace(True), stream=stream)

    def outputs(self, backward=True):
        out = {"o": self.o, "lse": self.lse}
        if backward:
            out |= {"dq": self.dq, "dk": self.dk_, "dv": self.dv_}
            if self.dbias is not None:
                out["dbias"] = self.dbias
        return out

    def check(self, what, backward=True):
        flat = lambda t: to_f64(t).reshape(t.shape[0], t.shape[1], -1)  # noqa: E731
        q, k, v, do = flat(self.q), flat(self.k), flat(self.v), flat(self.do)
        bias = None if self.bias is None else to_f64(self.bias)
        got = {n: to_f64(t) for n, t in self.outputs(backward).items()}
        for n in ("o", "dq", "dk", "dv"):
            if n in got:
                got[n] = got[n].reshape(got[n].shape[0], got[n].shape[1], -1)
        r = self.H // self.K
        sums = {n: np.zeros_like(got[n]) for n in got if n in ("dk", "dv", "dbias")}
        bounds = {n: np.zeros_like(got[n]) for n in sums}
        floor = 2.0 ** -25 if self.dt == F16 else 0.0
        worst = {}

        def hold(name, y, ref, bound):
            assert np.array_equal(np.isinf(y), np.isinf(ref)), f"{what}: {name}: infinities"
            ok = ~np.isinf(ref)
            err = np.abs(y[ok] - ref[ok])
            assert np.all(err <= bound[ok]), \
                f"{what}: {name}: off by {err.max():.3e}, {np.nanmax(err / np.maximum(bound[ok], 1e-300)):.2f} of the bound"
            if err.size:
                worst[name] = max(worst.get(name, 0.0), float(np.max(err / np.maximum(bound[ok], 1e-300))))

        for b in range(self.B):
            sq, sk = slice(self.off[b], self.off[b + 1]), slice(self.kv_off[b], self.kv_off[b + 1])
            for h in range(self.H):
                one = att.Head(q[sq, h], k[sk, h // r], v[sk, h // r], self.scale, self.causal,
                               None if bias is None else bias[h], self.reach)
                one.n_buckets = self.buckets
                if backward:
                    one.backward(do[sq, h], self.buckets)
                add = np.abs(bias[h][one.bucket]) if bias is not None else 0.0
                bd = head_bounds(one, self.dt, add, backward)
                hold("o", got["o"][sq, h], one.o, bd["o"])
                hold("lse", got["lse"][h, sq], one.lse, bd["lse"])
                if not backward:
                    continue
                hold("dq", got["dq"][sq, h], one.dq, 1.01 * bd["dq"] + np.maximum(U[self.dt] * np.abs(one.dq), floor))
                for n, at in (("dk", (sk, h // r)), ("dv", (sk, h // r)), ("dbias", h)):
                    if n in sums:
                        sums[n][at] += getattr(one, n)
                        bounds[n][at] += bd[n]
        seen = slice(0, self.kv_off[-1])
        for n in sums:
            at = seen if n != "dbias" else slice(None)
            extra = np.maximum(U[self.dt] * np.abs(sums[n]), floor) if n != "dbias" else (len(self.lens) + 4) * E * np.abs(sums[n])
            hold(n, got[n][at], sums[n][at], (1.01 * bounds[n] + extra)[at])
        # rows of no sequence stay as they were
        for n, end in (("o", self.off[-1]), ("dq", self.off[-1]), ("dk", self.kv_off[-1]), ("dv", self.kv_off[-1])):
            if n in got:
                assert np.all(got[n][end:] == 7.0), f"{what}: {name_of(n)} wrote behind the last sequence"
        assert np.all(got["lse"][:, self.off[-1]:] == 7.0)
        return worst


def name_of(n):
    return n
