"""Workloads of softmax attention on regular-representation features: prompts and training with a
learned relative position bias, single tokens over a paged key-value cache, and the cache's block
tables, slot maps and stores.

A feature is a record of N group elements per channel ([token][channel][N], group elements
innermost) and a head a run of d whole channels, d N numbers wide.  Scores sum over the group axis
and a bias by distance is the same for every group element, so attention commutes with a cyclic
shift of that axis.

Sizes follow this repository's layers: heads of 8 x 8 and 16 x 8 numbers of width 768 (64 images of
197 tokens), heads of 16 x 7 of width 1120 (32768 tokens).
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROWS = 1 << 27  # scores that the plain form holds at a time


def _case(op, name=None, **kw):
    c = {"op": op, **kw}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one short prompt of a request that has just come: latency
        _case("attend", "attend: short prompt", dtype="bf16", N=8, heads=12, kv=4, dk=8, dv=8, batch=1, tokens=50,
              ragged=False, causal=True, buckets=0, reach=0, fused=True),
        # a batch of images, every token seeing all others, distances learned
        _case("attend", "attend: images", dtype="bf16", N=8, heads=12, kv=12, dk=8, dv=8, batch=64, tokens=197,
              ragged=False, causal=False, buckets=32, reach=128, fused=True),
        # one long sequence
        _case("attend", "attend: long prompt", dtype="f16", N=7, heads=10, kv=10, dk=16, dv=16, batch=1, tokens=32768,
              ragged=False, causal=True, buckets=0, reach=0, fused=False),
        # training on packed images of different sizes, three query heads to a key, with the bias' gradient
        _case("train", "train: images", dtype="bf16", N=8, heads=12, kv=4, dk=8, dv=8, batch=64, tokens=197,
              ragged=True, causal=False, buckets=32, reach=128, fused=True),
        # training on long sequences
        _case("train", "train: long", dtype="bf16", N=8, heads=12, kv=4, dk=16, dv=16, batch=2, tokens=8192,
              ragged=False, causal=True, buckets=0, reach=0, fused=False),
        # a small model trained in fp32
        _case("train", "train: fp32", dtype="f32", N=8, heads=4, kv=4, dk=8, dv=8, batch=16, tokens=256,
              ragged=False, causal=True, buckets=32, reach=128, fused=False),
        # eight sequences being decoded
        _case("step", "step: of 8", dtype="bf16", N=8, heads=12, kv=12, dk=8, dv=8, batch=8, tokens=1000, ragged=True,
              causal=True, buckets=0, reach=0, block=16),
        # a full serving batch of unequal contexts
        _case("step", "step: of 256", dtype="bf16", N=8, heads=12, kv=4, dk=16, dv=16, batch=256, tokens=2048,
              ragged=True, causal=True, buckets=32, reach=128, block=16),
        # one sequence far into its context
        _case("step", "step: long context", dtype="f16", N=7, heads=10, kv=2, dk=16, dv=16, batch=1, tokens=131072,
              ragged=False, causal=True, buckets=0, reach=0, block=64),
        # the next token of eight sequences joins the cache
        _case("append", "append: 8 tokens", dtype="bf16", N=8, heads=12, kv=12, dk=8, dv=8, batch=8, tokens=1000,
              added=1, ragged=True, block=16),
        # prompts of new requests next to requests that decode
        _case("append", "append: prompts", dtype="bf16", N=8, heads=12, kv=4, dk=16, dv=16, batch=128, tokens=500,
              added=197, ragged=True, block=16),
        # a step of very many requests
        _case("append", "append: 2048 tokens", dtype="f16", N=7, heads=10, kv=2, dk=16, dv=16, batch=2048, tokens=200,
              added=1, ragged=True, block=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "train", "train", "step", "step", "append"])
    N = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 12, 16])
    top = max(1, 128 // N)
    least = min(top, -(-8 // N))
    kv = rng.choice([1, 2, 3, 4, 8])
    c = _case(op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), N=N, kv=kv, heads=kv * rng.choice([1, 1, 2, 3, 4]),
              dk=_log(rng, least, top))
    c["dv"] = c["dk"] if rng.random() < 0.7 else _log(rng, least, top)
    if op == "append":
        c["block"] = rng.choice([1, 7, 16, 32, 64])
        c["batch"], c["tokens"] = _log(rng, 1, 2048), _log(rng, 1, 1000)
        c["added"] = 1 if rng.random() < 0.5 else _log(rng, 1, 400)
        c["ragged"] = rng.random() < 0.7
    else:
        c["causal"] = op == "step" or rng.random() < 0.5
        c["buckets"], c["reach"] = (0, 0) if rng.random() < 0.4 else rng.choice([(8, 20), (32, 128), (64, 500), (128, 1024)])
        if op == "step":
            c["block"] = rng.choice([1, 7, 16, 32, 64, 256])
            if rng.random() < 0.3:
                c["batch"], c["tokens"] = 1, _log(rng, 1, 131072)
            else:
                c["batch"], c["tokens"] = _log(rng, 1, 256), _log(rng, 1, 4096)
        else:
            c["fused"] = rng.random() < 0.5
            if rng.random() < 0.3:
                c["batch"], c["tokens"] = 1, _log(rng, 1, 8192)
            else:
                c["batch"], c["tokens"] = _log(rng, 1, 64), _log(rng, 1, 1024)
        c["ragged"] = c["batch"] > 1 and rng.random() < 0.5
    most = [work(k) for k in listed()]
    most = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    while work(c)["bytes"] > most[0] or work(c)["flops"] > most[1]:
        c["batch" if c["batch"] > 1 else "tokens"] //= 2
    c["ragged"] = c["ragged"] and c["batch"] > 1
    return c


# --- what a case holds ------------------------------------------------------------------

def _uneven(total, parts, seed):
    """`parts` whole numbers of the given sum, unequal, with a 0 and a 1 among four or more."""
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(parts, generator=g, dtype=torch.float64) * 1.5 + 0.25
    n = (w / w.sum() * total).floor().to(torch.int64).tolist()
    if parts >= 4:
        n[1], n[2] = 0, 1
    n[-1] += total - sum(n)
    return [int(v) for v in n]


def lengths(case):
    """Tokens of each sequence (step, append: in the cache)."""
    B, S = case["batch"], case["tokens"]
    return _uneven(B * S, B, 1000 * B + S) if case["ragged"] else [S] * B


def additions(case):
    """append: new tokens of each request."""
    B, A = case["batch"], case["added"]
    if not case["ragged"] or A == 1:
        return [A] * B
    n = _uneven(B * A, B, 7000 * B + A)
    return n[::-1]


def _blocks(case):
    """Blocks of the cache and of a row of the table: what the sequences need and a few more."""
    need = lengths(case)
    if case["op"] == "append":
        need = [a + b for a, b in zip(need, additions(case))]
    rows = [-(-n // case["block"]) for n in need]
    return sum(rows) + 3, max(rows) + 1


def _pairs(case):
    """Pairs of a query and a key that it sees."""
    return sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lengths(case))


def work(case):
    T, N, B = case["batch"] * case["tokens"], case["N"], case["batch"]
    es = 4 if case["dtype"] == "f32" else 2
    H, K, Dk, Dv = case["heads"], case["kv"], case["dk"] * N, case["dv"] * N
    if case["op"] == "append":
        A = sum(additions(case))
        return {"bytes": 2 * es * A * K * (Dk + Dv) + 20 * A + 20 * B, "flops": 0}
    bias = es * H * case["buckets"]
    if case["op"] == "step":
        keys = sum(lengths(case))
        return {"bytes": es * (keys * K * (Dk + Dv) + B * H * (Dk + Dv)) + 4 * keys // case["block"] + bias,
                "flops": 2 * keys * H * (Dk + Dv)}
    q, k, v, o = T * H * Dk, T * K * Dk, T * K * Dv, T * H * Dv
    pairs = _pairs(case) * H
    if case["op"] == "attend":
        return {"bytes": es * (q + k + v + o) + bias, "flops": 2 * pairs * (Dk + Dv)}
    # o and the statistics out; o, do and the inputs in, gradients out
    return {"bytes": es * (3 * q + 3 * k + 3 * v + 3 * o) + 8 * T * H + 2 * bias,
            "flops": 2 * pairs * (4 * Dk + 3 * Dv)}


class _Maker:
    """Inputs from the seed alone."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(self, *shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=self.g, device="cuda") * std).to(dtype)

    def order(self, n):
        return torch.randperm(n, generator=self.g, device="cuda").to(torch.int32)


def _split(y, parts):
    at = 0
    for h, d in parts:
        yield y[:, at:at + h * d].unflatten(1, (h, d))
        at += h * d


def _heads(make, T, parts, N, fused):
    """Tensors [T, heads, channels, N] for (heads, channels) in parts: slices of one projection's output, or apart."""
    if not fused:
        return [make(T, h, d, N) for h, d in parts]
    return list(_split(make(T, sum(h * d for h, d in parts), N), parts))


def _offsets(n):
    at = [0]
    for v in n:
        at.append(at[-1] + v)
    return torch.tensor(at, dtype=torch.int64, device="cuda")


def prepare(case, seed):
    m = _Maker(seed)
    dt = DTYPES[case["dtype"]]
    B, N, H, K, dk, dv = (case[k] for k in ("batch", "N", "heads", "kv", "dk", "dv"))
    n = lengths(case)
    s = {"case": case, "scale": 1.0 / math.sqrt(dk * N), "bias": None}
    new = lambda *shape: m.normal(*shape, dtype=dt)  # noqa: E731
    out = lambda *shape: torch.empty(*shape, dtype=dt, device="cuda")  # noqa: E731
    if case.get("buckets"):
        s["bias"] = m.normal(H, case["buckets"], dtype=dt)
    if case["op"] in ("attend", "train"):
        T = s["T"] = sum(n)
        s["offsets"] = _offsets(n) if case["ragged"] else None
        parts = [(H, dk), (K, dk), (K, dv)]
        s["q"], s["k"], s["v"] = _heads(new, T, parts, N, case["fused"])
        s["o"] = out(T, H, dv, N)
        if case["op"] == "train":
            s["lse"] = torch.empty(H, T, device="cuda")
            s["do"] = new(T, H, dv, N)
            s["dq"], s["dk"], s["dv"] = _heads(out, T, parts, N, case["fused"])
            s["dbias"] = torch.empty(H, case["buckets"], device="cuda") if case["buckets"] else None
    else:
        blocks, row = _blocks(case)
        s["k_cache"], s["v_cache"] = new(blocks, case["block"], K, dk, N), new(blocks, case["block"], K, dv, N)
        order = m.order(blocks)
        held = [-(-v // case["block"]) for v in n]
        table = torch.full((B, row), -1, dtype=torch.int32)
        at, ids = 0, order.cpu()
        for b, h in enumerate(held):
            table[b, :h] = ids[at:at + h]
            at += h
        s["table"] = table.cuda()
        s["lengths"] = torch.tensor(n, dtype=torch.int32, device="cuda")
        if case["op"] == "step":
            s["q"], s["o"] = new(B, H, dk, N), out(B, H, dv, N)
        else:
            added = additions(case)
            T = s["T"] = sum(added)
            s["added"] = torch.tensor(added, dtype=torch.int32, device="cuda")
            s["k"], s["v"] = new(T, K, dk, N), new(T, K, dv, N)
            # the free list is the whole order, of which the sequences hold the first blocks
            s["free"], s["cursor"] = order, torch.tensor([at], dtype=torch.int32, device="cuda")
            s["new_lengths"], s["new_cursor"] = torch.empty_like(s["lengths"]), torch.empty_like(s["cursor"])
            s["slots"] = torch.empty(T, dtype=torch.int64, device="cuda")
            s["positions"] = torch.empty(T, dtype=torch.int32, device="cuda")
            s["offsets"] = torch.empty(B + 1, dtype=torch.int64, device="cuda")
    if own:
        _plan(s)
    return s


# --- the framework's operators --------------------------------------------------------------

def _plan(s):
    """What a user's program keeps: the plan, and the workspace that the library asks for."""
    import group_equivariant_linear_amd as eq
    c = s["case"]
    dt = {"f32": eq.EQL_F32, "bf16": eq.EQL_BF16, "f16": eq.EQL_F16}[c["dtype"]]
    s["eq"] = eq
    s["plan"] = eq.eqlinear_attention_plan(c["N"], c["heads"], c["kv"], c["dk"], c["dv"], dt,
                                           causal=c.get("causal", True), buckets=c.get("buckets", 0),
                                           max_distance=c.get("reach", 0))
    if c["op"] == "step":
        n = eq.eqlinear_attention_step_workspace(s["plan"], c["batch"])
    elif c["op"] == "append":
        n = eq.eqlinear_cache_tables_workspace(c["batch"])
    else:
        n = eq.eqlinear_attention_workspace(s["plan"], s["T"], s["T"], c["batch"], backward=c["op"] == "train")
    s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def _run_own(s):
    eq, c, plan = s["eq"], s["case"], s["plan"]
    if c["op"] == "append":
        eq.eqlinear_cache_tables(s["lengths"], s["added"], s["free"], s["cursor"], s["table"], c["block"],
                                 s["new_lengths"], s["new_cursor"], s["slots"], s["positions"], s["offsets"],
                                 workspace=s["workspace"])
        eq.eqlinear_cache_store(plan, s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
        return {"table": s["table"], "lengths": s["new_lengths"], "cursor": s["new_cursor"], "slots": s["slots"],
                "positions": s["positions"], "offsets": s["offsets"], "k": s["k_cache"], "v": s["v_cache"]}
    if c["op"] == "step":
        eq.eqlinear_attention_step(plan, s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["o"],
                                   scale=s["scale"], bias=s["bias"], workspace=s["workspace"])
        return {"o": s["o"]}
    train = c["op"] == "train"
    eq.eqlinear_attention(plan, s["q"], s["k"], s["v"], s["o"], scale=s["scale"], bias=s["bias"],
                          lse=s["lse"] if train else None, offsets=s["offsets"], batch=c["batch"],
                          workspace=s["workspace"])
    if not train:
        return {"o": s["o"]}
    eq.eqlinear_attention_backward(plan, s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["dq"], s["dk"], s["dv"],
                                   scale=s["scale"], bias=s["bias"], dbias=s["dbias"], offsets=s["offsets"],
                                   batch=c["batch"], workspace=s["workspace"])
    out = {"o": s["o"], "lse": s["lse"], "dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}
    if s["dbias"] is not None:
        out["dbias"] = s["dbias"]
    return out


# --- the plain forms ----------------------------------------------------------------------------

def _bucket_table(buckets, reach):
    """Bucket of the distances 0 .. reach on one side of `buckets`, in whole numbers: the first half one by one,
    then by equal steps of the logarithm up to reach."""
    exact = buckets // 2
    m = buckets - exact
    first = [n for n in range(exact)]
    of, b = [], 0
    for n in range(reach + 1):
        if n < exact:
            of.append(first[n])
            continue
        while b + 1 < m and n ** m >= exact ** (m - b - 1) * reach ** (b + 1):
            b += 1
        of.append(exact + b)
    return of


def _bucket(distance, case):
    """Buckets of distances (query's position less key's)."""
    side = case["buckets"] if case["causal"] else case["buckets"] // 2
    of = torch.tensor(_bucket_table(side, case["reach"]), device=distance.device)
    b = of[distance.abs().clamp(max=case["reach"])]
    return b if case["causal"] else torch.where(distance < 0, b + side, b)


class _Batch:
    """Packed tokens as sequences of one padded length."""

    def __init__(self, s):
        n = lengths(s["case"])
        self.B, self.S = len(n), max(1, max(n))
        off = s["offsets"] if s["offsets"] is not None else torch.arange(self.B + 1, device="cuda") * n[0]
        at = torch.arange(self.S, device="cuda")
        self.valid = at[None] < (off[1:] - off[:-1])[:, None]
        self.index = torch.where(self.valid, off[:-1, None] + at[None], 0)
        token = torch.arange(s["T"], device="cuda")
        seq = torch.searchsorted(off[1:].contiguous(), token, right=True)
        self.back = seq * self.S + token - off[seq]

    def take(self, x):
        """[T, H, d, N] -> [B, H, S, d N] in 32 bits, zeros past each end."""
        y = x.flatten(2).float()[self.index.reshape(-1)].reshape(self.B, self.S, x.shape[1], -1)
        return (y * self.valid[:, :, None, None]).transpose(1, 2).contiguous()

    def put(self, y):
        """[B, H, S, D] -> [T, H, D]."""
        return y.transpose(1, 2).reshape(self.B * self.S, y.shape[1], -1)[self.back]


def _attention(s):
    case = s["case"]
    g = _Batch(s)
    B, S, H, K = g.B, g.S, case["heads"], case["kv"]
    r = H // K
    scale = s["scale"]
    q, k, v = g.take(s["q"]), g.take(s["k"]), g.take(s["v"])
    train = case["op"] == "train"
    do = g.take(s["do"]) if train else None
    o = torch.empty(B, H, S, v.shape[-1], device="cuda")
    lse = torch.empty(B, H, S, device="cuda") if train else None
    if train:
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
        near = torch.zeros(H, 2 * S, device="cuda")  # gradients of the scores by distance
    at = torch.arange(S, device="cuda")
    # runs of sequences, of one kv head's query heads, of query rows: what ROWS scores hold
    nb = max(1, min(B, ROWS // (r * S * S)))
    rows = S if nb > 1 or r * S * S <= ROWS else max(1, ROWS // (r * S))
    for b0 in range(0, B, nb):
        b = slice(b0, min(B, b0 + nb))
        for h in range(K):
            hs = slice(h * r, (h + 1) * r)
            kh, vh = k[b, h:h + 1], v[b, h:h + 1]
            kt, vt = kh.transpose(-1, -2).contiguous(), vh.transpose(-1, -2).contiguous()
            for t0 in range(0, S, rows):
                t1 = min(S, t0 + rows)
                n = t1 if case["causal"] else S  # keys that any of these rows sees
                x = torch.matmul(q[b, hs, t0:t1], kt[..., :n]) * scale
                gap = at[t0:t1, None] - at[None, :n]
                if s["bias"] is not None:
                    x = x + s["bias"][hs].float()[:, _bucket(gap, case)]
                seen = g.valid[b, None, None, :n]
                if case["causal"]:
                    seen = seen & (gap >= 0)
                x = x.masked_fill(~seen, float("-inf"))
                top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
                x = torch.exp(x - top)
                total = x.sum(-1, keepdim=True)
                p = x / total.clamp(min=torch.finfo(torch.float32).tiny)
                o[b, hs, t0:t1] = torch.matmul(p, vh[:, :, :n])
                if not train:
                    continue
                lse[b, hs, t0:t1] = (top + torch.log(total))[..., 0]
                d = do[b, hs, t0:t1]
                dp = torch.matmul(d, vt[..., :n])
                ds = p * (dp - (p * dp).sum(-1, keepdim=True))
                dq[b, hs, t0:t1] = torch.matmul(ds, kh[:, :, :n]) * scale
                dk[b, h, :n] += (torch.matmul(ds.transpose(-1, -2).contiguous(), q[b, hs, t0:t1]) * scale).sum(1)
                dv[b, h, :n] += torch.matmul(p.transpose(-1, -2).contiguous(), d).sum(1)
                if s["bias"] is not None:
                    # rows read as rows one step longer: diagonals come under each other
                    ds = (ds * g.valid[b, None, t0:t1, None]).sum(0)
                    m = t1 - t0
                    z = torch.nn.functional.pad(ds, (0, m - 1)).flatten(1)
                    z = torch.nn.functional.pad(z, (0, m)).reshape(r, m, n + m).sum(1)
                    # columns: key less row, 0 .. n - 1, then -m .. -1
                    key = torch.arange(n + m, device="cuda")
                    key = torch.where(key < n, key, key - (n + m))
                    near[hs, t0 - key + S - 1] += z
    o = g.put(o).to(s["o"].dtype).reshape(s["o"].shape)
    if not train:
        return {"o": o}
    out = {"o": o, "lse": g.put(lse[..., None])[..., 0].t().contiguous()}
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        out[name] = g.put(x).to(s[name].dtype).reshape(s[name].shape)
    if s["bias"] is not None:
        of = _bucket(torch.arange(2 * S, device="cuda") - (S - 1), case)
        out["dbias"] = torch.matmul(near, (of[:, None] == torch.arange(case["buckets"], device="cuda")).float())
    return out


def _step(s):
    case = s["case"]
    r, bs = case["heads"] // case["kv"], case["block"]
    longest = max(lengths(case))
    at = torch.arange(max(1, longest), device="cuda")
    slot = s["table"].long().clamp(min=0)[:, at // bs] * bs + at % bs  # [B, S]
    o = torch.empty_like(s["o"])
    run = max(1, (1 << 28) // (at.numel() * case["kv"] * max(case["dk"], case["dv"]) * case["N"]))
    for b0 in range(0, case["batch"], run):
        b = slice(b0, b0 + run)
        n = s["lengths"][b, None]
        k = s["k_cache"].flatten(0, 1).flatten(2)[slot[b]].float()  # [B, S, K, D]
        v = s["v_cache"].flatten(0, 1).flatten(2)[slot[b]].float()
        q = s["q"][b].flatten(2).float().unflatten(1, (case["kv"], r))  # [B, K, r, D]
        x = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * s["scale"]
        if s["bias"] is not None:
            gap = (n - 1 - at).clamp(min=0)
            x = x + s["bias"].float()[:, _bucket(gap, case)].transpose(0, 1).unflatten(1, (case["kv"], r))
        seen = (at < n)[:, None, None, :]
        x = x.masked_fill(~seen, float("-inf"))
        x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
        p = x / x.sum(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)
        y = torch.matmul(p, v.transpose(1, 2).contiguous())
        o[b] = y.to(o.dtype).reshape(y.shape[0], *o.shape[1:])
    return {"o": o}


def _append(s):
    bs, T = s["case"]["block"], s["T"]
    n, a = s["lengths"].long(), s["added"].long()
    offsets = torch.cat([a.new_zeros(1), a.cumsum(0)])
    held = (n + bs - 1) // bs
    fresh = (n + a + bs - 1) // bs - held
    first = fresh.cumsum(0) - fresh + s["cursor"].long()  # place of a request's first new block in the free list
    token = torch.arange(T, device="cuda")
    seq = torch.searchsorted(offsets[1:].contiguous(), token, right=True)
    pos = n[seq] + token - offsets[seq]
    at = pos // bs
    old = s["table"][seq, at.clamp(max=s["table"].shape[1] - 1)]
    new = s["free"][(first[seq] + at - held[seq]).clamp(0, s["free"].numel() - 1)]
    block = torch.where(at < held[seq], old, new)
    s["table"][seq, at] = block
    s["slots"].copy_(block.long() * bs + pos % bs)
    s["positions"].copy_(pos)
    s["offsets"].copy_(offsets)
    s["new_lengths"].copy_(n + a)
    s["new_cursor"].copy_(s["cursor"] + fresh.sum())
    s["k_cache"].flatten(0, 1)[s["slots"]] = s["k"]
    s["v_cache"].flatten(0, 1)[s["slots"]] = s["v"]
    return {"table": s["table"], "lengths": s["new_lengths"], "cursor": s["new_cursor"], "slots": s["slots"],
            "positions": s["positions"], "offsets": s["offsets"], "k": s["k_cache"], "v": s["v_cache"]}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return _append(state) if op == "append" else _step(state) if op == "step" else _attention(state)


# --- the definition in 64 bits ------------------------------------------------------------------

def _distance_bias(bias, case, gap):
    """bias[h][bucket of gap] in 64 bits, the bucket from the powers that bound it."""
    side = case["buckets"] if case["causal"] else case["buckets"] // 2
    exact = side // 2
    m = side - exact
    far = gap.abs()
    b = far.clamp(max=exact)
    for j in range(1, m):
        # the least whole number whose m-th power reaches exact^(m-j) reach^j
        least = int((exact ** (1 - j / m)) * (case["reach"] ** (j / m))) - 1
        while least ** m < exact ** (m - j) * case["reach"] ** j:
            least += 1
        b = b + (far >= least)
    if not case["causal"]:
        b = b + side * (gap < 0)
    return bias.double()[:, b], b


def _exact_rows(q, k, v, bias, case, scale, first, do=None):
    """One sequence and its heads [H, n, D] (k and v repeated), query rows from `first` on: o and what follows."""
    n_q, n_k = q.shape[1], k.shape[1]
    gap = first + torch.arange(n_q, device=q.device)[:, None] - torch.arange(n_k, device=q.device)[None]
    x = (q @ k.transpose(1, 2)) * scale
    of = None
    if bias is not None:
        add, of = _distance_bias(bias, case, gap)
        x = x + add
    if case["causal"]:
        x = torch.where(gap >= 0, x, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    o = p @ v
    if do is None:
        return o, lse
    ds = p * (do @ v.transpose(1, 2) - (do * o).sum(-1, keepdim=True))
    dbias = None
    if bias is not None:
        dbias = torch.stack([(ds * (of == b)).sum((1, 2)) for b in range(case["buckets"])], 1)
    return o, lse, scale * (ds @ k), scale * (ds.transpose(1, 2) @ q), p.transpose(1, 2) @ do, dbias


def exact(case, seed):
    global own
    kept, own = own, False  # inputs alone
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    H, K, scale = case["heads"], case["kv"], s["scale"]
    r = H // K
    n = lengths(case)
    if case["op"] == "append":
        return None  # whole numbers and copies
    if case["op"] == "step":
        o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
        for b, m in enumerate(n):
            if m == 0:
                continue
            ids = s["table"][b, :-(-m // case["block"])].long()
            k, v = (s[c][ids].flatten(0, 1)[:m].flatten(2).transpose(0, 1) for c in ("k_cache", "v_cache"))
            for h in range(K):  # one kv head in 64 bits at a time
                hs = slice(h * r, h * r + r)
                y, _ = _exact_rows(s["q"][b, hs].flatten(1).double()[:, None], k[h:h + 1].double().expand(r, -1, -1),
                                   v[h:h + 1].double().expand(r, -1, -1), None if s["bias"] is None else s["bias"][hs],
                                   case, scale, m - 1)
                o[b, hs] = y.reshape(r, *o.shape[2:])
        return {"o": o}
    train = case["op"] == "train"
    if train and s["bias"] is not None and _pairs(case) * H * case["buckets"] > 1 << 36:
        return None
    T = s["T"]
    wide = lambda x: x.flatten(2).double()  # noqa: E731
    zeros = lambda x: torch.zeros(*x.shape[:2], x.shape[2] * x.shape[3], dtype=torch.float64, device="cuda")  # noqa: E731
    out = {"o": zeros(s["o"])}
    if train:
        out |= {"lse": torch.empty(H, T, dtype=torch.float64, device="cuda"), "dq": zeros(s["q"]), "dk": zeros(s["k"]),
                "dv": zeros(s["v"])}
        if s["bias"] is not None:
            out["dbias"] = torch.zeros(H, case["buckets"], dtype=torch.float64, device="cuda")
    t0 = 0
    for m in n:
        t = slice(t0, t0 + m)
        t0 += m
        if m == 0:
            continue
        for h in range(K):
            per = max(1, min(r, (1 << 27) // (m * m)))  # query heads at a time
            for h0 in range(h * r, h * r + r, per):
                hs = slice(h0, min(h0 + per, h * r + r))
                w = hs.stop - hs.start
                k, v = (s[c][t, h:h + 1].flatten(2).double().transpose(0, 1).expand(w, -1, -1) for c in "kv")
                q = wide(s["q"][t, hs]).transpose(0, 1)
                do = wide(s["do"][t, hs]).transpose(0, 1) if train else None
                bias = None if s["bias"] is None else s["bias"][hs]
                rows = max(1, min(m, (1 << 27) // m))
                for i in range(0, m, rows):
                    part = slice(i, min(m, i + rows))
                    got = _exact_rows(q[:, part], k, v, bias, case, scale, i, do[:, part] if train else None)
                    at = slice(t.start + part.start, t.start + part.stop)
                    out["o"][at, hs] = got[0].transpose(0, 1)
                    if train:
                        out["lse"][hs, at] = got[1]
                        out["dq"][at, hs] = got[2].transpose(0, 1)
                        out["dk"][t, h] += got[3].sum(0)
                        out["dv"][t, h] += got[4].sum(0)
                        if bias is not None:
                            out["dbias"][hs] += got[5]
    for name, like in (("o", "o"), ("dq", "q"), ("dk", "k"), ("dv", "v")):
        if name in out:
            out[name] = out[name].reshape(s[like].shape)
    return out
