"""Workloads of the token-mixing operators on regular-representation features: rotary
positions, linear attention with a decay for each head, and group norm with an activation.

A feature is a record of N group elements per channel, as the equivariant layers write it
([token][channel][N], group elements innermost).  Heads are runs of whole channels, so a head
of d channels is d N numbers wide.  All three operators commute with a cyclic shift of the
group axis: rotary turns channel pairs by an angle that is the same for every group element,
scores sum over it, and norm statistics run over it.

Sizes follow this repository's layers: width 768 (96 channels of C8) over 64 images of 197
tokens, width 1120 (160 channels of C7) over 32768 tokens, width 256 (32 channels of C8) over
4096 tokens.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CHUNK = 128  # tokens of one chunk of the plain linear attention


def _case(op, kind, name=None, **kw):
    c = {"op": op, "kind": kind, **kw}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # eight sequences being decoded, one new token each, far into their contexts
        _case("rotary", "forward", "rotary: 8 new tokens", dtype="bf16", N=8, heads=12, kv=12, d=8, rot=8,
              layout="half", scaling="banded", batch=8, tokens=1, context=32768, fused=True),
        # a prompt batch of images: half of each head's channels turned, keys shared by three query heads
        _case("rotary", "forward", "rotary: prompt", dtype="bf16", N=8, heads=12, kv=4, d=8, rot=4,
              layout="interleaved", scaling="none", batch=64, tokens=197, context=197, fused=True),
        # decoding: one token for each of a few sequences, the state read and written once
        _case("mix", "step", "mix: step of 8", dtype="bf16", N=8, heads=12, kv=12, dk=8, dv=8, batch=8, tokens=1,
              fused=True, ragged=False, state=True),
        # decoding at a large serving batch with wide shared heads
        _case("mix", "step", "mix: step of 512", dtype="bf16", N=8, heads=12, kv=4, dk=16, dv=16, batch=512, tokens=1,
              fused=True, ragged=False, state=True),
        # a prompt batch of images at the width of a base vision transformer
        _case("mix", "forward", "mix: prompt", dtype="bf16", N=8, heads=12, kv=12, dk=8, dv=8, batch=64, tokens=197,
              fused=True, ragged=False, state=False),
        # one long prompt of the odd-order layer, continued from a state
        _case("mix", "forward", "mix: long prompt", dtype="f16", N=7, heads=10, kv=10, dk=16, dv=16, batch=1,
              tokens=32768, fused=True, ragged=False, state=True),
        # a training step over packed images of unequal sizes, keys and values shared by three query heads
        _case("mix", "train", "mix: train, packed", dtype="bf16", N=8, heads=12, kv=4, dk=8, dv=8, batch=64,
              tokens=197, fused=True, ragged=True, state=True),
        # a training step in 32 bits at the narrow width
        _case("mix", "train", "mix: train, f32", dtype="f32", N=8, heads=4, kv=4, dk=8, dv=8, batch=16, tokens=256,
              fused=False, ragged=False, state=False),
        # the norm after mixing for new tokens: every token a sample of its own, a group for each head
        _case("norm", "forward", "norm: 8 new tokens", dtype="bf16", N=8, C=96, groups=12, act="silu", batch=8,
              tokens=1, ragged=False, fused=False),
        # the same norm in training, every token a sample
        _case("norm", "train", "norm: train, tokens", dtype="bf16", N=8, C=96, groups=12, act="silu", batch=64 * 197,
              tokens=1, ragged=False, fused=False),
        # statistics over whole images, packed, in training
        _case("norm", "train", "norm: train, images", dtype="bf16", N=8, C=96, groups=8, act="gelu", batch=64,
              tokens=197, ragged=True, fused=False),
        # one long map: the statistics of each group run over 32768 tokens
        _case("norm", "forward", "norm: long map", dtype="f16", N=7, C=160, groups=10, act="none", batch=1,
              tokens=32768, ragged=False, fused=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, kind = rng.choice([("rotary", "forward"), ("rotary", "inverse"), ("mix", "step"), ("mix", "forward"),
                           ("mix", "train"), ("norm", "forward"), ("norm", "train")])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    N = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 12, 16])
    top = max(2, 128 // N)
    c = _case(op, kind, dtype=dtype, N=N, fused=rng.random() < 0.5)
    if op == "norm":
        c["groups"] = rng.choice([1, 2, 4, 8, 12, 16])
        least = -(-16 // N)  # a group of one token holds 16 numbers at least: statistics of fewer say little
        c["C"] = c["groups"] * _log(rng, least, max(least, 1280 // (N * c["groups"])))
        c["act"] = rng.choice(["none", "gelu", "silu"])
        shape = rng.choice(["tokens", "samples", "one"])
        if shape == "tokens":
            c["batch"], c["tokens"] = _log(rng, 1, 32768), 1
        elif shape == "samples":
            c["batch"], c["tokens"] = _log(rng, 2, 128), _log(rng, 2, 1024)
        else:
            c["batch"], c["tokens"] = 1, _log(rng, 1, 32768)
        c["ragged"] = shape == "samples" and rng.random() < 0.5
    else:
        c["kv"] = rng.choice([1, 2, 3, 4, 8])
        c["heads"] = c["kv"] * rng.choice([1, 1, 2, 3, 4])
        if op == "rotary":
            c["d"] = max(2, _log(rng, 2, top))
            c["rot"] = 2 * rng.randint(1, c["d"] // 2)
            c["layout"] = rng.choice(["half", "interleaved"])
            c["scaling"] = rng.choice(["none", "linear", "raised", "banded"])
            c["batch"], c["tokens"] = (_log(rng, 1, 512), 1) if rng.random() < 0.4 else (_log(rng, 1, 64), _log(rng, 2, 1024))
            c["context"] = max(c["tokens"], _log(rng, 16, 131072))
        else:
            c["dk"], c["dv"] = (_log(rng, min(2, top), top) for _ in "kv")
            if kind == "step":
                c["batch"], c["tokens"] = _log(rng, 1, 512), 1
            elif rng.random() < 0.3:
                c["batch"], c["tokens"] = 1, _log(rng, 1, 32768)
            else:
                c["batch"], c["tokens"] = _log(rng, 1, 64), _log(rng, 1, 1024)
            c["ragged"] = kind != "step" and c["batch"] > 1 and rng.random() < 0.5
            c["state"] = kind == "step" or rng.random() < 0.5
    most = [work(k) for k in listed()]
    most = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    while work(c)["bytes"] > most[0] or work(c)["flops"] > most[1]:
        c["tokens" if c["tokens"] > 1 else "batch"] //= 2
        if "context" in c:
            c["context"] = max(c["context"], c["tokens"])
    return c


# --- what a case holds ------------------------------------------------------------------

def lengths(case):
    """Tokens of each sequence (or sample): equal, or unequal with an empty one and one of a single token."""
    B, S = case["batch"], case["tokens"]
    if not case.get("ragged"):
        return [S] * B
    g = torch.Generator().manual_seed(1000 * B + S)
    w = torch.rand(B, generator=g, dtype=torch.float64) * 1.5 + 0.25
    n = (w / w.sum() * (B * S)).floor().to(torch.int64).tolist()
    if B >= 4:
        n[1], n[2] = 0, 1
    n[-1] += B * S - sum(n)
    return [int(v) for v in n]


def work(case):
    T, N = case["batch"] * case["tokens"], case["N"]
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rotary":
        e = T * (case["heads"] + case["kv"]) * N
        return {"bytes": 2 * e * case["d"] * es + 4 * T, "flops": 3 * e * case["rot"]}
    if case["op"] == "norm":
        e = T * case["C"] * N
        if case["kind"] == "train":  # x in, y out; dy and x in, dx out
            return {"bytes": 5 * e * es, "flops": 30 * e}
        return {"bytes": 2 * e * es, "flops": 10 * e}
    Dk, Dv = case["dk"] * N, case["dv"] * N
    q, k, v, o = T * case["heads"] * Dk, T * case["kv"] * Dk, T * case["kv"] * Dv, T * case["heads"] * Dv
    s = case["batch"] * case["kv"] * Dk * Dv
    once = 2 * T * (case["heads"] + case["kv"]) * Dk * Dv  # the state read by every query, written by every key
    if case["kind"] == "step":
        return {"bytes": es * (q + k + v + o) + 8 * s, "flops": once}
    if case["kind"] == "forward":
        return {"bytes": es * (q + k + v + o) + (8 * s if case["state"] else 4 * s), "flops": once}
    grads = 2 * T * (2 * case["heads"] + 3 * case["kv"]) * Dk * Dv  # dq, and both states' updates; dk, dv
    return {"bytes": es * (3 * q + 3 * k + 3 * v + 2 * o) + (20 * s if case["state"] else 8 * s), "flops": once + grads}


class _Maker:
    """Inputs from the seed alone."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(self, *shape, dtype=torch.float32, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=self.g, device="cuda") * std + mean).to(dtype)


def _heads(m, T, parts, N, dtype, fused):
    """Tensors [T, heads, channels, N] for (heads, channels) in parts: slices of one projection's output, or apart."""
    if not fused:
        return [m.normal(T, h, d, N, dtype=dtype) for h, d in parts]
    y = m.normal(T, sum(h * d for h, d in parts), N, dtype=dtype)
    return list(_split(y, parts))


def _split(y, parts):
    at = 0
    for h, d in parts:
        yield y[:, at:at + h * d].unflatten(1, (h, d))
        at += h * d


def _like(T, parts, N, dtype, fused):
    if not fused:
        return [torch.empty(T, h, d, N, dtype=dtype, device="cuda") for h, d in parts]
    return list(_split(torch.empty(T, sum(h * d for h, d in parts), N, dtype=dtype, device="cuda"), parts))


def _offsets(case):
    at = [0]
    for n in lengths(case):
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int64, device="cuda")


def prepare(case, seed):
    m = _Maker(seed)
    dt = DTYPES[case["dtype"]]
    B, S, N = case["batch"], case["tokens"], case["N"]
    T = B * S
    s = {"case": case, "T": T, "offsets": _offsets(case) if case.get("ragged") else None}
    s["longest"] = max(lengths(case))
    if case["op"] == "rotary":
        H, K, d = case["heads"], case["kv"], case["d"]
        s["q"], s["k"] = _heads(m, T, [(H, d), (K, d)], N, dt, case["fused"])
        if S == 1:
            s["pos"] = torch.randint(0, case["context"], (T,), generator=m.g, device="cuda", dtype=torch.int32)
        else:
            first = torch.randint(0, case["context"] - S + 1, (B, 1), generator=m.g, device="cuda", dtype=torch.int32)
            s["pos"] = (first + torch.arange(S, device="cuda", dtype=torch.int32)).reshape(T).contiguous()
        s["q_out"], s["k_out"] = _like(T, [(H, d), (K, d)], N, dt, False)
    elif case["op"] == "mix":
        H, K, dk, dv = case["heads"], case["kv"], case["dk"], case["dv"]
        s["q"], s["k"], s["v"] = _heads(m, T, [(H, dk), (K, dk), (K, dv)], N, dt, case["fused"])
        # decays of a retentive layer: 1 - 2^-5, 1 - 2^-6, ..., from fast to slow over the heads
        h = torch.arange(K, dtype=torch.float64, device="cuda")
        s["log_decay"] = torch.log1p(-torch.exp2(-5.0 - h * (5.0 / max(1, K - 1)))).float()
        s["scale"] = 1.0 / math.sqrt(dk * N)
        s["o"] = torch.empty(T, H, dv, N, dtype=dt, device="cuda")
        s["state"] = m.normal(B, K, dk * N, dv * N, std=2.0) if case["state"] else None
        s["state_out"] = torch.empty(B, K, dk * N, dv * N, device="cuda")
        if case["kind"] == "train":
            s["do"] = m.normal(T, H, dv, N, dtype=dt)
            s["dq"], s["dk"], s["dv"] = _like(T, [(H, dk), (K, dk), (K, dv)], N, dt, case["fused"])
            s["dstate_out"] = m.normal(B, K, dk * N, dv * N, std=0.1) if case["state"] else None
            s["dstate"] = torch.empty(B, K, dk * N, dv * N, device="cuda") if case["state"] else None
    else:
        C = case["C"]
        # activations with a channel-dependent mean, as layers with biases give them
        if case["fused"]:
            y = m.normal(T, 2 * C, N) + m.normal(1, 2 * C, 1, std=0.5)
            s["x"] = y.to(dt)[:, C:]
        else:
            s["x"] = (m.normal(T, C, N) + m.normal(1, C, 1, std=0.5)).to(dt)
        s["gamma"], s["beta"] = m.normal(C, dtype=dt, std=0.2, mean=1.0), m.normal(C, dtype=dt, std=0.2)
        s["y"] = torch.empty(T, C, N, dtype=dt, device="cuda")
        if case["kind"] == "train":
            s["dy"] = m.normal(T, C, N, dtype=dt)
            s["dx"] = torch.empty(T, C, N, dtype=dt, device="cuda")
            s["dgamma"], s["dbeta"] = (torch.empty(C, device="cuda") for _ in "gb")
        s["eps"] = 1e-5
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
    if c["op"] == "rotary":
        layout = {"half": eq.EQL_ROTARY_HALF, "interleaved": eq.EQL_ROTARY_INTERLEAVED}[c["layout"]]
        s["plan"] = eq.eqlinear_rotary_plan(c["N"], c["heads"], c["kv"], c["d"], c["rot"], layout, dt,
                                            **_rotary_scaling(c, eq))
        return
    if c["op"] == "mix":
        s["plan"] = eq.eqlinear_mixer_plan(c["N"], c["heads"], c["kv"], c["dk"], c["dv"], dt)
        n = eq.eqlinear_linear_attention_workspace(s["plan"], s["T"], c["batch"], backward=c["kind"] == "train")
    else:
        act = {"none": eq.EQL_ACT_NONE, "gelu": eq.EQL_ACT_GELU, "silu": eq.EQL_ACT_SILU}[c["act"]]
        s["plan"] = eq.eqlinear_norm_plan(c["N"], c["C"], c["groups"], act, dt, eps=s["eps"])
        n = eq.eqlinear_group_norm_workspace(s["plan"], s["T"], c["batch"], backward=c["kind"] == "train")
        s["stats"] = torch.empty(c["batch"], c["groups"], 2, device="cuda") if c["kind"] == "train" else None
    s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def _rotary_scaling(c, eq):
    kind = {"none": eq.EQL_ROTARY_PLAIN, "linear": eq.EQL_ROTARY_LINEAR, "raised": eq.EQL_ROTARY_RAISED_BASE,
            "banded": eq.EQL_ROTARY_BANDED}[c["scaling"]]
    return {"base": BASE, "scaling": kind, "factor": FACTOR, "context": CONTEXT, "turns_slow": SLOW, "turns_fast": FAST,
            "magnitude": MAGNITUDE if c["scaling"] == "banded" else 1.0}


def _run_own(s):
    eq, c, plan = s["eq"], s["case"], s["plan"]
    if c["op"] == "rotary":
        eq.eqlinear_rotary(plan, s["q"], s["k"], s["pos"], s["q_out"], s["k_out"], inverse=c["kind"] == "inverse")
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "mix":
        if c["kind"] == "step":
            eq.eqlinear_linear_attention_step(plan, s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["o"],
                                              scale=s["scale"])
            return {"o": s["o"], "state": s["state"]}
        eq.eqlinear_linear_attention(plan, s["q"], s["k"], s["v"], s["log_decay"], s["o"], scale=s["scale"],
                                     offsets=s["offsets"], batch=c["batch"], state_in=s["state"],
                                     state_out=s["state_out"], workspace=s["workspace"])
        out = {"o": s["o"], "state": s["state_out"]}
        if c["kind"] == "train":
            eq.eqlinear_linear_attention_backward(plan, s["q"], s["k"], s["v"], s["do"], s["log_decay"], s["dq"],
                                                  s["dk"], s["dv"], scale=s["scale"], offsets=s["offsets"],
                                                  batch=c["batch"], state_in=s["state"], dstate_out=s["dstate_out"],
                                                  dstate_in=s["dstate"], workspace=s["workspace"])
            out |= {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}
            if s["dstate"] is not None:
                out["dstate"] = s["dstate"]
        return out
    train = c["kind"] == "train"
    eq.eqlinear_group_norm(plan, s["x"], s["gamma"], s["beta"], s["y"], stats=s["stats"], offsets=s["offsets"],
                           batch=c["batch"], workspace=s["workspace"])
    if not train:
        return {"y": s["y"]}
    eq.eqlinear_group_norm_backward(plan, s["dy"], s["x"], s["gamma"], s["beta"], s["stats"], s["dx"], s["dgamma"],
                                    s["dbeta"], offsets=s["offsets"], batch=c["batch"], workspace=s["workspace"])
    return {"y": s["y"], "dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}


# --- the plain forms ----------------------------------------------------------------------------

# rotary: the base, and a context of 4096 stretched eightfold
BASE, FACTOR, CONTEXT, SLOW, FAST, MAGNITUDE = 10000.0, 8.0, 4096, 1.0, 32.0, 0.1 * math.log(8.0) + 1.0


def _frequencies(case):
    """Angle per position of each channel pair, in 64 bits."""
    R = case["rot"]
    j = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    base = BASE * FACTOR ** (R / (R - 2)) if case["scaling"] == "raised" and R > 2 else BASE
    f = base ** (-2.0 * j / R)
    if case["scaling"] == "linear":
        f = f / FACTOR
    if case["scaling"] == "banded":
        # pairs that turn often within the trained context keep their pace, slow ones are stretched
        turns = CONTEXT * f / (2 * math.pi)
        keep = ((turns - SLOW) / (FAST - SLOW)).clamp(0.0, 1.0)
        f = f * keep + f / FACTOR * (1 - keep)
    return f


def _rotary(s):
    c = s["case"]
    # the angle in 64 bits: in 32 a large position loses the fraction of a turn
    ang = s["pos"].double()[:, None] * _frequencies(c)
    mag = MAGNITUDE if c["scaling"] == "banded" else 1.0
    cos, sin = (ang.cos() * mag).float()[:, None, :, None], (ang.sin() * mag).float()[:, None, :, None]
    if c["kind"] == "inverse":
        sin = -sin
    return {"q": _turn(s["q"], cos, sin, c), "k": _turn(s["k"], cos, sin, c)}


def _turn(x, cos, sin, c):
    R, y = c["rot"], x.float().clone()
    a, b = (slice(0, R // 2), slice(R // 2, R)) if c["layout"] == "half" else (slice(0, R, 2), slice(1, R, 2))
    xa, xb = y[:, :, a], y[:, :, b]
    ya, yb = xa * cos - xb * sin, xb * cos + xa * sin
    y[:, :, a], y[:, :, b] = ya, yb
    return y.to(x.dtype)


class _Batch:
    """Packed tokens as sequences of one padded length, a whole number of chunks."""

    def __init__(self, s):
        c = s["case"]
        self.B, self.T = c["batch"], s["T"]
        self.L = min(CHUNK, max(1, s["longest"]))
        self.S = max(1, -(-s["longest"] // self.L)) * self.L
        off = s["offsets"]
        if off is None:
            off = torch.arange(self.B + 1, device="cuda") * c["tokens"]
        self.len = off[1:] - off[:-1]
        at = torch.arange(self.S, device="cuda")
        self.valid = at[None] < self.len[:, None]
        self.index = torch.where(self.valid, off[:-1, None] + at[None], 0)
        token = torch.arange(self.T, device="cuda")
        seq = torch.searchsorted(off[1:].contiguous(), token, right=True)
        self.back = seq * self.S + token - off[seq]

    def take(self, x):
        """[T, H, d, N] -> [B, H, S, d N] in 32 bits, zeros past each end."""
        y = x.flatten(2).float()[self.index.reshape(-1)].reshape(self.B, self.S, x.shape[1], -1)
        return (y * self.valid[:, :, None, None]).transpose(1, 2).contiguous()

    def put(self, y, like):
        """[B, H, S, D] -> [T, H, d, N] in the type of `like`."""
        z = y.transpose(1, 2).reshape(self.B * self.S, y.shape[1], -1)[self.back]
        return z.to(like.dtype).unflatten(2, like.shape[2:])


def _decayed(a, b, c, la, L, reverse):
    """out[t] = sum over s <= t (s >= t if reverse) of exp(la |t - s|) (a[t] . b[s]) c[s], by chunks of L tokens."""
    B, H, S, _ = a.shape
    n = S // L
    a, b, c = (x.reshape(B, H, n, L, x.shape[-1]) for x in (a, b, c))
    i = torch.arange(L, device="cuda", dtype=torch.float32)
    la = la[:, None]
    gap = i[None, :] - i[:, None] if reverse else i[:, None] - i[None, :]
    near = torch.where(gap >= 0, torch.exp(la[:, :, None] * gap.clamp(min=0)), 0.0)  # [H, L, L]
    out = torch.matmul(torch.matmul(a, b.transpose(-1, -2).contiguous()) * near[None, :, None], c)
    if n == 1:
        return out.reshape(B, H, S, -1)
    carry = torch.exp(la * (i if reverse else L - 1 - i))  # [H, L]: a chunk's own state at its end
    kv = torch.matmul((b * carry[None, :, None, :, None]).transpose(-1, -2).contiguous(), c)  # [B, H, n, Da, Dc]
    j = torch.arange(n, device="cuda", dtype=torch.float32)
    far = (j[None, :] - j[:, None] if reverse else j[:, None] - j[None, :]) - 1
    far = torch.where(far >= 0, torch.exp(la[:, :, None] * (far.clamp(min=0) * L)), 0.0)  # [H, n, n]
    before = torch.matmul(far[None], kv.flatten(3)).reshape(kv.shape)
    reach = torch.exp(la * (L - i if reverse else i + 1))
    out = out + torch.matmul(a, before) * reach[None, :, None, :, None]
    return out.reshape(B, H, S, -1)


def _mix(s):
    case, la, scale = s["case"], s["log_decay"], s["scale"]
    g = _Batch(s)
    r = case["heads"] // case["kv"]
    wide = lambda x: x.repeat_interleave(r, dim=1)  # noqa: E731
    group = lambda x: x.unflatten(1, (case["kv"], r)).sum(2)  # noqa: E731
    q, k, v = g.take(s["q"]), g.take(s["k"]), g.take(s["v"])
    kw, vw, lw = wide(k), wide(v), la.repeat_interleave(r)
    at = torch.arange(g.S, device="cuda", dtype=torch.float32)
    last = (g.len[:, None] - 1 - at[None]).clamp(min=0).float()  # [B, S]: tokens after this one
    fade = torch.exp(la[None, :, None] * last[:, None])[..., None]  # [B, K, S, 1]
    grow = torch.exp(lw[:, None] * (at + 1))[None, :, :, None]
    full = torch.exp(la[None] * g.len[:, None].float())[..., None, None]  # [B, K, 1, 1]
    o = _decayed(q, kw, vw, lw, g.L, False)
    new = torch.matmul((k * fade).transpose(-1, -2).contiguous(), v)
    if s["state"] is not None:
        sw = wide(s["state"])
        o = o + torch.matmul(q, sw) * grow
        new = new + s["state"] * full
    out = {"o": g.put(o * scale, s["o"]), "state": new}
    if case["kind"] != "train":
        return out
    do = g.take(s["do"]) * scale
    dq = _decayed(do, vw, kw, lw, g.L, False)
    dk = group(_decayed(vw, do, q, lw, g.L, True))
    dv = group(_decayed(kw, q, do, lw, g.L, True))
    if s["state"] is not None:
        d = s["dstate_out"]
        dq = dq + torch.matmul(do, sw.transpose(-1, -2).contiguous()) * grow
        dk = dk + torch.matmul(v, d.transpose(-1, -2).contiguous()) * fade
        dv = dv + torch.matmul(k, d) * fade
        out["dstate"] = group(torch.matmul((q * grow).transpose(-1, -2).contiguous(), do)) + d * full
    return out | {"dq": g.put(dq, s["dq"]), "dk": g.put(dk, s["dk"]), "dv": g.put(dv, s["dv"])}


def _step(s):
    case = s["case"]
    r = case["heads"] // case["kv"]
    q, k, v = (s[n].flatten(2).float() for n in "qkv")
    S = s["state"]
    S.copy_(S * torch.exp(s["log_decay"])[None, :, None, None] + k[..., None] * v[:, :, None])
    o = (q[..., None] * S.repeat_interleave(r, dim=1)).sum(2) * s["scale"]
    return {"o": o.to(s["o"].dtype).unflatten(2, s["o"].shape[2:]), "state": S}


def _act(z, act):
    """The activation and its derivative."""
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return z, torch.ones_like(z)


def _norm(s):
    case, T = s["case"], s["T"]
    B, G, C, N = case["batch"], case["groups"], case["C"], case["N"]
    x = s["x"].float().reshape(T, G, -1)
    W = x.shape[2]
    if s["offsets"] is None:
        n = case["tokens"] * W

        def mean(z):  # over each sample's tokens and each group, for every token
            m = z.reshape(B, case["tokens"], G, W).sum((1, 3), keepdim=True) / n
            return m.expand(B, case["tokens"], G, 1).reshape(T, G, 1)
    else:
        off = s["offsets"]
        seq = torch.searchsorted(off[1:].contiguous(), torch.arange(T, device="cuda"), right=True)
        n = (off[1:] - off[:-1]).float()[seq][:, None, None] * W

        def mean(z):
            return torch.zeros(B, G, device="cuda").index_add_(0, seq, z.sum(2))[seq][..., None] / n
    c = x - mean(x)
    rstd = torch.rsqrt(mean(c * c) + s["eps"])
    xh = c * rstd
    gamma, beta = (s[p].float()[None, :, None] for p in ("gamma", "beta"))
    y, slope = _act(xh.reshape(T, C, N) * gamma + beta, case["act"])
    out = {"y": y.to(s["x"].dtype)}
    if case["kind"] != "train":
        return out
    dz = s["dy"].float() * slope
    out["dgamma"], out["dbeta"] = (dz * xh.reshape(T, C, N)).sum((0, 2)), dz.sum((0, 2))
    g = (dz * gamma).reshape(T, G, W)
    out["dx"] = ((g - mean(g) - xh * mean(g * xh)) * rstd).reshape(T, C, N).to(s["x"].dtype)
    return out


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "rotary":
        return _rotary(state)
    if c["op"] == "norm":
        return _norm(state)
    return _step(state) if c["kind"] == "step" else _mix(state)


# --- the definitions in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "mix": _exact_mix, "norm": _exact_norm}[case["op"]](s)


def _exact_rotary(s):
    """Every pair as a complex number times a complex unit."""
    c = s["case"]
    mag = MAGNITUDE if c["scaling"] == "banded" else 1.0
    turn = torch.polar(torch.full((s["T"], c["rot"] // 2), mag, dtype=torch.float64, device="cuda"),
                       s["pos"].double()[:, None] * _frequencies(c) * (-1 if c["kind"] == "inverse" else 1))
    out = {}
    for name in "qk":
        x = s[name].double()
        R = c["rot"]
        head = x[:, :, :R]
        pairs = head.unflatten(2, (2, R // 2)).transpose(2, 3) if c["layout"] == "half" else head.unflatten(2, (R // 2, 2))
        z = torch.complex(pairs[:, :, :, 0], pairs[:, :, :, 1]) * turn[:, None, :, None]
        z = torch.stack([z.real, z.imag], 2 if c["layout"] == "half" else 3).flatten(2, 3)
        out[name] = torch.cat([z, x[:, :, R:]], 2)
    return out


def _exact_mix(s):
    """Sequence by sequence, every query against every key before it, rows in blocks."""
    case = s["case"]
    r, scale = case["heads"] // case["kv"], s["scale"]
    train = case["kind"] == "train"
    q, k, v = (s[n].flatten(2).double().transpose(0, 1) for n in "qkv")  # [H, T, D]
    do = s["do"].flatten(2).double().transpose(0, 1) if train else None
    o = torch.zeros(case["heads"], s["T"], v.shape[2], dtype=torch.float64, device="cuda")
    grads = [torch.zeros_like(x) for x in (q, k, v)] if train else []
    la = s["log_decay"].double()
    ends, dends, at = [], [], 0
    for b, n in enumerate(lengths(case)):
        S0 = s["state"][b].double() if s["state"] is not None else torch.zeros(
            case["kv"], k.shape[2], v.shape[2], dtype=torch.float64, device="cuda")
        t = torch.arange(n, dtype=torch.float64, device="cuda")
        D1 = s["dstate_out"][b].double() if train and s["dstate_out"] is not None else torch.zeros_like(S0)
        fade = torch.exp(la[:, None] * (n - 1 - t))
        sl = slice(at, at + n)
        ends.append(S0 * torch.exp(la * n)[:, None, None] + (k[:, sl] * fade[..., None]).transpose(1, 2) @ v[:, sl])
        dS = D1 * torch.exp(la * n)[:, None, None]
        for g in range(case["kv"]):
            if train:
                grads[1][g, sl] += (v[g, sl] @ D1[g].T) * fade[g][:, None]
                grads[2][g, sl] += (k[g, sl] @ D1[g]) * fade[g][:, None]
        for h in range(case["heads"]):
            g = h // r
            for i in range(0, n, 2048):
                e = min(n, i + 2048)
                Q, K, V = q[h, at + i:at + e], k[g, at:at + e], v[g, at:at + e]
                gap = t[i:e, None] - t[None, :e]
                decay = torch.where(gap >= 0, torch.exp(la[g] * gap.clamp(min=0)), 0.0) * scale
                grow = torch.exp(la[g] * (t[i:e] + 1))[:, None] * scale
                P = Q @ K.T * decay
                o[h, at + i:at + e] = P @ V + (Q @ S0[g]) * grow
                if train:
                    dO = do[h, at + i:at + e]
                    dP = dO @ V.T * decay
                    grads[0][h, at + i:at + e] = dP @ K + (dO @ S0[g].T) * grow
                    grads[1][g, at:at + e] += dP.T @ Q
                    grads[2][g, at:at + e] += P.T @ dO
                    dS[g] += (Q * grow).T @ dO
        dends.append(dS)
        at += n
    back = lambda x, like: x.transpose(0, 1).unflatten(2, like.shape[2:])  # noqa: E731
    out = {"o": back(o, s["o"]), "state": torch.stack(ends)}
    if train:
        out |= {n: back(x, s[n]) for n, x in zip(("dq", "dk", "dv"), grads)}
        if s["dstate"] is not None:
            out["dstate"] = torch.stack(dends)
    return out


def _exact_norm(s):
    """The formula's forward, and autograd's gradients of it."""
    case = s["case"]
    T, B, G, C, N = s["T"], case["batch"], case["groups"], case["C"], case["N"]
    train = case["kind"] == "train"
    x, gamma, beta = (s[n].double().detach().clone().requires_grad_(train) for n in ("x", "gamma", "beta"))
    if case["ragged"]:
        parts = [p.reshape(1, n, G, -1) for p, n in zip(x.split(lengths(case)), lengths(case)) if n]
    else:
        parts = [x.reshape(B, case["tokens"], G, -1)]
    rows = []
    for p in parts:
        var, mean = torch.var_mean(p, (1, 3), correction=0, keepdim=True)
        rows.append(((p - mean) / torch.sqrt(var + s["eps"])).reshape(-1, C, N))
    z = torch.cat(rows) * gamma[None, :, None] + beta[None, :, None]
    y = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "none": lambda v: v}[case["act"]](z)
    out = {"y": y.detach()}
    if train:
        dx, dg, db = torch.autograd.grad(y, (x, gamma, beta), s["dy"].double())
        out |= {"dx": dx, "dgamma": dg, "dbeta": db}
    return out
