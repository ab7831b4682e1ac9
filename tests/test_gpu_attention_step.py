"""Attention of single tokens over a paged cache against its fp64 definition (bounds as in attention_util), the
cache's tables and stores against theirs (whole numbers and copies: equal), and a run of them together."""
import numpy as np
import pytest

from attention_util import BF16, E, F16, F32, U, Problem, eqdt
from gpu_util import to_f64, torch_dtype
from oracle import attention as att

pytestmark = pytest.mark.gpu
TYPES = [F32, BF16, F16]


@pytest.fixture(scope="module")
def eq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import group_equivariant_linear_amd as eq
    eq.load_library()
    return eq


class Step:
    def __init__(self, eq, dt, N, H, K, dk, dv, lens, block, buckets=0, reach=0, seed=0, layout="apart", std=1.0, spare=2):
        import torch
        self.eq, self.dt, self.reach = eq, dt, reach
        self.plan = eq.eqlinear_attention_plan(N, H, K, dk, dv, eqdt(eq, dt), causal=True, buckets=buckets, max_distance=reach)
        g = torch.Generator().manual_seed(seed)
        tdt = torch_dtype(dt)
        B = len(lens)
        held = [-(-n // block) for n in lens]
        blocks = sum(held) + spare
        rand = lambda *s: (torch.randn(*s, generator=g) * std).to(tdt).cuda()  # noqa: E731
        if layout == "turns":  # keys and values of a block in turn, heads before tokens
            assert dk == dv
            buf = rand(blocks, 2, K, block, dk, N)
            self.kc, self.vc = buf[:, 0].transpose(1, 2), buf[:, 1].transpose(1, 2)
        elif layout == "odd":
            mk = lambda d: rand(blocks * block * (K * (d * N + 1) + 1) + 1).as_strided(  # noqa: E731
                (blocks, block, K, d, N), (block * (K * (d * N + 1) + 1), K * (d * N + 1) + 1, d * N + 1, N, 1), 1)
            self.kc, self.vc = mk(dk), mk(dv)
        else:
            self.kc, self.vc = rand(blocks, block, K, dk, N), rand(blocks, block, K, dv, N)
        order = torch.randperm(blocks, generator=g).to(torch.int32).tolist()
        self.rows = max(held) + 1
        table = torch.full((B, self.rows), -1, dtype=torch.int32)
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = torch.tensor(order[at:at + h], dtype=torch.int32)
            at += h
        self.table = table.cuda()
        self.lengths = torch.tensor(lens, dtype=torch.int32).cuda()
        self.q = rand(B, H, dk, N)
        self.o = torch.full((B, H, dv, N), 7.0, dtype=tdt, device="cuda")
        self.lse = torch.full((H, B), 7.0, device="cuda")
        self.bias = rand(H, buckets) if buckets else None
        self.scale = float(np.float32(1 / np.sqrt(dk * N)))
        n = eq.eqlinear_attention_step_workspace(self.plan, B)
        self.ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") if n else None

    def run(self, stream=None):
        self.eq.eqlinear_attention_step(self.plan, self.q, self.kc, self.vc, self.table, self.lengths, self.o, scale=self.scale,
                                        bias=self.bias, lse=self.lse, workspace=self.ws, stream=stream)

    def check(self, what):
        flat = lambda t: to_f64(t).reshape(*t.shape[:-2], -1)  # noqa: E731
        q, kc, vc = flat(self.q), flat(self.kc), flat(self.vc)
        table, lens = self.table.cpu().numpy(), self.lengths.cpu().numpy()
        bias = None if self.bias is None else to_f64(self.bias)
        o, lse = att.step(q, kc, vc, table, lens, self.scale, bias, self.reach)
        u, up = U[self.dt], 0.0 if self.dt == F32 else U[self.dt]
        y, yl = flat(self.o), to_f64(self.lse)
        r, bs = q.shape[1] // kc.shape[2], kc.shape[1]
        for b in range(len(q)):
            at = np.arange(min(max(int(lens[b]), 0), table.shape[1] * bs))
            ids = table[b][at // bs] if len(at) else np.zeros(0, int)
            ok = (ids >= 0) & (ids < len(kc))
            k, v = kc[ids[ok], at[ok] % bs], vc[ids[ok], at[ok] % bs]
            for h in range(q.shape[1]):
                if not len(k):
                    assert np.all(y[b, h] == 0) and yl[h, b] == -np.inf, what
                    continue
                s = self.scale * k[:, h // r] @ q[b, h]
                add = np.zeros(len(s)) if bias is None else \
                    np.array([bias[h][att.bucket(len(at) - 1 - j, bias.shape[1], self.reach, True)] for j in at[ok]])
                s = s + add
                L = abs(lse[h, b])
                es = E * ((q.shape[2] + 4) * self.scale * (np.abs(k[:, h // r]) @ np.abs(q[b, h])) + 8 * np.abs(s) + 8 * np.abs(add))
                worst = (2 * (es + E * (8 + 2 * L))).max()  # (one exponential more, of the join)
                p = np.exp(s - lse[h, b])
                low = 2.0 ** -37 * p.max() * np.abs(v[:, h // r]).sum(0) if self.dt == F16 else 0.0
                bound = 1.01 * (p @ np.abs(v[:, h // r]) * (up + 2 * worst + 2 * (len(s) + 8) * E) + low)
                bound = bound + np.maximum(u * np.abs(o[b, h]), 2.0 ** -25 if self.dt == F16 else 0.0)
                err = np.abs(y[b, h] - o[b, h])
                assert np.all(err <= bound), f"{what}: b {b} h {h}: off by {err.max():.3e}, {(err / bound).max():.2f} of the bound"
                assert abs(yl[h, b] - lse[h, b]) <= 1.01 * (worst + (len(s) + 8) * E) + 4 * E * L, f"{what}: lse"


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("N,dk,dv", [(8, 8, 8), (7, 16, 16), (8, 16, 16), (1, 1, 1), (5, 9, 9), (3, 11, 7), (4, 8, 24), (16, 8, 2)])
def test_widths(eq, dt, N, dk, dv):
    s = Step(eq, dt, N, 4, 2, dk, dv, [70, 33, 1], 16, seed=N)
    s.run()
    s.check(f"{dt} {N} {dk} {dv}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("block", [1, 7, 16, 64, 300])
@pytest.mark.parametrize("buckets,reach", [(0, 0), (32, 128)])
def test_lengths_and_blocks(eq, dt, block, buckets, reach):
    s = Step(eq, dt, 8, 2, 1, 8, 8, [0, 1, 2, 31, 32, 33, 127, 128, 129, 300, 1000], block, buckets, reach, seed=block)
    s.run()
    s.check(f"{dt} {block}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("H,K", [(1, 1), (3, 3), (16, 1), (17, 1), (40, 2)])
def test_shared_heads(eq, dt, H, K):
    s = Step(eq, dt, 8, H, K, 4, 4, [200, 5], 16, 16, 50, seed=H)
    s.run()
    s.check(f"{dt} {H} {K}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("layout", ["turns", "odd"])
def test_layouts(eq, dt, layout):
    s = Step(eq, dt, 8, 4, 2, 8, 8, [100, 40], 16, layout=layout)
    s.run()
    s.check(f"{dt} {layout}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("batch", [1, 200])
def test_one_long_and_many(eq, dt, batch):
    lens = [9000] if batch == 1 else [3 * b + 1 for b in range(batch)]
    s = Step(eq, dt, 4, 4, 2, 8, 8, lens, 16, 32, 1024)
    s.run()
    s.check(f"{dt} {batch}")


@pytest.mark.parametrize("dt", TYPES)
def test_blocks_that_are_not_there(eq, dt):
    """Ids below 0 and past the cache: their keys count as not there; lengths past the table are held to it."""
    s = Step(eq, dt, 8, 2, 1, 8, 8, [100, 60, 40, 10, 5], 16)
    s.table[0, 2], s.table[1, :] = -5, 1 << 30
    s.table[2, 0] = s.kc.shape[0]
    s.table[3, 0] = 0
    s.lengths[3] = 1 << 29
    s.lengths[4] = -3
    s.run()
    s.check(f"{dt}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("empty", ["blocks", "table", "lengths"])
def test_no_cache(eq, dt, empty):
    """A cache of no blocks, a table of no entries, sequences of no keys."""
    import torch
    s = Step(eq, dt, 8, 2, 1, 8, 8, [3, 0, 1], 16)
    if empty == "blocks":
        s.kc, s.vc = s.kc[:0], s.vc[:0]
    elif empty == "table":
        s.table = s.table[:, :0].contiguous()
    else:
        s.lengths.zero_()
    s.run()
    assert (s.o == 0).all() and (s.lse == -float("inf")).all()


@pytest.mark.parametrize("dt", TYPES)
def test_nan_behind_the_last_key(eq, dt):
    """Values and keys past a sequence's length, in its own last block too, and in blocks of no sequence."""
    import torch
    s = Step(eq, dt, 8, 2, 1, 8, 8, [100, 35, 0], 16)
    s.run()
    o, lse = s.o.clone(), s.lse.clone()
    used = torch.zeros(s.kc.shape[:2], dtype=torch.bool)
    for b, n in enumerate(s.lengths.tolist()):
        for j in range(n):
            used[int(s.table[b, j // 16]), j % 16] = True
    for c in (s.kc, s.vc):
        c[~used.cuda()] = float("nan")
    s.run()
    assert torch.equal(s.o, o) and torch.equal(s.lse, lse)


@pytest.mark.parametrize("dt", TYPES)
def test_infinities_that_are_seen(eq, dt):
    import torch
    s = Step(eq, dt, 8, 2, 2, 8, 8, [100, 100], 16)
    block, at = int(s.table[0, 3]), 5
    s.vc[block, at, 0, 1, 1] = float("inf")
    s.kc[int(s.table[1, 0]), 3, 1] = float("nan")
    s.run()
    assert s.o[0, 0, 1, 1] == float("inf") and torch.isnan(s.o[1, 1].float()).all()
    s.o[0, 0, 1, 1] = 0
    s.o[1, 1] = 0
    assert torch.isfinite(s.o.float()).all()


@pytest.mark.parametrize("dt", [BF16])
def test_a_cache_past_32_bits(eq, dt):
    """Blocks whose element offsets pass 2^32 (a cache of 9 GB, used at its ends)."""
    import torch
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("memory")
    blocks, block, d = 9 << 15, 128, 128  # 128 x 128 numbers a block
    s = Step(eq, dt, 1, 2, 1, d, d, [300, 200], block, spare=1)
    ids = torch.tensor([[0, blocks - 1, blocks // 2, -1], [blocks - 2, 5, -1, -1]], dtype=torch.int32).cuda()
    small_k, small_v, small_table = s.kc, s.vc, s.table
    s.kc = torch.zeros(blocks, block, 1, d, 1, dtype=torch.bfloat16, device="cuda")
    s.vc = torch.zeros_like(s.kc)
    for b in range(2):
        for j in range(3 - b):
            s.kc[ids[b, j].long()] = small_k[small_table[b, j].long()]
            s.vc[ids[b, j].long()] = small_v[small_table[b, j].long()]
    s.run()
    want = s.o.clone(), s.lse.clone()  # of the far blocks
    s.table = ids
    s.run()
    far = s.o.clone(), s.lse.clone()
    s.kc, s.vc, s.table = small_k, small_v, small_table
    s.run()
    assert torch.equal(far[0], s.o) and torch.equal(far[1], s.lse) and want[0].shape == s.o.shape


def test_captured(eq):
    import torch
    s = Step(eq, BF16, 8, 4, 2, 8, 8, [400, 90, 7], 16, 16, 60)
    s.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = s.o.clone()
    s.o.fill_(7.0)
    s.run(stream=side)
    side.synchronize()
    assert torch.equal(s.o, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for n in (399, 33, 1):
        s.lengths[0] = n
        g.replay()
        torch.cuda.synchronize()
        got = s.o.clone()
        s.run()
        torch.cuda.synchronize()
        assert torch.equal(s.o, got)
        s.check(f"{n}")


# --- tables and stores ------------------------------------------------------------------

def run_tables(eq, lengths, added, free, cursor, table, bs, T, in_place=False, stream=None):
    import torch
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    n, a, f, c, t = i32(lengths), i32(added), i32(free), i32([cursor]), i32(table)
    out, cout = (n, c) if in_place else (torch.empty_like(n), torch.empty_like(c))
    slots, pos = torch.full((T,), 77, dtype=torch.int64, device="cuda"), torch.full((T,), 77, dtype=torch.int32, device="cuda")
    off = torch.full((len(lengths) + 1,), 77, dtype=torch.int64, device="cuda")
    ws = torch.full((eq.eqlinear_cache_tables_workspace(len(lengths)),), 0xff, dtype=torch.uint8, device="cuda")
    eq.eqlinear_cache_tables(n, a, f, c, t, bs, out, cout, slots, pos, off, workspace=ws, stream=stream)
    return [x.cpu().numpy() for x in (t, out, cout, slots, pos, off)]


@pytest.mark.parametrize("batch", [1, 3, 64, 1023, 1024, 1025, 3000])
@pytest.mark.parametrize("bs", [1, 7, 16])
@pytest.mark.parametrize("kind", ["one", "ragged"])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables(eq, batch, bs, kind, in_place):
    rng = np.random.default_rng(batch + bs)
    lengths = rng.integers(0, 60, batch)
    added = np.ones(batch, int) if kind == "one" else rng.integers(0, 20, batch)
    max_blocks = -(-80 // bs)
    table = rng.integers(0, 10000, (batch, max_blocks))
    T = int(added.sum()) + (0 if kind == "one" else 5)
    need = int((-(-(lengths + added) // bs) - -(-lengths // bs)).sum())
    free = rng.permutation(need + 10)
    got = run_tables(eq, lengths, added, free, 4, table, bs, T, in_place)
    want = att.tables(lengths, added, free, 4, table, bs, T)
    for g, w, n in zip(got, want, ("table", "lengths", "cursor", "slots", "positions", "offsets")):
        assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1)), n


@pytest.mark.parametrize("case", ["short list", "past the table", "past T", "no tokens", "negative", "holes", "cursor"])
def test_tables_at_their_limits(eq, case):
    lengths, added, free, cursor, bs, T = [5, 0, 17, 8], [10, 30, 1, 8], list(range(100, 130)), 0, 4, 49
    table = np.arange(4 * 16).reshape(4, 16)
    if case == "short list":
        free = free[:5]
    elif case == "past the table":
        table = table[:, :5].copy()
    elif case == "past T":
        T = 20
    elif case == "no tokens":
        added, T = [0] * 4, 0
    elif case == "negative":
        lengths, added = [-3, 0, 17, 8], [10, -2, 1, 8]
    elif case == "holes":
        table[0, 1] = table[2, 4] = -1
    else:
        cursor = 28
    got = run_tables(eq, lengths, added, free, cursor, table, bs, T)
    want = att.tables(lengths, added, free, cursor, table, bs, T)
    for g, w, n in zip(got, want, ("table", "lengths", "cursor", "slots", "positions", "offsets")):
        assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1)), n


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("N,dk,dv,layout", [(8, 8, 8, "apart"), (8, 8, 8, "turns"), (5, 3, 7, "apart"), (7, 16, 16, "tokens"), (3, 5, 5, "odd")])
def test_store(eq, dt, N, dk, dv, layout):
    import torch
    K, blocks, bs, T = 3, 6, 16, 40
    tdt = torch_dtype(dt)
    plan = eq.eqlinear_attention_plan(N, K, K, dk, dv, eqdt(eq, dt))
    g = torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g).to(tdt).cuda()  # noqa: E731
    if layout == "turns":
        buf = rand(blocks, 2, K, bs, dk, N)
        kc, vc = buf[:, 0].transpose(1, 2), buf[:, 1].transpose(1, 2)
    elif layout == "tokens":
        buf = rand(blocks, bs, 2, K, dk, N)
        kc, vc = buf[:, :, 0], buf[:, :, 1]
    elif layout == "odd":
        mk = lambda d: rand(blocks * bs * (K * d * N + 1) + 1).as_strided(  # noqa: E731
            (blocks, bs, K, d, N), (bs * (K * d * N + 1), K * d * N + 1, d * N, N, 1), 1)
        kc, vc = mk(dk), mk(dv)
    else:
        kc, vc = rand(blocks, bs, K, dk, N), rand(blocks, bs, K, dv, N)
    rows = rand(T, K * (dk + dv), N)
    k, v = rows[:, :K * dk].unflatten(1, (K, dk)), rows[:, K * dk:].unflatten(1, (K, dv))
    slots = torch.randperm(blocks * bs, generator=g)[:T]
    slots[3], slots[9], slots[11] = -1, blocks * bs, 1 << 50
    want_k, want_v = kc.clone(), vc.clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < blocks * bs:
            want_k[s // bs, s % bs], want_v[s // bs, s % bs] = k[t], v[t]
    eq.eqlinear_cache_store(plan, k, v, slots.cuda(), kc, vc)
    bits = torch.int32 if dt == F32 else torch.int16
    assert torch.equal(kc.contiguous().view(bits), want_k.contiguous().view(bits))
    assert torch.equal(vc.contiguous().view(bits), want_v.contiguous().view(bits))


@pytest.mark.parametrize("dt", TYPES)
def test_serving(eq, dt):
    """Prompts, then single tokens: tables, rotary positions, stores and attention as one loop; every step's output
    is the row of one causal attention over the whole sequence."""
    import torch
    N, H, K, d, bs, B = 8, 4, 2, 8, 16, 3
    tdt, lens, steps = torch_dtype(dt), [21, 1, 40], 20
    plan = eq.eqlinear_attention_plan(N, H, K, d, d, eqdt(eq, dt), causal=True, buckets=8, max_distance=30)
    rot = eq.eqlinear_rotary_plan(N, H, K, d, d, eq.EQL_ROTARY_HALF, eqdt(eq, dt))
    g = torch.Generator().manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=g).to(tdt).cuda()  # noqa: E731
    total = [n + steps for n in lens]
    q, k, v = ([rand(n, h, d, N) for n in total] for h in (H, K, K))
    bias = rand(H, 8)
    scale = float(np.float32(1 / 8))
    kc, vc = rand(16, bs, K, d, N), rand(16, bs, K, d, N)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    lengths, cursor, table = i32([0] * B), i32([0]), torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(16, generator=g).to(torch.int32).cuda()
    ws = torch.empty(eq.eqlinear_cache_tables_workspace(B), dtype=torch.uint8, device="cuda")
    sws = torch.empty(max(1, eq.eqlinear_attention_step_workspace(plan, B)), dtype=torch.uint8, device="cuda")
    outs = [[] for _ in range(B)]
    for step in range(-1, steps):
        new = lens if step < 0 else [1] * B
        T = sum(new)
        slots, pos = torch.empty(T, dtype=torch.int64, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")
        off = torch.empty(B + 1, dtype=torch.int64, device="cuda")
        eq.eqlinear_cache_tables(lengths, i32(new), free, cursor, table, bs, lengths, cursor, slots, pos, off, workspace=ws)
        rows = [slice(0, n) if step < 0 else slice(n + step, n + step + 1) for n in lens]
        qs, ks, vs = (torch.cat([x[r] for x, r in zip(t, rows)]) for t in (q, k, v))
        eq.eqlinear_rotary(rot, qs, ks, pos, qs, ks)
        eq.eqlinear_cache_store(plan, ks, vs, slots, kc, vc)
        o = torch.empty(T, H, d, N, dtype=tdt, device="cuda")
        if step < 0:
            eq.eqlinear_attention(plan, qs, ks, vs, o, scale=scale, bias=bias, offsets=off)
        else:
            eq.eqlinear_attention_step(plan, qs, kc, vc, table, lengths, o, scale=scale, bias=bias, workspace=sws)
        at = 0
        for b, n in enumerate(new):
            outs[b].append(o[at:at + n])
            at += n
    assert lengths.tolist() == total
    for b, n in enumerate(total):
        p = Problem(eq, dt, N, H, K, d, d, [n], causal=True, buckets=8, reach=30, scale=scale)
        p.q, p.k, p.v, p.bias = q[b].clone(), k[b].clone(), v[b].clone(), bias
        eq.eqlinear_rotary(rot, p.q, p.k, torch.arange(n, dtype=torch.int32, device="cuda"), p.q, p.k)
        p.forward()
        p.check("whole", backward=False)
        p.o = torch.cat(outs[b])
        p.check("steps", backward=False)
