"""More sequences, heads, biases or numbers of softmax attention and its cache than one launch of 2^32 threads takes:
every one of them is answered.  (A larger grid starts its workgroups modulo 2^32 threads and reports no error.)"""
import pytest

from test_gpu_operator_counts import WGS, eq, give_back, room  # noqa: F401

pytestmark = pytest.mark.gpu


def workspace(n):
    import torch
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def test_step_of_many_heads(eq):  # noqa: F811
    """2048 sequences of 2^14 heads: 2^25 workgroups of 128 threads join the parts of items that were cut.  Values are
    the sequence's own number (whole, below 2^11), so every mean of them is that number, to 2^-24 (n + 8) of it."""
    import torch
    room(8)
    B, H, n = 2048, 1 << 14, 300
    plan = eq.eqlinear_attention_plan(1, H, 1, 1, 1, eq.EQL_F32, causal=True)
    q = torch.randn(B, H, 1, 1, device="cuda")
    k = torch.randn(B, n, 1, 1, 1, device="cuda")
    number = torch.arange(1, B + 1, device="cuda", dtype=torch.float32)
    v = number.view(B, 1, 1, 1, 1).expand_as(k).contiguous()
    table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    lengths = torch.full((B,), n, dtype=torch.int32, device="cuda")
    o, lse = torch.full_like(q, 7.5), torch.full((H, B), float("nan"), device="cuda")
    eq.eqlinear_attention_step(plan, q, k, v, table, lengths, o, scale=1.0, lse=lse,
                               workspace=workspace(eq.eqlinear_attention_step_workspace(plan, B)))
    off = (o.view(B, H) - number[:, None]).abs() / number[:, None]
    assert float(off.max()) <= 2.0 ** -24 * 2 * (n + 8)
    assert bool(torch.isfinite(lse).all())


def test_step_of_many_sequences(eq):  # noqa: F811
    import torch
    room(4)
    B = WGS + 11
    plan = eq.eqlinear_attention_plan(1, 1, 1, 1, 1, eq.EQL_F32, causal=True)
    q, o = torch.randn(B, 1, 1, 1, device="cuda"), torch.full((B, 1, 1, 1), 7.5, device="cuda")
    k, v = torch.randn(B, 1, 1, 1, 1, device="cuda"), torch.randn(B, 1, 1, 1, 1, device="cuda")
    table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    lengths = torch.ones(B, dtype=torch.int32, device="cuda")
    eq.eqlinear_attention_step(plan, q, k, v, table, lengths, o, scale=1.0,
                               workspace=workspace(eq.eqlinear_attention_step_workspace(plan, B)))
    assert torch.equal(o.view(-1), v.view(-1))  # one key, met first: its probability is 1 to the bit


def test_attention_of_many_sequences(eq):  # noqa: F811
    """Sequences of one token each: o = v and dv = do within the rounding of lse (2^-24 |lse| and 2^-23 of the
    exponentials), dq = dk = 0."""
    import torch
    room(8)
    B = WGS + 9
    plan = eq.eqlinear_attention_plan(1, 1, 1, 1, 1, eq.EQL_F32)
    q, k, v, do = (torch.rand(B, 1, 1, 1, device="cuda") + 0.5 for _ in range(4))
    o, dq, dk, dv = (torch.full_like(q, 7.5) for _ in range(4))
    lse = torch.full((1, B), 7.5, device="cuda")
    eq.eqlinear_attention(plan, q, k, v, o, scale=1.0, lse=lse, batch=B)
    eq.eqlinear_attention_backward(plan, q, k, v, o, do, lse, dq, dk, dv, scale=1.0, batch=B,
                                   workspace=workspace(eq.eqlinear_attention_workspace(plan, B, B, B, True)))
    assert float((o - v).abs().max()) <= 2.0 ** -20
    assert float((dv - do).abs().max()) <= 2.0 ** -20
    assert float((lse.view(-1) - (q * k).view(-1)).abs().max()) <= 2.0 ** -20
    assert bool((dq == 0).all()) and bool((dk == 0).all())


def test_biases_of_many_heads(eq):  # noqa: F811
    """2^16 heads of 256 buckets: 2^24 sums of 256 threads.  Two causal tokens: the second sees distances 1 and 0, with
    probabilities p and 1 - p; dS = +-p (1 - p) (dP_0 - dP_1) in their buckets and 0 in all others."""
    import torch
    room(8)
    H = 1 << 16
    plan = eq.eqlinear_attention_plan(1, H, H, 1, 1, eq.EQL_F32, causal=True, buckets=256, max_distance=300)
    q, k, v, do = (torch.rand(2, H, 1, 1, device="cuda") + 0.5 for _ in range(4))
    o, dq, dk, dv = (torch.full_like(q, 7.5) for _ in range(4))
    bias = torch.randn(H, 256, device="cuda")
    lse, dbias = torch.empty(H, 2, device="cuda"), torch.full((H, 256), 7.5, device="cuda")
    eq.eqlinear_attention(plan, q, k, v, o, scale=1.0, bias=bias, lse=lse)
    eq.eqlinear_attention_backward(plan, q, k, v, o, do, lse, dq, dk, dv, scale=1.0, bias=bias, dbias=dbias,
                                   workspace=workspace(eq.eqlinear_attention_workspace(plan, 2, 2, 1, True)))
    Q, K, V, G = (t.double().view(2, H) for t in (q, k, v, do))
    s1, s0 = Q[1] * K[0] + bias[:, 1].double(), Q[1] * K[1] + bias[:, 0].double()
    p = torch.sigmoid(s1 - s0)
    ds = p * (1 - p) * G[1] * (V[0] - V[1])
    # scores of at most 8 in size, so exponentials off by 2^-24 (8 * 8 + 8); products and differences of numbers up to 2.25
    assert float((dbias[:, 1].double() - ds).abs().max()) <= 2.0 ** -17
    assert float((dbias[:, 0].double() + ds).abs().max()) <= 2.0 ** -17
    assert bool((dbias[:, 2:] == 0).all())


def test_a_store_past_32_bits(eq):  # noqa: F811
    """A cache of 2^32 numbers and more, row by row (rows off 16 bytes: a thread a number, more of them than a launch
    takes); single tokens read them back from its far blocks."""
    import torch
    room(60)
    d, bs = 130 // 2, 128
    blocks = (1 << 32) // (d * bs) + 3
    T = blocks * bs
    plan = eq.eqlinear_attention_plan(1, 1, 1, d, d, eq.EQL_BF16, causal=True)
    bits = lambda n: torch.randint(0, 1 << 14, (n,), dtype=torch.int16, device="cuda")  # noqa: E731 (finite numbers)
    k, v = (bits(T * d).view(torch.bfloat16).view(T, 1, d, 1) for _ in range(2))
    kc, vc = (torch.zeros(blocks, bs, 1, d, 1, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.arange(T - 1, -1, -1, dtype=torch.int64, device="cuda")
    slots[5] = -1
    eq.eqlinear_cache_store(plan, k, v, slots, kc, vc)
    for c, x in ((kc, k), (vc, v)):
        c, x = c.view(T, d).view(torch.int16), x.view(T, d).view(torch.int16)
        assert bool((c[T - 6] == 0).all())
        for i in range(0, T, 1 << 20):
            n = min(1 << 20, T - i)
            a, b = c[T - i - n:T - i].flip(0), x[i:i + n]
            if i == 0:
                a, b = torch.cat([a[:5], a[6:]]), torch.cat([b[:5], b[6:]])
            assert torch.equal(a, b), i
    # the last block's keys and the first's, against a cache of just these
    table = torch.tensor([[blocks - 1, 0]], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, d, 1, device="cuda").to(torch.bfloat16)
    ws = workspace(eq.eqlinear_attention_step_workspace(plan, 1))
    far, near = torch.empty_like(q), torch.empty_like(q)
    lengths = torch.tensor([bs + 77], dtype=torch.int32, device="cuda")
    eq.eqlinear_attention_step(plan, q, kc, vc, table, lengths, far, scale=0.125, workspace=ws)
    few = [c[[blocks - 1, 0]].contiguous() for c in (kc, vc)]
    eq.eqlinear_attention_step(plan, q, *few, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), lengths, near, scale=0.125,
                               workspace=ws)
    assert torch.equal(far, near) and bool((far != 0).any())
