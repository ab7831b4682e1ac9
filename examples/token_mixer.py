"""An equivariant token mixer: the layers and the operators between them as one residual block.

    h = norm(x)                              every token's channels, in groups
    q, k, v = EQ-Linear(h)                   one projection, heads are slices of its rows
    q, k = rotary(q, k)                      in place
    o = linear attention(q, k, v)            decay exp(log_decay) per kv head, fp32 state
    y = x + EQ-Linear(silu(norm(o)))         a group for each head

x and y are [T][C][N].  Every step commutes with a cyclic shift of the group axis, so the block
does.  forward() takes packed sequences, backward() gives every gradient, step() adds one token
to each of a batch of sequences, reading nothing of the past but the state.

    python examples/token_mixer.py
"""
from __future__ import annotations

import math
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import group_equivariant_linear_amd as eq  # noqa: E402


class TokenMixer:
    """Weights, spectra and plans of one block."""

    def __init__(self, N=8, C=96, heads=12, kv_heads=4, d=8, dtype=eq.EQL_BF16, seed=0):
        self.N, self.C, self.H, self.K, self.d = N, C, heads, kv_heads, d
        wide = (heads + 2 * kv_heads) * d
        self.into = eq.eqlinear_plan(N, C, wide, dtype)
        self.out = eq.eqlinear_plan(N, heads * d, C, dtype)
        self.norm_x = eq.eqlinear_norm_plan(N, C, 1, eq.EQL_ACT_NONE, dtype)
        self.norm_o = eq.eqlinear_norm_plan(N, heads * d, heads, eq.EQL_ACT_SILU, dtype)
        self.rotary = eq.eqlinear_rotary_plan(N, heads, kv_heads, d, d, eq.EQL_ROTARY_HALF, dtype)
        self.mixer = eq.eqlinear_mixer_plan(N, heads, kv_heads, d, d, dtype)
        self.scale = 1.0 / math.sqrt(d * N)
        # half-lives from about 20 tokens up, doubling from head to head
        self.log_decay = torch.log1p(-torch.exp2(-5.0 - torch.arange(kv_heads))).float().cuda()

        g = torch.Generator().manual_seed(seed)
        dt = self.norm_x.torch_dtype
        self.w_in = (torch.randn(wide, C, N, generator=g) / math.sqrt(C * N)).to(dt).cuda()
        self.w_out = (torch.randn(C, heads * d, N, generator=g) / math.sqrt(heads * d * N)).to(dt).cuda()
        self.gamma_x, self.beta_x, self.gamma_o, self.beta_o = (
            (a + 0.1 * torch.randn(n, generator=g)).to(dt).cuda()
            for n, a in ((C, 1.0), (C, 0.0), (heads * d, 1.0), (heads * d, 0.0)))
        self.update()

    def update(self):
        """The spectra of the weights: after every change of w_in or w_out."""
        self.hat, self.adjoint = [], []
        for plan, w in ((self.into, self.w_in), (self.out, self.w_out)):
            hat, adj = torch.empty_like(w).view(-1), torch.empty_like(w).view(-1)
            eq.eqlinear_weight_fft(plan, w, hat)
            eq.eqlinear_w_hat_adjoint(plan, hat, adj)
            self.hat.append(hat)
            self.adjoint.append(adj)

    def new_state(self, batch):
        D = self.d * self.N
        return torch.zeros(batch, self.K, D, D, device="cuda")

    def _norm(self, plan, x, gamma, beta, stats=None):
        y = torch.empty_like(x)
        ws = self._workspace(eq.eqlinear_group_norm_workspace(plan, len(x), len(x)))
        eq.eqlinear_group_norm(plan, x, gamma, beta, y, stats=stats, batch=len(x), workspace=ws)
        return y

    def _heads(self, u):
        return u[:, :self.H], u[:, self.H:self.H + self.K], u[:, self.H + self.K:]

    def _project(self, h, positions):
        u = torch.empty(len(h), self.H + 2 * self.K, self.d, self.N, dtype=h.dtype, device="cuda")
        eq.eqlinear_forward(self.into, h, self.hat[0], u)
        q, k, v = self._heads(u)
        eq.eqlinear_rotary(self.rotary, q, k, positions, q, k)
        return u, q, k, v

    def _finish(self, x, n):
        y = torch.empty_like(x)
        eq.eqlinear_forward(self.out, n, self.hat[1], y)
        return y.add_(x)

    @staticmethod
    def _workspace(n):
        return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")

    def forward(self, x, offsets, positions, state=None):
        """x [T][C][N]; sequence b is tokens offsets[b] .. offsets[b + 1]; positions int32 [T]; state: of the
        tokens before (None: none).  Returns y, the state after the last tokens, and what backward() needs."""
        T, B = len(x), offsets.numel() - 1
        stats_x = torch.empty(T, 1, 2, device="cuda")
        stats_o = torch.empty(T, self.H, 2, device="cuda")
        h = self._norm(self.norm_x, x, self.gamma_x, self.beta_x, stats_x)
        u, q, k, v = self._project(h, positions)
        o = torch.empty(T, self.H, self.d, self.N, dtype=x.dtype, device="cuda")
        after = self.new_state(B)
        ws = self._workspace(eq.eqlinear_linear_attention_workspace(self.mixer, T, B))
        eq.eqlinear_linear_attention(self.mixer, q, k, v, self.log_decay, o, self.scale, offsets=offsets,
                                     state_in=state, state_out=after, workspace=ws)
        o = o.view(T, self.H * self.d, self.N)
        n = self._norm(self.norm_o, o, self.gamma_o, self.beta_o, stats_o)
        return self._finish(x, n), after, (x, offsets, positions, state, stats_x, stats_o, h, u, o, n)

    def _norm_backward(self, plan, dy, x, gamma, beta, stats):
        dx = torch.empty_like(x)
        dg, db = (torch.empty(x.shape[1], device="cuda") for _ in range(2))
        ws = self._workspace(eq.eqlinear_group_norm_workspace(plan, len(x), len(x), True))
        eq.eqlinear_group_norm_backward(plan, dy, x, gamma, beta, stats, dx, dg, db, batch=len(x), workspace=ws)
        return dx, dg, db

    def _layer_backward(self, plan, adjoint, x, dy):
        dx = torch.empty_like(x)
        dw = torch.empty(dy.numel() // len(dy) // self.N, x.shape[1], self.N, device="cuda")
        eq.eqlinear_backward_data(plan, dy, adjoint, dx)
        ws = self._workspace(eq.eqlinear_backward_weight_workspace(plan, len(x)))
        eq.eqlinear_backward_weight(plan, x, dy, dw, ws)
        return dx, dw

    def backward(self, dy, saved, dstate_after=None):
        """Gradients of a sum of dy y (and dstate_after state): a dict by name, weights' and norms' in fp32."""
        x, offsets, positions, state, stats_x, stats_o, h, u, o, n = saved
        T, B, g = len(x), offsets.numel() - 1, {}
        dn, g["w_out"] = self._layer_backward(self.out, self.adjoint[1], n, dy)
        do, g["gamma_o"], g["beta_o"] = self._norm_backward(self.norm_o, dn, o, self.gamma_o, self.beta_o, stats_o)
        du = torch.empty_like(u)
        (q, k, v), (dq, dk, dv) = self._heads(u), self._heads(du)
        if state is not None:
            g["state"] = torch.empty_like(state)
        ws = self._workspace(eq.eqlinear_linear_attention_workspace(self.mixer, T, B, True))
        eq.eqlinear_linear_attention_backward(
            self.mixer, q, k, v, do.view(T, self.H, self.d, self.N), self.log_decay, dq, dk, dv, self.scale,
            offsets=offsets, state_in=state, dstate_out=dstate_after, dstate_in=g.get("state"), workspace=ws)
        eq.eqlinear_rotary(self.rotary, dq, dk, positions, dq, dk, inverse=True)  # a turn's transpose
        dh, g["w_in"] = self._layer_backward(self.into, self.adjoint[0], h, du)
        dx, g["gamma_x"], g["beta_x"] = self._norm_backward(self.norm_x, dh, x, self.gamma_x, self.beta_x, stats_x)
        g["x"] = dx.add_(dy)
        return g

    def step(self, x, positions, state):
        """One token of each sequence, x [B][C][N]: y, and state [B] in place.  Launches only: a HIP graph may
        hold it."""
        h = self._norm(self.norm_x, x, self.gamma_x, self.beta_x)
        _, q, k, v = self._project(h, positions)
        o = torch.empty(len(x), self.H, self.d, self.N, dtype=x.dtype, device="cuda")
        eq.eqlinear_linear_attention_step(self.mixer, q, k, v, self.log_decay, state, o, self.scale)
        n = self._norm(self.norm_o, o.view(len(x), self.H * self.d, self.N), self.gamma_o, self.beta_o)
        return self._finish(x, n)


def packed(lens):
    """(offsets, positions) of sequences of these lengths, one after the other, on the GPU."""
    offsets = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int64).cuda()
    positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    return offsets, positions


def main():
    torch.manual_seed(0)
    block, lens = TokenMixer(), [197, 50, 1, 144]
    offsets, positions = packed(lens)
    x = torch.randn(sum(lens), block.C, block.N, device="cuda").to(block.w_in.dtype)
    y, state, saved = block.forward(x, offsets, positions)
    turned = block.forward(x.roll(3, 2), offsets, positions)[0]
    off = (turned.float() - y.roll(3, 2).float()).norm() / y.float().norm()
    print(f"prompt: {len(lens)} sequences, {len(x)} tokens; a shift of the group axis passes through to {off:.1e}")

    grads = block.backward(torch.randn_like(y), saved)
    print("gradients: " + ", ".join(f"{n} {tuple(t.shape)}" for n, t in grads.items()))

    at = torch.tensor(lens, dtype=torch.int32).cuda()
    token = y[offsets[1:] - 1].contiguous()
    for _ in range(8):
        token = block.step(token, at, state)
        at += 1
    torch.cuda.synchronize()
    print(f"8 tokens more for each: positions {at.tolist()}, state {tuple(state.shape)}")


if __name__ == "__main__":
    main()
