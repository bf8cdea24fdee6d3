"""A sequence mixer built on the linear-attention operators, as a model would use them: trained on
whole sequences, then given prompts of different lengths, then one token at a time for the sequences
of a state pool.

    python examples/linear_attention_layer.py        (needs a GB300)

Per head:  S_t = exp(g_t) S_{t-1} + k_t v_t^T,  y_t = q_t S_t / sqrt(N);  the heads' outputs are
normalised one by one, gated with silu(z), and projected back.  The projections are torch's.
"""

from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mamba_selective_scan_fwd_gb300 as ss  # noqa: E402


class LinearAttention(torch.autograd.Function):
    """ss_la_fwd with its gradient; the backward recomputes the states it needs."""

    @staticmethod
    def forward(ctx, q, k, v, g, scale, h0, lengths):
        y, last = ss.ss_la_fwd(q, k, v, g, scale=scale, h0=h0, lengths=lengths)
        ctx.save_for_backward(q, k, v, g, h0, lengths)
        ctx.scale = scale
        return y, last

    @staticmethod
    def backward(ctx, dy, dlast):
        q, k, v, g, h0, lengths = ctx.saved_tensors
        d = ss.ss_la_bwd(q, k, v, g, dy.contiguous(), scale=ctx.scale, h0=h0, dlast_state=dlast.contiguous(),
                         lengths=lengths)
        return d["dq"], d["dk"], d["dv"], d["dg"], None, d["dh0"], None


class GatedNorm(torch.autograd.Function):
    """norm(x) * silu(z), one group of channels per head."""

    @staticmethod
    def forward(ctx, x, weight, bias, z, groups):
        ctx.save_for_backward(x, weight, bias, z)
        ctx.groups = groups
        return ss.ss_gnorm_fwd(x, weight, bias, z, groups=groups)

    @staticmethod
    def backward(ctx, dout):
        x, weight, bias, z = ctx.saved_tensors
        d = ss.ss_gnorm_bwd(x, weight, bias, dout.contiguous(), z=z, groups=ctx.groups)
        return d["dx"], d["dweight"], d["dbias"], d["dz"], None


class Mixer(torch.nn.Module):
    """H heads of P value channels; G of them share their queries and keys of N channels."""

    def __init__(self, model, H, G, N, P, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.H, self.G, self.N, self.P = H, G, N, P
        to = {"dtype": dtype, "device": device}
        self.qkv = torch.nn.Linear(model, 2 * G * N + H * P, bias=False, **to)
        self.z = torch.nn.Linear(model, H * P, bias=False, **to)
        self.dt = torch.nn.Linear(model, H, bias=False, **to)
        self.out = torch.nn.Linear(H * P, model, bias=False, **to)
        f32 = {"dtype": torch.float32, "device": device}
        self.dt_bias = torch.nn.Parameter(torch.linspace(-5.0, -2.0, H, **f32))
        self.A_log = torch.nn.Parameter(torch.linspace(1.0, 8.0, H, **f32).log())
        self.norm_weight = torch.nn.Parameter(torch.ones(H * P, **f32))
        self.norm_bias = torch.nn.Parameter(torch.zeros(H * P, **f32))

    def inputs(self, x):
        """q, k, v: slices of one projection's output, which the operators read where they lie; and
        the log decays, <= 0."""
        q, k, v = self.qkv(x).split([self.G * self.N, self.G * self.N, self.H * self.P], -1)
        g = -self.A_log.exp() * F.softplus(self.dt(x).float() + self.dt_bias)
        return q.unflatten(-1, (self.G, self.N)), k.unflatten(-1, (self.G, self.N)), v.unflatten(-1, (self.H, self.P)), g

    def outputs(self, y, x):
        return self.out(GatedNorm.apply(y.flatten(-2), self.norm_weight, self.norm_bias, self.z(x), self.H))

    def forward(self, x, h0=None, lengths=None):
        """x [Bsz, L, model] -> (the same shape, the states after each row's last token)."""
        q, k, v, g = self.inputs(x)
        y, last = LinearAttention.apply(q, k, v, g, self.N ** -0.5, h0, lengths)
        return self.outputs(y, x), last

    def step(self, x, pool, slots):
        """One token x [Bsz, model] of the sequences whose states are pool[slots], updated in place."""
        q, k, v, g = self.inputs(x)
        return self.outputs(ss.ss_la_step(q, k, v, g, pool, scale=self.N ** -0.5, slots=slots), x)


def main():
    torch.manual_seed(0)
    mixer = Mixer(512, H=8, G=2, N=64, P=64)
    Bsz, L = 4, 300

    # train: fit one batch of random targets
    optim = torch.optim.Adam(mixer.parameters(), lr=2e-3)
    x, target = torch.randn(2, Bsz, L, 512, device="cuda", dtype=torch.bfloat16)
    for i in range(60):
        y, _ = mixer(x)
        loss = F.mse_loss(y.float(), target.float())
        optim.zero_grad()
        loss.backward()
        optim.step()
        if i % 20 == 0 or i == 59:
            print(f"training step {i}: loss {loss.item():.3f}")

    # serve: prompts of different lengths into the slots of a pool, then token by token
    with torch.no_grad():
        lengths = torch.tensor([300, 17, 128, 1], dtype=torch.int32, device="cuda")
        slots = torch.tensor([5, 0, 3, 6], dtype=torch.int32, device="cuda")
        pool = torch.zeros(8, mixer.H, mixer.N, mixer.P, device="cuda")
        _, last = mixer(x, lengths=lengths)
        pool[slots.long()] = last
        for _ in range(4):
            y = mixer.step(torch.randn(Bsz, 512, device="cuda", dtype=torch.bfloat16), pool, slots)
        print(f"after 4 tokens: outputs {tuple(y.shape)}, state norms {pool[slots.long()].flatten(1).norm(dim=1).tolist()}")
    status = ss.device_status()
    if status != ss.SS_OK:
        raise RuntimeError(ss.status_string(status))


if __name__ == "__main__":
    main()
