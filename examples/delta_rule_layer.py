"""A sequence mixer built on the gated delta rule, as a model would use it: trained on whole
sequences, then given prompts of different lengths, then one token at a time for the sequences of a
state pool.

    python examples/delta_rule_layer.py        (needs a GB300)

Per head, with q and k normalised and turned by their position:  u_t = beta_t (v_t - e^{g_t} S_{t-1}^T k_t),
S_t = e^{g_t} S_{t-1} + k_t u_t^T,  y_t = q_t S_t / sqrt(N);  the heads' outputs are normalised one by
one, gated with silu(z), and projected back.  The projections are torch's.
"""

from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mamba_selective_scan_fwd_gb300 as ss  # noqa: E402
from linear_attention_layer import GatedNorm  # noqa: E402


class QKNorm(torch.autograd.Function):
    """ss_qknorm_fwd with its gradient: unit queries and keys, turned by their positions."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, freqs):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, freqs)
        return ss.ss_qknorm_fwd(q, k, q_weight, k_weight, positions, freqs, l2=True)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        q, k, q_weight, k_weight, positions, freqs = ctx.saved_tensors
        d = ss.ss_qknorm_bwd(q, k, dq.contiguous(), dk.contiguous(), q_weight, k_weight, positions, freqs, l2=True)
        return d["dq"], d["dk"], d["dq_weight"], d["dk_weight"], None, None


class GatedDeltaRule(torch.autograd.Function):
    """ss_gdr_fwd with its gradient; the backward recomputes the states it needs."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, scale, h0, lengths):
        y, last = ss.ss_gdr_fwd(q, k, v, g, beta, scale=scale, h0=h0, lengths=lengths)
        ctx.save_for_backward(q, k, v, g, beta, h0, lengths)
        ctx.scale = scale
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dlast):
        q, k, v, g, beta, h0, lengths = ctx.saved_tensors
        d = ss.ss_gdr_bwd(q, k, v, g, beta, dy.contiguous(), scale=ctx.scale, h0=h0, dlast_state=dlast.contiguous(),
                          lengths=lengths)
        return d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"], None, d["dh0"], None


class DeltaMixer(torch.nn.Module):
    """H heads of P value channels; G of them share their queries and keys of N channels."""

    def __init__(self, model, H, G, N, P, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.H, self.G, self.N, self.P = H, G, N, P
        to = {"dtype": dtype, "device": device}
        self.qkv = torch.nn.Linear(model, 2 * G * N + H * P, bias=False, **to)
        self.z = torch.nn.Linear(model, H * P, bias=False, **to)
        self.rates = torch.nn.Linear(model, 2 * H, bias=False, **to)
        self.out = torch.nn.Linear(H * P, model, bias=False, **to)
        f32 = {"dtype": torch.float32, "device": device}
        self.dt_bias = torch.nn.Parameter(torch.linspace(-5.0, -2.0, H, **f32))
        self.A_log = torch.nn.Parameter(torch.linspace(1.0, 8.0, H, **f32).log())
        self.q_weight = torch.nn.Parameter(torch.ones(N, **f32))
        self.k_weight = torch.nn.Parameter(torch.ones(N, **f32))
        self.norm_weight = torch.nn.Parameter(torch.ones(H * P, **f32))
        self.norm_bias = torch.nn.Parameter(torch.zeros(H * P, **f32))
        # a quarter of the channels turn, by up to a radian a token
        self.register_buffer("freqs", 1e4 ** (-torch.arange(N // 8, **f32) / (N // 8)))

    def inputs(self, x, positions):
        """q, k (normalised and turned) and v, a slice of one projection's output, which the operators
        read where it lies; the log decays, <= 0; the rates in (0, 1).  x [Bsz, L, model]."""
        q, k, v = self.qkv(x).split([self.G * self.N, self.G * self.N, self.H * self.P], -1)
        q, k = QKNorm.apply(q.unflatten(-1, (self.G, self.N)), k.unflatten(-1, (self.G, self.N)), self.q_weight, self.k_weight,
                            positions, self.freqs)
        a, b = self.rates(x).float().split(self.H, -1)
        g = -self.A_log.exp() * F.softplus(a + self.dt_bias)
        return q, k, v.unflatten(-1, (self.H, self.P)), g, torch.sigmoid(b)

    def outputs(self, y, x):
        return self.out(GatedNorm.apply(y.flatten(-2), self.norm_weight, self.norm_bias, self.z(x), self.H))

    def forward(self, x, h0=None, lengths=None):
        """x [Bsz, L, model] -> (the same shape, the states after each row's last token)."""
        y, last = GatedDeltaRule.apply(*self.inputs(x, None), self.N ** -0.5, h0, lengths)
        return self.outputs(y, x), last

    def step(self, x, positions, pool, slots):
        """One token x [Bsz, model] at ``positions`` (int32 [Bsz]) of the sequences whose states are
        pool[slots], updated in place."""
        q, k, v, g, beta = (t[:, 0] for t in self.inputs(x[:, None], positions[:, None]))
        return self.outputs(ss.ss_gdr_step(q, k, v, g, beta, pool, scale=self.N ** -0.5, slots=slots), x)


def main():
    torch.manual_seed(0)
    mixer = DeltaMixer(512, H=8, G=4, N=64, P=64)
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
        for i in range(4):
            y = mixer.step(torch.randn(Bsz, 512, device="cuda", dtype=torch.bfloat16), lengths + i, pool, slots)
        print(f"after 4 tokens: outputs {tuple(y.shape)}, state norms {pool[slots.long()].flatten(1).norm(dim=1).tolist()}")
    status = ss.device_status()
    if status != ss.SS_OK:
        raise RuntimeError(ss.status_string(status))


if __name__ == "__main__":
    main()
