"""The delta rule and the norm of its queries and keys together, in the layer of
examples/delta_rule_layer.py.

Tolerances (normwise, f32): the operators hold 1e-5 one by one; a gradient passes through four
projections, two norms and the delta rule, each of which adds its own and none of which is worse
conditioned than 10 at these sizes: 1e-4.  TF32 is off."""

import os
import subprocess
import sys

import pytest
import torch
import torch.nn.functional as F

import mamba_selective_scan_fwd_gb300 as ss
from gpu_util import normwise

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
from delta_rule_layer import DeltaMixer  # noqa: E402

pytestmark = pytest.mark.gpu
TOL = 1e-4


def host(t):
    return t.detach().double().cpu().numpy()


def plain(m, x, h0, lengths):
    """The layer in f64 torch operations, token by token (autograd gives its gradient)."""
    p = {n: w.detach().double().requires_grad_() for n, w in m.named_parameters()}
    H, G, N, P = m.H, m.G, m.N, m.P
    L = x.shape[1]
    q, k, v = (x @ p["qkv.weight"].T).split([G * N, G * N, H * P], -1)
    angle = torch.arange(L, device=x.device).double()[:, None, None] * m.freqs.double()
    pairs = len(m.freqs)

    def normed(t, w):
        t = t.unflatten(-1, (G, N))
        t = t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt() * w
        a, b, rest = t.split([pairs, pairs, N - 2 * pairs], -1)
        t = torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin(), rest], -1)
        return t.repeat_interleave(H // G, -2)

    q, k, v = normed(q, p["q_weight"]), normed(k, p["k_weight"]), v.unflatten(-1, (H, P))
    a, b = (x @ p["rates.weight"].T).split(H, -1)
    g, beta = -p["A_log"].exp() * F.softplus(a + p["dt_bias"]), torch.sigmoid(b)
    S, ys = h0, []
    for t in range(L):
        live = (t < lengths)[:, None, None, None]
        old = g[:, t].exp()[..., None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhn,bhnp->bhp", k[:, t], old))
        S = torch.where(live, old + k[:, t, ..., None] * u[:, :, None, :], S)
        ys.append(torch.where(live[..., 0], N ** -0.5 * torch.einsum("bhn,bhnp->bhp", q[:, t], S), 0.0))
    y = torch.stack(ys, 1)
    y = (y - y.mean(-1, keepdim=True)) / (y.var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    y = y.flatten(-2) * p["norm_weight"] + p["norm_bias"]
    return (y * F.silu(x @ p["z.weight"].T)) @ p["out.weight"].T, S, p


def test_layer_and_its_gradients():
    torch.manual_seed(1)
    m = DeltaMixer(48, H=4, G=2, N=16, P=32, dtype=torch.float32)
    x = torch.randn(3, 70, 48, device="cuda", requires_grad=True)
    h0 = torch.randn(3, 4, 16, 32, device="cuda", requires_grad=True)
    lengths = torch.tensor([70, 33, 1], dtype=torch.int32, device="cuda")
    dy, dlast = torch.randn(3, 70, 48, device="cuda"), torch.randn(3, 4, 16, 32, device="cuda")
    # the tokens past a row's length have outputs too (of y = 0): the loss leaves them out
    dy *= (torch.arange(70, device="cuda") < lengths[:, None])[..., None]
    y, last = m(x, h0, lengths)
    ((y * dy).sum() + (last * dlast).sum()).backward()
    x64, h64 = (t.detach().double().requires_grad_() for t in (x, h0))
    y64, last64, p64 = plain(m, x64, h64, lengths)
    ((y64 * dy.double()).sum() + (last64 * dlast.double()).sum()).backward()
    live = dy != 0
    got = {"y": y * live, "last": last, "dx": x.grad, "dh0": h0.grad}
    want = {"y": y64 * live, "last": last64, "dx": x64.grad, "dh0": h64.grad}
    for n, w in m.named_parameters():
        got[n], want[n] = w.grad, p64[n].grad
    assert ss.device_status() == ss.SS_OK
    bad = {n: e for n in got if not (e := normwise(host(got[n]), host(want[n]))) <= TOL}
    assert not bad, bad


def test_prompt_then_tokens():
    torch.manual_seed(2)
    m = DeltaMixer(48, H=4, G=2, N=32, P=24, dtype=torch.float32)
    lengths = torch.tensor([40, 9, 0], dtype=torch.int32, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    x, more = torch.randn(3, 40, 48, device="cuda"), torch.randn(3, 5, 48, device="cuda")
    with torch.no_grad():
        pool = torch.full((6, 4, 32, 24), 7.0, device="cuda")
        _, last = m(x, lengths=lengths)
        pool[slots.long()] = last
        ys = torch.stack([m.step(more[:, t], lengths + t, pool, slots) for t in range(5)], 1)
        for b, n in enumerate(lengths.tolist()):
            y, last = m(torch.cat([x[b:b + 1, :n], more[b:b + 1]], 1))
            assert normwise(host(ys[b]), host(y[0, n:])) <= TOL
            assert normwise(host(pool[slots[b].item()]), host(last[0])) <= TOL
    assert (pool[[1, 3, 5]] == 7.0).all()  # states of other sequences
    assert ss.device_status() == ss.SS_OK


def test_example_runs():
    subprocess.run([sys.executable, os.path.join(ROOT, "examples", "delta_rule_layer.py")], check=True, timeout=300)
