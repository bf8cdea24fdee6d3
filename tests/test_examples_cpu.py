"""The examples' autograd functions without a GPU, their operators replaced by stand-ins: a second derivative, which no
operator here has, is refused and not left out."""

import os
import sys

import pytest
import torch

import mamba_selective_scan_fwd_gb300 as ss

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import delta_rule_layer as dl  # noqa: E402
import linear_attention_layer as la  # noqa: E402

B, L, H, G, N, P = 2, 3, 4, 2, 8, 6


def leaf(*shape):
    return torch.ones(shape, requires_grad=True)


def qk():
    return leaf(B, L, G, N), leaf(B, L, G, N)


CASES = {
    "QKNorm": (dl.QKNorm, lambda: (*qk(), leaf(N), leaf(N), None, torch.ones(2))),
    "GatedDeltaRule": (dl.GatedDeltaRule, lambda: (*qk(), leaf(B, L, H, P), leaf(B, L, H), leaf(B, L, H), 1.0, leaf(B, H, N, P), None)),
    "LinearAttention": (la.LinearAttention, lambda: (*qk(), leaf(B, L, H, P), leaf(B, L, H), 1.0, leaf(B, H, N, P), None)),
    "GatedNorm": (la.GatedNorm, lambda: (leaf(B, L, H * P), leaf(H * P), leaf(H * P), leaf(B, L, H * P), H)),
}


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    def like(**names):
        return {n: torch.ones_like(t) for n, t in names.items()}

    monkeypatch.setattr(ss, "ss_qknorm_fwd", lambda q, k, *_, **__: (q + 0, k + 0))
    monkeypatch.setattr(ss, "ss_qknorm_bwd", lambda q, k, dq, dk, qw, kw, *_, **__: like(dq=q, dk=k, dq_weight=qw, dk_weight=kw))
    monkeypatch.setattr(ss, "ss_gdr_fwd", lambda q, k, v, g, beta, scale, h0, lengths: (v + 0, h0 + 0))
    monkeypatch.setattr(ss, "ss_gdr_bwd", lambda q, k, v, g, beta, dy, scale, h0, dlast_state, lengths:
                        like(dq=q, dk=k, dv=v, dg=g, dbeta=beta, dh0=h0))
    monkeypatch.setattr(ss, "ss_la_fwd", lambda q, k, v, g, scale, h0, lengths: (v + 0, h0 + 0))
    monkeypatch.setattr(ss, "ss_la_bwd", lambda q, k, v, g, dy, scale, h0, dlast_state, lengths: like(dq=q, dk=k, dv=v, dg=g, dh0=h0))
    monkeypatch.setattr(ss, "ss_gnorm_fwd", lambda x, w, b, z, groups: x + 0)
    monkeypatch.setattr(ss, "ss_gnorm_bwd", lambda x, w, b, dout, z, groups: like(dx=x, dweight=w, dbias=b, dz=z))


@pytest.mark.parametrize("name", CASES)
def test_second_derivatives_are_refused(name):
    fn, make = CASES[name]
    args = make()
    leaves = [t for t in args if isinstance(t, torch.Tensor) and t.requires_grad]
    out = fn.apply(*args)
    loss = sum((t * t).sum() for t in (out if isinstance(out, tuple) else (out,)))
    grads = torch.autograd.grad(loss, leaves, create_graph=True)
    assert all(g.shape == t.shape for g, t in zip(grads, leaves))
    with pytest.raises(RuntimeError, match="once_differentiable|differentiate twice"):
        sum((g * t).sum() for g, t in zip(grads, leaves)).backward()


@pytest.mark.parametrize("name", CASES)
def test_first_derivatives_reach_every_leaf(name):
    fn, make = CASES[name]
    args = make()
    out = fn.apply(*args)
    sum(t.sum() for t in (out if isinstance(out, tuple) else (out,))).backward()
    assert all(t.grad is not None for t in args if isinstance(t, torch.Tensor) and t.requires_grad)
