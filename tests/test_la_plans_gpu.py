"""Parity of the time-cut plans on the tensor cores: whole units beside cut ones, carried starts in every 16-bit
type, N beyond 64, padded rows (tolerances: those of test_la_gpu; test_la_plans_cpu asks the planner that these
shapes are cut so)."""

import numpy as np
import pytest
import torch

import la_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from gpu_util import normwise
from test_la_gpu import check_bwd, check_fwd, on_gpu, tol_bwd, tol_fwd
from test_la_plans_cpu import SHAPES

pytestmark = pytest.mark.gpu


def walk64(t, scale, lengths):
    """The recurrence and its reverse token by token in 64 bits on the GPU, all heads at once.  dg from the sums of
    q.dq and k.dk of the tokens from t on: exact to 1e-12 in 64 bits."""
    q, k, v, g, dy, h0, dlast = (t[n].double() for n in ("q", "k", "v", "g", "dy", "h0", "dlast"))
    Bsz, L, H, P = v.shape
    G = q.shape[2]
    of = torch.arange(H, device=v.device) // (H // G)
    n = torch.as_tensor(lengths, device=v.device)
    on = (torch.arange(L, device=v.device) < n[:, None])
    S, y, dq = h0, torch.zeros_like(v), torch.zeros(Bsz, L, H, q.shape[3], dtype=torch.float64, device=v.device)
    for i in range(L):
        new = g[:, i].exp()[:, :, None, None] * S + k[:, i, of][..., None] * v[:, i][:, :, None]
        S = torch.where(on[:, i, None, None, None], new, S)
        y[:, i] = scale * torch.einsum("bhn,bhnp->bhp", q[:, i, of], S)
        dq[:, i] = scale * torch.einsum("bhnp,bhp->bhn", S, dy[:, i])
    last, end = S, (S * dlast).sum((-1, -2))
    R, dk, dv = dlast, torch.zeros_like(dq), torch.zeros_like(v)
    for i in reversed(range(L)):
        live = on[:, i, None, None, None]
        R = torch.where(live, R + scale * q[:, i, of][..., None] * dy[:, i][:, :, None], R)
        dk[:, i] = torch.einsum("bhnp,bhp->bhn", R, v[:, i])
        dv[:, i] = torch.einsum("bhnp,bhn->bhp", R, k[:, i, of])
        R = torch.where(live, g[:, i].exp()[:, :, None, None] * R, R)
    live = on[..., None, None]
    y, dq, dk, dv = (x * live for x in (y, dq, dk, dv))
    dg = ((q[:, :, of] * dq - k[:, :, of] * dk).sum(-1).flip(1).cumsum(1).flip(1) + end[:, None]) * on[..., None]
    groups = lambda x: x.unflatten(2, (G, -1)).sum(3)
    return {"y": y, "last": last, "dq": groups(dq), "dk": groups(dk), "dv": dv, "dg": dg, "dh0": R}


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_whole_units_beside_cut_ones(shape, io):
    Bsz, L = shape[:2]
    t, _ = on_gpu(ref.la_inputs(*shape, h0=True, seed=sum(shape)), io)
    lengths = [L, 1111][:Bsz]
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, last = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], scale=0.5, h0=t["h0"], lengths=n)
    got = ss.ss_la_bwd(t["q"], t["k"], t["v"], t["g"], t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"], lengths=n)
    assert ss.device_status() == ss.SS_OK
    want = {name: x.cpu().numpy() for name, x in walk64(t, 0.5, lengths).items()}
    assert normwise(y, want["y"]) <= tol_fwd(io, "y") and normwise(last, want["last"]) <= tol_fwd(io, "last")
    for name, x in got.items():
        assert normwise(x, want[name]) <= tol_bwd(io, name), name


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("N,P", [(16, 16), (64, 64), (128, 64), (72, 80)])
def test_few_heads_cut_in_time(N, P, io):
    x = ref.la_inputs(1, 3000, 2, 1, N, P, h0=True, seed=N + P)
    check_fwd(x, io)
    check_bwd(x, io)


def test_the_walk_agrees_with_the_reference():
    x = ref.la_inputs(2, 30, 4, 2, 16, 8, h0=True, seed=51)
    t, r = on_gpu(x, "f32")
    lengths = [30, 11]
    got = walk64(t, 0.5, lengths)
    y, last = ref.la_fwd(r["q"], r["k"], r["v"], r["g"], 0.5, r["h0"], lengths)
    want = ref.la_bwd(r["q"], r["k"], r["v"], r["g"], r["dy"], 0.5, r["h0"], r["dlast"], lengths)
    for name, w in {"y": y, "last": last, **want}.items():
        assert np.max(np.abs(got[name].cpu().numpy() - w)) <= 1e-11 * np.max(np.abs(w)), name
