"""Which pointers of the delta rule's calls may start anywhere, and which on 16 bytes: as the header says."""

import pytest
import torch

import gdr_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from gpu_util import normwise
from test_gdr_gpu import on_gpu, tol_bwd, tol_fwd

pytestmark = pytest.mark.gpu

SHAPE = (2, 70, 3, 1, 7, 5)  # H N P is odd: the states of a pool do not all start on 16 bytes


def moved(t):
    """The same values one element behind an aligned start."""
    if t is None:
        return None
    space = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
    space.copy_(t)
    return space


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [SHAPE, (2, 70, 2, 1, 64, 64)], ids=str)
def test_inputs_may_start_at_any_element(shape, io):
    t, _ = on_gpu(ref.gdr_inputs(*shape, seed=91), io)
    names = ("q", "k", "v", "g", "beta")
    y, last = ss.ss_gdr_fwd(*[t[n] for n in names], scale=0.5, h0=t["h0"])
    d = ss.ss_gdr_bwd(*[t[n] for n in names], t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"])
    y2, last2 = ss.ss_gdr_fwd(*[moved(t[n]) for n in names], scale=0.5, h0=t["h0"])
    d2 = ss.ss_gdr_bwd(*[moved(t[n]) for n in names], moved(t["dy"]), scale=0.5, h0=t["h0"], dlast_state=t["dlast"])
    # (16-bit inputs move to other units: two results within tolerance of the truth)
    assert normwise(y2, y.double().cpu().numpy()) <= 2 * tol_fwd(io, "y")
    assert normwise(last2, last.double().cpu().numpy()) <= 2 * tol_fwd(io, "last")
    for n in d:
        assert normwise(d2[n], d[n].double().cpu().numpy()) <= 2 * tol_bwd(io, n), n
    # only g and beta moved: the same units, the same bits
    y3, last3 = ss.ss_gdr_fwd(t["q"], t["k"], t["v"], moved(t["g"]), moved(t["beta"]), scale=0.5, h0=t["h0"])
    assert torch.equal(y3, y) and torch.equal(last3, last)


def test_states_that_start_off_16_bytes_are_refused():
    B, L, H, G, N, P = SHAPE
    t, _ = on_gpu(ref.gdr_inputs(*SHAPE, seed=92), "f32")
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    pool = torch.zeros(5, H, N, P, device="cuda")
    with pytest.raises(ss.SSError, match="UNSUPPORTED"):
        ss.ss_gdr_fwd(*args, h0=pool[1:3])
    with pytest.raises(ss.SSError, match="UNSUPPORTED"):
        ss.ss_gdr_fwd(*args, last_state=pool[1:3])
    with pytest.raises(ss.SSError, match="UNSUPPORTED"):
        ss.ss_gdr_bwd(*args, t["dy"], dlast_state=pool[1:3])
    with pytest.raises(ss.SSError, match="UNSUPPORTED"):
        ss.ss_gdr_bwd(*args, t["dy"], out={"dbeta": moved(t["beta"])})
    with pytest.raises(ss.SSError, match="UNSUPPORTED"):
        ss.ss_gdr_step(*[a[:, 0].contiguous() for a in args], pool[1:3])
    with pytest.raises(ss.SSError, match="UNSUPPORTED"):
        ss.ss_gdr_step(*[a[:, 0].contiguous() for a in args], pool, y=moved(t["v"][:, 0].contiguous()))
    ss.ss_gdr_fwd(*args, h0=pool[:2], last_state=pool[:2].clone())
    assert not pool.any()
