"""The gated delta rule under positive log decays, up to the documented limit: runs of tokens inside 64 that add up to 60.

16-bit outputs, and f32 io: the tolerances of test_gdr_gpu.  f32 outputs of 16-bit io: its 22-bit operands leave 1e-6 of the norm, four
times that by the largest element; a chunk's decay is the exponential of one rounded number of up to 60: 60 x 2^-24 = 3.6e-6;
1e-5 for both.  y by the largest value of its own token (bf16; f16 cannot hold such ranges): half a step, 2^-8, and what is a
2^-18 of values that are up to eight times the token's: 2^-15."""

import numpy as np
import pytest
import torch

import gdr_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from gpu_util import normwise
from test_gdr_gpu import check_bwd, check_fwd, on_gpu

pytestmark = pytest.mark.gpu

B, L, H, G, N, P = 2, 150, 4, 2, 64, 64


def inputs(kind, grow, size=1.0, shape=(B, L, H, G, N, P)):
    x = ref.gdr_inputs(*shape, seed=81)
    L = shape[1]
    g = np.full(L, -0.01)
    if kind == "ramp":  # one chunk's every token
        g[:64] = grow / 64
    elif kind == "burst":  # three tokens amid a chunk
        g[30:33] = grow / 3
    elif kind == "across":  # two chunks' tokens
        g[40:104] = grow / 64
    elif kind == "dip":  # a chunk that decays first, then grows as much
        g[10:20], g[45:50] = -grow / 10, grow / 5
    elif kind == "saw":  # up and down by turns
        g[:] = np.where(np.arange(L) % 2, -grow / 32, grow / 32)
    elif kind == "reset":  # growth from an empty state
        g[20], g[40:50] = -np.inf, grow / 10
    x["g"][:] = g[None, :, None].astype(np.float32)
    x["g"][:, :, 1] = ref.gdr_inputs(*shape, seed=82)["g"][:, :, 1]  # a head without growth beside them
    for n in ("v", "h0", "dy", "dlast"):
        x[n] *= np.float32(size)
    return x


KINDS = ["ramp", "burst", "across", "dip", "saw", "reset"]


@pytest.mark.parametrize("io,grow,size", [("f32", 58, 1e-6), ("bf16", 12, 1.0), ("bf16", 30, 1.0), ("bf16", 58, 1e-6), ("f16", 12, 2e-3)])
@pytest.mark.parametrize("kind", KINDS)
def test_growth(kind, io, grow, size):
    x = inputs(kind, grow, size)
    for lengths in (None, [L, 47]):
        y, last = check_fwd(x, io, lengths=lengths)
        d = check_bwd(x, io, lengths=lengths)
        assert all(torch.isfinite(z).all() for z in (y, last, *(d[n] for n in d)))
        _, r = on_gpu(x, io)
        rargs = [r[n] for n in ("q", "k", "v", "g", "beta")]
        wy, wl = ref.gdr_fwd(*rargs, 0.5, r["h0"], lengths)
        w = ref.gdr_bwd(*rargs, r["dy"], 0.5, r["h0"], r["dlast"], lengths)
        assert normwise(last, wl) <= 1e-5
        assert {n: e for n in ("dg", "dbeta", "dh0") if not (e := normwise(d[n], w[n])) <= 1e-5} == {}
        if io != "f16":
            off, most = np.abs(y.double().cpu().numpy() - wy).max(-1), np.abs(wy).max(-1)
            assert (off <= ((1.01 * 2.0 ** -8 if io == "bf16" else 0.0) + 2.0 ** -15) * most).all()


@pytest.mark.parametrize("kind", KINDS)
def test_growth_in_sequences_cut_in_time(kind):
    check_fwd(inputs(kind, 40, 1e-4, (1, 4100, 2, 1, 64, 64)), "bf16")
    check_bwd(inputs(kind, 40, 1e-4, (1, 2700, 2, 1, 64, 64)), "bf16")


def test_heads_without_growth_keep_their_bits():
    """A head's results do not change when another one's decays grow."""
    x = inputs("across", 30)
    t, _ = on_gpu(x, "bf16")
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    y, last = ss.ss_gdr_fwd(*args, scale=0.5, h0=t["h0"])
    d = ss.ss_gdr_bwd(*args, t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"])
    t["g"][:, :, [0, 2, 3]] = -0.1
    y2, last2 = ss.ss_gdr_fwd(*args, scale=0.5, h0=t["h0"])
    d2 = ss.ss_gdr_bwd(*args, t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"])
    assert torch.equal(y[:, :, 1], y2[:, :, 1]) and torch.equal(last[:, 1], last2[:, 1])
    for n in ("dv", "dg", "dbeta"):
        assert torch.equal(d[n][:, :, 1], d2[n][:, :, 1])


@pytest.mark.parametrize("io,rate", [("f32", 10.0), ("bf16", 5.0)])
def test_rates_that_let_the_state_grow(io, rate):
    """beta |k|^2 beyond two: the state grows by some 2^16 (5) or 2^50 (10) inside 64 tokens."""
    x = ref.gdr_inputs(1, 128, 2, 1, 64, 64, gate=False, seed=4)
    x["beta"][:] = rate
    for n in ("v", "h0", "dy", "dlast"):
        x[n] *= np.float32(1e-3)
    check_fwd(x, io)
    check_bwd(x, io)
