"""Strong decays, where nothing hides what is left of the old state: v is zero after the first tokens, and every
token's y and the states are held to their own size.

Tolerance 1e-5 (f32 outputs; bf16 y: 3 u): the cumulative log decays stay above -80, so that their rounding to
log2 units, 2^-24 of at most 115, moves the result by 4.8e-6 and the exponential by 2^-22 more."""

import numpy as np
import pytest

import la_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from gpu_util import normwise
from test_la_gpu import on_gpu, tol_fwd

pytestmark = pytest.mark.gpu

G = [-0.2, -0.6, -0.8, -2.0, -8.0, -12.0, -17.0, -30.0, -75.0]


def off(got, want):
    """Largest error of a token, by the token's own largest value ([tokens, ...])."""
    got, want = got.double().cpu().numpy().reshape(len(want), -1), want.reshape(len(want), -1)
    return np.max(np.max(np.abs(got - want), 1) / np.max(np.abs(want), 1))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N", [24, 64, 128])
@pytest.mark.parametrize("g", G)
def test_what_is_left_of_the_first_state(g, N, io):
    L = int(min(40, 80 / -g))
    x = ref.la_inputs(1, L, 2, 1, N, 64, h0=True, seed=3)
    x["v"][:] = 0
    x["g"][:] = g
    t, r = on_gpu(x, io)
    y, last = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], h0=t["h0"])
    wy, wl = ref.la_fwd(r["q"], r["k"], r["v"], r["g"], 1.0, r["h0"])
    assert off(y[0], wy[0]) <= tol_fwd(io, "y")
    assert off(last, wl) <= 1e-5
    state = t["h0"].clone()
    for i in range(L):
        y = ss.ss_la_step(t["q"][:, i], t["k"][:, i], t["v"][:, i], t["g"][:, i].contiguous(), state)
        assert off(y, wy[:, i]) <= tol_fwd(io, "y")
    assert off(state, wl) <= 1e-5


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [24, 64, 128])
@pytest.mark.parametrize("g", [-8.0, -17.0, -30.0])
def test_sequences_cut_in_time(g, N, io):
    """One strong decay soon after (forward) or before (backward) the only tokens that add to the states."""
    L = 2000
    x = ref.la_inputs(1, L, 1, 1, N, 64, seed=4)
    x["g"][:] = 0
    x["g"][0, 40] = x["g"][0, L - 41] = g
    x["v"][0, 3:] = 0
    x["dy"][0, :-3] = 0
    x["h0"] = np.zeros((1, 1, N, 64))
    t, r = on_gpu(x, io)
    y, last = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], h0=t["h0"])
    wy, wl = ref.la_fwd(r["q"], r["k"], r["v"], r["g"], 1.0, r["h0"])
    assert off(last, wl) <= 1e-5
    if io != "f16":  # (whose range ends above e^-17)
        # a q nearly orthogonal to the three k leaves a small y of large terms: by the stretches between the decays
        for part in (slice(0, 40), slice(40, L - 41), slice(L - 41, L)):
            assert normwise(y[0, part], wy[0, part]) <= tol_fwd(io, "y")
    got = ss.ss_la_bwd(t["q"], t["k"], t["v"], t["g"], t["dy"], h0=t["h0"])
    want = ref.la_bwd(r["q"], r["k"], r["v"], r["g"], r["dy"], 1.0, r["h0"])
    assert off(got["dh0"], want["dh0"]) <= 1e-5
