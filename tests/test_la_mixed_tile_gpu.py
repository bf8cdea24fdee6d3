"""The f32 forward where log decays of both signs meet in one tile.

Tolerance: 1e-5 of each token's largest value; what is left of the tokens before is nothing or within an
exponential's rounding (g of at most 50: 2^-24 x 50 = 3e-6)."""

import numpy as np
import pytest
import torch

import la_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from test_la_gpu import on_gpu
from test_la_strong_decay_gpu import off

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [24, 64, 100])
def test_f32_dip_and_rise_in_one_tile(N):
    """Decays of -100 and back in one tile: every token but the last, where the exact state leaves f32's range."""
    x = ref.la_inputs(1, 4, 2, 1, N, 64, seed=5)
    x["g"][0, :, :] = np.array([-50.0, -50.0, 48.0, 48.5])[:, None]
    t, r = on_gpu(x, "f32")
    y, _ = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"])
    with np.errstate(over="ignore", invalid="ignore"):
        wy, _ = ref.la_fwd(r["q"], r["k"], r["v"], r["g"])
    assert torch.isfinite(y[0, :3]).all()
    assert off(y[0, :3], wy[0, :3]) <= 1e-5
