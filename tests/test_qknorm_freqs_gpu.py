"""Frequencies around zero: the angles that they make are the reference's (tolerances: those of test_qknorm_gpu)."""

import pytest
import torch

import mamba_selective_scan_fwd_gb300 as ss
from test_qknorm_gpu import check, inputs

pytestmark = pytest.mark.gpu

# just below zero a frequency's distance to the whole turn below it rounds to a whole turn in 64 bits (at -3.4e-16 the last such)
TINY = [-1e-17, -0.0, 0.0, -1e-30, -1.4e-45, -3.4e-16, -3.5e-16, -1e-15, 1e-17, 1.4e-45, -1e-12, -1e-7, 1e-12, 1e-7, -0.5, 0.5]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("far", [0, 2_000_000_000, -2_000_000_000])
def test_frequencies_around_zero(far, interleaved):
    x = inputs(2, 30, 2, 1, 2 * len(TINY), len(TINY), True, "f32", seed=8, far=far)
    x["freqs"] = torch.tensor(TINY, device="cuda")
    out, d = check(x, "f32", interleaved=interleaved)
    assert all(torch.isfinite(t).all() for t in (*out, *d.values()))


@pytest.mark.parametrize("sign", [1, -1])
def test_whole_and_half_turns(sign):
    """Frequencies of a half turn and of whole turns a token, and their neighbours, either way round."""
    turn = 6.2831855
    x = inputs(2, 30, 2, 1, 16, 8, True, "f32", seed=9)
    f = torch.tensor([turn / 2, turn, 3 * turn / 2, 2 * turn], device="cuda")
    x["freqs"] = sign * torch.cat([f, torch.nextafter(f, torch.zeros_like(f))])
    check(x, "f32")


def test_frequencies_that_are_not_finite_spoil_their_channels_only():
    x = inputs(1, 9, 2, 1, 16, 4, False, "f32", seed=10)
    want, _ = check(x, "f32")
    for bad in (float("nan"), float("inf"), -float("inf")):
        x["freqs"][1] = bad
        got = ss.ss_qknorm_fwd(x["q"], x["k"], positions=x["positions"], freqs=x["freqs"])
        for a, b in zip(got, want):
            assert torch.isnan(a[..., [1, 5]]).all()
            rest = [c for c in range(16) if c not in (1, 5)]
            assert torch.equal(a[..., rest], b[..., rest])
