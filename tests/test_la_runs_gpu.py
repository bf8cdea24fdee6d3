"""The 16-bit backward where its blocks take runs of several heads that cut groups in two or more
parts, or hold whole groups, and the f32 forward's two kinds of tiles, against the 64-bit reference
(tolerances: those of test_la_gpu)."""

import pytest
import torch

import la_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from test_la_gpu import check_bwd, check_fwd

pytestmark = pytest.mark.gpu

# Bsz, L, H, G, N, P: more heads of chunks than SMs (152), so that runs are longer than one
SHAPES = [
    (3, 1000, 10, 2, 32, 64),    # 240: runs of one or two heads, groups of five in three to five parts
    (2, 700, 30, 1, 128, 32),    # 360, two or three a run
    (2, 1000, 38, 2, 16, 64),    # 608: exactly four a run
    (4, 640, 76, 19, 16, 32),    # 1520: ten a run, groups of four
    (1, 2500, 8, 8, 64, 80),     # groups of one head, two value tiles
]


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward_in_runs(shape, io):
    check_bwd(ref.la_inputs(*shape, h0=True, seed=sum(shape)), io)
    assert ss.device_status() == ss.SS_OK


def test_runs_repeat_bit_for_bit():
    x = ref.la_inputs(2, 700, 30, 1, 64, 64, seed=5)
    t = {n: torch.from_numpy(x[n]).to("cuda", torch.float32 if n == "g" else torch.bfloat16) for n in ("q", "k", "v", "g", "dy")}
    a, b = (ss.ss_la_bwd(t["q"], t["k"], t["v"], t["g"], t["dy"]) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in ("dq", "dk", "dv", "dg"))


@pytest.mark.parametrize("g", [-0.2, -0.25, -0.2500001, -0.3, 0.0, 0.01])
@pytest.mark.parametrize("N", [24, 64, 100])
def test_f32_on_either_side_of_a_slow_tile(g, N):
    """The f32 forward takes tiles of 16 tokens (8 for N > 64) by their decay, e^-4 or weaker or not."""
    x = ref.la_inputs(1, 150, 2, 1, N, 70, h0=True, seed=N)
    x["g"][:] = g
    x["g"][0, 40:80] *= 2  # both kinds in one sequence
    check_fwd(x, "f32")
