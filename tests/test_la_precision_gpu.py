"""The precision of what the tensor-core kernels keep in f32, tighter than the parity bounds: tight enough that a
part of the operands left out (w v without its last part: 2e-6 of the state; states without their third: 2.4e-6
of dg; without their second: 2^-9) does not pass.

Tolerances (normwise):
* last_state, dh0: w v holds 22 bits (f16) or 24 (bf16), 2^-22; a chunk's sum is accumulated in f32, with the 8
  steps of the largest part at full size, 8 x 2^-24 where they all round one way; the exponential has 2^-22:
  2^-20 together.
* dg: every term has two f32 scores (2^-23), an exponential (2^-22) and products, 2^-20 together at worst for one
  term, half as much again for the sums over tokens: 1.5 x 2^-20 where the states keep 22 bits or more.  bf16 with
  N > 64: states of 16 bits, 2^-17 of each of the N P terms, of random signs: 2^-18.
* f32 io: the same arithmetic on the FP32 units, 2^-20 for every output."""

import pytest
import torch

import la_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from gpu_util import normwise
from test_la_gpu import on_gpu

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1000, 8, 1, 64, 64), (1, 700, 4, 2, 128, 64), (2, 500, 4, 4, 32, 80)]


def dg_bound(io, N):
    return 2.0 ** -18 if io == "bf16" and N > 64 else 1.5 * 2.0 ** -20


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_f32_outputs(shape, io):
    t, r = on_gpu(ref.la_inputs(*shape, h0=True, seed=sum(shape)), io)
    y, last = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], scale=0.125, h0=t["h0"])
    got = ss.ss_la_bwd(t["q"], t["k"], t["v"], t["g"], t["dy"], scale=0.125, h0=t["h0"], dlast_state=t["dlast"])
    torch.cuda.synchronize()
    assert ss.device_status() == ss.SS_OK
    wy, wl = ref.la_fwd(r["q"], r["k"], r["v"], r["g"], 0.125, r["h0"])
    want = ref.la_bwd(r["q"], r["k"], r["v"], r["g"], r["dy"], 0.125, r["h0"], r["dlast"])
    errors = {"last": normwise(last, wl)}
    errors.update({n: normwise(x, want[n]) for n, x in got.items() if io == "f32" or n in ("dg", "dh0")})
    if io == "f32":
        errors["y"] = normwise(y, wy)
    print(io, shape, {n: f"{e:.1e}" for n, e in errors.items()})
    bounds = {n: dg_bound(io, shape[4]) if n == "dg" else 2.0 ** -20 for n in errors}
    assert not {n: e for n, e in errors.items() if not e <= bounds[n]}


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("every", [2, 3, 11, 100])
def test_resets_cost_no_precision(every, io):
    """Sequences packed into one row: dg, and dq, dk, dv where nothing is rounded to 16 bits."""
    x = ref.la_inputs(1, 300, 4, 2, 64, 64, h0=True, seed=every)
    x["g"][0, ::every, :] = -float("inf")
    x["g"][0, 5::every, 1] = -110.0
    t, r = on_gpu(x, io)
    got = ss.ss_la_bwd(t["q"], t["k"], t["v"], t["g"], t["dy"], scale=0.125, h0=t["h0"], dlast_state=t["dlast"])
    want = ref.la_bwd(r["q"], r["k"], r["v"], r["g"], r["dy"], 0.125, r["h0"], r["dlast"])
    assert ss.device_status() == ss.SS_OK
    for n in ("dg", "dq", "dk", "dv") if io == "f32" else ("dg",):
        assert normwise(got[n], want[n]) <= (dg_bound(io, 64) if n == "dg" else 2.0 ** -20), n
