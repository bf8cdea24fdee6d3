"""GPU parity of the gated group norm, forward and backward, with its 64-bit reference.

Tolerances (normwise).  The arithmetic is f32 throughout and the inputs are exact, so 16-bit outputs
differ by their one rounding, u = 2^-8 (bf16) or 2^-11 (f16), doubled for values at a rounding border;
f32 outputs and the parameter sums by f32 rounding and the exponential's few ulp: 1e-5."""

import numpy as np
import pytest
import torch

import la_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from gpu_util import normwise

pytestmark = pytest.mark.gpu

IO = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TOL = {"f32": 1e-5, "bf16": 2 * 2.0 ** -8, "f16": 2 * 2.0 ** -11}

# (M, C, groups): groups of 1 to 8192 channels, whole 16-byte runs or not
SHAPES = [(1, 64, 1), (3, 1024, 16), (37, 640, 20), (9, 144, 2), (5, 35, 7), (17, 7, 7), (2, 999, 1), (4, 1280, 1), (3, 5120, 1),
          (70, 512, 2), (2, 8192, 1), (1, 8191, 1), (300, 5120, 80), (3, 2500, 4)]


def inputs(M, C, mode, io, seed):
    r = np.random.default_rng(seed)
    x = {"x": 2 * r.normal(size=(M, C)) + 0.3, "z": r.normal(size=(M, C)), "dout": r.normal(size=(M, C)),
         "weight": 1 + 0.2 * r.normal(size=C), "bias": 0.1 * r.normal(size=C)}
    if mode == "act":
        x["z"] = None
    t = {k: None if v is None else torch.from_numpy(v).to(IO[io] if v.ndim == 2 else torch.float32).cuda() for k, v in x.items()}
    return t, {k: None if v is None else v.double().cpu().numpy() for k, v in t.items()}


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("mode", ["gate", "act", "gate_first"])
@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_both_directions(shape, io, mode, center):
    M, C, groups = shape
    if mode == "gate_first" and center and C // groups == 1:
        pytest.skip("a centred group of one channel is constant")
    t, r = inputs(M, C, mode, io, M + C)
    kw = dict(groups=groups, center=center, gate_first=mode == "gate_first")
    out = ss.ss_gnorm_fwd(t["x"], t["weight"], t["bias"], t["z"], **kw)
    got = ss.ss_gnorm_bwd(t["x"], t["weight"], t["bias"], t["dout"], z=t["z"], **kw)
    want = ref.gnorm_fwd(r["x"], r["weight"], r["bias"], r["z"], groups, 1e-5, center, mode == "gate_first")
    assert normwise(out, want) <= TOL[io]
    want = ref.gnorm_bwd(r["x"], r["weight"], r["bias"], r["dout"], r["z"], groups, 1e-5, center, mode == "gate_first")
    for name, g in got.items():
        if name == "dz" and mode == "act":
            assert g is None
            continue
        # a group of one channel (rms: sign(x), no gradient): compared with the gradient's scale, not with zero
        scale = max(1.0, 1.0 / max(np.max(np.abs(want[name])), 1e-300)) if C == groups else 1.0
        assert normwise(g, want[name]) <= (1e-5 if name in ("dweight", "dbias") else TOL[io]) * scale, name


def test_without_parameters_and_misaligned():
    """No weight or bias; tensors that start off a 16-byte border."""
    t, r = inputs(33, 128, "gate", "bf16", 1)
    want = ref.gnorm_fwd(r["x"], None, None, r["z"], 4, 1e-5, True, False)
    assert normwise(ss.ss_gnorm_fwd(t["x"], z=t["z"], groups=4), want) <= TOL["bf16"]
    buf = torch.empty(33 * 128 + 1, dtype=torch.bfloat16, device="cuda")
    off = buf[1:].view(33, 128)
    off.copy_(t["x"])
    assert normwise(ss.ss_gnorm_fwd(off, z=t["z"], groups=4), want) <= TOL["bf16"]
    got = ss.ss_gnorm_bwd(off, None, None, t["dout"], z=t["z"], groups=4)
    assert got["dweight"] is None and got["dbias"] is None
    want = ref.gnorm_bwd(r["x"], None, None, r["dout"], r["z"], 4, 1e-5, True, False)
    assert normwise(got["dx"], want["dx"]) <= TOL["bf16"] and normwise(got["dz"], want["dz"]) <= TOL["bf16"]


def test_constant_and_offset_groups():
    """A constant group gives its bias (no division by zero); a mean far above the deviations loses nothing to
    cancellation beyond the input's own rounding."""
    x = torch.full((4, 64), 3.0, device="cuda")
    b = torch.randn(64, device="cuda")
    out = ss.ss_gnorm_fwd(x, None, b, groups=2)
    want = b.double() * torch.sigmoid(b.double())
    assert normwise(out, want.expand(4, 64).cpu().numpy()) <= 1e-5
    x = 1000 + torch.randn(8, 256, device="cuda")
    want = ref.gnorm_fwd(x.double().cpu().numpy(), None, None, None, 1, 1e-5, True, False)
    # the mean carries a rounding of 2^-24 * 1000 = 6e-5 against deviations of order one
    assert normwise(ss.ss_gnorm_fwd(x), want) <= 2e-4


def test_no_tokens():
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    assert ss.ss_gnorm_fwd(x, w, w, x).shape == (0, 64)
    got = ss.ss_gnorm_bwd(x, w, w, x, z=x)
    assert not got["dweight"].any() and not got["dbias"].any()


def test_repeats_bit_for_bit():
    t, _ = inputs(1000, 1024, "gate", "bf16", 2)
    a = ss.ss_gnorm_bwd(t["x"], t["weight"], t["bias"], t["dout"], z=t["z"], groups=16)
    b = ss.ss_gnorm_bwd(t["x"], t["weight"], t["bias"], t["dout"], z=t["z"], groups=16)
    assert all(torch.equal(a[k], b[k]) for k in a)
