"""The gated group norm without an epsilon (tolerances: those of test_gnorm_gpu)."""

import pytest

import la_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from gpu_util import normwise
from test_gnorm_gpu import TOL, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("mode", ["gate", "act", "gate_first"])
@pytest.mark.parametrize("C,groups", [(64, 4), (128, 2), (640, 20), (256, 1), (1024, 2), (2048, 1), (70, 2)])
@pytest.mark.parametrize("M", [1, 7, 8, 9])
def test_eps_zero(M, C, groups, mode, center):
    """Rows beyond the last of a block's eight have nothing to divide by."""
    t, r = inputs(M, C, mode, "f32", M + C)
    kw = dict(groups=groups, eps=0.0, center=center, gate_first=mode == "gate_first")
    out = ss.ss_gnorm_fwd(t["x"], t["weight"], t["bias"], t["z"], **kw)
    got = ss.ss_gnorm_bwd(t["x"], t["weight"], t["bias"], t["dout"], z=t["z"], **kw)
    form = (groups, 0.0, center, mode == "gate_first")
    assert normwise(out, ref.gnorm_fwd(r["x"], r["weight"], r["bias"], r["z"], *form)) <= TOL["f32"]
    want = ref.gnorm_bwd(r["x"], r["weight"], r["bias"], r["dout"], r["z"], *form)
    for name, g in got.items():
        if name == "dz" and mode == "act":
            assert g is None
        else:
            assert normwise(g, want[name]) <= TOL["f32"], name
