"""Tokens past a row's length are zeros and other rows are untouched whatever the row's own tokens hold, NaN and
infinities included, on the tensor cores and on the FP32 units."""

import numpy as np
import pytest
import torch

import la_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from test_la_gpu import IO

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v", "dy", "g", "h0", "dlast"])
@pytest.mark.parametrize("io,P", [("f32", 64), ("bf16", 64), ("f16", 64), ("bf16", 66)])
def test_padding_is_zero(io, P, where, bad):
    Bsz, L, H, G, N = 3, 300, 4, 2, 64
    x = ref.la_inputs(Bsz, L, H, G, N, P, h0=True, seed=31)
    t = {n: torch.from_numpy(v).to("cuda", IO[io] if n in ("q", "k", "v", "dy") else torch.float32) for n, v in x.items()}
    lengths = torch.tensor([L, 150, 70], dtype=torch.int32, device="cuda")

    def run():
        y, last = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], scale=0.5, h0=t["h0"], lengths=lengths)
        d = ss.ss_la_bwd(t["q"], t["k"], t["v"], t["g"], t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"], lengths=lengths)
        return {"y": y, "last": last, **d}

    clean = run()
    if where in ("h0", "dlast"):
        t[where][1] = bad
    else:
        t[where][1, 149] = bad  # the row's last token
    got = run()
    assert ss.device_status() == ss.SS_OK
    for name, v in got.items():
        if name not in ("last", "dh0"):
            for b, n in enumerate(lengths.tolist()):
                assert not v[b, n:].any(), (name, b)  # (NaN counts as any)
        for b in (0, 2):
            assert torch.equal(v[b], clean[name][b]), (name, b)
    assert not all(torch.isfinite(v).all() for v in got.values())


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_an_empty_row_keeps_a_state_that_is_not_finite(io):
    x = ref.la_inputs(2, 130, 2, 1, 64, 64, h0=True, seed=32)
    t = {n: torch.from_numpy(v).to("cuda", IO[io] if n in ("q", "k", "v", "dy") else torch.float32) for n, v in x.items()}
    t["h0"][0, 0, 3, 5] = np.inf
    y, last = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], h0=t["h0"],
                           lengths=torch.tensor([0, 130], dtype=torch.int32, device="cuda"))
    assert not y[0].any() and torch.isfinite(y[1]).all()
