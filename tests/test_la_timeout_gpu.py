"""A wait of a tensor-core block that runs out after the block's other parts are over (a barrier nothing completes,
1 ms) reaches the status word, and the context and its tensor memory stay usable."""

import pytest
import torch

import la_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from test_la_gpu import check_bwd, check_fwd

pytestmark = pytest.mark.gpu


def test_late_timeout_is_reported_and_context_survives():
    assert ss.device_status() == ss.SS_OK
    for limit in (1_000_000, 0):
        ss.la_selftest_wait_timeout(limit)
        assert ss.device_status() == ss.SS_ERR_DEVICE_TIMEOUT
        assert ss.device_status() == ss.SS_OK  # the read cleared it
    # (two of the forward's blocks take all of an SM's tensor memory, one of the backward's)
    x = ref.la_inputs(1, 300, 8, 2, 64, 64, h0=True, seed=41)
    check_fwd(x, "bf16")
    check_bwd(x, "bf16")
    torch.cuda.synchronize()
