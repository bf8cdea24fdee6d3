"""What the gated group norm refuses, through Python."""

import pytest
import torch

import mamba_selective_scan_fwd_gb300 as ss

pytestmark = pytest.mark.gpu


def test_groups_beyond_8192_channels():
    x = torch.zeros(2, 2 * 8200, device="cuda")
    for groups in (1, 2):
        with pytest.raises(ss.SSError, match="unsupported"):
            ss.ss_gnorm_fwd(x, groups=groups)
        with pytest.raises(ss.SSError, match="unsupported"):
            ss.ss_gnorm_bwd(x, None, None, x, groups=groups)


@pytest.mark.parametrize("shape", [(2, 0), ()])
def test_no_channels(shape):
    x = torch.zeros(shape, device="cuda")
    with pytest.raises(ValueError, match="groups"):
        ss.ss_gnorm_fwd(x)
    with pytest.raises(ValueError, match="groups"):
        ss.ss_gnorm_bwd(x, None, None, x)


def test_negative_epsilon():
    x = torch.zeros(2, 8, device="cuda")
    with pytest.raises(ss.SSError, match="invalid"):
        ss.ss_gnorm_fwd(x, eps=-1.0)
    with pytest.raises(ss.SSError, match="invalid"):
        ss.ss_gnorm_bwd(x, None, None, x, eps=-1.0)
