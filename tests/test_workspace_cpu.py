"""A workspace that a caller gives is checked before its address reaches a kernel (no GPU: the check alone)."""

import pytest
import torch

from mamba_selective_scan_fwd_gb300.binding import _workspace

GPU = torch.device("cuda", 0)


def test_memory_of_another_device_is_refused():
    with pytest.raises(ValueError, match="workspace is on cpu, expected cuda:0"):
        _workspace(64, GPU, torch.empty(64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace is on cpu"):
        _workspace(0, GPU, torch.empty(64, dtype=torch.uint8))


def test_memory_with_gaps_is_refused():
    space = torch.empty(128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        _workspace(64, space.device, space[::2])


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float32])
def test_given_and_missing_workspaces(dtype):
    space = torch.empty(32, dtype=dtype)
    assert _workspace(16, space.device, space) == (space, 32 * space.element_size())
    assert _workspace(0, space.device, None) == (None, 0)
    made, size = _workspace(48, space.device, None)
    assert size == 48 == made.numel()
