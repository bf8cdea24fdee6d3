"""The limits of the linear attention's own wait test are checked before the first CUDA call."""

import mamba_selective_scan_fwd_gb300 as ss

INVALID = 1


def test_wait_limit_checked_before_any_launch():
    assert ss.lib().ss_la_selftest_wait_timeout(-1, None) == INVALID
    assert ss.lib().ss_la_selftest_wait_timeout(2_000_000_001, None) == INVALID
