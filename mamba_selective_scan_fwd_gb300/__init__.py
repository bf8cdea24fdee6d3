"""GB300 (sm_103a) Mamba-1 selective scan, forward and backward; linear attention with one
decay per head and the gated group norm of its output (``linear_attention``); the gated delta
rule and the norm with rotation of its queries and keys (``delta_rule``).

The compute lives in ``libss.so`` (CUDA kernels behind the C ABI of ``include/ss.h``,
``include/ss_la.h`` and ``include/ss_gdr.h``); ``binding`` marshals torch CUDA tensors into it.  The
library is loaded on first use and every entry point raises if it is
missing -- there is no other implementation to fall back on.
"""

from .binding import (SS_BF16, SS_ERR_DEVICE_TIMEOUT, SS_F16, SS_F32, SS_OK, SSError, bwd_saved_workspace_bytes,
                      bwd_workspace_bytes, device_status, fwd_workspace_bytes, lib, plan_info, saved_bytes,
                      selftest_wait_timeout, set_copies_only, ss_bwd, ss_bwd_ex, ss_bwd_saved, ss_decode_step, ss_fwd,
                      ss_fwd_ex, ss_fwd_noalloc, ss_fwd_save, staging_uses_tma, status_string)
from .delta_rule import (gdr_bwd_workspace_bytes, gdr_fwd_workspace_bytes, ss_gdr_bwd, ss_gdr_fwd, ss_gdr_step,
                         ss_qknorm_bwd, ss_qknorm_fwd)
from .linear_attention import (la_bwd_workspace_bytes, la_fwd_workspace_bytes, la_selftest_wait_timeout, ss_gnorm_bwd,
                               ss_gnorm_fwd, ss_la_bwd, ss_la_fwd, ss_la_step)

__all__ = ["ss_fwd", "ss_fwd_save", "ss_fwd_ex", "ss_fwd_noalloc", "ss_bwd", "ss_bwd_saved", "ss_bwd_ex",
           "ss_decode_step",
           "fwd_workspace_bytes", "bwd_workspace_bytes", "saved_bytes", "bwd_saved_workspace_bytes", "status_string",
           "plan_info", "lib", "SSError", "SS_F32", "SS_F16", "SS_BF16", "SS_OK", "SS_ERR_DEVICE_TIMEOUT",
           "ss_la_fwd", "ss_la_bwd", "ss_la_step", "ss_gnorm_fwd", "ss_gnorm_bwd", "la_fwd_workspace_bytes",
           "la_bwd_workspace_bytes", "la_selftest_wait_timeout",
           "ss_gdr_fwd", "ss_gdr_bwd", "ss_gdr_step", "ss_qknorm_fwd", "ss_qknorm_bwd", "gdr_fwd_workspace_bytes",
           "gdr_bwd_workspace_bytes",
           "device_status", "selftest_wait_timeout", "set_copies_only", "staging_uses_tma"]
