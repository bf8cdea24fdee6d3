"""Gated delta rule and q / k norm: checks that need no GPU.  The references agree with central
differences of their own forward, the descriptors match the header, and bad arguments are refused
before the first CUDA call."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

import gdr_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from mamba_selective_scan_fwd_gb300 import delta_rule as dr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call here fails validation first


def _difference(loss, x, key, rng):
    """(<gradient, direction> by central differences, the direction) of loss(x) along a random direction of x[key]."""
    d = rng.normal(size=x[key].shape)
    eps = 1e-6
    hi, lo = dict(x), dict(x)
    hi[key], lo[key] = x[key] + eps * d, x[key] - eps * d
    return (loss(hi) - loss(lo)) / (2 * eps), d


@pytest.mark.parametrize("gate", [False, True])
def test_gdr_reference_gradient_matches_differences(gate):
    x = ref.gdr_inputs(2, 9, 4, 2, 5, 3, gate=gate, seed=1)
    x = {k: None if v is None else v.astype(np.float64) for k, v in x.items()}
    lengths = np.array([9, 4])

    def loss(x):
        y, S = ref.gdr_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.7, x["h0"], lengths)
        return np.sum(y * x["dy"]) + np.sum(S * x["dlast"])

    got = ref.gdr_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["dy"], 0.7, x["h0"], x["dlast"], lengths)
    rng = np.random.default_rng(2)
    for key in ("q", "k", "v", "beta", "h0") + (("g",) if gate else ()):
        want, d = _difference(loss, x, key, rng)
        # central differences of a smooth function at 1e-6: truncation 1e-12, cancellation 2^-53 / 1e-6 of the loss
        assert abs(np.sum(got["d" + key] * d) - want) <= 1e-7 * max(1.0, abs(loss(x))), key


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("l2", [False, True])
def test_norm_reference_gradient_matches_differences(l2, interleaved):
    rng = np.random.default_rng(3)
    x = {"x": rng.normal(size=(2, 3, 4, 10)), "weight": rng.normal(size=10), "dout": rng.normal(size=(2, 3, 4, 10))}
    positions, freqs = rng.integers(0, 50, size=(2, 3)), rng.normal(size=3)

    def loss(x):
        return np.sum(x["dout"] * ref.norm_fwd(x["x"], x["weight"], positions, freqs, l2, 1e-6, interleaved))

    got = dict(zip(("x", "weight"), ref.norm_bwd(x["x"], x["weight"], x["dout"], positions, freqs, l2, 1e-6, interleaved)))
    for key in ("x", "weight"):
        want, d = _difference(loss, x, key, rng)
        assert abs(np.sum(got[key] * d) - want) <= 1e-6 * max(1.0, abs(loss(x))), key


def test_descriptor_layouts_match_the_header(tmp_path):
    structs = [("ss_gdr_fwd_desc", dr.GdrFwdDesc), ("ss_gdr_bwd_desc", dr.GdrBwdDesc), ("ss_gdr_step_desc", dr.GdrStepDesc),
               ("ss_qknorm_fwd_desc", dr.QkNormFwdDesc), ("ss_qknorm_bwd_desc", dr.QkNormBwdDesc)]
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "ss_gdr.h"', "int main(void) {"]
    want = []
    for name, cls in structs:
        src.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            src.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    c = tmp_path / "layout.c"
    c.write_text("\n".join(src + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(c)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == want


def _fwd(**kw):
    d = dr.GdrFwdDesc(**{f: FAKE for f in ("q", "k", "v", "g", "beta", "y", "workspace")}, workspace_bytes=1 << 40, Bsz=2, L=100,
                      H=4, G=2, N=64, P=64, q_token=128, q_batch=12800, k_token=128, k_batch=12800, v_token=256,
                      v_batch=25600, scale=1.0, dtype=ss.SS_F32)
    for k, v in kw.items():
        setattr(d, k, v)
    return ss.lib().ss_gdr_fwd(ctypes.byref(d), None)


@pytest.mark.parametrize("kw,want", [
    (dict(H=3), INVALID), (dict(G=0), INVALID), (dict(Bsz=-1), INVALID), (dict(L=-1), INVALID), (dict(N=0), INVALID),
    (dict(P=0), INVALID), (dict(N=129), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED), (dict(beta=None), INVALID),
    (dict(q=None), INVALID), (dict(y=None), INVALID), (dict(q_token=-1), INVALID), (dict(y=FAKE + 4), UNSUPPORTED),
    (dict(h0=FAKE + 8), UNSUPPORTED), (dict(last_state=FAKE + 8), UNSUPPORTED), (dict(workspace=FAKE + 8), UNSUPPORTED),
    (dict(L=1 << 40), UNSUPPORTED), (dict(Bsz=1 << 20, H=1 << 10), UNSUPPORTED)])
def test_forward_refusals(kw, want):
    assert _fwd(**kw) == want


def _bwd(**kw):
    names = ("q", "k", "v", "g", "beta", "dy", "dq", "dk", "dv", "dg", "dbeta", "workspace")
    d = dr.GdrBwdDesc(**{f: FAKE for f in names}, workspace_bytes=1 << 40, Bsz=2, L=100, H=4, G=2, N=64, P=64, q_token=128,
                      q_batch=12800, k_token=128, k_batch=12800, v_token=256, v_batch=25600, dy_token=256, dy_batch=25600,
                      scale=1.0, dtype=ss.SS_F32)
    for k, v in kw.items():
        setattr(d, k, v)
    return ss.lib().ss_gdr_bwd(ctypes.byref(d), None)


@pytest.mark.parametrize("kw,want", [
    (dict(h0=FAKE), INVALID), (dict(dh0=FAKE), INVALID), (dict(dg=None), INVALID), (dict(g=None), INVALID),
    (dict(dbeta=None), INVALID), (dict(dq=None), INVALID), (dict(dq=FAKE + 4), UNSUPPORTED), (dict(workspace_bytes=16), WS_SMALL),
    (dict(workspace=None), WS_SMALL), (dict(N=200), UNSUPPORTED), (dict(dy_batch=-5), INVALID)])
def test_backward_refusals(kw, want):
    assert _bwd(**kw) == want


def _step(**kw):
    d = dr.GdrStepDesc(**{f: FAKE for f in ("q", "k", "v", "g", "beta", "state", "y")}, q_batch=128, k_batch=128, v_batch=256, Bsz=2,
                       H=4, G=2, N=64, P=64, pool=2, scale=1.0, dtype=ss.SS_BF16)
    for k, v in kw.items():
        setattr(d, k, v)
    return ss.lib().ss_gdr_step(ctypes.byref(d), None)


@pytest.mark.parametrize("kw,want", [
    (dict(pool=1), INVALID), (dict(pool=-1), INVALID), (dict(beta=None), INVALID), (dict(state=FAKE + 4), UNSUPPORTED),
    (dict(N=130), UNSUPPORTED), (dict(v_batch=-1), INVALID), (dict(state=None), INVALID), (dict(Bsz=0), OK)])
def test_step_refusals(kw, want):
    assert _step(**kw) == want


def _norm(back, **kw):
    cls = dr.QkNormBwdDesc if back else dr.QkNormFwdDesc
    names = ("q", "k", "freqs", "dq_out", "dk_out", "dq", "dk", "workspace") if back else ("q", "k", "freqs", "q_out", "k_out")
    d = cls(**{f: FAKE for f in names}, q_token=256, q_batch=25600, k_token=128, k_batch=12800, Bsz=2, L=100, Hq=4, Hk=2, N=64,
            pairs=32, eps=1e-6, dtype=ss.SS_BF16)
    if back:
        d.workspace_bytes = 1 << 40
    for k, v in kw.items():
        setattr(d, k, v)
    return getattr(ss.lib(), "ss_qknorm_bwd" if back else "ss_qknorm_fwd")(ctypes.byref(d), None)


COMMON = [(dict(pairs=33), INVALID), (dict(pairs=-1), INVALID), (dict(freqs=None), INVALID), (dict(N=257), UNSUPPORTED),
          (dict(Hk=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(flags=4), INVALID),
          (dict(dtype=3), UNSUPPORTED), (dict(q=None), INVALID), (dict(q_batch=-1), INVALID)]


@pytest.mark.parametrize("kw,want", COMMON + [(dict(q_out=None), INVALID), (dict(Bsz=0), OK)])
def test_norm_refusals(kw, want):
    assert _norm(False, **kw) == want


@pytest.mark.parametrize("kw,want", COMMON + [(dict(dq=None), INVALID), (dict(q_weight=FAKE), INVALID),
                                              (dict(dk_weight=FAKE), INVALID), (dict(workspace_bytes=8), WS_SMALL),
                                              (dict(workspace=None), WS_SMALL), (dict(workspace=FAKE + 4), UNSUPPORTED)])
def test_norm_backward_refusals(kw, want):
    assert _norm(True, **kw) == want


def test_python_refusals_name_the_argument():
    import torch

    q, k, v = torch.zeros(2, 5, 2, 8), torch.zeros(2, 5, 2, 8), torch.zeros(2, 5, 4, 8)
    g = beta = torch.zeros(2, 5, 4)
    with pytest.raises(ValueError, match="CUDA"):
        ss.ss_gdr_fwd(q, k, v, g, beta)
    with pytest.raises(ValueError, match="beta"):
        ss.ss_gdr_fwd(q, k, v, g, beta[:, :4])
    with pytest.raises(ValueError, match="share"):
        ss.ss_gdr_fwd(q, k, v[:, :, :3], g, beta)
    with pytest.raises(TypeError, match="k: dtype"):
        ss.ss_gdr_fwd(q, k.bfloat16(), v, g, beta)
    with pytest.raises(ValueError, match="dy"):
        ss.ss_gdr_bwd(q, k, v, g, beta, v[:, :4])
    with pytest.raises(ValueError, match="states"):
        ss.ss_gdr_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0].contiguous(), beta[:, 0].contiguous(), torch.zeros(1, 4, 8, 8))
    with pytest.raises(ValueError, match="frequencies"):
        ss.ss_qknorm_fwd(q, k, freqs=torch.zeros(5))
    with pytest.raises(ValueError, match="positions"):
        ss.ss_qknorm_fwd(q, k, positions=torch.zeros(2, 5, dtype=torch.int32))
    with pytest.raises(ValueError, match="last two"):
        ss.ss_qknorm_fwd(torch.zeros(2, 5, 8, 2).transpose(2, 3), k)
    with pytest.raises(ValueError, match="k_weight"):
        ss.ss_qknorm_bwd(q, k, q, k, k_weight=torch.zeros(7))


def test_workspace_sizes():
    assert ss.gdr_bwd_workspace_bytes(0, 100, 4, 2, 64, 64, ss.SS_F32) == 0
    assert ss.gdr_bwd_workspace_bytes(2, 0, 4, 2, 64, 64, ss.SS_F32) == 0
    assert ss.gdr_bwd_workspace_bytes(2, 100, 4, 3, 64, 64, ss.SS_F32) == 0
    assert ss.gdr_bwd_workspace_bytes(2, 100, 4, 2, 64, 64, ss.SS_F32) > 0
