"""Linear attention and gated group norm: checks that need no GPU.  The references agree with
central differences of their own forward, the descriptors match the header, and bad arguments
are refused before the first CUDA call."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

import la_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from mamba_selective_scan_fwd_gb300 import linear_attention as la

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


@pytest.mark.parametrize("per_head", [False, True])
def test_la_reference_gradient_matches_differences(per_head):
    x = ref.la_inputs(2, 9, 4, 2, 5, 3, per_head=per_head, h0=True, seed=1)
    lengths = np.array([9, 4])

    def loss(x):
        y, S = ref.la_fwd(x["q"], x["k"], x["v"], x["g"], 0.7, x["h0"], lengths)
        return np.sum(y * x["dy"]) + np.sum(S * x["dlast"])

    got = ref.la_bwd(x["q"], x["k"], x["v"], x["g"], x["dy"], 0.7, x["h0"], x["dlast"], lengths)
    rng = np.random.default_rng(2)
    for key in ("q", "k", "v", "g", "h0"):
        want, d = _difference(loss, x, key, rng)
        # central differences of a smooth function at 1e-6: truncation 1e-12, cancellation 2^-53 / 1e-6 of the loss
        assert abs(np.sum(got["d" + key] * d) - want) <= 1e-7 * max(1.0, abs(loss(x))), key


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("mode", ["gate", "act", "gate_first"])
def test_gnorm_reference_gradient_matches_differences(mode, center):
    rng = np.random.default_rng(3)
    x = {"x": rng.normal(size=(5, 12)), "z": rng.normal(size=(5, 12)), "weight": rng.normal(size=12),
         "bias": rng.normal(size=12), "dout": rng.normal(size=(5, 12))}
    first = mode == "gate_first"

    def z(x):
        return None if mode == "act" else x["z"]

    def loss(x):
        return np.sum(x["dout"] * ref.gnorm_fwd(x["x"], x["weight"], x["bias"], z(x), 3, 1e-5, center, first))

    got = ref.gnorm_bwd(x["x"], x["weight"], x["bias"], x["dout"], z(x), 3, 1e-5, center, first)
    for key in ("x", "weight", "bias") + (() if mode == "act" else ("z",)):
        want, d = _difference(loss, x, key, rng)
        assert abs(np.sum(got["d" + key] * d) - want) <= 1e-6 * max(1.0, abs(loss(x))), key


def test_descriptor_layouts_match_the_header(tmp_path):
    structs = [("ss_la_fwd_desc", la.LaFwdDesc), ("ss_la_bwd_desc", la.LaBwdDesc), ("ss_la_step_desc", la.LaStepDesc)]
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "ss_la.h"', "int main(void) {"]
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
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in out] == want


def _fwd(**kw):
    d = la.LaFwdDesc()
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, y=FAKE, workspace=FAKE, workspace_bytes=1 << 40, q_token=16, q_batch=256,
             k_token=16, k_batch=256, v_token=32, v_batch=512, Bsz=2, L=16, H=4, G=2, N=8, P=8, scale=1.0, dtype=2)
    a.update(kw)
    for key, v in a.items():
        setattr(d, key, v)
    return ss.lib().ss_la_fwd(ctypes.byref(d), None)


@pytest.mark.parametrize("kw,code", [
    (dict(Bsz=-1), INVALID), (dict(L=-1), INVALID), (dict(H=0), INVALID), (dict(G=0), INVALID), (dict(G=3), INVALID),
    (dict(N=0), INVALID), (dict(P=0), INVALID), (dict(N=129), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(P=1 << 17), UNSUPPORTED), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(g=None), INVALID), (dict(y=None), INVALID), (dict(y=FAKE + 8), UNSUPPORTED), (dict(h0=FAKE + 4), UNSUPPORTED),
    (dict(q_token=-16), INVALID), (dict(v_batch=-1), INVALID),
    (dict(Bsz=1, L=1 << 17, workspace_bytes=0), WS_SMALL), (dict(Bsz=1, L=1 << 17, workspace=None), WS_SMALL),
])
def test_la_fwd_rejects(kw, code):
    assert _fwd(**kw) == code


def _bwd(**kw):
    d = la.LaBwdDesc()
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, dy=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE, workspace=FAKE,
             workspace_bytes=1 << 40, q_token=16, q_batch=256, k_token=16, k_batch=256, v_token=32, v_batch=512,
             dy_token=32, dy_batch=512, Bsz=2, L=16, H=4, G=2, N=8, P=8, scale=1.0, dtype=2)
    a.update(kw)
    for key, v in a.items():
        setattr(d, key, v)
    return ss.lib().ss_la_bwd(ctypes.byref(d), None)


@pytest.mark.parametrize("kw,code", [
    (dict(L=-1), INVALID), (dict(G=3), INVALID), (dict(N=129), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED),
    (dict(h0=FAKE), INVALID), (dict(dh0=FAKE), INVALID), (dict(dy=None), INVALID), (dict(dq=None), INVALID),
    (dict(dk=None), INVALID), (dict(dv=None), INVALID), (dict(dg=None), INVALID), (dict(dv=FAKE + 2), UNSUPPORTED),
    (dict(dlast_state=FAKE + 4), UNSUPPORTED), (dict(dy_token=-1), INVALID), (dict(workspace=None), WS_SMALL),
    (dict(workspace_bytes=64), WS_SMALL), (dict(L=0, g_per_head=1, dg=None), INVALID),
])
def test_la_bwd_rejects(kw, code):
    assert _bwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(N=129), UNSUPPORTED), (dict(G=3), INVALID), (dict(pool=-1), INVALID), (dict(pool=1), INVALID),
    (dict(state=None), INVALID), (dict(state=FAKE + 8), UNSUPPORTED), (dict(q=None), INVALID), (dict(y=None), INVALID),
    (dict(v_batch=-8), INVALID), (dict(dtype=5), UNSUPPORTED), (dict(Bsz=0), OK),
])
def test_la_step_rejects(kw, code):
    d = la.LaStepDesc()
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, state=FAKE, y=FAKE, q_batch=16, k_batch=16, v_batch=32, Bsz=2, H=4, G=2,
             N=8, P=8, pool=2, scale=1.0, dtype=2)
    a.update(kw)
    for key, v in a.items():
        setattr(d, key, v)
    assert ss.lib().ss_la_step(ctypes.byref(d), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(groups=0), INVALID), (dict(groups=5), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(flags=4), INVALID), (dict(flags=2, z=None), INVALID), (dict(dtype=3), UNSUPPORTED),
    (dict(C=16400, groups=1), UNSUPPORTED), (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(M=0), OK),
])
def test_gnorm_fwd_rejects(kw, code):
    a = dict(x=FAKE, weight=None, bias=None, z=FAKE, out=FAKE, M=4, C=64, groups=4, eps=1e-5, flags=1, dtype=0)
    a.update(kw)
    assert ss.lib().ss_gnorm_fwd(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dz=None), INVALID), (dict(z=None), INVALID), (dict(dweight=None), INVALID), (dict(weight=None), INVALID),
    (dict(dbias=FAKE), INVALID), (dict(dout=None), INVALID), (dict(dx=None), INVALID), (dict(ws=None), WS_SMALL),
    (dict(wsb=16), WS_SMALL), (dict(ws=FAKE + 4), UNSUPPORTED), (dict(groups=3), INVALID),
])
def test_gnorm_bwd_rejects(kw, code):
    a = dict(x=FAKE, weight=FAKE, bias=None, z=FAKE, dout=FAKE, dx=FAKE, dz=FAKE, dweight=FAKE, dbias=None, M=4, C=64,
             groups=4, eps=1e-5, flags=1, dtype=0, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    assert ss.lib().ss_gnorm_bwd(*a.values(), None) == code


def test_binding_refuses_malformed_tensors():
    import torch

    q, v, g = torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 4, 8), torch.zeros(1, 4, 4)
    with pytest.raises(ValueError, match="share"):
        ss.ss_la_fwd(torch.zeros(1, 4, 3, 8), torch.zeros(1, 4, 3, 8), v, g)
    with pytest.raises(ValueError, match="shape"):
        ss.ss_la_fwd(q, q[:, :3], v, g)
    with pytest.raises(TypeError, match="dtype"):
        ss.ss_la_fwd(q, q.half(), v, g)
    with pytest.raises(ValueError, match="contiguous"):
        ss.ss_la_fwd(q, torch.zeros(1, 4, 8, 2).transpose(2, 3), v, g)
    with pytest.raises(TypeError, match="lengths"):
        ss.ss_la_fwd(q, q, v, g, lengths=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        ss.ss_la_fwd(q, q, v, g)
    with pytest.raises(ValueError, match="CUDA"):
        ss.ss_la_bwd(q, q, v, g, v)
    with pytest.raises(ValueError, match="states for"):
        ss.ss_la_step(q[:, 0], q[:, 0], v[:, 0], g[:, 0], torch.zeros(0, 4, 8, 8))
    with pytest.raises(ValueError, match="groups"):
        ss.ss_gnorm_fwd(torch.zeros(2, 10), groups=3)
    with pytest.raises(ValueError, match="gate"):
        ss.ss_gnorm_fwd(torch.zeros(2, 10), groups=2, gate_first=True)
    with pytest.raises(ValueError, match="CUDA"):
        ss.ss_gnorm_fwd(torch.zeros(2, 10), groups=2)


def test_workspaces_are_pure_and_bounded():
    # nothing to keep when the heads fill the GPU; segment states when one sequence is cut in time
    assert ss.la_fwd_workspace_bytes(64, 4096, 80, 1, 128, 64, ss.SS_F32) == 0
    one = ss.la_fwd_workspace_bytes(1, 131072, 16, 16, 64, 64, ss.SS_F32)
    assert one == ss.la_fwd_workspace_bytes(1, 131072, 16, 16, 64, 64, ss.SS_F32) > 0
    assert ss.la_fwd_workspace_bytes(1, 0, 16, 16, 64, 64, ss.SS_F32) == 0
    assert ss.la_fwd_workspace_bytes(1, 16, 16, 3, 64, 64, ss.SS_F32) == 0
    # the backward keeps two states per chunk of at least 64 tokens
    n = ss.la_bwd_workspace_bytes(1, 640, 4, 4, 64, 64, ss.SS_F32)
    assert n >= 2 * 4 * 5 * 64 * 64 * 4
