"""Linear attention under positive log decays, resets and decays of mixed sign in every io type: finite and
within the bounds of test_la_gpu wherever the exact result is representable.

The 16-bit bounds there rest on relative roundings of each operand, which positive decays change nothing about:
the sums are dominated by other terms, not by more of them.  f32: the exponents of a chunk reach 128 x 0.05 x 1.44
= 9.2 and carry two-float precision, so the exponential's own 2^-22 stays the largest part."""

import numpy as np
import pytest

import la_reference as ref
from test_la_gpu import check_bwd, check_fwd

pytestmark = pytest.mark.gpu

# scale: keeps y and the gradients below f16's 65504 (states grow to e^7 here)
SCALE = 0.05


def grown(kind, L, H=2, N=64, seed=0, **kw):
    """Inputs whose g is constant and positive, per token or per head, or changes sign from chunk to chunk or
    from token to token."""
    x = ref.la_inputs(1, L, H, 1, N, 64, per_head=kind == "head", seed=seed, **kw)
    r = np.random.default_rng(seed + 1)
    t = np.arange(L)
    x["g"][:] = {"0.02": 0.02, "0.05": 0.05, "head": 0.03,
                 "chunks": np.where(t // 128 % 2 == 0, 0.04, -0.04)[None, :, None],
                 "tokens": r.normal(scale=0.3, size=(1, L, 1))}[kind]
    return x


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind,L,N", [("0.02", 300, 64), ("0.05", 140, 64), ("0.05", 128, 128), ("head", 200, 16), ("tokens", 140, 64),
                                      ("chunks", 500, 128), ("chunks", 3300, 16)])
def test_positive_decays(kind, L, N, io):
    x = grown(kind, L, N=N, h0=True, seed=L)
    check_fwd(x, io, scale=SCALE)
    check_bwd(x, io, scale=SCALE)


def test_resets_and_extreme_decays_in_f16():
    x = ref.la_inputs(1, 260, 3, 1, 32, 32, h0=True, seed=7)
    x["g"][0, [3, 100, 101, 200], 0] = -np.inf
    x["g"][0, [0, 127, 128], 1] = np.finfo(np.float32).min
    x["g"][0, 60, 1] = -1000.0
    x["g"][0, :, 2] = 0.0
    check_fwd(x, "f16")
    check_bwd(x, "f16")


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_every_other_token_resets(io):
    """Sequences of two tokens packed into one row: a run of 32 tokens holds 16 resets."""
    x = ref.la_inputs(1, 200, 2, 1, 64, 64, h0=True, seed=9)
    x["g"][0, ::2, :] = -np.inf
    check_fwd(x, io)
    check_bwd(x, io)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [64, 128])
def test_growth_near_the_documented_limit(N, io):
    """128 tokens that add up to 57, of 60 that a chunk takes; the scale brings e^57 back into f16's range."""
    x = ref.la_inputs(1, 128, 2, 1, N, 64, seed=61)
    x["g"][:] = 0.45
    check_fwd(x, io, scale=1e-24)
    check_bwd(x, io, scale=1e-24)
