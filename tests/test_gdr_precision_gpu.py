"""The gated delta rule's precision: 16-bit outputs are the exact values rounded once, f32 outputs good to 10^-6 of their norm.

Operands that the tensor cores take are f16 in two parts: 22 bits, 2^-23 of a value at most.
* 16-bit outputs, each element: half a step of its own, and beside it what the operands' roundings leave.  A y passes some
  seven of them (S, X, M, U, P and the two products that leave out low times low) and sums of f32; the correction's
  inverse doubles them at these inputs (unit keys in 64 and more dimensions, rates below one): 2 (7 + 2) 2^-23 = 2.1e-6 of
  the largest y, 2^-18 allowed.  Gradients join two such chains: 2^-17.  (One part, 11 bits, is 2^-12: 2e-4.)
* f32 outputs, norm of the error over the norm: roundings of 2^-24.8 root mean square, twenty of them in quadrature (dg
  and dbeta join two walks), doubled as above: 3e-7; the products' f32 sums, cut after each 16 terms: up to twenty-four
  of 2^-24 one way, 1.4e-6 if all fell on every value alike, half of which stays for steps of both signs: 1e-6 in all.
  (16 bits' two parts, 2^-17, would be 4e-6; scales from bounds that are 2^10 high, 2e-6.)  f32 io: 2^-24 each, the same bound.
"""

import numpy as np
import pytest
import torch

import gdr_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from test_gdr_gpu import lengths_on_gpu, on_gpu

pytestmark = pytest.mark.gpu

BITS = {"bf16": 8, "f16": 11}


def beyond_half_a_step(got, want, io):
    """By how much the worst element is off beyond half a step of its type, over the largest value."""
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    e = np.floor(np.log2(np.where(want == 0, 1.0, np.abs(want))))
    if io == "f16":
        e = np.maximum(e, -14)
    half = np.where(want == 0, 0.0, 2.0 ** (e - BITS[io]))
    return (np.abs(got - want) - half).max() / np.abs(want).max()


def off(got, want):
    return np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)


# (Bsz, L, H, G, N, P): whole tiles, heads that share keys, several value tiles, odd multiples of eight, cut in time
SHAPES = [(2, 300, 4, 2, 128, 128), (1, 200, 2, 2, 64, 200), (3, 130, 6, 2, 72, 40), (1, 3001, 2, 1, 64, 64)]


def run(shape, io, lengths=None):
    x = ref.gdr_inputs(*shape, seed=71)
    t, r = on_gpu(x, io)
    args, rargs = ([z[n] for n in ("q", "k", "v", "g", "beta")] for z in (t, r))
    n = lengths_on_gpu(lengths)
    y, last = ss.ss_gdr_fwd(*args, scale=0.5, h0=t["h0"], lengths=n)
    got = ss.ss_gdr_bwd(*args, t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"], lengths=n)
    got.update(y=y, last=last)
    want = ref.gdr_bwd(*rargs, r["dy"], 0.5, r["h0"], r["dlast"], lengths)
    want["y"], want["last"] = ref.gdr_fwd(*rargs, 0.5, r["h0"], lengths)
    assert ss.device_status() == ss.SS_OK
    return got, want


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("lengths", [None, "ragged"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_y_is_rounded_once(shape, lengths, io):
    B, L = shape[:2]
    got, want = run(shape, io, lengths and [(2 * L // 3, 0, L)[i % 3] for i in range(B)])
    assert beyond_half_a_step(got["y"], want["y"], io) <= 2.0 ** -18


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("lengths", [None, "ragged"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients_are_rounded_once(shape, lengths, io):
    B, L = shape[:2]
    got, want = run(shape, io, lengths and [(2 * L // 3, 0, L)[i % 3] for i in range(B)])
    bad = {n: e for n in ("dq", "dk", "dv") if not (e := beyond_half_a_step(got[n], want[n], io)) <= 2.0 ** -17}
    assert not bad, bad


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_states_and_gradients_in_32_bits(shape, io):
    got, want = run(shape, io)
    names = ("last", "dh0", "dg", "dbeta") + (("y", "dq", "dk", "dv") if io == "f32" else ())
    bad = {n: e for n in names if not (e := off(got[n], want[n])) <= 1e-6}
    assert not bad, bad


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_states_and_gradients_in_32_bits_of_ragged_rows(io):
    got, want = run((4, 200, 4, 2, 64, 64), io, [200, 0, 77, 129])
    bad = {n: e for n in ("last", "dh0", "dg", "dbeta") if not (e := off(got[n], want[n])) <= 1e-6}
    assert not bad, bad
