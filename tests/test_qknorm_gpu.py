"""GPU parity of the per-head norm of q and k with rotation, both directions, with the 64-bit
reference on the same values.

Tolerances (normwise).  f32: the sum of N <= 256 squares by lanes (2^-21), rsqrt (2^-22), the
angle's cosine (2^-23), two products: 1e-6.  dx = r (d - n m) is a difference, and at N = 1 with a small
eps of equal numbers: its roundings go with |r d|, not with dx, so 1e-5 of the larger of the two.
16-bit outputs: half a step of their own rounding beside it, u = 2^-8 or 2^-11 (1.01 u: the f32 part).
Weights' gradients are f32 sums of up to some thousand terms of both signs: 1e-5."""

import numpy as np
import pytest
import torch

import gdr_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from gpu_util import normwise

pytestmark = pytest.mark.gpu

IO = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def inputs(B, L, Hq, Hk, N, pairs, weight, io, seed=0, far=0):
    rng = np.random.default_rng(seed)

    def t(*shape):
        return torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(IO[io]).cuda()

    x = {"q": t(B, L, Hq, N), "k": t(B, L, Hk, N), "dq": t(B, L, Hq, N), "dk": t(B, L, Hk, N)}
    x["qw"], x["kw"] = (torch.from_numpy(1 + 0.2 * rng.normal(size=N).astype(np.float32)).cuda() if weight else None for _ in "qk")
    x["positions"] = x["freqs"] = None
    if pairs:
        x["positions"] = torch.from_numpy(far + rng.integers(0, 1000, size=(B, L))).to(torch.int32).cuda()
        x["freqs"] = torch.from_numpy(np.exp(-np.arange(pairs) * 9.2 / pairs).astype(np.float32)).cuda()
    return x


def check(x, io, l2=False, interleaved=False, eps=1e-6):
    kw = dict(q_weight=x["qw"], k_weight=x["kw"], positions=x["positions"], freqs=x["freqs"], l2=l2, eps=eps, interleaved=interleaved)
    out = ss.ss_qknorm_fwd(x["q"], x["k"], **kw)
    d = ss.ss_qknorm_bwd(x["q"], x["k"], x["dq"], x["dk"], **kw)
    r = {k: None if v is None else v.double().cpu().numpy() for k, v in x.items()}
    for i, (n, w, dn, dw) in enumerate((("q", "qw", "dq", "dq_weight"), ("k", "kw", "dk", "dk_weight"))):
        want = ref.norm_fwd(r[n], r[w], r["positions"], r["freqs"], l2, eps, interleaved)
        assert normwise(out[i], want) <= 1e-6 + 1.01 * U[io]
        dx, dweight = ref.norm_bwd(r[n], r[w], r[dn], r["positions"], r["freqs"], l2, eps, interleaved)
        off = np.abs(d[dn].double().cpu().numpy() - dx).max()
        rd = np.abs(ref._rstd(r[n], l2, eps) * np.abs(r[dn]) * (1 if r[w] is None else np.abs(r[w]))).max()
        assert off <= 1e-5 * max(rd, np.abs(dx).max()) + 1.01 * U[io] * np.abs(dx).max()
        if dweight is None:
            assert d[dw] is None
        else:
            assert normwise(d[dw], dweight) <= 1e-5
    return out, d


# (B, L, Hq, Hk, N, pairs)
SHAPES = [(1, 1, 1, 1, 128, 64), (2, 3, 4, 2, 64, 16), (2, 37, 16, 16, 128, 32), (1, 5, 3, 1, 80, 20), (1, 9, 2, 2, 80, 40),
          (2, 7, 4, 1, 256, 128), (1, 130, 1, 1, 32, 0), (1, 4, 3, 2, 33, 16), (1, 3, 2, 1, 7, 2), (1, 2, 1, 1, 1, 0),
          (1, 6, 2, 2, 250, 125), (3, 700, 8, 2, 64, 32), (1, 11, 2, 1, 192, 48), (2, 8, 2, 1, 16, 8)]


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_parity(shape, interleaved, io):
    l2 = shape[1] % 2 == 0
    check(inputs(*shape, weight=shape[2] != 3, io=io, seed=shape[1]), io, l2=l2, interleaved=interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_keep_their_angle(interleaved):
    """At two thousand million tokens a product in 32 bits would be off by a hundred radians."""
    check(inputs(1, 50, 2, 1, 64, 32, True, "f32", far=2_000_000_000), "f32", interleaved=interleaved)
    check(inputs(1, 50, 2, 1, 64, 32, True, "f32", far=-5_000), "f32", interleaved=interleaved)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_slices_offsets_and_in_place(io):
    B, L, Hq, Hk, N = 2, 21, 4, 2, 64
    x = inputs(B, L, Hq, Hk, N, 32, True, io)
    (q, k), d = check(x, io)
    kw = dict(q_weight=x["qw"], k_weight=x["kw"], positions=x["positions"], freqs=x["freqs"])
    for pad in (0, 8, 4, 1):
        wide = torch.zeros(B, L + 2, (Hq + Hk) * N + pad, dtype=IO[io], device="cuda")[:, :L]
        qs, ks = wide[:, :, pad:pad + Hq * N].unflatten(2, (Hq, N)), wide[:, :, pad + Hq * N:].unflatten(2, (Hk, N))
        qs.copy_(x["q"])
        ks.copy_(x["k"])
        q2, k2 = ss.ss_qknorm_fwd(qs, ks, **kw)
        d2 = ss.ss_qknorm_bwd(qs, ks, x["dq"], x["dk"], **kw)
        # (a row's sum runs over other lanes where runs are narrower)
        for a, b in ((q2, q), (k2, k), (d2["dq"], d["dq"]), (d2["dk_weight"], d["dk_weight"])):
            assert normwise(a, b.double().cpu().numpy()) <= 2e-5 + 2.02 * U[io] * (a.dtype != torch.float32)
    qi, ki = x["q"].clone(), x["k"].clone()
    ss.ss_qknorm_fwd(qi, ki, **kw, q_out=qi, k_out=ki)
    assert torch.equal(qi, q) and torch.equal(ki, k)


def test_default_positions_count_from_zero():
    x = inputs(2, 40, 2, 1, 64, 32, False, "f32")
    x["positions"] = torch.arange(40, dtype=torch.int32, device="cuda").repeat(2, 1)
    want, _ = check(x, "f32")
    got = ss.ss_qknorm_fwd(x["q"], x["k"], freqs=x["freqs"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_tokens_and_zero_rows():
    x = inputs(2, 0, 2, 1, 64, 32, True, "bf16")
    q, _ = ss.ss_qknorm_fwd(x["q"], x["k"], x["qw"], x["kw"])
    d = ss.ss_qknorm_bwd(x["q"], x["k"], x["dq"], x["dk"], x["qw"], x["kw"])
    assert q.numel() == 0 and not d["dq_weight"].any() and not d["dk_weight"].any()
    x = inputs(1, 4, 2, 1, 64, 32, True, "f32")
    x["q"].zero_()
    check(x, "f32", l2=True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_graph_stream_and_repeats(io):
    x = inputs(2, 300, 8, 4, 128, 64, True, io)
    kw = dict(q_weight=x["qw"], k_weight=x["kw"], positions=x["positions"], freqs=x["freqs"])
    out, d = check(x, io)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2 = ss.ss_qknorm_fwd(x["q"], x["k"], **kw, stream=side)
    d2 = ss.ss_qknorm_bwd(x["q"], x["k"], x["dq"], x["dk"], **kw, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out3 = ss.ss_qknorm_fwd(x["q"], x["k"], **kw)
        d3 = ss.ss_qknorm_bwd(x["q"], x["k"], x["dq"], x["dk"], **kw)
    graph.replay()
    torch.cuda.synchronize()
    for o, e in ((out2, d2), (out3, d3)):
        assert all(torch.equal(a, b) for a, b in zip(o, out)) and all(torch.equal(e[n], d[n]) for n in d)


# one head of 64 channels: 32 tokens a tile, 64 rows at once, so that slots without a row go through every tile; 60011
# tokens: three tiles a block, all three tables.  700 rows of 7 tokens: tiles over several rows' ends, without positions
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 60011, 1, 1, 64, 32), (700, 7, 1, 2, 64, 16), (3, 5000, 1, 3, 32, 16), (900, 1, 4, 1, 80, 40)], ids=str)
def test_many_tiles_a_block(shape, io):
    x = inputs(*shape, weight=True, io=io, seed=5)
    check(x, io)
    B, L = shape[:2]
    x["positions"] = torch.arange(L, dtype=torch.int32, device="cuda").repeat(B, 1)
    (q, k), _ = check(x, io)
    got = ss.ss_qknorm_fwd(x["q"], x["k"], x["qw"], x["kw"], freqs=x["freqs"])
    assert torch.equal(got[0], q) and torch.equal(got[1], k)


def test_in_place_over_many_tiles():
    """Rows are read a tile ahead of the writes."""
    x = inputs(2, 9000, 3, 2, 128, 32, True, "bf16", seed=6)
    kw = dict(q_weight=x["qw"], k_weight=x["kw"], positions=x["positions"], freqs=x["freqs"])
    q, k = ss.ss_qknorm_fwd(x["q"], x["k"], **kw)
    ss.ss_qknorm_fwd(x["q"], x["k"], **kw, q_out=x["q"], k_out=x["k"])
    assert torch.equal(x["q"], q) and torch.equal(x["k"], k)
