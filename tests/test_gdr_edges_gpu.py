"""Gated delta rule at the edges of its ranges: sizes of the values, decays that grow, sequences cut in time, values
that are not finite, pools beyond 2^31 elements, workspaces that calls share (tolerances: those of test_gdr_gpu)."""

import numpy as np
import pytest
import torch

import gdr_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from gpu_util import normwise
from test_gdr_gpu import IO, check_bwd, check_fwd, lengths_on_gpu, on_gpu, tol_bwd, tol_fwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io,size", [("bf16", 1e-18), ("bf16", 1e18), ("f32", 1e-12), ("f32", 1e12), ("f16", 1e-3), ("f16", 1e3)])
def test_values_of_any_size(io, size):
    """The rule is linear in v and the start, and q's and dy's sizes only scale what they multiply."""
    x = ref.gdr_inputs(1, 150, 2, 1, 64, 64, seed=21)
    for key in ("v", "h0"):
        x[key] = (x[key] * size).astype(np.float32)
    x["dy"] = (x["dy"] * np.float32(1e-2)).astype(np.float32)
    check_fwd(x, io)
    check_bwd(x, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("big,small", [("v", "dy"), ("dy", "v")])
def test_values_near_the_largest_of_32_bits(io, big, small):
    """What the rule makes of values of 10^36 stays below 3.4 10^38, bounds on it need not.  (The small ones keep their
    products with them in range.)"""
    x = ref.gdr_inputs(1, 200, 2, 1, 128, 128, seed=31)
    for key, size in ((big, 1e36), (small, 1e-6)):
        x[key] = (x[key] * np.float32(size)).astype(np.float32)
        state = {"v": "h0", "dy": "dlast"}[key]
        x[state] = (x[state] * np.float32(size)).astype(np.float32)
    check_fwd(x, io)
    check_bwd(x, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("how", ["decays", "corrections"])
def test_small_states_after_large_ones(io, how):
    """Values fall by 10^5 inside a chunk, and decays of e^-25 or corrections in eight dimensions take the larger
    state out: what is left has to be good by its own size."""
    x = ref.gdr_inputs(3, 128, 2, 1, 8, 64, seed=33)
    x["v"][:, 80:] *= np.float32(1e-5)
    if how == "decays":
        x["g"] = (x["g"] * np.float32(50)).astype(np.float32)
    check_fwd(x, io)
    check_bwd(x, io)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_long_keys_with_small_rates(io):
    """Keys of length 5 and rates that keep beta |k|^2 below one; queries of length 30."""
    x = ref.gdr_inputs(2, 130, 2, 2, 64, 64, seed=22)
    x["k"] *= 5
    x["q"] *= 30
    x["beta"] *= np.float32(0.04)
    check_fwd(x, io)
    check_bwd(x, io)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_decays_that_grow(io):
    """Positive log decays: the state grows by e^3 in 64 tokens."""
    x = ref.gdr_inputs(1, 130, 2, 1, 32, 32, seed=23)
    x["g"] = np.full_like(x["g"], 3 / 64)
    check_fwd(x, io)
    check_bwd(x, io)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_negative_rates_and_zero_rows(io):
    x = ref.gdr_inputs(1, 100, 2, 1, 32, 32, seed=24)
    x["beta"][:, ::3] *= -0.3
    x["k"][:, 10:20] = 0
    x["q"][:, 30:40] = 0
    x["v"][:, 50:60] = 0
    x["dy"][:, 64:] = 0
    check_fwd(x, io)
    check_bwd(x, io)


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 9000, 2, 1, 128, 128), (2, 5001, 1, 1, 64, 200), (1, 4097, 3, 3, 16, 64)], ids=str)
def test_sequences_cut_in_time(shape, io):
    """Few heads and many tokens: the forward walks segments from carried states.  Against the same values at an odd offset,
    which run on the FP32 units: both are within their tolerance of the truth.  One row is padded."""
    B, L, H, G, N, P = shape
    x = ref.gdr_inputs(*shape, seed=L)
    t, _ = on_gpu(x, io)
    lengths = lengths_on_gpu([L - 1500] + [L] * (B - 1))
    y, last = ss.ss_gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], scale=0.5, h0=t["h0"], lengths=lengths)
    odd = torch.empty(B, L, 2 * G * N + H * P + 1, dtype=IO[io], device="cuda")[:, :, 1:]
    q, k, v = odd.split([G * N, G * N, H * P], -1)
    q, k, v = q.unflatten(2, (G, N)), k.unflatten(2, (G, N)), v.unflatten(2, (H, P))
    for to, key in ((q, "q"), (k, "k"), (v, "v")):
        to.copy_(t[key])
    y2, last2 = ss.ss_gdr_fwd(q, k, v, t["g"], t["beta"], scale=0.5, h0=t["h0"], lengths=lengths)
    assert ss.device_status() == ss.SS_OK
    assert normwise(last, last2.double().cpu().numpy()) <= tol_fwd(io, "last") + 1e-5
    assert normwise(y, y2.double().cpu().numpy()) <= 2 * tol_fwd(io, "y")
    assert not y[0, L - 1500:].any()


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_values_that_are_not_finite_stay_in_their_row_and_head(io):
    x = ref.gdr_inputs(3, 150, 4, 2, 64, 64, seed=25)
    t, _ = on_gpu(x, io)
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    y, last = ss.ss_gdr_fwd(*args, scale=0.5, h0=t["h0"])
    d = ss.ss_gdr_bwd(*args, t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"])
    t["v"][1, 70, 2] = float("nan")
    t["v"][1, 80, 2] = float("inf")
    y2, last2 = ss.ss_gdr_fwd(*args, scale=0.5, h0=t["h0"])
    d2 = ss.ss_gdr_bwd(*args, t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"])
    assert torch.isnan(last2[1, 2]).any() and not torch.isfinite(y2[1, 128:, 2]).all()
    assert torch.equal(y2[:, :, [0, 1, 3]], y[:, :, [0, 1, 3]]) and torch.equal(y2[[0, 2]], y[[0, 2]])
    assert torch.equal(y2[1, :64], y[1, :64])  # tokens of earlier 64s
    assert torch.equal(last2[[0, 2]], last[[0, 2]]) and torch.equal(last2[1, [0, 1, 3]], last[1, [0, 1, 3]])
    for n in ("dv", "dbeta", "dg"):
        assert torch.equal(d2[n][[0, 2]], d[n][[0, 2]]) and torch.equal(d2[n][:, :, [0, 1, 3]], d[n][:, :, [0, 1, 3]])
    for n in ("dq", "dk"):
        assert torch.equal(d2[n][[0, 2]], d[n][[0, 2]]) and torch.equal(d2[n][:, :, 0], d[n][:, :, 0])


def test_pool_beyond_two_to_the_31_elements():
    H, N, P = 32, 128, 128
    pool = 2 ** 31 // (H * N * P) + 8
    x = ref.gdr_inputs(3, 1, H, 16, N, P, seed=26)
    t, r = on_gpu(x, "bf16")
    state = torch.zeros(pool, H, N, P, device="cuda")
    slots = torch.tensor([pool - 1, 5, pool - 3], dtype=torch.int32, device="cuda")
    state[slots.long()] = t["h0"]
    args = [t[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")]
    y = ss.ss_gdr_step(*args, state, scale=0.5, slots=slots)
    wy, ws = ref.gdr_step(*[r[n][:, 0] for n in ("q", "k", "v", "g", "beta")], r["h0"], 0.5)
    assert normwise(y, wy) <= 2 * 2.0 ** -8
    assert normwise(state[slots.long()], ws) <= 1e-5
    assert not state[6:pool - 3].any()


def test_without_tma_the_results_stay_within_tolerance():
    x = ref.gdr_inputs(2, 140, 4, 2, 64, 64, seed=27)
    before = ss.set_copies_only(True)
    try:
        check_fwd(x, "bf16")
        check_bwd(x, "bf16")
    finally:
        ss.set_copies_only(before)


def test_a_workspace_serves_calls_and_graphs_in_turn():
    """One workspace for a forward, a backward and two captured graphs of them, replayed one after the other."""
    x = ref.gdr_inputs(2, 200, 4, 2, 64, 64, seed=28)
    t, _ = on_gpu(x, "bf16")
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    need = max(ss.gdr_fwd_workspace_bytes(2, 200, 4, 2, 64, 64, ss.SS_BF16), ss.gdr_bwd_workspace_bytes(2, 200, 4, 2, 64, 64, ss.SS_BF16))
    space = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # (NaN where it would be read unwritten)
    y, last = ss.ss_gdr_fwd(*args, scale=0.5, h0=t["h0"])
    d = ss.ss_gdr_bwd(*args, t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"])
    graphs, outs = [], []
    for back in (False, True):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(ss.ss_gdr_bwd(*args, t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"], workspace=space) if back else
                        ss.ss_gdr_fwd(*args, scale=0.5, h0=t["h0"], workspace=space))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], y) and torch.equal(outs[0][1], last)
    assert all(torch.equal(outs[1][n], d[n]) for n in d)
    with pytest.raises(ss.SSError, match="WORKSPACE"):
        ss.ss_gdr_bwd(*args, t["dy"], h0=t["h0"], dlast_state=t["dlast"], workspace=space[:1024])


def test_given_outputs_are_used_and_checked():
    x = ref.gdr_inputs(1, 40, 2, 1, 16, 16, seed=29)
    t, _ = on_gpu(x, "f32")
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    y, last = torch.empty_like(t["v"]), torch.empty_like(t["h0"])
    y2, last2 = ss.ss_gdr_fwd(*args, y=y, last_state=last)
    assert y2 is y and last2 is last
    assert ss.ss_gdr_fwd(*args, return_last_state=False)[1] is None
    out = {"dq": torch.empty_like(t["q"]), "dbeta": torch.empty_like(t["beta"])}
    d = ss.ss_gdr_bwd(*args, t["dy"], out=out)
    assert d["dq"] is out["dq"] and d["dbeta"] is out["dbeta"] and d["dh0"] is None
    with pytest.raises(ValueError, match="dk"):
        ss.ss_gdr_bwd(*args, t["dy"], out={"dk": torch.empty(1, 40, 1, 8, device="cuda")})


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(70, 140, 4, 2, 64, 64), (30, 200, 6, 2, 128, 136)], ids=str)
def test_many_ragged_rows(shape, io):
    """More chunks than the chunk kernel has blocks, so that each takes several, some of them without a token."""
    B, L = shape[:2]
    lengths = [(0, L, 1, 64, 65, 128, 129, 17)[i % 8] for i in range(B)]
    x = ref.gdr_inputs(*shape, seed=41)
    check_fwd(x, io, lengths=lengths)
    got = check_bwd(x, io, lengths=lengths)
    for name in ("dq", "dk", "dv", "dg", "dbeta"):
        for b in range(0, B, 8):
            assert not got[name][b].any(), name


@pytest.mark.parametrize("io,shape", [("f32", (1, 3000, 2, 1, 64, 64)), ("f32", (2, 1501, 1, 1, 128, 40)), ("f32", (1, 1200, 1, 1, 16, 130)),
                                      ("f32", (3, 999, 1, 1, 32, 8)), ("bf16", (1, 1100, 2, 2, 33, 66)), ("f16", (2, 900, 2, 1, 5, 7))], ids=str)
def test_sequences_cut_in_time_without_tensor_cores(io, shape):
    """Few heads of many tokens: segments, their sums and both carries; with and without rows that end early or hold nothing."""
    B, L = shape[:2]
    x = ref.gdr_inputs(*shape, seed=51)
    check_fwd(x, io)
    check_bwd(x, io)
    for lengths in ([L // 3] * B, [0] * B, [(L, 130, 64)[i % 3] for i in range(B)]):
        check_fwd(x, io, lengths=lengths)
        check_bwd(x, io, lengths=lengths)
    for key in ("h0", "dlast", "g"):
        x[key] = None
    check_fwd(x, io)
    check_bwd(x, io)


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 3001, 2, 1, 128, 128), (2, 2900, 1, 1, 64, 200), (1, 4097, 3, 3, 16, 64)], ids=str)
def test_backward_of_sequences_cut_in_time(shape, io):
    """Segments of both directions, rows that end in the first one or hold nothing, and no states at either end."""
    B, L = shape[:2]
    x = ref.gdr_inputs(*shape, seed=61)
    check_bwd(x, io)
    check_bwd(x, io, lengths=[(L // 4, 0)[i % 2] for i in range(B)])
    check_bwd(x, io, lengths=[L - 70] * B)
    for key in ("h0", "dlast"):
        x[key] = None
    check_bwd(x, io)
