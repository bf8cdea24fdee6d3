"""GPU parity of the linear attention (forward, backward, single token) with the 64-bit
token-by-token reference on the same values.

Tolerances (normwise: max |got - ref| / max |ref|), with u the unit roundoff of the io type
(2^-8 for bf16, 2^-11 for f16):
* f32 outputs (states, dg, dh0; everything for f32 io): the scan's own, 1e-5 forward and 1e-4
  backward.  They are sums in 32 bits of products that keep 16 bits or more.
* 16-bit y: one rounding each of a score (or of the state) and of the result, and all terms of
  one sign at worst: 3 u.  dq, dk, dv: a score, a scaled operand and the result, and once more
  where a head's share joins others: 4 u.
"""

import numpy as np
import pytest
import torch

import la_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from gpu_util import normwise

pytestmark = pytest.mark.gpu

IO = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def tol_fwd(io, name):
    return 1e-5 if io == "f32" or name == "last" else 3 * U[io]


def tol_bwd(io, name):
    return 1e-4 if io == "f32" or name in ("dg", "dh0") else 4 * U[io]


def on_gpu(x, io):
    """Tensors of the inputs, and the values they hold in 64 bits."""
    t, r = {}, {}
    for key, v in x.items():
        if v is None:
            t[key] = r[key] = None
            continue
        t[key] = torch.from_numpy(v).to(IO[io] if key in ("q", "k", "v", "dy") else torch.float32).cuda()
        r[key] = t[key].double().cpu().numpy()
    return t, r


def check_fwd(x, io, scale=0.5, lengths=None, stream=None):
    t, r = on_gpu(x, io)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, last = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], scale=scale, h0=t["h0"], lengths=n)
    torch.cuda.synchronize()
    assert ss.device_status() == ss.SS_OK
    wy, wl = ref.la_fwd(r["q"], r["k"], r["v"], r["g"], scale, r["h0"], lengths)
    assert normwise(y, wy) <= tol_fwd(io, "y")
    assert normwise(last, wl) <= tol_fwd(io, "last")
    return y, last


def check_bwd(x, io, scale=0.5, lengths=None):
    t, r = on_gpu(x, io)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    got = ss.ss_la_bwd(t["q"], t["k"], t["v"], t["g"], t["dy"], scale=scale, h0=t["h0"], dlast_state=t["dlast"], lengths=n)
    torch.cuda.synchronize()
    assert ss.device_status() == ss.SS_OK
    want = ref.la_bwd(r["q"], r["k"], r["v"], r["g"], r["dy"], scale, r["h0"], r["dlast"], lengths)
    for name, g in got.items():
        if name == "dh0" and x["h0"] is None:
            assert g is None
            continue
        assert normwise(g, want[name]) <= tol_bwd(io, name), name
    return got


# (Bsz, L, H, G, N, P)
SHAPES = [(1, 1, 1, 1, 16, 16), (2, 2, 2, 1, 64, 64), (1, 63, 4, 2, 64, 64), (2, 64, 3, 3, 32, 40), (1, 65, 4, 1, 128, 64),
          (1, 127, 2, 2, 128, 128), (2, 128, 2, 1, 16, 200), (1, 129, 6, 2, 72, 8), (1, 300, 5, 1, 64, 80), (1, 257, 2, 2, 8, 64),
          (2, 131, 3, 1, 5, 7), (1, 90, 2, 1, 33, 66)]
IDS = ["x".join(map(str, s)) for s in SHAPES]


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape, io):
    check_fwd(ref.la_inputs(*shape, per_head=shape[1] % 2 == 0, h0=shape[1] != 128, seed=shape[1]), io)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape, io):
    check_bwd(ref.la_inputs(*shape, per_head=shape[1] % 2 == 0, h0=shape[1] != 128, seed=10 + shape[1]), io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_long_sequence_is_cut_in_time(io):
    x = ref.la_inputs(1, 3000, 2, 1, 16, 16, h0=True, seed=5)
    check_fwd(x, io)
    check_bwd(x, io)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_lengths_leave_rows_empty_and_padding_unread(io):
    """Rows of 0, 1, some, all and (clamped) too many tokens; whatever the padding holds, NaN included."""
    x = ref.la_inputs(6, 200, 2, 1, 64, 64, h0=True, seed=6)
    lengths = np.array([0, 1, 77, 128, 200, 999])
    for b, n in enumerate(lengths):
        for key in ("q", "k", "v", "dy"):
            x[key][b, n:] = np.nan
        x["g"][b, n:] = np.nan
    clean = {k: np.nan_to_num(v) for k, v in x.items()}
    t, _ = on_gpu(x, io)
    _, r = on_gpu(clean, io)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, last = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], scale=0.5, h0=t["h0"], lengths=n)
    got = ss.ss_la_bwd(t["q"], t["k"], t["v"], t["g"], t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"], lengths=n)
    wy, wl = ref.la_fwd(r["q"], r["k"], r["v"], r["g"], 0.5, r["h0"], lengths)
    want = ref.la_bwd(r["q"], r["k"], r["v"], r["g"], r["dy"], 0.5, r["h0"], r["dlast"], lengths)
    assert normwise(y, wy) <= tol_fwd(io, "y") and normwise(last, wl) <= tol_fwd(io, "last")
    for name in want:
        assert normwise(got[name], want[name]) <= tol_bwd(io, name), name
    assert torch.equal(last[0], t["h0"][0]) and not y[0].any() and not got["dv"][0].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_resets_and_extreme_decays(io):
    """exp(g) = 0 at -inf, at the type's lowest value and at -1000 cuts the sequence there; g = 0 forgets
    nothing; tokens right after a reset keep full accuracy."""
    x = ref.la_inputs(1, 260, 3, 1, 32, 32, h0=True, seed=7)
    x["g"][0, [3, 100, 101, 200], 0] = -np.inf
    x["g"][0, [0, 127, 128], 1] = np.finfo(np.float32).min
    x["g"][0, 60, 1] = -1000.0
    x["g"][0, :, 2] = 0.0
    check_fwd(x, io)
    check_bwd(x, io)


def test_large_values_stay_finite_in_f16():
    """Scores and states beyond f16's range: the result is finite whenever it is representable."""
    x = ref.la_inputs(1, 150, 2, 1, 64, 64, h0=True, seed=8)
    x["q"] *= 64
    x["k"] *= 64
    x["v"] *= 0.01
    x["h0"] *= 1e6
    x["h0"][:, :, :, 1::2] *= 1e-6
    y, _ = check_fwd(x, "f16", scale=1e-6)
    assert torch.isfinite(y).all()
    check_bwd(x, "f16", scale=1e-6)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_inputs_may_be_slices(io):
    """q, k, v, dy cut out of wider tensors, at offsets of whole and of odd numbers of elements."""
    Bsz, L, H, G, N, P = 2, 140, 4, 2, 64, 64
    x = ref.la_inputs(Bsz, L, H, G, N, P, seed=9)
    t, _ = on_gpu(x, io)
    want = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"])
    back = ss.ss_la_bwd(t["q"], t["k"], t["v"], t["g"], t["dy"])
    # equal or not to the last bit depends on the path (odd offsets leave the tensor cores): the parity bounds
    for lead in (0, 8, 3):
        wide = torch.full((Bsz, L + 1, lead + 2 * G * N + 2 * H * P + 5 + (-lead - 5) % 8), float("nan"), dtype=IO[io],
                          device="cuda")
        cuts, at = {}, lead
        for key, w in (("q", G * N), ("k", G * N), ("v", H * P), ("dy", H * P)):
            cuts[key] = wide[:, :L, at:at + w].unflatten(2, (-1, N if key in "qk" else P))
            cuts[key].copy_(t[key])
            at += w
        y, last = ss.ss_la_fwd(cuts["q"], cuts["k"], cuts["v"], t["g"])
        assert normwise(y, want[0].double().cpu().numpy()) <= tol_fwd(io, "y")
        assert normwise(last, want[1].double().cpu().numpy()) <= 1e-5
        got = ss.ss_la_bwd(cuts["q"], cuts["k"], cuts["v"], t["g"], cuts["dy"])
        for name in ("dq", "dk", "dv", "dg"):
            assert normwise(got[name], back[name].double().cpu().numpy()) <= tol_bwd(io, name), name


def test_batch_stride_beyond_32_bits():
    """Rows 2^31 + 64 elements apart."""
    Bsz, L, H, G, N, P = 2, 70, 2, 1, 64, 64
    x = ref.la_inputs(Bsz, L, H, G, N, P, seed=11)
    t, r = on_gpu(x, "bf16")
    far = torch.empty((1 << 31) + 64 + L * H * P, dtype=torch.bfloat16, device="cuda")
    v = far.as_strided((Bsz, L, H, P), ((1 << 31) + 64, H * P, P, 1))
    v.copy_(t["v"])
    y, last = ss.ss_la_fwd(t["q"], t["k"], v, t["g"])
    wy, wl = ref.la_fwd(r["q"], r["k"], r["v"], r["g"])
    assert normwise(y, wy) <= tol_fwd("bf16", "y") and normwise(last, wl) <= 1e-5


@pytest.mark.parametrize("per_head", [False, True])
def test_backward_matches_differences(per_head):
    """<gradient, direction> against central differences of the 64-bit forward (f32 gradients: 1e-4 of
    the norms' product, as the parity bound allows for each element)."""
    x = ref.la_inputs(1, 70, 4, 2, 16, 24, per_head=per_head, h0=True, seed=12)
    t, r = on_gpu(x, "f32")
    got = ss.ss_la_bwd(t["q"], t["k"], t["v"], t["g"], t["dy"], scale=0.7, h0=t["h0"], dlast_state=t["dlast"])

    def loss(x):
        y, S = ref.la_fwd(x["q"], x["k"], x["v"], x["g"], 0.7, x["h0"])
        return np.sum(y * x["dy"]) + np.sum(S * x["dlast"])

    rng = np.random.default_rng(13)
    for key in ("q", "k", "v", "g", "h0"):
        d = rng.normal(size=r[key].shape)
        hi, lo = dict(r), dict(r)
        hi[key], lo[key] = r[key] + 1e-6 * d, r[key] - 1e-6 * d
        want = (loss(hi) - loss(lo)) / 2e-6
        grad = got["d" + key].double().cpu().numpy()
        assert abs(np.sum(grad * d) - want) <= 1e-4 * np.linalg.norm(grad) * np.linalg.norm(d) / np.sqrt(d.size) + 1e-4 * abs(want)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_segments_chain(io):
    """A sequence run in two calls (state handed on, its gradient handed back) equals one call."""
    x = ref.la_inputs(2, 330, 4, 2, 64, 64, h0=True, seed=14)
    t, _ = on_gpu(x, io)
    args = [t[n] for n in ("q", "k", "v", "g")]
    y, last = ss.ss_la_fwd(*args, h0=t["h0"])
    whole = ss.ss_la_bwd(*args, t["dy"], h0=t["h0"], dlast_state=t["dlast"])
    cut = 201
    a, b = [x[:, :cut].contiguous() for x in args], [x[:, cut:].contiguous() for x in args]
    y1, mid = ss.ss_la_fwd(*a, h0=t["h0"])
    y2, last2 = ss.ss_la_fwd(*b, h0=mid)
    g2 = ss.ss_la_bwd(*b, t["dy"][:, cut:].contiguous(), h0=mid, dlast_state=t["dlast"])
    g1 = ss.ss_la_bwd(*a, t["dy"][:, :cut].contiguous(), h0=t["h0"], dlast_state=g2["dh0"])
    assert normwise(torch.cat([y1, y2], 1), y.double().cpu().numpy()) <= tol_fwd(io, "y")
    assert normwise(last2, last.double().cpu().numpy()) <= 1e-5
    for name in ("dq", "dk", "dv", "dg"):
        got = torch.cat([g1[name], g2[name]], 1)
        assert normwise(got, whole[name].double().cpu().numpy()) <= tol_bwd(io, name), name
    assert normwise(g1["dh0"], whole["dh0"].double().cpu().numpy()) <= 1e-4


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 24, 1, 128, 64), (5, 4, 2, 64, 80), (64, 16, 16, 64, 64), (3, 2, 1, 5, 7), (2, 3, 3, 72, 8)],
                         ids=lambda s: "x".join(map(str, s)))
def test_step(shape, io):
    """One token on a pool of states, rows on scattered slots, one of them padding."""
    Bsz, H, G, N, P = shape
    x = ref.la_inputs(Bsz, 1, H, G, N, P, seed=15)
    t, r = on_gpu(x, io)
    rng = np.random.default_rng(16)
    pool = Bsz + 3
    slots = rng.permutation(pool)[:Bsz].astype(np.int32)
    pad = Bsz // 2 if Bsz > 1 else None
    if pad is not None:
        slots[pad] = -1
    state = torch.randn(pool, H, N, P, device="cuda")
    before = state.double().cpu().numpy()
    y = ss.ss_la_step(t["q"][:, 0], t["k"][:, 0], t["v"][:, 0], t["g"][:, 0], state, scale=0.5,
                      slots=torch.from_numpy(slots).cuda())
    want = before.copy()
    wy, wS = ref.la_fwd(r["q"], r["k"], r["v"], r["g"], 0.5, before[np.maximum(slots, 0)])
    for b in range(Bsz):
        if b == pad:
            wy[b] = 0
        else:
            want[slots[b]] = wS[b]
    assert normwise(y, wy[:, 0]) <= tol_fwd(io, "y")
    assert normwise(state, want) <= 1e-5
    untouched = [s for s in range(pool) if s not in slots]
    assert np.array_equal(state.double().cpu().numpy()[untouched], before[untouched])


def test_step_ignores_slots_outside_the_pool():
    x = ref.la_inputs(3, 1, 2, 1, 16, 16, seed=17)
    t, _ = on_gpu(x, "f32")
    state = torch.randn(2, 2, 16, 16, device="cuda")
    keep = state.clone()
    y = ss.ss_la_step(t["q"][:, 0], t["k"][:, 0], t["v"][:, 0], t["g"][:, 0], state,
                      slots=torch.tensor([2, -1, 1 << 30], dtype=torch.int32, device="cuda"))
    assert torch.equal(state, keep) and not y.any()


def test_step_on_a_pool_beyond_32_bits():
    H, N, P = 64, 128, 128
    pool = (1 << 31) // (H * N * P) + 2
    state = torch.empty(pool, H, N, P, device="cuda")
    x = ref.la_inputs(2, 1, H, 1, N, P, seed=18)
    t, r = on_gpu(x, "bf16")
    state[pool - 1].normal_()
    state[0].normal_()
    before = state[[pool - 1, 0]].double().cpu().numpy()
    y = ss.ss_la_step(t["q"][:, 0], t["k"][:, 0], t["v"][:, 0], t["g"][:, 0], state,
                      slots=torch.tensor([pool - 1, 0], dtype=torch.int32, device="cuda"))
    wy, wS = ref.la_fwd(r["q"], r["k"], r["v"], r["g"], 1.0, before)
    assert normwise(y, wy[:, 0]) <= tol_fwd("bf16", "y")
    assert normwise(state[[pool - 1, 0]], wS) <= 1e-5


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_steps_continue_a_prompt(io):
    x = ref.la_inputs(2, 140, 4, 1, 64, 64, seed=19)
    t, _ = on_gpu(x, io)
    args = [t[n] for n in ("q", "k", "v", "g")]
    y, last = ss.ss_la_fwd(*args)
    n = 131
    y0, state = ss.ss_la_fwd(*[a[:, :n] for a in args[:3]], args[3][:, :n].contiguous())
    got = [ss.ss_la_step(*[a[:, i] for a in args[:3]], args[3][:, i].contiguous(), state) for i in range(n, 140)]
    assert normwise(torch.cat([y0, torch.stack(got, 1)], 1), y.double().cpu().numpy()) <= tol_fwd(io, "y")
    assert normwise(state, last.double().cpu().numpy()) <= 1e-5


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_runs_repeat_bit_for_bit_and_on_other_streams(io):
    x = ref.la_inputs(2, 700, 6, 2, 64, 64, h0=True, seed=20)
    t, _ = on_gpu(x, io)

    def call(stream=None):
        f = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], h0=t["h0"], stream=stream)
        b = ss.ss_la_bwd(t["q"], t["k"], t["v"], t["g"], t["dy"], h0=t["h0"], dlast_state=t["dlast"], stream=stream)
        return list(f) + list(b.values())

    first = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = call()
    torch.cuda.synchronize()
    third = call(s)
    torch.cuda.synchronize()
    for a, b, c in zip(first, again, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_graph_replay():
    x = ref.la_inputs(1, 300, 4, 1, 64, 64, seed=21)
    t, _ = on_gpu(x, "bf16")
    dt = ss.SS_BF16
    ws = torch.empty(max(16, ss.la_fwd_workspace_bytes(1, 300, 4, 1, 64, 64, dt)), dtype=torch.uint8, device="cuda")
    y, last = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], workspace=ws)
    y2, last2 = torch.empty_like(y), torch.empty_like(last)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], y=y2, last_state=last2, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(last, last2)


def test_empty_sequences_pass_the_state_through():
    h0 = torch.randn(2, 4, 8, 8, device="cuda")
    q, v = torch.empty(2, 0, 1, 8, device="cuda"), torch.empty(2, 0, 4, 8, device="cuda")
    g = torch.empty(2, 0, 4, device="cuda")
    y, last = ss.ss_la_fwd(q, q, v, g, h0=h0)
    assert y.shape == (2, 0, 4, 8) and torch.equal(last, h0)
    assert not ss.ss_la_fwd(q, q, v, g)[1].any()
    back = ss.ss_la_bwd(q, q, v, g, v, h0=h0, dlast_state=h0)
    assert torch.equal(back["dh0"], h0)
    back = ss.ss_la_bwd(q, q, v, -torch.ones(4, device="cuda"), v)
    assert not back["dg"].any()
