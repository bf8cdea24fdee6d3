"""GPU parity of the gated delta rule (forward, backward, single token) with the 64-bit
token-by-token reference on the same values.

Tolerances (normwise: max |got - ref| / max |ref|), with u the unit roundoff of the io type
(2^-8 for bf16, 2^-11 for f16):
* f32 outputs of f32 io: the scan's own, 1e-5 forward and 1e-4 backward.  16-bit io: operands of
  16 bits or more enter products as two parts (2^-17 each), a chunk's chain is four products
  long: 4 x 2^-17 = 3e-5 forward; the backward joins two such chains and sums: 1e-4.
* 16-bit y: one rounding each of a score, of u and of the result: 3 u.  dq, dk, dv: a score, an
  operand, the result, and once more where a head's share joins others: 4 u.
"""

import numpy as np
import pytest
import torch

import gdr_reference as ref
import mamba_selective_scan_fwd_gb300 as ss
from gpu_util import normwise

pytestmark = pytest.mark.gpu

IO = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def tol_fwd(io, name):
    return 1e-5 if io == "f32" else 3e-5 if name == "last" else 3 * U[io]


def tol_bwd(io, name):
    return 1e-4 if io == "f32" or name in ("dg", "dbeta", "dh0") else 4 * U[io]


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


def lengths_on_gpu(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")


def check_fwd(x, io, scale=0.5, lengths=None):
    t, r = on_gpu(x, io)
    y, last = ss.ss_gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], scale=scale, h0=t["h0"], lengths=lengths_on_gpu(lengths))
    torch.cuda.synchronize()
    assert ss.device_status() == ss.SS_OK
    wy, wl = ref.gdr_fwd(r["q"], r["k"], r["v"], r["g"], r["beta"], scale, r["h0"], lengths)
    assert normwise(y, wy) <= tol_fwd(io, "y")
    assert normwise(last, wl) <= tol_fwd(io, "last")
    return y, last


def check_bwd(x, io, scale=0.5, lengths=None):
    t, r = on_gpu(x, io)
    got = ss.ss_gdr_bwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["dy"], scale=scale, h0=t["h0"], dlast_state=t["dlast"],
                        lengths=lengths_on_gpu(lengths))
    torch.cuda.synchronize()
    assert ss.device_status() == ss.SS_OK
    want = ref.gdr_bwd(r["q"], r["k"], r["v"], r["g"], r["beta"], r["dy"], scale, r["h0"], r["dlast"], lengths)
    for name, g in got.items():
        if want[name] is None:
            assert g is None
            continue
        assert normwise(g, want[name]) <= tol_bwd(io, name), name
    return got


# (Bsz, L, H, G, N, P)
SHAPES = [(1, 1, 1, 1, 16, 16), (2, 2, 2, 1, 64, 64), (1, 63, 4, 2, 64, 64), (2, 64, 3, 3, 32, 40), (1, 65, 4, 1, 128, 64),
          (1, 127, 2, 2, 128, 128), (2, 128, 2, 1, 16, 200), (1, 129, 6, 2, 72, 8), (1, 300, 5, 1, 64, 80), (1, 257, 2, 2, 8, 64),
          (1, 200, 2, 1, 128, 256), (2, 131, 3, 1, 5, 7), (1, 90, 2, 1, 33, 66)]
IDS = ["x".join(map(str, s)) for s in SHAPES]


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape, io):
    check_fwd(ref.gdr_inputs(*shape, gate=shape[1] % 3 != 0, h0=shape[1] != 128, seed=shape[1]), io)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape, io):
    check_bwd(ref.gdr_inputs(*shape, gate=shape[1] % 3 != 0, h0=shape[1] != 128, seed=10 + shape[1]), io)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_long_sequence(io):
    x = ref.gdr_inputs(1, 3000, 2, 1, 16, 16, seed=5)
    check_fwd(x, io)
    check_bwd(x, io)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_lengths_leave_rows_empty_and_padding_unread(io):
    """Rows of 0, 1, some, all and (clamped) too many tokens; whatever the padding holds, NaN included."""
    x = ref.gdr_inputs(6, 200, 2, 1, 64, 64, seed=6)
    lengths = np.array([0, 1, 77, 128, 200, 999])
    for b, n in enumerate(lengths):
        for key in ("q", "k", "v", "dy", "g", "beta"):
            x[key][b, n:] = np.nan
    clean = {k: np.nan_to_num(v) for k, v in x.items()}
    t, _ = on_gpu(x, io)
    _, r = on_gpu(clean, io)
    n = lengths_on_gpu(lengths)
    y, last = ss.ss_gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], scale=0.5, h0=t["h0"], lengths=n)
    wy, wl = ref.gdr_fwd(r["q"], r["k"], r["v"], r["g"], r["beta"], 0.5, r["h0"], lengths)
    assert normwise(y, wy) <= tol_fwd(io, "y") and normwise(last, wl) <= tol_fwd(io, "last")
    assert torch.equal(last[0], t["h0"][0])
    got = ss.ss_gdr_bwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"], lengths=n)
    want = ref.gdr_bwd(r["q"], r["k"], r["v"], r["g"], r["beta"], r["dy"], 0.5, r["h0"], r["dlast"], lengths)
    for name, g in got.items():
        assert normwise(g, want[name]) <= tol_bwd(io, name), name
    for b, m in enumerate(lengths):
        for z in (y, got["dq"], got["dk"], got["dv"], got["dg"], got["dbeta"]):
            assert not z[b, m:].any()
    assert torch.equal(got["dh0"][0], t["dlast"][0])


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_strong_decays_and_resets(io):
    """Every kind of decay in one chunk: none, strong ones, and tokens that reset the state (-inf, -200)."""
    x = ref.gdr_inputs(1, 150, 2, 1, 32, 32, seed=7)
    rng = np.random.default_rng(8)
    x["g"] = rng.choice([0.0, -1e-6, -0.5, -8.0, -30.0], size=x["g"].shape).astype(np.float32)
    x["g"][:, ::37] = -np.inf
    x["g"][:, 50] = -200.0
    check_fwd(x, io)
    got = check_bwd(x, io)
    assert torch.isfinite(got["dg"]).all()


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_equal_keys_and_rates_of_zero_one_and_two(io):
    """Keys that are all the same (each token overwrites what the last one wrote) and rates at the ends of their range."""
    x = ref.gdr_inputs(1, 140, 2, 1, 32, 32, seed=9)
    x["k"][:] = x["k"][:, :1]
    x["beta"][:, :, 0] = 1.0
    x["beta"][:, ::2, 1] = 0.0
    check_fwd(x, io)
    check_bwd(x, io)
    x = ref.gdr_inputs(1, 140, 2, 1, 32, 32, gate=False, seed=10)
    x["beta"][:] = 2.0  # reflections: the state neither grows nor decays
    check_fwd(x, io)
    check_bwd(x, io)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_strides_and_misaligned_slices_give_the_same(io):
    """Slices of one projection, at aligned and odd offsets, against contiguous copies."""
    B, L, H, G, N, P = 2, 100, 4, 2, 64, 64
    x = ref.gdr_inputs(B, L, H, G, N, P, seed=11)
    t, _ = on_gpu(x, io)
    want = check_fwd(x, io)
    dwant = check_bwd(x, io)
    for pad in (0, 8, 1):
        wide = torch.zeros(B, L + 3, H * P + 2 * G * N + 2 * pad, dtype=IO[io], device="cuda")[:, :L]
        at = pad
        parts = []
        for key, heads, width in (("v", H, P), ("k", G, N), ("q", G, N)):
            s = wide[:, :, at:at + heads * width].unflatten(2, (heads, width))
            s.copy_(t[key])
            parts.append(s)
            at += heads * width
        v, k, q = parts
        y, last = ss.ss_gdr_fwd(q, k, v, t["g"], t["beta"], scale=0.5, h0=t["h0"])
        got = ss.ss_gdr_bwd(q, k, v, t["g"], t["beta"], t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"])
        # (odd offsets of 16-bit inputs run on other units: the tolerances' sum instead of equal bits)
        same = torch.equal if pad != 1 or io == "f32" else None
        if same:
            assert same(y, want[0]) and same(last, want[1])
            assert all(same(got[n], dwant[n]) for n in got)
        else:
            assert normwise(y, want[0].double().cpu().numpy()) <= 2 * tol_fwd(io, "y")
            assert all(normwise(got[n], dwant[n].double().cpu().numpy()) <= 2 * tol_bwd(io, n) for n in got)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_no_tokens(io):
    x = ref.gdr_inputs(2, 0, 2, 1, 16, 16, seed=12)
    t, _ = on_gpu(x, io)
    y, last = ss.ss_gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], h0=t["h0"])
    assert y.shape == (2, 0, 2, 16) and torch.equal(last, t["h0"])
    _, last = ss.ss_gdr_fwd(t["q"], t["k"], t["v"], None, t["beta"])
    assert not last.any()
    got = ss.ss_gdr_bwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["dy"], h0=t["h0"], dlast_state=t["dlast"])
    assert torch.equal(got["dh0"], t["dlast"]) and got["dbeta"].numel() == 0


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 2, 1, 128, 128), (7, 4, 2, 64, 80), (3, 3, 1, 5, 7), (40, 8, 4, 128, 128), (2, 2, 2, 33, 66),
                                   (40, 8, 4, 64, 64), (60, 4, 4, 40, 72), (30, 6, 1, 16, 132)],
                         ids=str)
def test_step(shape, io):
    B, H, G, N, P = shape
    x = ref.gdr_inputs(B, 1, H, G, N, P, gate=B != 7, seed=B)
    t, r = on_gpu(x, io)
    pool = B + 3
    state = torch.randn(pool, H, N, P, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    slots = torch.randperm(pool)[:B].to(torch.int32)
    if B > 1:
        slots[1] = -1
    args = [None if t[n] is None else t[n][:, 0] for n in ("q", "k", "v", "g", "beta")]
    rargs = [None if r[n] is None else r[n][:, 0] for n in ("q", "k", "v", "g", "beta")]
    wy, ws = ref.gdr_step(*rargs, state.double().cpu().numpy(), 0.5, slots.numpy())
    before = state.clone()
    y = ss.ss_gdr_step(*[None if a is None else a.contiguous() for a in args], state, scale=0.5, slots=slots.cuda())
    assert normwise(y, wy) <= (1e-5 if io == "f32" else 2 * U[io])
    assert normwise(state, ws) <= 1e-5
    idle = sorted(set(range(pool)) - set(slots.tolist()))
    assert torch.equal(state[idle], before[idle])


def test_steps_continue_a_prompt():
    """A prompt's last state, carried on token by token, is the whole sequence's."""
    B, L, H, G, N, P = 2, 70, 4, 2, 64, 64
    x = ref.gdr_inputs(B, L, H, G, N, P, seed=13)
    t, _ = on_gpu(x, "f32")
    y, last = ss.ss_gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], scale=0.5, h0=t["h0"])
    cut = 61
    head = {n: t[n][:, :cut].contiguous() for n in ("q", "k", "v", "g", "beta")}
    _, state = ss.ss_gdr_fwd(head["q"], head["k"], head["v"], head["g"], head["beta"], scale=0.5, h0=t["h0"])
    for i in range(cut, L):
        yt = ss.ss_gdr_step(*[t[n][:, i].contiguous() for n in ("q", "k", "v", "g", "beta")], state, scale=0.5)
        assert normwise(yt, y[:, i].double().cpu().numpy()) <= 2e-5
    assert normwise(state, last.double().cpu().numpy()) <= 2e-5


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradients_match_differences_of_the_kernel_itself(io):
    """<gradient, direction> against the forward kernel's own central differences, along the f32 inputs
    (g, beta, h0).  Truncation of a step of 2^-6: 1e-3 of |gradient| |direction|.  The loss is <last_state,
    dlast> with each state off by r of itself and its own way: 2 r |last * dlast| / 2^-5 in the difference, r a
    dozen roundings to 2^-24 (f32), two parts' 2^-17 (bf16).  (Under these decays h0's gradient is 1e-4: what
    the difference shows of it is that it is small.)"""
    x = ref.gdr_inputs(1, 100, 2, 1, 32, 32, seed=14)
    t, _ = on_gpu(x, io)
    zero = torch.zeros_like(t["dy"])
    got = ss.ss_gdr_bwd(t["q"], t["k"], t["v"], t["g"], t["beta"], zero, scale=0.5, h0=t["h0"], dlast_state=t["dlast"])
    gen = torch.Generator("cuda").manual_seed(3)
    for key in ("g", "beta", "h0"):
        d = torch.randn(t[key].shape, device="cuda", generator=gen) * (0.05 if key != "h0" else 1.0)
        loss = []
        for sign in (1, -1):
            a = dict(t)
            a[key] = t[key] + sign * 2.0 ** -6 * d
            _, last = ss.ss_gdr_fwd(a["q"], a["k"], a["v"], a["g"], a["beta"], scale=0.5, h0=a["h0"])
            loss.append((last.double() * t["dlast"].double()).sum().item())
        want = (loss[0] - loss[1]) * 2.0 ** 5
        g = got["d" + key].double()
        noise = 2.0 ** 6 * (2.0 ** -21 if io == "f32" else 2.0 ** -17) * (last * t["dlast"]).double().norm().item()
        assert abs((g * d.double()).sum().item() - want) <= 1e-3 * (g.norm() * d.double().norm()).item() + noise, key


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_streams_graphs_and_repeats(io):
    """Another stream, a captured and replayed forward and backward, and equal bits every time."""
    x = ref.gdr_inputs(2, 150, 4, 2, 64, 64, seed=15)
    t, _ = on_gpu(x, io)
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    y, last = ss.ss_gdr_fwd(*args, scale=0.5, h0=t["h0"])
    d = ss.ss_gdr_bwd(*args, t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, last2 = ss.ss_gdr_fwd(*args, scale=0.5, h0=t["h0"], stream=side)
    d2 = ss.ss_gdr_bwd(*args, t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(last, last2) and all(torch.equal(d[n], d2[n]) for n in d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, last3 = ss.ss_gdr_fwd(*args, scale=0.5, h0=t["h0"])
        d3 = ss.ss_gdr_bwd(*args, t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"])
    t["v"].mul_(2.0)
    t["h0"].mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    # the state is linear in v and the start
    assert torch.equal(y3, 2 * y) and torch.equal(last3, 2 * last)
    assert torch.equal(d3["dq"], 2 * d["dq"]) and torch.equal(d3["dbeta"], 2 * d["dbeta"])


def test_two_calls_at_once_do_not_disturb_each_other():
    x = ref.gdr_inputs(2, 300, 4, 2, 64, 64, seed=16)
    t, _ = on_gpu(x, "bf16")
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    want = ss.ss_gdr_bwd(*args, t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(3):
        for s in streams:
            outs.append(ss.ss_gdr_bwd(*args, t["dy"], scale=0.5, h0=t["h0"], dlast_state=t["dlast"], stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o[n], want[n]) for o in outs for n in want)
