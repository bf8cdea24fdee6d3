"""Cases, plain forms and 64-bit values of the gated delta rule and of the per-head norm with rotation of q and k.

The operators (per batch row b and head h, N key and P value channels, state S of N x P):

  gated delta rule   u_t = beta_t (v_t - e^{g_t} S_{t-1}^T k_t),  S_t = e^{g_t} S_{t-1} + k_t u_t^T,  y_t = scale * q_t S_t
                     ("fwd", its gradient "bwd", and one token in place on a pool of states "step")
  q / k norm         n = x / sqrt(mean(x^2) + eps) * weight, or x / sqrt(sum(x^2) + eps), over each head's channels,
                     then pairs of the first `rot` channels turned by position * freq ("qknorm", its gradient "dqknorm")

q and k have G heads, each shared by H / G of the H heads of v.  g is one f32 log decay per token and head or absent,
beta one f32 rate per token and head.  lengths, where given, cuts each batch row: later tokens give zeros and leave the
state alone.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CHUNK = 64  # tokens per chunk of the plain chunked form
EPS = 1e-6


def listed():
    return [
        # the next turn of one conversation: a few dozen tokens after a kept state, where latency counts
        dict(name="fwd-turn", op="fwd", io="bf16", B=1, L=37, H=32, G=16, N=128, P=128, gate=True, h0=True,
             ragged=False, packed=True),
        # prompts of a layer of 4096 value channels in heads of 128, two of them to a q/k head, sliced from one projection
        dict(name="fwd-layer", op="fwd", io="bf16", B=4, L=4096, H=32, G=16, N=128, P=128, gate=True, h0=False,
             ragged=False, packed=True),
        # one very long sequence on few heads
        dict(name="fwd-long", op="fwd", io="bf16", B=1, L=65536, H=8, G=4, N=128, P=128, gate=True, h0=False,
             ragged=False, packed=False),
        # padded batch of prompts of unequal length (one of them empty) that continue kept states
        dict(name="fwd-ragged-f16", op="fwd", io="f16", B=8, L=2047, H=16, G=8, N=64, P=128, gate=True, h0=True,
             ragged=True, packed=False),
        # full-precision prompt of 1536 value channels
        dict(name="fwd-f32", op="fwd", io="f32", B=2, L=1000, H=24, G=24, N=64, P=64, gate=True, h0=False,
             ragged=False, packed=False),
        # training step of the 4096-channel layer
        dict(name="bwd-layer", op="bwd", io="bf16", B=2, L=4096, H=32, G=16, N=128, P=128, gate=True, h0=False,
             ragged=False, packed=True),
        # small half-precision training batch, padded, without a gate (the plain delta rule)
        dict(name="bwd-ragged-f16", op="bwd", io="f16", B=3, L=509, H=8, G=2, N=64, P=80, gate=False, h0=True,
             ragged=True, packed=False),
        # full-precision gradient of a sequence segment between two others (state gradients in and out)
        dict(name="bwd-f32", op="bwd", io="f32", B=1, L=777, H=16, G=4, N=32, P=64, gate=True, h0=True,
             ragged=False, packed=False),
        # one token of one sequence
        dict(name="step-one", op="step", io="bf16", B=1, H=32, G=16, N=128, P=128, gate=True, pool=4),
        # one token of each of 256 running sequences, their states anywhere in a larger pool
        dict(name="step-batch", op="step", io="bf16", B=256, H=32, G=16, N=128, P=128, gate=True, pool=300),
        # q and k of the layer's prompts: root mean square norm with a weight, half the channels turned
        dict(name="qknorm-layer", op="qknorm", io="bf16", B=4, L=4096, Hq=16, Hk=16, N=128, rot=64, l2=False,
             interleaved=False, packed=True),
        # their gradient in training
        dict(name="dqknorm-layer", op="dqknorm", io="bf16", B=2, L=4096, Hq=16, Hk=16, N=128, rot=64, l2=False,
             interleaved=False, packed=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "fwd", "bwd", "bwd", "bwd", "step", "qknorm", "dqknorm"))
    io = rng.choice(("bf16", "bf16", "f16", "f32"))
    packed = rng.choice((True, False))
    if op in ("qknorm", "dqknorm"):
        N = rng.choice((32, 64, 64, 80, 128, 128, 192, 256))
        Hq = rng.choice((1, 4, 8, 16, 24, 32))
        Hk = rng.choice([h for h in (1, 2, 4, 8, 16, 24, 32) if h <= Hq])
        l2 = rng.choice((True, False))
        rot = rng.choice((0, N // 2, N))
        L = _log(rng, 1, 16384)
        B = max(1, min(_log(rng, 1, 16), 40_000_000 // ((Hq + Hk) * N * L)))
        return dict(op=op, io=io, B=B, L=L, Hq=Hq, Hk=Hk, N=N, rot=rot, l2=l2, interleaved=rng.choice((True, False)),
                    packed=packed)
    G = rng.choice((1, 2, 4, 8, 16))
    H = G * rng.choice((1, 1, 2, 4))
    N = rng.choice((16, 32, 64, 64, 128, 128))
    P = rng.choice((32, 64, 80, 128, 128, 256))
    gate = rng.choice((True, True, False))
    if op == "step":
        B = _log(rng, 1, max(1, min(600, 130_000_000 // (H * N * P))))
        return dict(op=op, io=io, B=B, H=H, G=G, N=N, P=P, gate=gate, pool=B + rng.randrange(0, 9))
    most = 60_000_000 // (H * max(N + P, 128)) // (1 if op == "fwd" else 4)  # tokens
    L = min(_log(rng, 1, 20000), most)
    B = max(1, min(_log(rng, 1, 8), most // L))
    return dict(op=op, io=io, B=B, L=L, H=H, G=G, N=N, P=P, gate=gate, h0=rng.choice((True, False)),
                ragged=rng.choice((True, False)), packed=packed)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    io = DTYPES[case["io"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    s = {"case": case}
    if case["op"] in ("qknorm", "dqknorm"):
        B, L, Hq, Hk, N, rot = (case[n] for n in ("B", "L", "Hq", "Hk", "N", "rot"))
        if case["packed"]:
            x = (1.5 * normal(B, L, (Hq + Hk) * N)).to(io)
            s["q"], s["k"] = x[:, :, :Hq * N].unflatten(2, (Hq, N)), x[:, :, Hq * N:].unflatten(2, (Hk, N))
        else:
            s["q"], s["k"] = (1.5 * normal(B, L, Hq, N)).to(io), (1.5 * normal(B, L, Hk, N)).to(io)
        s["qw"], s["kw"] = (None, None) if case["l2"] else (1 + 0.2 * normal(N), 1 + 0.2 * normal(N))
        s["positions"] = s["freqs"] = None
        if rot:
            # every row somewhere in a context of up to a million tokens
            start = torch.randint(0, 1_000_000, (B, 1), generator=gen, device=dev)
            s["positions"] = (start + torch.arange(L, device=dev)).to(torch.int32)
            s["freqs"] = torch.exp(torch.arange(rot // 2, device=dev).double() * (-2 * math.log(1e6) / rot)).float()
        if case["op"] == "dqknorm":
            s["dq"], s["dk"] = normal(B, L, Hq, N).to(io), normal(B, L, Hk, N).to(io)
        return s
    B, H, G, N, P = (case[n] for n in "BHGNP")
    lead = (B,) if case["op"] == "step" else (B, case["L"])

    def unit(x):
        """What a norm of q and k per head leaves: unit vectors in the io type."""
        x = x.float()
        return (x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)).to(io)

    s["scale"] = 1.0 / math.sqrt(N)
    if case.get("packed"):
        # one buffer for the layer's q, k and v, as its projection and convolution leave it
        x = normal(*lead, H * P + 2 * G * N).to(io)
        s["v"] = x[..., :H * P].unflatten(-1, (H, P))
        s["k"] = x[..., H * P:H * P + G * N].unflatten(-1, (G, N))
        s["q"] = x[..., H * P + G * N:].unflatten(-1, (G, N))
        s["k"].copy_(unit(s["k"]))
        s["q"].copy_(unit(s["q"]))
    else:
        s["q"], s["k"], s["v"] = unit(normal(*lead, G, N)), unit(normal(*lead, G, N)), normal(*lead, H, P).to(io)
    s["beta"] = torch.sigmoid(normal(*lead, H))
    s["g"] = None
    if case["gate"]:
        # -dt * A with dt log-uniform in [1e-3, 1e-1] and A in [1, 16] per head
        A = 1 + 15 * torch.rand(H, generator=gen, device=dev)
        s["g"] = -torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand((*lead, H), generator=gen, device=dev)) * A
    if case["op"] == "step":
        s["state"] = 0.5 * normal(case["pool"], H, N, P)
        s["slots"] = torch.randperm(case["pool"], generator=gen, device=dev)[:B].to(torch.int32)
        return s
    s["h0"] = 0.5 * normal(B, H, N, P) if case["h0"] else None
    s["lengths"] = None
    if case["ragged"]:
        lengths = torch.randint(0, case["L"] + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        lengths[0] = case["L"]
        if B > 1:
            lengths[-1] = 0
        s["lengths"] = lengths
    if case["op"] == "bwd":
        s["dy"] = normal(*lead, H, P).to(io)
        s["dlast"] = normal(B, H, N, P) if case["h0"] else None
    return s


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    import mamba_selective_scan_fwd_gb300 as ss

    op = s["case"]["op"]
    if op == "fwd":
        return ss.ss_gdr_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], h0=s["h0"],
                             lengths=s["lengths"])
    if op == "bwd":
        return ss.ss_gdr_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dy"], scale=s["scale"], h0=s["h0"],
                             dlast_state=s["dlast"], lengths=s["lengths"])
    if op == "step":
        y = ss.ss_gdr_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], scale=s["scale"], slots=s["slots"])
        return {"y": y, "state": s["state"]}
    kind = dict(q_weight=s["qw"], k_weight=s["kw"], positions=s["positions"], freqs=s["freqs"], l2=s["case"]["l2"],
                eps=EPS, interleaved=s["case"]["interleaved"])
    if op == "qknorm":
        return ss.ss_qknorm_fwd(s["q"], s["k"], **kind)
    return ss.ss_qknorm_bwd(s["q"], s["k"], s["dq"], s["dk"], **kind)


# ------------------------------------------------------------------ plain forms (32 bits)

def _inverse(x):
    """Inverse of unit lower triangular matrices [..., n, n], n a power of two, by halves."""
    n = x.shape[-1]
    if n == 1:
        return torch.ones_like(x)
    h = n // 2
    a, b = _inverse(torch.stack([x[..., :h, :h], x[..., h:, h:]])).unbind(0)
    c = -(b @ x[..., h:, :h] @ a)
    return torch.cat([torch.cat([a, torch.zeros_like(a)], -1), torch.cat([c, b], -1)], -2)


def _starts(phi, e, s0):
    """States before each chunk of S' = phi S + e: [B, H, c, N, P]; pairs of chunks joined, then opened again."""
    c = e.shape[2]
    if c == 1:
        return s0.unsqueeze(2)
    if c % 2:  # the chunk after the last is never opened
        phi, e = (torch.cat([t, torch.zeros_like(t[:, :, :1])], 2) for t in (phi, e))
    p0, p1, e0, e1 = phi[:, :, 0::2], phi[:, :, 1::2], e[:, :, 0::2], e[:, :, 1::2]
    even = _starts(p1 @ p0, p1 @ e0 + e1, s0)
    return torch.stack([even, p0 @ even + e0], 3).flatten(2, 3)[:, :, :c]


def _chunked(s, dy=None):
    """The inputs in 32 bits, cut into chunks [B, H, c, T, .], zero past each row's length; decays and the inverse."""
    q, k, v, beta = s["q"].float(), s["k"].float(), s["v"].float(), s["beta"]
    B, L, H, P = v.shape
    g = torch.zeros_like(beta) if s["g"] is None else s["g"]
    rep = H // q.shape[2]
    xs = [q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2), v, g.unsqueeze(-1), beta.unsqueeze(-1)]
    xs += [] if dy is None else [dy.float()]
    if s["lengths"] is not None:
        on = (torch.arange(L, device=v.device) < s["lengths"].unsqueeze(1))[:, :, None, None]
        xs = [x.masked_fill(~on, 0.0) for x in xs]
    pad = -L % CHUNK
    xs = [torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).unflatten(1, (-1, CHUNK)).permute(0, 3, 1, 2, 4) for x in xs]
    d = dict(zip(("q", "k", "v", "g", "beta", "dy"), xs))
    c = torch.cumsum(d["g"].squeeze(-1).double(), -1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device).tril()
    d["gam"] = torch.exp((c.unsqueeze(-1) - c.unsqueeze(-2)).masked_fill(~low, -math.inf)).float()
    d["up"] = torch.exp(c).float().unsqueeze(-1)                      # from the chunk's start
    d["down"] = torch.exp(c[..., -1:] - c).float().unsqueeze(-1)      # to its end
    d["through"] = torch.exp(c[..., -1]).float()[..., None, None]
    kk = (d["k"] @ d["k"].transpose(-1, -2)) * d["gam"]
    d["inv"] = _inverse(torch.eye(CHUNK, device=v.device) + (d["beta"] * kk).tril(-1))
    d["w"] = d["inv"] @ (d["beta"] * d["up"] * d["k"])
    d["pairs"] = (d["q"] @ d["k"].transpose(-1, -2)) * d["gam"]
    d["kd"] = d["down"] * d["k"]
    d["phi"] = d["through"] * torch.eye(q.shape[3], device=v.device) - d["kd"].transpose(-1, -2) @ d["w"]
    return d


def _states(d, h0):
    """U of a zero start, the states before each chunk and the one after the last."""
    u0 = d["inv"] @ (d["beta"] * d["v"])
    e = d["kd"].transpose(-1, -2) @ u0
    if h0 is None:
        h0 = torch.zeros_like(e[:, :, 0])
    h = _starts(d["phi"], e, h0)
    return u0, h, d["phi"][:, :, -1] @ h[:, :, -1] + e[:, :, -1]


def _tokens(x, L):
    """[B, H, c, T, .] -> [B, L, H, .]"""
    return x.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :L]


def _plain_fwd(s):
    L = s["v"].shape[1]
    d = _chunked(s)
    u0, h, last = _states(d, s["h0"])
    u = u0 - d["w"] @ h
    y = s["scale"] * (d["up"] * (d["q"] @ h) + d["pairs"] @ u)
    return _tokens(y, L).to(s["v"].dtype).contiguous(), last.contiguous()


def _plain_bwd(s):
    L, io, scale = s["v"].shape[1], s["v"].dtype, s["scale"]
    G, N = s["q"].shape[2:]
    d = _chunked(s, s["dy"])
    q, k, beta, dy, gam, up, down = (d[n] for n in ("q", "k", "beta", "dy", "gam", "up", "down"))
    u0, h, _ = _states(d, s["h0"])
    u = u0 - d["w"] @ h
    miss = d["v"] - up * (k @ h) - ((k @ k.transpose(-1, -2)) * gam).tril(-1) @ u           # u = beta * miss
    # adjoints of the states after each chunk, last chunk first
    du0 = scale * (d["pairs"].transpose(-1, -2) @ dy)
    e = scale * ((up * q).transpose(-1, -2) @ dy) - d["w"].transpose(-1, -2) @ du0
    r0 = torch.zeros_like(e[:, :, 0]) if s["dlast"] is None else s["dlast"]
    back = d["phi"].transpose(-1, -2)
    r = _starts(back.flip(2), e.flip(2), r0).flip(2)
    dh0 = back[:, :, 0] @ r[:, :, 0] + e[:, :, 0]
    x = d["inv"].transpose(-1, -2) @ (du0 + d["kd"] @ r)
    ht = h.transpose(-1, -2)
    es = scale * gam * (dy @ u.transpose(-1, -2))
    fs = -(beta * gam * (x @ u.transpose(-1, -2))).tril(-1)
    dq1, dk1, dk2 = scale * up * (dy @ ht), -beta * up * (x @ ht), down * (u @ r.transpose(-1, -2))
    dq = dq1 + es @ k
    dk = dk1 + dk2 + fs @ k + es.transpose(-1, -2) @ q + fs.transpose(-1, -2) @ k
    a = (q * dq1).sum(-1) + (k * dk1).sum(-1)
    b = (k * dk2).sum(-1)
    spans = es * (q @ k.transpose(-1, -2)) + fs * (k @ k.transpose(-1, -2))
    # dg_t: every path that crosses token t, by its two ends
    low = torch.cumsum(spans, -1) - spans                                              # sum over j < column
    dg = low.flip(-2).cumsum(-2).flip(-2).diagonal(dim1=-2, dim2=-1)                   # and over i >= t, at t
    dg = dg + a.flip(-1).cumsum(-1).flip(-1) + torch.cumsum(b, -1) - b
    dg = dg + (d["through"] * h * r).sum((-1, -2)).unsqueeze(-1)
    outs = [_tokens(t, L) for t in (dq, dk, beta * x, dg.unsqueeze(-1), (x * miss).sum(-1, keepdim=True))]
    if s["lengths"] is not None:
        on = (torch.arange(L, device=dy.device) < s["lengths"].unsqueeze(1))[:, :, None, None]
        outs = [t.masked_fill(~on, 0.0) for t in outs]
    dq, dk, dv, dg, dbeta = outs
    return {"dq": dq.unflatten(2, (G, -1)).sum(3).to(io), "dk": dk.unflatten(2, (G, -1)).sum(3).to(io),
            "dv": dv.to(io).contiguous(), "dg": None if s["g"] is None else dg.squeeze(-1).contiguous(),
            "dbeta": dbeta.squeeze(-1).contiguous(), "dh0": None if s["h0"] is None else dh0.contiguous()}


def _plain_step(s):
    rep = s["v"].shape[1] // s["q"].shape[1]
    q, k = s["q"].float().repeat_interleave(rep, 1), s["k"].float().repeat_interleave(rep, 1)
    at = s["slots"].long()
    old = s["state"][at]
    if s["g"] is not None:
        old = torch.exp(s["g"])[:, :, None, None] * old
    u = s["beta"].unsqueeze(-1) * (s["v"].float() - (k.unsqueeze(-1) * old).sum(-2))
    new = old + k.unsqueeze(-1) * u.unsqueeze(-2)
    s["state"][at] = new
    y = s["scale"] * (q.unsqueeze(-1) * new).sum(-2)
    return {"y": y.to(s["v"].dtype), "state": s["state"]}


def _turns(s):
    """cos and sin [B, L, 1, rot / 2]; the angles of far positions need 64 bits."""
    angle = s["positions"].double()[:, :, None, None] * s["freqs"].double()
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    x, rest = x[..., :rot], x[..., rot:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    x = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([x, rest], -1)


def _unit(x, case):
    m = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((m if case["l2"] else m / x.shape[-1]) + EPS)


def _plain_qknorm(s):
    case = s["case"]
    cs = None if s["freqs"] is None else _turns(s)

    def one(x, w):
        n = x.float()
        n = n * _unit(n, case)
        n = n if w is None else n * w
        return (n if cs is None else _rotate(n, *cs, case["interleaved"])).to(x.dtype)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _plain_dqknorm(s):
    case = s["case"]
    cs = None if s["freqs"] is None else _turns(s)

    def one(x, w, d):
        io, x, d = x.dtype, x.float(), d.float()
        if cs is not None:
            d = _rotate(d, cs[0], -cs[1], case["interleaved"])
        r = _unit(x, case)
        n = x * r
        dw = None if w is None else (d * n).sum((0, 1, 2))
        d = d if w is None else d * w
        m = (d * n).sum(-1, keepdim=True)
        return (r * (d - n * (m if case["l2"] else m / x.shape[-1]))).to(io), dw

    (dq, dqw), (dk, dkw) = one(s["q"], s["qw"], s["dq"]), one(s["k"], s["kw"], s["dk"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def run(state):
    if own:
        return _run_own(state)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "qknorm": _plain_qknorm,
            "dqknorm": _plain_dqknorm}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    e = 4 if case["io"] == "f32" else 2
    if case["op"] in ("qknorm", "dqknorm"):
        tokens, back = case["B"] * case["L"], case["op"] == "dqknorm"
        n = tokens * (case["Hq"] + case["Hk"]) * case["N"]
        weights = 0 if case["l2"] else 8 * case["N"]
        return {"bytes": (3 if back else 2) * e * n + (2 if back else 1) * weights + (4 * tokens if case["rot"] else 0),
                "flops": (14 if back else 7) * n}
    B, H, G, N, P = (case[n] for n in "BHGNP")
    gates = 2 if case["gate"] else 1
    if case["op"] == "step":
        return {"bytes": 8 * B * H * N * P + e * B * (2 * G * N + 2 * H * P) + 4 * gates * B * H, "flops": 7 * B * H * N * P}
    L = case["L"]
    state = 4 * B * H * N * P
    if case["op"] == "fwd":
        return {"bytes": e * B * L * (2 * G * N + 2 * H * P) + 4 * gates * B * L * H + state * (2 if case["h0"] else 1),
                "flops": 6 * B * L * H * N * P}
    return {"bytes": e * B * L * (4 * G * N + 3 * H * P) + 8 * gates * B * L * H + state * (3 if case["h0"] else 0),
            "flops": 16 * B * L * H * N * P}


# ------------------------------------------------------------------ 64 bits, token by token

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("qknorm", "dqknorm"):
        return _exact_qknorm(case, s)
    if case["op"] == "step":
        return _exact_step(case, s)
    if case["L"] > 20000 or case["B"] * case["L"] * case["H"] * case["N"] * case["P"] > 12_000_000_000:
        return None
    B, L, H, P = s["v"].shape
    of = torch.arange(H, device=s["v"].device) // (H // case["G"])
    q, k, v = s["q"].double()[:, :, of], s["k"].double()[:, :, of], s["v"].double()
    beta, g = s["beta"].double(), torch.zeros(B, L, H, dtype=torch.float64, device=v.device)
    if s["g"] is not None:
        g = s["g"].double()
    if s["lengths"] is not None:
        off = torch.arange(L, device=v.device) >= s["lengths"].unsqueeze(1)
        beta, g = beta.masked_fill(off[..., None], 0.0), g.masked_fill(off[..., None], 0.0)
        q = q.masked_fill(off[..., None, None], 0.0)
    a = torch.exp(g)
    S = torch.zeros(B, H, case["N"], P, dtype=torch.float64, device=v.device) if s["h0"] is None else s["h0"].double()

    def forward(S, t):
        S = S * a[:, t, :, None, None]
        miss = v[:, t] - torch.matmul(k[:, t].unsqueeze(-2), S).squeeze(-2)
        u = beta[:, t].unsqueeze(-1) * miss
        return torch.addcmul(S, k[:, t].unsqueeze(-1), u.unsqueeze(-2)), u, miss

    if case["op"] == "fwd":
        y = torch.zeros_like(v)
        for t in range(L):
            S, _, _ = forward(S, t)
            y[:, t] = s["scale"] * torch.matmul(q[:, t].unsqueeze(-2), S).squeeze(-2)
        return y, S
    every = 64
    kept = []
    for t in range(L):
        if t % every == 0:
            kept.append(S)
        S, _, _ = forward(S, t)
    R = torch.zeros_like(S) if s["dlast"] is None else s["dlast"].double()
    dy = s["dy"].double()
    if s["lengths"] is not None:
        dy = dy.masked_fill(off[..., None, None], 0.0)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(beta), torch.zeros_like(beta)
    for c in reversed(range(len(kept))):
        t0 = c * every
        run_, us, misses = [kept.pop()], [], []
        for t in range(t0, min(L, t0 + every)):
            S, u, miss = forward(run_[-1], t)
            run_.append(S)
            us.append(u)
            misses.append(miss)
        for t in reversed(range(t0, min(L, t0 + every))):
            old, new, u, miss = run_[t - t0], run_[t - t0 + 1], us[t - t0], misses[t - t0]
            kt, dyt, b = k[:, t].unsqueeze(-1), dy[:, t].unsqueeze(-2), beta[:, t, :, None, None]
            dq[:, t] = s["scale"] * (new * dyt).sum(-1)
            R = R + s["scale"] * q[:, t].unsqueeze(-1) * dyt
            x = (R * kt).sum(-2, keepdim=True)
            dv[:, t] = (b * x).squeeze(-2)
            dbeta[:, t] = (x.squeeze(-2) * miss).sum(-1)
            dk[:, t] = (R * u.unsqueeze(-2)).sum(-1) - (b * a[:, t, :, None, None] * old * x).sum(-1)
            R = a[:, t, :, None, None] * (R - b * kt * x)
            dg[:, t] = (R * old).sum((-1, -2))
    if s["lengths"] is not None:
        dk, dv = dk.masked_fill(off[..., None, None], 0.0), dv.masked_fill(off[..., None, None], 0.0)
        dg, dbeta = dg.masked_fill(off[..., None], 0.0), dbeta.masked_fill(off[..., None], 0.0)
    G = case["G"]
    return {"dq": dq.unflatten(2, (G, -1)).sum(3), "dk": dk.unflatten(2, (G, -1)).sum(3), "dv": dv,
            "dg": None if s["g"] is None else dg, "dbeta": dbeta, "dh0": None if s["h0"] is None else R}


def _exact_step(case, s):
    per = case["H"] // case["G"]
    state = s["state"].double()
    at = s["slots"].long()
    q, k = (s[n].double().unsqueeze(2).expand(-1, -1, per, -1).flatten(1, 2) for n in "qk")
    decay = 1.0 if s["g"] is None else torch.exp(s["g"].double())[..., None, None]
    old = state[at]
    # the other form: e^g (I - beta k k^T) S + beta k v^T
    rank1 = s["beta"].double()[..., None, None] * k[..., :, None]
    new = decay * (old - rank1 * torch.matmul(k[..., None, :], old)) + rank1 * s["v"].double()[..., None, :]
    state[at] = new
    return {"y": s["scale"] * torch.matmul(q[..., None, :], new).squeeze(-2), "state": state}


def _exact_qknorm(case, s):
    back = case["op"] == "dqknorm"
    turn = None
    if s["freqs"] is not None:
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=s["q"].device),
                           s["positions"].double()[..., None] * s["freqs"].double()).unsqueeze(2)

    def one(x, w):
        length = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2
        n = x / torch.sqrt((length if case["l2"] else length / x.shape[-1]) + EPS)
        n = n if w is None else n * w
        if turn is None:
            return n
        rot = case["rot"]
        z = n[..., :rot].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
        z = (z if case["interleaved"] else z.transpose(-1, -2)).contiguous()
        z = torch.view_as_real(torch.view_as_complex(z) * turn)
        z = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        return torch.cat([z, n[..., rot:]], -1)

    outs = []
    for x, w, d in ((s["q"], s["qw"], s.get("dq")), (s["k"], s["kw"], s.get("dk"))):
        x = x.double().requires_grad_(back)
        w = None if w is None else w.double().requires_grad_(back)
        y = one(x, w)
        outs.append(torch.autograd.grad(y, [x] + ([] if w is None else [w]), d.double()) if back else y)
    if not back:
        return tuple(outs)
    (dq, *dqw), (dk, *dkw) = outs
    return {"dq": dq, "dk": dk, "dq_weight": dqw[0] if dqw else None, "dk_weight": dkw[0] if dkw else None}
