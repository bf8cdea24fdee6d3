"""Cases, plain forms and 64-bit values of the head-decay linear attention and of the gated group norm.

The operators (per batch row b and head h, N key and P value channels, state S of N x P):

  linear attention   S_t = exp(g_t) S_{t-1} + k_t v_t^T,  y_t = scale * q_t S_t     ("fwd", its gradient "bwd",
                     and one token in place on a pool of states "step")
  group norm         n = (x - mean) * rstd * weight + bias over groups of adjacent channels of one token,
                     out = n * silu(z), silu(n), or the norm of x * silu(z)          ("norm", its gradient "dnorm")

q and k have G heads, each shared by H / G of the H heads of v.  g is one f32 log decay per token and head, or one
per head.  lengths, where given, cuts each batch row: later tokens give zeros and leave the state alone.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CHUNK = 128  # tokens per chunk of the plain chunked form


def listed():
    return [
        # the next turn of one conversation: a few dozen tokens after a kept state, where latency counts
        dict(name="fwd-turn", op="fwd", io="bf16", B=1, L=37, H=16, G=1, N=128, P=64, decay="token", h0=True,
             ragged=False, packed=True),
        # prompt of a layer of 5120 channels in heads of 64 that share one q/k, sliced from one projection
        dict(name="fwd-layer", op="fwd", io="bf16", B=4, L=4096, H=80, G=1, N=128, P=64, decay="token", h0=False,
             ragged=False, packed=True),
        # one very long sequence, 1024 channels, a fixed decay per head, q/k of every head its own
        dict(name="fwd-long", op="fwd", io="bf16", B=1, L=131072, H=16, G=16, N=64, P=64, decay="head", h0=False,
             ragged=False, packed=False),
        # padded batch of prompts of unequal length (one of them empty) that continue kept states
        dict(name="fwd-ragged-f16", op="fwd", io="f16", B=8, L=2047, H=20, G=4, N=64, P=128, decay="token", h0=True,
             ragged=True, packed=False),
        # full-precision prompt of 1536 channels
        dict(name="fwd-f32", op="fwd", io="f32", B=2, L=1000, H=24, G=24, N=64, P=64, decay="token", h0=False,
             ragged=False, packed=False),
        # training step of the 5120-channel layer
        dict(name="bwd-layer", op="bwd", io="bf16", B=2, L=4096, H=80, G=1, N=128, P=64, decay="token", h0=False,
             ragged=False, packed=True),
        # small half-precision training batch, padded, with the gradient of one decay per head
        dict(name="bwd-ragged-f16", op="bwd", io="f16", B=3, L=509, H=8, G=2, N=64, P=80, decay="head", h0=True,
             ragged=True, packed=False),
        # full-precision gradient of a sequence segment between two others (state gradients in and out)
        dict(name="bwd-f32", op="bwd", io="f32", B=1, L=777, H=16, G=4, N=32, P=64, decay="token", h0=True,
             ragged=False, packed=False),
        # one token of one sequence
        dict(name="step-one", op="step", io="bf16", B=1, H=24, G=1, N=128, P=64, decay="token", pool=4),
        # one token of each of 256 running sequences, their states anywhere in a larger pool
        dict(name="step-batch", op="step", io="bf16", B=256, H=80, G=1, N=128, P=64, decay="token", pool=300),
        # output norm of the 5120-channel layer's prompt, one group per head, gated
        dict(name="norm-layer", op="norm", io="bf16", M=16384, C=5120, groups=80, mode="gate", center=True),
        # its gradient in training
        dict(name="dnorm-layer", op="dnorm", io="bf16", M=8192, C=5120, groups=80, mode="gate", center=True),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n - (n == 3072)


def draw(rng):
    op = rng.choice(("fwd", "fwd", "fwd", "bwd", "bwd", "bwd", "step", "norm", "dnorm"))
    io = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op in ("norm", "dnorm"):
        groups = rng.choice((1, 2, 8, 16, 20, 80))
        per = rng.choice((32, 64, 72, 80, 128, 256)) if groups > 2 else rng.choice((768, 1024, 1280, 2560, 5120))
        m = _log(rng, 1, max(1, 40_000_000 // (groups * per)))
        return dict(op=op, io=io, M=m, C=groups * per, groups=groups, mode=rng.choice(("gate", "act", "gate_first")),
                    center=rng.choice((True, False)))
    G = rng.choice((1, 1, 2, 4, 8))
    H = G * rng.choice((1, 2, 5, 8, 16))
    N = rng.choice((16, 32, 64, 64, 128, 128))
    P = rng.choice((32, 64, 64, 80, 128))
    decay = rng.choice(("token", "token", "head"))
    if op == "step":
        B = _log(rng, 1, max(1, min(600, 160_000_000 // (H * N * P))))
        return dict(op=op, io=io, B=B, H=H, G=G, N=N, P=P, decay=decay, pool=B + rng.randrange(0, 9))
    most = 120_000_000 // (H * (N + P)) // (1 if op == "fwd" else 4)  # tokens
    L = min(_log(rng, 1, 20000), most)
    B = max(1, min(_log(rng, 1, 8), most // L))
    return dict(op=op, io=io, B=B, L=L, H=H, G=G, N=N, P=P, decay=decay, h0=rng.choice((True, False)),
                ragged=rng.choice((True, False)), packed=rng.choice((True, False)))


def _decay(case, gen, shape, dev):
    """Log decays: -dt * A with dt log-uniform in [1e-3, 1e-1] and A in [1, 16] per head, or one per head that
    forgets over 2^5 to 2^12 tokens."""
    H = case["H"]
    if case["decay"] == "head":
        t = torch.arange(H, dtype=torch.float32, device=dev) / max(H, 1)
        r = torch.rand(H, generator=gen, device=dev)
        return torch.log1p(-torch.exp2(-(5 + 6 * t + r)))
    A = 1 + 15 * torch.rand(H, generator=gen, device=dev)
    dt = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(shape, generator=gen, device=dev))
    return -dt * A


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    io = DTYPES[case["io"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    s = {"case": case}
    if case["op"] in ("norm", "dnorm"):
        M, C = case["M"], case["C"]
        s["x"] = (2 * normal(M, C) + 0.3).to(io)
        s["z"] = normal(M, C).to(io) if case["mode"] != "act" else None
        s["weight"] = 1 + 0.2 * normal(C)
        s["bias"] = 0.1 * normal(C)
        if case["op"] == "dnorm":
            s["dout"] = normal(M, C).to(io)
        return s
    B, H, G, N, P = (case[k] for k in "BHGNP")
    s["scale"] = 1.0 / math.sqrt(N)
    if case["op"] == "step":
        s["q"], s["k"], s["v"] = normal(B, G, N).to(io), normal(B, G, N).to(io), normal(B, H, P).to(io)
        s["g"] = _decay(case, gen, (B, H), dev)
        s["state"] = 3 * normal(case["pool"], H, N, P)
        s["slots"] = torch.randperm(case["pool"], generator=gen, device=dev)[:B].to(torch.int32)
        return s
    L = case["L"]
    if case["packed"]:
        x = normal(B, L, H * P + 2 * G * N).to(io)
        s["v"] = x[:, :, :H * P].unflatten(2, (H, P))
        s["k"] = x[:, :, H * P:H * P + G * N].unflatten(2, (G, N))
        s["q"] = x[:, :, H * P + G * N:].unflatten(2, (G, N))
    else:
        s["q"], s["k"], s["v"] = normal(B, L, G, N).to(io), normal(B, L, G, N).to(io), normal(B, L, H, P).to(io)
    s["g"] = _decay(case, gen, (B, L, H), dev)
    s["h0"] = normal(B, H, N, P) if case["h0"] else None
    s["lengths"] = None
    if case["ragged"]:
        lengths = torch.randint(0, L + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        lengths[0] = L
        if B > 1:
            lengths[-1] = 0
        s["lengths"] = lengths
    if case["op"] == "bwd":
        s["dy"] = normal(B, L, H, P).to(io)
        s["dlast"] = normal(B, H, N, P) if case["h0"] else None
    return s


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    import mamba_selective_scan_fwd_gb300 as ss

    op = s["case"]["op"]
    if op == "fwd":
        return ss.ss_la_fwd(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], h0=s["h0"], lengths=s["lengths"])
    if op == "bwd":
        return ss.ss_la_bwd(s["q"], s["k"], s["v"], s["g"], s["dy"], scale=s["scale"], h0=s["h0"],
                            dlast_state=s["dlast"], lengths=s["lengths"])
    if op == "step":
        y = ss.ss_la_step(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"], slots=s["slots"])
        return {"y": y, "state": s["state"]}
    kind = dict(z=s["z"], groups=s["case"]["groups"], center=s["case"]["center"],
                gate_first=s["case"]["mode"] == "gate_first")
    if op == "norm":
        return ss.ss_gnorm_fwd(s["x"], s["weight"], s["bias"], **kind)
    return ss.ss_gnorm_bwd(s["x"], s["weight"], s["bias"], s["dout"], **kind)


# ------------------------------------------------------------------ plain forms (32 bits)

def _segments(g):
    """sum of g over (j, i] for j <= i and -inf for j > i, of the last axis: [..., T] -> [..., T, T] (i, j).
    Summed over each segment itself, so that a long sequence's sums do not cancel."""
    T = g.shape[-1]
    x = g.unsqueeze(-1).expand(*g.shape, T)
    low = torch.ones(T, T, dtype=torch.bool, device=g.device).tril(-1)
    x = torch.cumsum(x.masked_fill(~low, 0.0), -2)
    return x.masked_fill(~torch.ones(T, T, dtype=torch.bool, device=g.device).tril(), -math.inf)


def _chunked(s):
    """The inputs in 32 bits, cut into chunks: q, k, v [B, c, T, H, .], g [B, c, H, T]; zero past each length."""
    q, k, v, g = s["q"].float(), s["k"].float(), s["v"].float(), s["g"]
    B, L, H, P = v.shape
    T = min(CHUNK, max(1, L))
    pad = -L % T
    g = g.expand(B, L, H)
    if s["lengths"] is not None:
        on = torch.arange(L, device=v.device) < s["lengths"].unsqueeze(1)
        q, k, v = (t.masked_fill(~on[:, :, None, None], 0.0) for t in (q, k, v))
        g = g.masked_fill(~on[:, :, None], 0.0)

    def cut(t):
        t = torch.nn.functional.pad(t, (0, 0) * (t.dim() - 2) + (0, pad))
        return t.unflatten(1, (-1, T))

    rep = H // q.shape[2]
    q, k = cut(q).repeat_interleave(rep, 3), cut(k).repeat_interleave(rep, 3)
    return q, k, cut(v), cut(g).transpose(2, 3), cut


def _states(k, v, g, h0):
    """States before each chunk and after the last: [B, c + 1, H, N, P]."""
    cum = torch.cumsum(g, -1)
    total = cum[..., -1]
    w = torch.exp(total.unsqueeze(-1) - cum)
    new = torch.einsum("bcthn,bcht,bcthp->bchnp", k, w, v)
    if h0 is None:
        h0 = torch.zeros_like(new[:, 0])
    new = torch.cat([h0.unsqueeze(1), new], 1)
    d = torch.exp(_segments(torch.nn.functional.pad(total, (0, 0, 1, 0)).transpose(1, 2)))
    return torch.einsum("bhij,bjhnp->bihnp", d, new)


def _plain_fwd(s):
    q, k, v, g, _ = _chunked(s)
    B, L, H, P = s["v"].shape
    states = _states(k, v, g, s["h0"])
    inside = torch.einsum("bcihn,bcjhn->bchij", q, k) * torch.exp(_segments(g))
    y = torch.einsum("bchij,bcjhp->bcihp", inside, v)
    del inside
    decay = torch.exp(torch.cumsum(g, -1)).transpose(2, 3).unsqueeze(-1)
    y = s["scale"] * (y + decay * torch.einsum("bcihn,bchnp->bcihp", q, states[:, :-1]))
    return y.flatten(1, 2)[:, :L].to(s["v"].dtype), states[:, -1].contiguous()


def _plain_bwd(s):
    q, k, v, g, cut = _chunked(s)
    B, L, H, P = s["v"].shape
    G, N = s["q"].shape[2:]
    scale = s["scale"]
    dy = s["dy"].float()
    if s["lengths"] is not None:
        on = torch.arange(L, device=dy.device) < s["lengths"].unsqueeze(1)
        dy = dy.masked_fill(~on[:, :, None, None], 0.0)
    dy = cut(dy)
    before = _states(k, v, g, s["h0"])[:, :-1]
    cum = torch.cumsum(g, -1)
    total = cum[..., -1]
    up = torch.exp(cum).transpose(2, 3).unsqueeze(-1)                              # from the chunk's start
    down = torch.exp(total.unsqueeze(-1) - cum).transpose(2, 3).unsqueeze(-1)      # to its end
    # adjoints of the states after each chunk, last chunk first, then of the state before the first
    add = scale * torch.einsum("bcthn,bcthp->bchnp", q * up, dy).flip(1)
    last = torch.zeros_like(add[:, 0]) if s["dlast"] is None else s["dlast"]
    add = torch.cat([last.unsqueeze(1), add], 1)
    d = torch.exp(_segments(torch.nn.functional.pad(total.flip(1), (0, 0, 1, 0)).transpose(1, 2)))
    adj = torch.einsum("bhij,bjhnp->bihnp", d, add).flip(1)
    dh0, after = adj[:, 0], adj[:, 1:]
    m = scale * torch.exp(_segments(g))
    qk = torch.einsum("bcihn,bcjhn->bchij", q, k)
    e = torch.einsum("bcihp,bcjhp->bchij", dy, v) * m
    dv = torch.einsum("bchij,bcihp->bcjhp", qk * m, dy)
    spans = e * qk
    del qk, m
    dq = torch.einsum("bchij,bcjhn->bcihn", e, k)
    dk = torch.einsum("bchij,bcihn->bcjhn", e, q)
    del e
    from_before = scale * up * torch.einsum("bchnp,bcihp->bcihn", before, dy)
    to_after = down * torch.einsum("bchnp,bcjhp->bcjhn", after, v)
    dv = dv + down * torch.einsum("bchnp,bcjhn->bcjhp", after, k)
    a = (q * from_before).sum(-1).transpose(2, 3)
    b = (k * to_after).sum(-1).transpose(2, 3)
    through = torch.exp(total) * (before * after).sum((-1, -2))
    # dg_t: everything that reaches across token t, by its two ends
    low = torch.cumsum(spans, -1)                                                  # sum over j <= column
    low = torch.nn.functional.pad(low, (1, 0))[..., :-1]                           # sum over j < column
    dg = low.flip(-2).cumsum(-2).flip(-2).diagonal(dim1=-2, dim2=-1)               # and over i >= t, at t
    dg = dg + a.flip(-1).cumsum(-1).flip(-1) + torch.cumsum(b, -1) - b + through.unsqueeze(-1)
    dg = dg.transpose(2, 3).flatten(1, 2)[:, :L]
    if s["lengths"] is not None:
        dg = dg.masked_fill(~on[:, :, None], 0.0)
    io = s["v"].dtype

    def whole(t, heads, width):
        t = t.flatten(1, 2)[:, :L]
        return t.unflatten(2, (heads, -1)).sum(3).to(io) if heads != H else t.to(io)

    return {"dq": whole(dq + from_before, G, N), "dk": whole(dk + to_after, G, N), "dv": whole(dv, H, P),
            "dg": dg.sum((0, 1)) if s["g"].dim() == 1 else dg.contiguous(),
            "dh0": None if s["h0"] is None else dh0.contiguous()}


def _plain_step(s):
    rep = s["v"].shape[1] // s["q"].shape[1]
    q, k = s["q"].float().repeat_interleave(rep, 1), s["k"].float().repeat_interleave(rep, 1)
    at = s["slots"].long()
    a = torch.exp(s["g"]).expand(q.shape[:2])[:, :, None, None]
    new = a * s["state"][at] + k.unsqueeze(-1) * s["v"].float().unsqueeze(-2)
    s["state"][at] = new
    y = s["scale"] * torch.einsum("bhn,bhnp->bhp", q, new)
    return {"y": y.to(s["v"].dtype), "state": s["state"]}


EPS = 1e-5


def _normed(x, case):
    x = x.unflatten(1, (case["groups"], -1))
    if case["center"]:
        x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return (x * rstd).flatten(1), rstd


def _plain_norm(s):
    case, x, z = s["case"], s["x"].float(), s["z"]
    f = None if z is None else z.float() * torch.sigmoid(z.float())
    if case["mode"] == "gate_first":
        x = x * f
    n = _normed(x, case)[0] * s["weight"] + s["bias"]
    if case["mode"] == "gate":
        n = n * f
    if case["mode"] == "act":
        n = n * torch.sigmoid(n)
    return n.to(s["x"].dtype)


def _plain_dnorm(s):
    case, x, z, d = s["case"], s["x"].float(), s["z"], s["dout"].float()
    io = s["x"].dtype
    dz = None
    if z is not None:
        zf = z.float()
        sig = torch.sigmoid(zf)
        f, df = zf * sig, sig * (1 + zf * (1 - sig))
    u = x * f if case["mode"] == "gate_first" else x
    xhat, rstd = _normed(u, case)
    n = xhat * s["weight"] + s["bias"]
    if case["mode"] == "gate":
        dz = (d * n * df).to(io)
        d = d * f
    if case["mode"] == "act":
        sig = torch.sigmoid(n)
        d = d * sig * (1 + n * (1 - sig))
    dw, db = (d * xhat).sum(0), d.sum(0)
    t = (d * s["weight"]).unflatten(1, (case["groups"], -1))
    xg = xhat.unflatten(1, (case["groups"], -1))
    du = t - xg * (t * xg).mean(-1, keepdim=True)
    if case["center"]:
        du = du - t.mean(-1, keepdim=True)
    du = (du * rstd).flatten(1)
    if case["mode"] == "gate_first":
        dz = (du * x * df).to(io)
        du = du * f
    return {"dx": du.to(io), "dz": dz, "dweight": dw, "dbias": db}


def run(state):
    if own:
        return _run_own(state)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm": _plain_norm,
            "dnorm": _plain_dnorm}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    e = 4 if case["io"] == "f32" else 2
    if case["op"] in ("norm", "dnorm"):
        n = case["M"] * case["C"]
        wide = (2 if case["op"] == "norm" else 3) + (0 if case["mode"] == "act" else 1 if case["op"] == "norm" else 2)
        return {"bytes": wide * e * n + 4 * case["C"] * (2 if case["op"] == "norm" else 4),
                "flops": (12 if case["op"] == "norm" else 30) * n}
    B, H, G, N, P = (case[k] for k in "BHGNP")
    if case["op"] == "step":
        return {"bytes": 8 * B * H * N * P + e * B * (2 * G * N + 2 * H * P) + 4 * H * (B if case["decay"] == "token" else 1),
                "flops": 5 * B * H * N * P}
    L = case["L"]
    g = 4 * H * (B * L if case["decay"] == "token" else 1)
    state = 4 * B * H * N * P
    if case["op"] == "fwd":
        return {"bytes": e * B * L * (2 * G * N + 2 * H * P) + g + state * (2 if case["h0"] else 1),
                "flops": 4 * B * L * H * N * P}
    return {"bytes": e * B * L * (4 * G * N + 3 * H * P) + 2 * g + state * (3 if case["h0"] else 0),
            "flops": 10 * B * L * H * N * P}


# ------------------------------------------------------------------ 64 bits, token by token

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "dnorm"):
        return _exact_norm(case, s)
    if case["op"] == "step":
        return _exact_step(case, s)
    if case["B"] * case["L"] * case["H"] * case["N"] * case["P"] > 12_000_000_000:
        return None
    q, k, v = (s[n].double() for n in "qkv")
    B, L, H, P = v.shape
    G, N = q.shape[2:]
    of = torch.arange(H, device=v.device) // (H // G)
    a = torch.exp(s["g"].double()).expand(B, L, H)
    n = torch.full((B,), L, device=v.device) if s["lengths"] is None else s["lengths"].long()
    S = torch.zeros(B, H, N, P, dtype=torch.float64, device=v.device) if s["h0"] is None else s["h0"].double()
    back = case["op"] == "bwd"
    dy = s["dy"].double() if back else None
    out = torch.zeros(B, L, H, N if back else P, dtype=torch.float64, device=v.device)
    full = s["lengths"] is None
    for t in range(L):
        new = S * a[:, t, :, None, None]
        new.addcmul_(k[:, t][:, of].unsqueeze(-1), v[:, t].unsqueeze(-2))
        S = new if full else torch.where((t < n)[:, None, None, None], new, S)
        if back:
            out[:, t] = (S * dy[:, t].unsqueeze(-2)).sum(-1)
        else:
            out[:, t] = (S * q[:, t][:, of].unsqueeze(-1)).sum(-2)
    on = (torch.arange(L, device=v.device) < n.unsqueeze(1))[:, :, None, None]
    out = s["scale"] * out * on
    if not back:
        return out, S
    R = torch.zeros_like(S) if s["dlast"] is None else s["dlast"].double()
    end = (R * S).sum((-1, -2))
    dk, dv = torch.zeros(B, L, H, N, dtype=torch.float64, device=v.device), torch.zeros_like(v)
    for t in reversed(range(L)):
        new = torch.addcmul(R, s["scale"] * q[:, t][:, of].unsqueeze(-1), dy[:, t].unsqueeze(-2))
        R = new if full else torch.where((t < n)[:, None, None, None], new, R)
        dk[:, t] = (R * v[:, t].unsqueeze(-2)).sum(-1)
        dv[:, t] = (R * k[:, t][:, of].unsqueeze(-1)).sum(-2)
        new = R * a[:, t, :, None, None]
        R = new if full else torch.where((t < n)[:, None, None, None], new, R)
    dk, dv = dk * on, dv * on
    # in 64 bits the difference of the two ends' sums loses nothing that shows
    dg = (q[:, :, of] * out - k[:, :, of] * dk).sum(-1).flip(1).cumsum(1).flip(1) + end.unsqueeze(1)
    dg = dg * on[..., 0]
    return {"dq": out.unflatten(2, (G, -1)).sum(3), "dk": dk.unflatten(2, (G, -1)).sum(3), "dv": dv,
            "dg": dg.sum((0, 1)) if s["g"].dim() == 1 else dg, "dh0": None if s["h0"] is None else R}


def _exact_step(case, s):
    per = case["H"] // case["G"]
    state = s["state"].double()
    at = s["slots"].long()
    q, k = (s[n].double().unsqueeze(2).expand(-1, -1, per, -1).flatten(1, 2) for n in "qk")
    new = state[at] * torch.exp(s["g"].double()).expand(case["B"], case["H"])[..., None, None]
    new = new + k[..., None] * s["v"].double()[..., None, :]
    state[at] = new
    return {"y": s["scale"] * (new * q[..., None]).sum(-2), "state": state}


def _exact_norm(case, s):
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    if case["op"] == "dnorm":
        x, w, b = x.requires_grad_(), w.requires_grad_(), b.requires_grad_()
    z = None if s["z"] is None else s["z"].double().requires_grad_(case["op"] == "dnorm")
    u = x * z / (1 + torch.exp(-z)) if case["mode"] == "gate_first" else x
    u = u.reshape(x.shape[0], case["groups"], -1)
    mean = u.sum(-1, keepdim=True) / u.shape[-1] if case["center"] else 0.0
    var = ((u - mean) ** 2).sum(-1, keepdim=True) / u.shape[-1]
    n = ((u - mean) / torch.sqrt(var + EPS)).reshape(x.shape) * w + b
    out = n / (1 + torch.exp(-n)) if case["mode"] == "act" else n * z / (1 + torch.exp(-z)) if case["mode"] == "gate" else n
    if case["op"] == "norm":
        return out
    want = [x, w, b] + ([] if z is None else [z])
    got = torch.autograd.grad(out, want, s["dout"].double())
    return {"dx": got[0], "dz": None if z is None else got[3], "dweight": got[1], "dbias": got[2]}
