"""Plain 64-bit numpy references of the linear attention and the gated group norm, token by
token from their definitions (no chunks, no cumulative decays)."""

from __future__ import annotations

import numpy as np


def la_inputs(Bsz, L, H, G, N, P, per_head=False, h0=False, seed=0):
    """f64 arrays with the layer's distributions: q, k, v, dy ~ N(0, 1), g = -dt A."""
    r = np.random.default_rng(seed)
    x = {"q": r.normal(size=(Bsz, L, G, N)), "k": r.normal(size=(Bsz, L, G, N)), "v": r.normal(size=(Bsz, L, H, P)),
         "dy": r.normal(size=(Bsz, L, H, P))}
    A = r.uniform(1, 16, size=H)
    dt = np.exp(r.uniform(np.log(1e-3), np.log(1e-1), size=(Bsz, L, H)))
    x["g"] = -0.02 * A if per_head else -dt * A
    x["h0"] = r.normal(size=(Bsz, H, N, P)) if h0 else None
    x["dlast"] = r.normal(size=(Bsz, H, N, P)) if h0 else None
    return x


def la_fwd(q, k, v, g, scale=1.0, h0=None, lengths=None):
    Bsz, L, H, P = v.shape
    G, N = q.shape[2:]
    of = np.arange(H) // (H // G)
    n = np.full(Bsz, L) if lengths is None else np.clip(lengths, 0, L)
    S = np.zeros((Bsz, H, N, P)) if h0 is None else h0.astype(np.float64).copy()
    y = np.zeros(v.shape)
    g = np.broadcast_to(g, (Bsz, L, H))
    for b in range(Bsz):
        for t in range(n[b]):
            S[b] = np.exp(g[b, t])[:, None, None] * S[b] + k[b, t, of][:, :, None] * v[b, t][:, None, :]
            y[b, t] = scale * np.einsum("hn,hnp->hp", q[b, t, of], S[b])
    return y, S


def la_bwd(q, k, v, g, dy, scale=1.0, h0=None, dlast=None, lengths=None):
    """Reverse walk with every state kept: dq, dk (per shared head), dv, dg, dh0."""
    Bsz, L, H, P = v.shape
    G, N = q.shape[2:]
    of = np.arange(H) // (H // G)
    n = np.full(Bsz, L) if lengths is None else np.clip(lengths, 0, L)
    gb = np.broadcast_to(g, (Bsz, L, H))
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dg = np.zeros((Bsz, L, H))
    dh0 = np.zeros((Bsz, H, N, P))
    for b in range(Bsz):
        S = [np.zeros((H, N, P)) if h0 is None else h0[b].astype(np.float64)]
        for t in range(n[b]):
            S.append(np.exp(gb[b, t])[:, None, None] * S[-1] + k[b, t, of][:, :, None] * v[b, t][:, None, :])
        R = np.zeros((H, N, P)) if dlast is None else dlast[b].astype(np.float64).copy()
        for t in reversed(range(n[b])):
            R = R + scale * q[b, t, of][:, :, None] * dy[b, t][:, None, :]
            np.add.at(dq[b, t], of, scale * np.einsum("hnp,hp->hn", S[t + 1], dy[b, t]))
            np.add.at(dk[b, t], of, np.einsum("hnp,hp->hn", R, v[b, t]))
            dv[b, t] = np.einsum("hnp,hn->hp", R, k[b, t, of])
            R = np.exp(gb[b, t])[:, None, None] * R
            dg[b, t] = np.sum(R * S[t], axis=(1, 2))
        dh0[b] = R
    return {"dq": dq, "dk": dk, "dv": dv, "dg": dg.sum((0, 1)) if g.ndim == 1 else dg, "dh0": dh0}


def _silu(z):
    s = 1 / (1 + np.exp(-z))
    return z * s, s * (1 + z * (1 - s))


def gnorm_fwd(x, weight, bias, z, groups, eps, center, gate_first):
    M, C = x.shape
    u = x * _silu(z)[0] if gate_first else x
    u = u.reshape(M, groups, -1)
    if center:
        u = u - u.mean(-1, keepdims=True)
    n = (u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)).reshape(M, C)
    n = n * (1 if weight is None else weight) + (0 if bias is None else bias)
    if z is None:
        return _silu(n)[0]
    return n if gate_first else n * _silu(z)[0]


def gnorm_bwd(x, weight, bias, dout, z, groups, eps, center, gate_first):
    M, C = x.shape
    w = np.ones(C) if weight is None else weight
    b = np.zeros(C) if bias is None else bias
    f, df = (None, None) if z is None else _silu(z)
    u = (x * f if gate_first else x).reshape(M, groups, -1)
    if center:
        u = u - u.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    xh = u * rstd
    n = xh.reshape(M, C) * w + b
    d, dz = dout, None
    if z is None:
        d = dout * _silu(n)[1]
    elif not gate_first:
        dz = dout * n * df
        d = dout * f
    t = (d * w).reshape(M, groups, -1)
    du = t - xh * (t * xh).mean(-1, keepdims=True)
    if center:
        du = du - t.mean(-1, keepdims=True)
    du = (du * rstd).reshape(M, C)
    dx = du
    if gate_first:
        dx, dz = du * f, du * x * df
    return {"dx": dx, "dz": dz, "dweight": (d * xh.reshape(M, C)).sum(0), "dbias": d.sum(0)}
