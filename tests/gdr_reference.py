"""64-bit references of the gated delta rule (token by token) and of the q / k norm with rotation,
and inputs for both."""

import numpy as np


def gdr_inputs(Bsz, L, H, G, N, P, gate=True, h0=True, seed=0):
    """q, k of about unit length, rates in (0, 1), decays between none and a few tokens' memory."""
    rng = np.random.default_rng(seed)

    def unit(*shape):
        x = rng.normal(size=shape)
        return x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6)

    x = {"q": unit(Bsz, L, G, N), "k": unit(Bsz, L, G, N), "v": rng.normal(size=(Bsz, L, H, P)),
         "g": -np.exp(rng.uniform(np.log(1e-3), np.log(1.0), size=(Bsz, L, H))) if gate else None,
         "beta": rng.uniform(0.05, 0.95, size=(Bsz, L, H)),
         "h0": rng.normal(size=(Bsz, H, N, P)) if h0 else None,
         "dy": rng.normal(size=(Bsz, L, H, P)), "dlast": rng.normal(size=(Bsz, H, N, P)) if h0 else None}
    return {k: None if v is None else v.astype(np.float32) for k, v in x.items()}


def _rows(q, k, v, g, beta, lengths):
    """Heads spread out, and what each token does: rates and log decays zero past the lengths."""
    Bsz, L, H, _ = v.shape
    rep = H // q.shape[2]
    q, k = np.repeat(np.asarray(q, np.float64), rep, 2), np.repeat(np.asarray(k, np.float64), rep, 2)
    v, beta = np.array(v, np.float64), np.array(beta, np.float64)
    g = np.zeros((Bsz, L, H)) if g is None else np.array(g, np.float64)
    on = np.ones((Bsz, L), bool)
    if lengths is not None:
        on = np.arange(L) < np.clip(np.asarray(lengths), 0, L)[:, None]
        q, k, v = (np.where(on[:, :, None, None], x, 0.0) for x in (q, k, v))
        g, beta = (np.where(on[:, :, None], x, 0.0) for x in (g, beta))
    return q, k, v, np.exp(g), beta, on


def _walk(q, k, v, a, beta, h0):
    """States after each token (index t + 1; 0: the start), u and v - a S^T k."""
    Bsz, L, H, P = v.shape
    S = [np.zeros((Bsz, H, q.shape[3], P)) if h0 is None else np.asarray(h0, np.float64)]
    us, misses = [], []
    for t in range(L):
        old = a[:, t, :, None, None] * S[-1]
        miss = v[:, t] - np.einsum("bhn,bhnp->bhp", k[:, t], old)
        u = beta[:, t, :, None] * miss
        S.append(old + k[:, t, :, :, None] * u[:, :, None, :])
        us.append(u)
        misses.append(miss)
    return S, us, misses


def gdr_fwd(q, k, v, g, beta, scale, h0=None, lengths=None):
    q, k, v, a, beta, on = _rows(q, k, v, g, beta, lengths)
    S, _, _ = _walk(q, k, v, a, beta, h0)
    y = np.zeros_like(v)
    for t in range(v.shape[1]):
        y[:, t] = scale * np.einsum("bhn,bhnp->bhp", q[:, t], S[t + 1])
    return y, S[-1]


def gdr_bwd(q, k, v, g, beta, dy, scale, h0=None, dlast=None, lengths=None):
    G, gated = np.asarray(q).shape[2], g is not None
    q, k, v, a, beta, on = _rows(q, k, v, g, beta, lengths)
    dy = np.where(on[:, :, None, None], np.asarray(dy, np.float64), 0.0)
    S, us, misses = _walk(q, k, v, a, beta, h0)
    Bsz, L, H, P = v.shape
    R = np.zeros_like(S[0]) if dlast is None else np.array(dlast, np.float64)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg, dbeta = np.zeros_like(beta), np.zeros_like(beta)
    for t in reversed(range(L)):
        dq[:, t] = scale * np.einsum("bhnp,bhp->bhn", S[t + 1], dy[:, t])
        R = R + scale * q[:, t, :, :, None] * dy[:, t, :, None, :]
        x = np.einsum("bhn,bhnp->bhp", k[:, t], R)
        b, at = beta[:, t, :, None], a[:, t, :, None, None]
        dv[:, t] = b * x
        dbeta[:, t] = (x * misses[t]).sum(-1)
        dk[:, t] = np.einsum("bhnp,bhp->bhn", R, us[t]) - np.einsum("bhnp,bhp->bhn", at * S[t], b * x)
        R = at * (R - k[:, t, :, :, None] * (b * x)[:, :, None, :])
        dg[:, t] = (R * S[t]).sum((-1, -2))
    dk, dv, dg, dbeta = (np.where(on.reshape(on.shape + (1,) * (x.ndim - 2)), x, 0.0) for x in (dk, dv, dg, dbeta))

    def shared(x):
        return x.reshape(Bsz, L, G, H // G, -1).sum(3)

    return {"dq": shared(dq), "dk": shared(dk), "dv": dv, "dg": dg if gated else None, "dbeta": dbeta,
            "dh0": None if h0 is None else R}


def gdr_step(q, k, v, g, beta, state, scale, slots=None):
    """(y, the pool after the step)."""
    state = np.array(state, np.float64)
    rep = v.shape[1] // q.shape[1]
    q, k = np.repeat(np.asarray(q, np.float64), rep, 1), np.repeat(np.asarray(k, np.float64), rep, 1)
    y = np.zeros(v.shape)
    for b in range(v.shape[0]):
        s = b if slots is None else int(slots[b])
        if not 0 <= s < state.shape[0]:
            continue
        old = state[s] if g is None else np.exp(np.asarray(g[b], np.float64))[:, None, None] * state[s]
        u = np.asarray(beta[b], np.float64)[:, None] * (v[b] - np.einsum("hn,hnp->hp", k[b], old))
        state[s] = old + k[b][:, :, None] * u[:, None, :]
        y[b] = scale * np.einsum("hn,hnp->hp", q[b], state[s])
    return y, state


# ------------------------------------------------------------------ q / k norm, one of the two

def _turned(n, positions, freqs, interleaved, back=False):
    if freqs is None:
        return n
    pairs = len(freqs)
    angle = np.asarray(positions, np.float64)[:, :, None, None] * np.asarray(freqs, np.float64)
    c, s = np.cos(angle), np.sin(angle) * (-1 if back else 1)
    out = n.copy()
    first = np.arange(pairs) * (2 if interleaved else 1)
    second = first + (1 if interleaved else pairs)
    out[..., first] = n[..., first] * c - n[..., second] * s
    out[..., second] = n[..., second] * c + n[..., first] * s
    return out


def _rstd(x, l2, eps):
    m = (x * x).sum(-1, keepdims=True)
    return 1 / np.sqrt((m if l2 else m / x.shape[-1]) + eps)


def norm_fwd(x, weight, positions, freqs, l2, eps, interleaved):
    x = np.asarray(x, np.float64)
    n = x * _rstd(x, l2, eps)
    return _turned(n if weight is None else n * weight, positions, freqs, interleaved)


def norm_bwd(x, weight, dout, positions, freqs, l2, eps, interleaved):
    """(dx, dweight)"""
    x = np.asarray(x, np.float64)
    r = _rstd(x, l2, eps)
    n = x * r
    d = _turned(np.asarray(dout, np.float64), positions, freqs, interleaved, back=True)
    dw = None if weight is None else (d * n).sum((0, 1, 2))
    d = d if weight is None else d * weight
    m = (d * n).sum(-1, keepdims=True)
    return r * (d - n * (m if l2 else m / x.shape[-1])), dw
