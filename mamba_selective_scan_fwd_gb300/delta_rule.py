"""Gated delta rule, and the norm with rotation of its queries and keys (C ABI in
include/ss_gdr.h).  Argument marshalling only, like ``binding``:

    u_t = beta_t (v_t - e^{g_t} S_{t-1}^T k_t),   S_t = e^{g_t} S_{t-1} + k_t u_t^T,   y_t = scale * q_t S_t

per batch row and head.  q, k are [Bsz, L, G, N], v is [Bsz, L, H, P] (f32, bf16 or f16; H / G
heads of v share a head of q and k), g (log decay, or None) and beta are f32 [Bsz, L, H]; states
are f32 [Bsz, H, N, P], laid out as ``linear_attention``'s, so that both may live in one pool.
"""

from __future__ import annotations

import ctypes
import functools

from .binding import _I32, _I64, _P, _SZ, _workspace, dtype_id, lib
from .linear_attention import _call, _gpu, _heads, _in_stream, _new, _optional, _sliced, _whole

QKNORM_L2, QKNORM_INTERLEAVED = 1, 2


class GdrFwdDesc(ctypes.Structure):
    """ss_gdr_fwd_desc of include/ss_gdr.h (same field order and types)."""
    _fields_ = [(n, _P) for n in ("q", "k", "v", "g", "beta", "h0", "lengths", "y", "last_state", "workspace")] + [
        ("workspace_bytes", _SZ)] + [
        (n, _I64) for n in ("q_token", "q_batch", "k_token", "k_batch", "v_token", "v_batch", "Bsz", "L", "H", "G", "N",
                            "P")] + [
        ("scale", ctypes.c_float), ("dtype", _I32)]


class GdrBwdDesc(ctypes.Structure):
    """ss_gdr_bwd_desc of include/ss_gdr.h (same field order and types)."""
    _fields_ = [(n, _P) for n in ("q", "k", "v", "g", "beta", "h0", "lengths", "dy", "dlast_state", "dq", "dk", "dv",
                                  "dg", "dbeta", "dh0", "workspace")] + [
        ("workspace_bytes", _SZ)] + [
        (n, _I64) for n in ("q_token", "q_batch", "k_token", "k_batch", "v_token", "v_batch", "dy_token", "dy_batch",
                            "Bsz", "L", "H", "G", "N", "P")] + [
        ("scale", ctypes.c_float), ("dtype", _I32)]


class GdrStepDesc(ctypes.Structure):
    """ss_gdr_step_desc of include/ss_gdr.h (same field order and types)."""
    _fields_ = [(n, _P) for n in ("q", "k", "v", "g", "beta", "state", "slots", "y")] + [
        (n, _I64) for n in ("q_batch", "k_batch", "v_batch", "Bsz", "H", "G", "N", "P", "pool")] + [
        ("scale", ctypes.c_float), ("dtype", _I32)]


class QkNormFwdDesc(ctypes.Structure):
    """ss_qknorm_fwd_desc of include/ss_gdr.h (same field order and types)."""
    _fields_ = [(n, _P) for n in ("q", "k", "q_weight", "k_weight", "positions", "freqs", "q_out", "k_out")] + [
        (n, _I64) for n in ("q_token", "q_batch", "k_token", "k_batch", "Bsz", "L", "Hq", "Hk", "N", "pairs")] + [
        ("eps", ctypes.c_float), ("flags", _I32), ("dtype", _I32), ("reserved", _I32)]


class QkNormBwdDesc(ctypes.Structure):
    """ss_qknorm_bwd_desc of include/ss_gdr.h (same field order and types)."""
    _fields_ = [(n, _P) for n in ("q", "k", "q_weight", "k_weight", "positions", "freqs", "dq_out", "dk_out", "dq", "dk",
                                  "dq_weight", "dk_weight", "workspace")] + [
        ("workspace_bytes", _SZ)] + [
        (n, _I64) for n in ("q_token", "q_batch", "k_token", "k_batch", "dq_token", "dq_batch", "dk_token", "dk_batch",
                            "Bsz", "L", "Hq", "Hk", "N", "pairs")] + [
        ("eps", ctypes.c_float), ("flags", _I32), ("dtype", _I32), ("reserved", _I32)]


@functools.lru_cache(maxsize=256)
def gdr_fwd_workspace_bytes(Bsz, L, H, G, N, P, dtype) -> int:
    return int(lib().ss_gdr_fwd_workspace_bytes(Bsz, L, H, G, N, P, dtype))


@functools.lru_cache(maxsize=256)
def gdr_bwd_workspace_bytes(Bsz, L, H, G, N, P, dtype) -> int:
    return int(lib().ss_gdr_bwd_workspace_bytes(Bsz, L, H, G, N, P, dtype))


@functools.lru_cache(maxsize=256)
def _qknorm_workspace_bytes(Bsz, L, Hq, Hk, N, dtype) -> int:
    return int(lib().ss_qknorm_bwd_workspace_bytes(Bsz, L, Hq, Hk, N, dtype))


def ss_gdr_fwd(q, k, v, g, beta, scale=1.0, h0=None, lengths=None, y=None, last_state=None, return_last_state=True,
               workspace=None, stream=None):
    """Gated delta rule over whole sequences.  ``g``: log decays, or None for the rule without a
    gate; ``h0``: state to start from; ``lengths`` (int32 [Bsz]): tokens of each row that count.
    q, k, v may be slices of one projection's output.  Returns (y, last_state or None)."""
    import torch

    if stream is not None:
        return _in_stream(stream, v, ss_gdr_fwd, q, k, v, g, beta, scale, h0, lengths, y, last_state, return_last_state,
                          workspace)
    Bsz, L, H, P = v.shape
    G, N = q.shape[2:]
    dev, io, f32 = v.device, v.dtype, torch.float32
    _heads(H, G)
    qs = _sliced(q, "q", (Bsz, L, G, N), io, dev)
    ks = _sliced(k, "k", (Bsz, L, G, N), io, dev)
    vs = _sliced(v, "v", (Bsz, L, H, P), io, dev)
    g_p = _optional(g, "g", (Bsz, L, H), f32, dev)
    _whole(beta, "beta", (Bsz, L, H), f32, dev)
    state = (Bsz, H, N, P)
    lengths_p = _optional(lengths, "lengths", (Bsz,), torch.int32, dev)
    h0_p = _optional(h0, "h0", state, f32, dev)
    _gpu(v)
    if y is None:
        y = _new(Bsz, L, H, P, io, dev)
    else:
        _whole(y, "y", (Bsz, L, H, P), io, dev)
    if last_state is None and return_last_state:
        last_state = _new(Bsz, H, N, P, f32, dev)
    last = _optional(last_state, "last_state", state, f32, dev)
    dt = dtype_id(v)
    workspace, wsb = _workspace(gdr_fwd_workspace_bytes(Bsz, L, H, G, N, P, dt), dev, workspace)
    d = GdrFwdDesc(q.data_ptr(), k.data_ptr(), v.data_ptr(), g_p, beta.data_ptr(), h0_p, lengths_p, y.data_ptr(), last,
                   None if workspace is None else workspace.data_ptr(), wsb, qs[1], qs[0], ks[1], ks[0], vs[1], vs[0],
                   Bsz, L, H, G, N, P, scale, dt)
    _call("ss_gdr_fwd", v, ctypes.byref(d))
    return y, last_state


def ss_gdr_bwd(q, k, v, g, beta, dy, scale=1.0, h0=None, dlast_state=None, lengths=None, out=None, workspace=None,
               stream=None):
    """Gradient of sum(dy * y) + sum(dlast_state * last_state).  Returns a dict: dq, dk (summed over
    the heads that share them) and dv in the io type, dg (None without g), dbeta and dh0 (None
    without h0) f32."""
    import torch

    if stream is not None:
        return _in_stream(stream, v, ss_gdr_bwd, q, k, v, g, beta, dy, scale, h0, dlast_state, lengths, out, workspace)
    Bsz, L, H, P = v.shape
    G, N = q.shape[2:]
    dev, io, f32 = v.device, v.dtype, torch.float32
    _heads(H, G)
    qs = _sliced(q, "q", (Bsz, L, G, N), io, dev)
    ks = _sliced(k, "k", (Bsz, L, G, N), io, dev)
    vs = _sliced(v, "v", (Bsz, L, H, P), io, dev)
    ys = _sliced(dy, "dy", (Bsz, L, H, P), io, dev)
    g_p = _optional(g, "g", (Bsz, L, H), f32, dev)
    _whole(beta, "beta", (Bsz, L, H), f32, dev)
    state = (Bsz, H, N, P)
    lengths_p = _optional(lengths, "lengths", (Bsz,), torch.int32, dev)
    h0_p = _optional(h0, "h0", state, f32, dev)
    dlast_p = _optional(dlast_state, "dlast_state", state, f32, dev)
    _gpu(v)
    shapes = {"dq": ((Bsz, L, G, N), io), "dk": ((Bsz, L, G, N), io), "dv": ((Bsz, L, H, P), io),
              "dg": ((Bsz, L, H), f32), "dbeta": ((Bsz, L, H), f32), "dh0": (state, f32)}
    absent = {"dg": g is None, "dh0": h0 is None}
    out = dict(out or {})
    for name, (shape, dtype) in shapes.items():
        if absent.get(name):
            out[name] = None
        elif out.get(name) is None:
            out[name] = torch.empty(shape, dtype=dtype, device=dev)
        else:
            _whole(out[name], name, shape, dtype, dev)
    ptr = {name: None if out[name] is None else out[name].data_ptr() for name in shapes}
    dt = dtype_id(v)
    workspace, wsb = _workspace(gdr_bwd_workspace_bytes(Bsz, L, H, G, N, P, dt), dev, workspace)
    d = GdrBwdDesc(q.data_ptr(), k.data_ptr(), v.data_ptr(), g_p, beta.data_ptr(), h0_p, lengths_p, dy.data_ptr(), dlast_p,
                   ptr["dq"], ptr["dk"], ptr["dv"], ptr["dg"], ptr["dbeta"], ptr["dh0"],
                   None if workspace is None else workspace.data_ptr(), wsb, qs[1], qs[0], ks[1], ks[0], vs[1], vs[0],
                   ys[1], ys[0], Bsz, L, H, G, N, P, scale, dt)
    _call("ss_gdr_bwd", v, ctypes.byref(d))
    return out


def ss_gdr_step(q, k, v, g, beta, state, scale=1.0, slots=None, y=None, stream=None):
    """One token of each sequence, in place on ``state`` [pool, H, N, P] f32: q, k [Bsz, G, N], v
    [Bsz, H, P], g (or None) and beta [Bsz, H].  ``slots`` (int32 [Bsz]): the state each row owns,
    -1 for a padding row (y = 0); without it row b owns state b.  Returns y [Bsz, H, P]."""
    import torch

    if stream is not None:
        return _in_stream(stream, v, ss_gdr_step, q, k, v, g, beta, state, scale, slots, y)
    Bsz, H, P = v.shape
    G, N = q.shape[1:]
    dev, io, f32 = v.device, v.dtype, torch.float32
    _heads(H, G)
    qs = _sliced(q, "q", (Bsz, G, N), io, dev)
    ks = _sliced(k, "k", (Bsz, G, N), io, dev)
    vs = _sliced(v, "v", (Bsz, H, P), io, dev)
    g_p = _optional(g, "g", (Bsz, H), f32, dev)
    _whole(beta, "beta", (Bsz, H), f32, dev)
    pool = state.shape[0]
    _whole(state, "state", (pool, H, N, P), f32, dev)
    if slots is None and pool < Bsz:
        raise ValueError(f"state holds {pool} states for {Bsz} rows")
    slots_p = _optional(slots, "slots", (Bsz,), torch.int32, dev)
    _gpu(v)
    if y is None:
        y = torch.empty_strided((Bsz, H, P), (H * P, P, 1), dtype=io, device=dev)
    else:
        _whole(y, "y", (Bsz, H, P), io, dev)
    d = GdrStepDesc(q.data_ptr(), k.data_ptr(), v.data_ptr(), g_p, beta.data_ptr(), state.data_ptr(), slots_p,
                    y.data_ptr(), qs[0], ks[0], vs[0], Bsz, H, G, N, P, pool, scale, dtype_id(v))
    _call("ss_gdr_step", v, ctypes.byref(d))
    return y


def _qknorm_prepare(q, k, q_weight, k_weight, positions, freqs, l2, interleaved):
    """Check what both directions share; returns the sizes, strides, pointers and flags."""
    import torch

    Bsz, L, Hq, N = q.shape
    Hk, dev, io, f32 = k.shape[2], q.device, q.dtype, torch.float32
    qs = _sliced(q, "q", (Bsz, L, Hq, N), io, dev)
    ks = _sliced(k, "k", (Bsz, L, Hk, N), io, dev)
    pairs = 0 if freqs is None else freqs.shape[0]
    if 2 * pairs > N:
        raise ValueError(f"{pairs} frequencies turn {2 * pairs} channels, heads have {N}")
    if positions is not None and freqs is None:
        raise ValueError("positions need freqs")
    pointers = (_optional(q_weight, "q_weight", (N,), f32, dev), _optional(k_weight, "k_weight", (N,), f32, dev),
                _optional(positions, "positions", (Bsz, L), torch.int32, dev),
                _optional(freqs, "freqs", (pairs,), f32, dev))
    _gpu(q)
    return (Bsz, L, Hq, Hk, N, pairs), qs, ks, pointers, (QKNORM_L2 if l2 else 0) | (QKNORM_INTERLEAVED if interleaved else 0)


def ss_qknorm_fwd(q, k, q_weight=None, k_weight=None, positions=None, freqs=None, l2=False, eps=1e-6, interleaved=False,
                  q_out=None, k_out=None, stream=None):
    """Norm of each head's channels of q [Bsz, L, Hq, N] and k [Bsz, L, Hk, N], then the rotation by
    position, in one pass.  The norm divides by the root of the mean square, or with ``l2`` by the
    length (|x| = 1 after it), and multiplies by the weight (f32 [N]).  ``freqs`` (f32 [pairs],
    radians a token): channels i and i + pairs (``interleaved``: 2 i and 2 i + 1) turn by position *
    freqs[i]; ``positions`` int32 [Bsz, L], token t stands at t without it.  N <= 256.
    q and k may be slices of one projection's output; q_out and k_out may be q and k.
    Returns (q_out, k_out)."""
    if stream is not None:
        return _in_stream(stream, q, ss_qknorm_fwd, q, k, q_weight, k_weight, positions, freqs, l2, eps, interleaved, q_out,
                          k_out)
    sizes, qs, ks, pointers, flags = _qknorm_prepare(q, k, q_weight, k_weight, positions, freqs, l2, interleaved)
    Bsz, L, Hq, Hk, N, pairs = sizes
    if q_out is None:
        q_out = _new(Bsz, L, Hq, N, q.dtype, q.device)
    else:
        _whole(q_out, "q_out", (Bsz, L, Hq, N), q.dtype, q.device)
    if k_out is None:
        k_out = _new(Bsz, L, Hk, N, q.dtype, q.device)
    else:
        _whole(k_out, "k_out", (Bsz, L, Hk, N), q.dtype, q.device)
    d = QkNormFwdDesc(q.data_ptr(), k.data_ptr(), *pointers, q_out.data_ptr(), k_out.data_ptr(), qs[1], qs[0], ks[1], ks[0],
                      *sizes, eps, flags, dtype_id(q), 0)
    _call("ss_qknorm_fwd", q, ctypes.byref(d))
    return q_out, k_out


def ss_qknorm_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, positions=None, freqs=None, l2=False, eps=1e-6,
                  interleaved=False, out=None, workspace=None, stream=None):
    """Gradient of sum(dq_out * q_out) + sum(dk_out * k_out) of ss_qknorm_fwd.  Returns a dict: dq, dk
    (io type) and dq_weight, dk_weight (f32, None without the weight)."""
    import torch

    if stream is not None:
        return _in_stream(stream, q, ss_qknorm_bwd, q, k, dq_out, dk_out, q_weight, k_weight, positions, freqs, l2, eps,
                          interleaved, out, workspace)
    sizes, qs, ks, pointers, flags = _qknorm_prepare(q, k, q_weight, k_weight, positions, freqs, l2, interleaved)
    Bsz, L, Hq, Hk, N, pairs = sizes
    dev, io, f32 = q.device, q.dtype, torch.float32
    dqs = _sliced(dq_out, "dq_out", (Bsz, L, Hq, N), io, dev)
    dks = _sliced(dk_out, "dk_out", (Bsz, L, Hk, N), io, dev)
    shapes = {"dq": ((Bsz, L, Hq, N), io), "dk": ((Bsz, L, Hk, N), io), "dq_weight": ((N,), f32), "dk_weight": ((N,), f32)}
    absent = {"dq_weight": q_weight is None, "dk_weight": k_weight is None}
    out = dict(out or {})
    for name, (shape, dtype) in shapes.items():
        if absent.get(name):
            out[name] = None
        elif out.get(name) is None:
            out[name] = torch.empty(shape, dtype=dtype, device=dev)
        else:
            _whole(out[name], name, shape, dtype, dev)
    ptr = {name: None if out[name] is None else out[name].data_ptr() for name in shapes}
    dt = dtype_id(q)
    workspace, wsb = _workspace(_qknorm_workspace_bytes(Bsz, L, Hq, Hk, N, dt), dev, workspace)
    d = QkNormBwdDesc(q.data_ptr(), k.data_ptr(), *pointers, dq_out.data_ptr(), dk_out.data_ptr(), ptr["dq"], ptr["dk"],
                      ptr["dq_weight"], ptr["dk_weight"], None if workspace is None else workspace.data_ptr(), wsb,
                      qs[1], qs[0], ks[1], ks[0], dqs[1], dqs[0], dks[1], dks[0], *sizes, eps, flags, dt, 0)
    _call("ss_qknorm_bwd", q, ctypes.byref(d))
    return out
