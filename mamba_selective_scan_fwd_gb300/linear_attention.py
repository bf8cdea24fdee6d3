"""Linear attention with one decay per head, and the gated group norm of its output
(C ABI in include/ss_la.h).  Argument marshalling only, like ``binding``:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,   y_t = scale * q_t S_t        per batch row and head

q, k are [Bsz, L, G, N], v is [Bsz, L, H, P] (f32, bf16 or f16; H / G heads of v share a head
of q and k), g is f32 [Bsz, L, H], or [H] for one decay per head; states are f32 [Bsz, H, N, P].
"""

from __future__ import annotations

import ctypes

from .binding import (_I32, _I64, _P, _SZ, _check, _nbytes, _on_device, _p, _require, _state_arg, _workspace, dtype_id,
                      lib, stream_handle)

GNORM_CENTER, GNORM_GATE_FIRST = 1, 2


class LaFwdDesc(ctypes.Structure):
    """ss_la_fwd_desc of include/ss_la.h (same field order and types)."""
    _fields_ = [(n, _P) for n in ("q", "k", "v", "g", "h0", "lengths", "y", "last_state", "workspace")] + [
        ("workspace_bytes", _SZ)] + [
        (n, _I64) for n in ("q_token", "q_batch", "k_token", "k_batch", "v_token", "v_batch", "Bsz", "L", "H", "G", "N",
                            "P")] + [
        ("scale", ctypes.c_float), ("dtype", _I32), ("g_per_head", _I32), ("reserved", _I32)]


class LaBwdDesc(ctypes.Structure):
    """ss_la_bwd_desc of include/ss_la.h (same field order and types)."""
    _fields_ = [(n, _P) for n in ("q", "k", "v", "g", "h0", "lengths", "dy", "dlast_state", "dq", "dk", "dv", "dg",
                                  "dh0", "workspace")] + [
        ("workspace_bytes", _SZ)] + [
        (n, _I64) for n in ("q_token", "q_batch", "k_token", "k_batch", "v_token", "v_batch", "dy_token", "dy_batch",
                            "Bsz", "L", "H", "G", "N", "P")] + [
        ("scale", ctypes.c_float), ("dtype", _I32), ("g_per_head", _I32), ("reserved", _I32)]


class LaStepDesc(ctypes.Structure):
    """ss_la_step_desc of include/ss_la.h (same field order and types)."""
    _fields_ = [(n, _P) for n in ("q", "k", "v", "g", "state", "slots", "y")] + [
        (n, _I64) for n in ("q_batch", "k_batch", "v_batch", "Bsz", "H", "G", "N", "P", "pool")] + [
        ("scale", ctypes.c_float), ("dtype", _I32), ("g_per_head", _I32), ("reserved", _I32)]


def la_fwd_workspace_bytes(Bsz, L, H, G, N, P, dtype) -> int:
    return int(lib().ss_la_fwd_workspace_bytes(Bsz, L, H, G, N, P, dtype))


def la_bwd_workspace_bytes(Bsz, L, H, G, N, P, dtype) -> int:
    return int(lib().ss_la_bwd_workspace_bytes(Bsz, L, H, G, N, P, dtype))


def _require_sliced(t, name, shape, dtype, device, inner):
    """Like _require, but only the last ``inner`` dimensions must be contiguous: the
    others may step over a wider tensor's other columns."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype} != {dtype}")
    want = 1
    for d in reversed(range(len(shape) - inner, len(shape))):
        if shape[d] > 1 and t.stride(d) != want:
            raise ValueError(f"{name}: the last {inner} dimensions must be contiguous")
        want *= shape[d]
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _set(desc, tensors):
    for name, t in tensors.items():
        setattr(desc, name, None if t is None else t.data_ptr())


def _set_strides(desc, tensors):
    for name, t in tensors.items():
        setattr(desc, f"{name}_batch", t.stride(0) if t.shape[0] > 1 else 0)
        if t.dim() == 4:
            setattr(desc, f"{name}_token", t.stride(1) if t.shape[1] > 1 else 0)


def _la_prepare(q, k, v, g, lengths):
    """Check the shared inputs of the forward and the backward; returns the sizes."""
    import torch

    Bsz, L, H, P = v.shape
    G, N = q.shape[2:]
    dev, io = v.device, v.dtype
    if G < 1 or H % G != 0:
        raise ValueError(f"{H} heads of v cannot share {G} heads of q and k evenly")
    _require_sliced(q, "q", (Bsz, L, G, N), io, dev, 2)
    _require_sliced(k, "k", (Bsz, L, G, N), io, dev, 2)
    _require_sliced(v, "v", (Bsz, L, H, P), io, dev, 2)
    _require(g, "g", (H,) if g.dim() == 1 else (Bsz, L, H), torch.float32, dev)
    if lengths is not None:
        _require(lengths, "lengths", (Bsz,), torch.int32, dev)
    return Bsz, L, H, G, N, P


def _set_sizes(d, sizes, scale, dtype, g):
    d.Bsz, d.L, d.H, d.G, d.N, d.P = sizes
    d.scale, d.dtype, d.g_per_head, d.reserved = float(scale), dtype, int(g.dim() == 1), 0


def ss_la_fwd(q, k, v, g, scale=1.0, h0=None, lengths=None, y=None, last_state=None, return_last_state=True,
              workspace=None, stream=None):
    """Linear attention over whole sequences.  ``h0``: state to start from; ``lengths`` (int32
    [Bsz]): tokens of each row that count.  q, k, v may be slices of one projection's output.
    Returns (y, last_state or None)."""
    import torch

    sizes = _la_prepare(q, k, v, g, lengths)
    Bsz, L, H, G, N, P = sizes
    dev, dt = v.device, dtype_id(v)
    _state_arg(h0, "h0", (Bsz, H, N, P), dev)
    if y is None:
        y = torch.empty((Bsz, L, H, P), dtype=v.dtype, device=dev)
    _require(y, "y", (Bsz, L, H, P), v.dtype, dev)
    if last_state is None and return_last_state:
        last_state = torch.empty((Bsz, H, N, P), dtype=torch.float32, device=dev)
    _state_arg(last_state, "last_state", (Bsz, H, N, P), dev)
    with _on_device(v, stream):
        workspace, wsb = _workspace(la_fwd_workspace_bytes(*sizes, dt), dev, workspace)
        d = LaFwdDesc()
        _set(d, dict(q=q, k=k, v=v, g=g, h0=h0, lengths=lengths, y=y, last_state=last_state, workspace=workspace))
        _set_strides(d, dict(q=q, k=k, v=v))
        _set_sizes(d, sizes, scale, dt, g)
        d.workspace_bytes = wsb
        rc = lib().ss_la_fwd(ctypes.byref(d), stream_handle(stream, dev))
    _check("ss_la_fwd", rc)
    return y, last_state


def ss_la_bwd(q, k, v, g, dy, scale=1.0, h0=None, dlast_state=None, lengths=None, out=None, workspace=None,
              stream=None):
    """Gradient of sum(dy * y) + sum(dlast_state * last_state).  Returns a dict: dq, dk (summed over
    the heads that share them) and dv in the io type, dg (g's shape) and dh0 (None without h0) f32."""
    import torch

    sizes = _la_prepare(q, k, v, g, lengths)
    Bsz, L, H, G, N, P = sizes
    dev, dt, f32 = v.device, dtype_id(v), torch.float32
    _require_sliced(dy, "dy", (Bsz, L, H, P), v.dtype, dev, 2)
    _state_arg(h0, "h0", (Bsz, H, N, P), dev)
    _state_arg(dlast_state, "dlast_state", (Bsz, H, N, P), dev)
    shapes = {"dq": ((Bsz, L, G, N), v.dtype), "dk": ((Bsz, L, G, N), v.dtype), "dv": ((Bsz, L, H, P), v.dtype),
              "dg": (tuple(g.shape), f32), "dh0": ((Bsz, H, N, P), f32)}
    out = dict(out or {})
    for name, (shape, dtype) in shapes.items():
        if name == "dh0" and h0 is None:
            out[name] = None
            continue
        if out.get(name) is None:
            out[name] = torch.empty(shape, dtype=dtype, device=dev)
        _require(out[name], name, shape, dtype, dev)
    with _on_device(v, stream):
        workspace, wsb = _workspace(la_bwd_workspace_bytes(*sizes, dt), dev, workspace)
        d = LaBwdDesc()
        _set(d, dict(q=q, k=k, v=v, g=g, h0=h0, lengths=lengths, dy=dy, dlast_state=dlast_state, workspace=workspace,
                     **{n: out[n] for n in shapes}))
        _set_strides(d, dict(q=q, k=k, v=v, dy=dy))
        _set_sizes(d, sizes, scale, dt, g)
        d.workspace_bytes = wsb
        rc = lib().ss_la_bwd(ctypes.byref(d), stream_handle(stream, dev))
    _check("ss_la_bwd", rc)
    return out


def ss_la_step(q, k, v, g, state, scale=1.0, slots=None, y=None, stream=None):
    """One token of each sequence, in place on ``state`` [pool, H, N, P] f32: q, k [Bsz, G, N], v
    [Bsz, H, P], g [Bsz, H] or [H].  ``slots`` (int32 [Bsz]): the state each row owns, -1 for a
    padding row (y = 0); without it row b owns state b.  Returns y [Bsz, H, P]."""
    import torch

    Bsz, H, P = v.shape
    G, N = q.shape[1:]
    dev, io = v.device, v.dtype
    if G < 1 or H % G != 0:
        raise ValueError(f"{H} heads of v cannot share {G} heads of q and k evenly")
    _require_sliced(q, "q", (Bsz, G, N), io, dev, 2)
    _require_sliced(k, "k", (Bsz, G, N), io, dev, 2)
    _require_sliced(v, "v", (Bsz, H, P), io, dev, 2)
    _require(g, "g", (H,) if g.dim() == 1 else (Bsz, H), torch.float32, dev)
    _require(state, "state", (state.shape[0], H, N, P), torch.float32, dev)
    if slots is not None:
        _require(slots, "slots", (Bsz,), torch.int32, dev)
    elif state.shape[0] < Bsz:
        raise ValueError(f"state holds {state.shape[0]} states for {Bsz} rows")
    if y is None:
        y = torch.empty((Bsz, H, P), dtype=io, device=dev)
    _require(y, "y", (Bsz, H, P), io, dev)
    with _on_device(v, stream):
        d = LaStepDesc()
        _set(d, dict(q=q, k=k, v=v, g=g, state=state, slots=slots, y=y))
        _set_strides(d, dict(q=q, k=k, v=v))
        d.Bsz, d.H, d.G, d.N, d.P, d.pool = Bsz, H, G, N, P, state.shape[0]
        d.scale, d.dtype, d.g_per_head, d.reserved = float(scale), dtype_id(v), int(g.dim() == 1), 0
        rc = lib().ss_la_step(ctypes.byref(d), stream_handle(stream, dev))
    _check("ss_la_step", rc)
    return y


def _gnorm_prepare(x, weight, bias, z, groups):
    import torch

    C = x.shape[-1]
    if groups < 1 or C % groups != 0:
        raise ValueError(f"{C} channels cannot form {groups} groups")
    _require(x, "x", x.shape, x.dtype, x.device)
    if z is not None:
        _require(z, "z", x.shape, x.dtype, x.device)
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _require(t, name, (C,), torch.float32, x.device)
    return x.numel() // C, C


def _gnorm_flags(z, center, gate_first):
    if gate_first and z is None:
        raise ValueError("gate_first needs a gate z")
    return (GNORM_CENTER if center else 0) | (GNORM_GATE_FIRST if gate_first else 0)


def ss_gnorm_fwd(x, weight=None, bias=None, z=None, groups=1, eps=1e-5, center=True, gate_first=False, out=None,
                 stream=None):
    """Group norm of each token's channels (the last dimension, ``groups`` runs of adjacent
    channels), then an activation: norm(x) * silu(z); norm(x * silu(z)) with ``gate_first``;
    silu(norm(x)) without z.  ``center=False`` divides by the root mean square instead.
    Returns out (x's shape and dtype)."""
    import torch

    M, C = _gnorm_prepare(x, weight, bias, z, groups)
    flags = _gnorm_flags(z, center, gate_first)
    if out is None:
        out = torch.empty_like(x)
    _require(out, "out", x.shape, x.dtype, x.device)
    with _on_device(x, stream):
        rc = lib().ss_gnorm_fwd(_p(x), _p(weight), _p(bias), _p(z), _p(out), M, C, groups, float(eps), flags,
                                dtype_id(x), stream_handle(stream, x.device))
    _check("ss_gnorm_fwd", rc)
    return out


def ss_gnorm_bwd(x, weight, bias, dout, z=None, groups=1, eps=1e-5, center=True, gate_first=False, out=None,
                 workspace=None, stream=None):
    """Gradient of sum(dout * ss_gnorm_fwd(...)).  Returns a dict: dx, dz (io type), dweight, dbias
    (f32); dz, dweight and dbias are None when their input is."""
    import torch

    M, C = _gnorm_prepare(x, weight, bias, z, groups)
    flags = _gnorm_flags(z, center, gate_first)
    _require(dout, "dout", x.shape, x.dtype, x.device)
    shapes = {"dx": (x.shape, x.dtype), "dz": (x.shape, x.dtype), "dweight": ((C,), torch.float32),
              "dbias": ((C,), torch.float32)}
    present = {"dz": z is not None, "dweight": weight is not None, "dbias": bias is not None}
    res = dict(out or {})
    for name, (shape, dtype) in shapes.items():
        if not present.get(name, True):
            res[name] = None
            continue
        if res.get(name) is None:
            res[name] = torch.empty(shape, dtype=dtype, device=x.device)
        _require(res[name], name, shape, dtype, x.device)
    dt = dtype_id(x)
    with _on_device(x, stream):
        workspace, _ = _workspace(int(lib().ss_gnorm_bwd_workspace_bytes(M, C, groups, dt)), x.device, workspace)
        rc = lib().ss_gnorm_bwd(_p(x), _p(weight), _p(bias), _p(z), _p(dout), _p(res["dx"]), _p(res["dz"]),
                                _p(res["dweight"]), _p(res["dbias"]), M, C, groups, float(eps), flags, dt,
                                _p(workspace), _nbytes(workspace), stream_handle(stream, x.device))
    _check("ss_gnorm_bwd", rc)
    return res
