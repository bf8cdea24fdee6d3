"""Linear attention with one decay per head, and the gated group norm of its output
(C ABI in include/ss_la.h).  Argument marshalling only, like ``binding``:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,   y_t = scale * q_t S_t        per batch row and head

q, k are [Bsz, L, G, N], v is [Bsz, L, H, P] (f32, bf16 or f16; H / G heads of v share a head
of q and k), g is f32 [Bsz, L, H], or [H] for one decay per head; states are f32 [Bsz, H, N, P].
"""

from __future__ import annotations

import ctypes
import functools

from .binding import _I32, _I64, _P, _SZ, _check, _on_device, _require, _workspace, dtype_id, lib, stream_handle

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


@functools.lru_cache(maxsize=256)
def la_fwd_workspace_bytes(Bsz, L, H, G, N, P, dtype) -> int:
    return int(lib().ss_la_fwd_workspace_bytes(Bsz, L, H, G, N, P, dtype))


@functools.lru_cache(maxsize=256)
def la_bwd_workspace_bytes(Bsz, L, H, G, N, P, dtype) -> int:
    return int(lib().ss_la_bwd_workspace_bytes(Bsz, L, H, G, N, P, dtype))


# The checks below answer the ordinary case with a few comparisons (a single-token call takes
# as long to check as to run) and leave the wording of a refusal to _require.


def _whole(t, name, shape, dtype, device):
    if not (t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.device == device):
        _require(t, name, shape, dtype, device)


def _optional(t, name, shape, dtype, device):
    """The checked tensor's address.  The caller keeps the tensor: one that only the call holds must
    not be freed, and its memory handed to an output, before the launch."""
    if t is None:
        return None
    _whole(t, name, shape, dtype, device)
    return t.data_ptr()


def _sliced(t, name, shape, dtype, device):
    """Check a tensor whose last two dimensions are contiguous; the others may step over a wider
    tensor's other columns.  Returns its strides."""
    stride = t.stride()
    if t.shape == shape and t.dtype is dtype and stride[-1] == 1 and stride[-2] == shape[-1] and t.device == device:
        return stride
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype} != {dtype}")
    if t.numel() and ((shape[-1] > 1 and stride[-1] != 1) or (shape[-2] > 1 and stride[-2] != shape[-1])):
        raise ValueError(f"{name}: the last two dimensions must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return stride


def _call(fn, t, *args):
    """Run a library call on t's device and that device's current stream."""
    import torch

    device = t.device
    if device.index == torch._C._cuda_getDevice():
        rc = getattr(lib(), fn)(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            rc = getattr(lib(), fn)(*args, torch.cuda.current_stream(device).cuda_stream)
    if rc:
        _check(fn, rc)


def _in_stream(stream, t, fn, *args):
    """fn with ``stream`` as the current stream: what it allocates (workspaces, outputs) then belongs
    to the stream that uses it, and is not handed out again while that still runs."""
    import torch

    with _on_device(t, stream), torch.cuda.stream(stream):
        return fn(*args)


def _new(a, b, c, d, dtype, device):
    """An uninitialised contiguous tensor [a, b, c, d] (torch.empty takes twice as long)."""
    import torch

    return torch.empty_strided((a, b, c, d), (b * c * d, c * d, d, 1), dtype=dtype, device=device)


def _heads(H, G):
    if G < 1 or H % G != 0:
        raise ValueError(f"{H} heads of v cannot share {G} heads of q and k evenly")


def _gpu(t):
    if t.device.type != "cuda":
        raise ValueError(f"tensors must be CUDA tensors, got {t.device}")


def ss_la_fwd(q, k, v, g, scale=1.0, h0=None, lengths=None, y=None, last_state=None, return_last_state=True,
              workspace=None, stream=None):
    """Linear attention over whole sequences.  ``h0``: state to start from; ``lengths`` (int32
    [Bsz]): tokens of each row that count.  q, k, v may be slices of one projection's output.
    Returns (y, last_state or None)."""
    import torch

    if stream is not None:
        return _in_stream(stream, v, ss_la_fwd, q, k, v, g, scale, h0, lengths, y, last_state, return_last_state,
                          workspace)
    Bsz, L, H, P = v.shape
    G, N = q.shape[2:]
    dev, io, f32 = v.device, v.dtype, torch.float32
    _heads(H, G)
    qs = _sliced(q, "q", (Bsz, L, G, N), io, dev)
    ks = _sliced(k, "k", (Bsz, L, G, N), io, dev)
    vs = _sliced(v, "v", (Bsz, L, H, P), io, dev)
    per_head = g.dim() == 1
    _whole(g, "g", (H,) if per_head else (Bsz, L, H), f32, dev)
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
    need = la_fwd_workspace_bytes(Bsz, L, H, G, N, P, dt)
    workspace, wsb = _workspace(need, dev, workspace)
    d = LaFwdDesc(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), h0_p, lengths_p, y.data_ptr(), last,
                  None if workspace is None else workspace.data_ptr(), wsb, qs[1], qs[0], ks[1], ks[0], vs[1], vs[0],
                  Bsz, L, H, G, N, P, scale, dt, per_head, 0)
    _call("ss_la_fwd", v, ctypes.byref(d))
    return y, last_state


def ss_la_bwd(q, k, v, g, dy, scale=1.0, h0=None, dlast_state=None, lengths=None, out=None, workspace=None,
              stream=None):
    """Gradient of sum(dy * y) + sum(dlast_state * last_state).  Returns a dict: dq, dk (summed over
    the heads that share them) and dv in the io type, dg (g's shape) and dh0 (None without h0) f32."""
    import torch

    if stream is not None:
        return _in_stream(stream, v, ss_la_bwd, q, k, v, g, dy, scale, h0, dlast_state, lengths, out, workspace)
    Bsz, L, H, P = v.shape
    G, N = q.shape[2:]
    dev, io, f32 = v.device, v.dtype, torch.float32
    _heads(H, G)
    qs = _sliced(q, "q", (Bsz, L, G, N), io, dev)
    ks = _sliced(k, "k", (Bsz, L, G, N), io, dev)
    vs = _sliced(v, "v", (Bsz, L, H, P), io, dev)
    ys = _sliced(dy, "dy", (Bsz, L, H, P), io, dev)
    per_head = g.dim() == 1
    _whole(g, "g", (H,) if per_head else (Bsz, L, H), f32, dev)
    state = (Bsz, H, N, P)
    lengths_p = _optional(lengths, "lengths", (Bsz,), torch.int32, dev)
    h0_p = _optional(h0, "h0", state, f32, dev)
    dlast_p = _optional(dlast_state, "dlast_state", state, f32, dev)
    _gpu(v)
    if out:
        shapes = {"dq": ((Bsz, L, G, N), io), "dk": ((Bsz, L, G, N), io), "dv": ((Bsz, L, H, P), io),
                  "dg": (tuple(g.shape), f32), "dh0": (state, f32)}
        out = dict(out)
        for name, (shape, dtype) in shapes.items():
            if name == "dh0" and h0 is None:
                out[name] = None
            elif out.get(name) is None:
                out[name] = torch.empty(shape, dtype=dtype, device=dev)
            else:
                _whole(out[name], name, shape, dtype, dev)
    else:
        out = {"dq": _new(Bsz, L, G, N, io, dev), "dk": _new(Bsz, L, G, N, io, dev), "dv": _new(Bsz, L, H, P, io, dev),
               "dg": torch.empty_like(g), "dh0": None if h0 is None else torch.empty_like(h0)}
    dt = dtype_id(v)
    need = la_bwd_workspace_bytes(Bsz, L, H, G, N, P, dt)
    workspace, wsb = _workspace(need, dev, workspace)
    d = LaBwdDesc(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), h0_p, lengths_p, dy.data_ptr(), dlast_p,
                  out["dq"].data_ptr(), out["dk"].data_ptr(), out["dv"].data_ptr(), out["dg"].data_ptr(),
                  None if out["dh0"] is None else out["dh0"].data_ptr(),
                  None if workspace is None else workspace.data_ptr(), wsb, qs[1], qs[0], ks[1], ks[0], vs[1], vs[0],
                  ys[1], ys[0], Bsz, L, H, G, N, P, scale, dt, per_head, 0)
    _call("ss_la_bwd", v, ctypes.byref(d))
    return out


def ss_la_step(q, k, v, g, state, scale=1.0, slots=None, y=None, stream=None):
    """One token of each sequence, in place on ``state`` [pool, H, N, P] f32: q, k [Bsz, G, N], v
    [Bsz, H, P], g [Bsz, H] or [H].  ``slots`` (int32 [Bsz]): the state each row owns, -1 for a
    padding row (y = 0); without it row b owns state b.  Returns y [Bsz, H, P]."""
    import torch

    if stream is not None:
        return _in_stream(stream, v, ss_la_step, q, k, v, g, state, scale, slots, y)
    Bsz, H, P = v.shape
    G, N = q.shape[1:]
    dev, io, f32 = v.device, v.dtype, torch.float32
    _heads(H, G)
    qs = _sliced(q, "q", (Bsz, G, N), io, dev)
    ks = _sliced(k, "k", (Bsz, G, N), io, dev)
    vs = _sliced(v, "v", (Bsz, H, P), io, dev)
    per_head = g.dim() == 1
    _whole(g, "g", (H,) if per_head else (Bsz, H), f32, dev)
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
    d = LaStepDesc(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), state.data_ptr(), slots_p, y.data_ptr(),
                   qs[0], ks[0], vs[0], Bsz, H, G, N, P, pool, scale, dtype_id(v), per_head, 0)
    _call("ss_la_step", v, ctypes.byref(d))
    return y


def la_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Launch one block, built like the tensor-core kernels', one part of which waits limit_ns for
    nothing after the others are over; it records the failure in the device status word."""
    _check("ss_la_selftest_wait_timeout", lib().ss_la_selftest_wait_timeout(int(limit_ns), stream_handle(stream)))


def _gnorm_prepare(x, weight, bias, z, groups, center, gate_first):
    """Check the shared inputs of both directions; returns M, C, flags and the inputs' pointers."""
    import torch

    C, dev, f32 = x.shape[-1] if x.dim() else 0, x.device, torch.float32
    if groups < 1 or C < 1 or C % groups != 0:
        raise ValueError(f"{C} channels cannot form {groups} groups")
    if gate_first and z is None:
        raise ValueError("gate_first needs a gate z")
    _whole(x, "x", x.shape, x.dtype, dev)
    flags = (GNORM_CENTER if center else 0) | (GNORM_GATE_FIRST if gate_first else 0)
    pointers = (_optional(weight, "weight", (C,), f32, dev), _optional(bias, "bias", (C,), f32, dev),
                _optional(z, "z", x.shape, x.dtype, dev))
    _gpu(x)
    return x.numel() // C, C, flags, *pointers


def ss_gnorm_fwd(x, weight=None, bias=None, z=None, groups=1, eps=1e-5, center=True, gate_first=False, out=None,
                 stream=None):
    """Group norm of each token's channels (the last dimension, ``groups`` runs of at most 8192
    adjacent channels), then an activation: norm(x) * silu(z); norm(x * silu(z)) with ``gate_first``;
    silu(norm(x)) without z.  ``center=False`` divides by the root mean square instead.
    Returns out (x's shape and dtype)."""
    import torch

    if stream is not None:
        return _in_stream(stream, x, ss_gnorm_fwd, x, weight, bias, z, groups, eps, center, gate_first, out)
    M, C, flags, wp, bp, zp = _gnorm_prepare(x, weight, bias, z, groups, center, gate_first)
    if out is None:
        out = torch.empty_like(x)
    else:
        _whole(out, "out", x.shape, x.dtype, x.device)
    _call("ss_gnorm_fwd", x, x.data_ptr(), wp, bp, zp, out.data_ptr(), M, C, groups, eps, flags, dtype_id(x))
    return out


def ss_gnorm_bwd(x, weight, bias, dout, z=None, groups=1, eps=1e-5, center=True, gate_first=False, out=None,
                 workspace=None, stream=None):
    """Gradient of sum(dout * ss_gnorm_fwd(...)).  Returns a dict: dx, dz (io type), dweight, dbias
    (f32); dz, dweight and dbias are None when their input is."""
    import torch

    if stream is not None:
        return _in_stream(stream, x, ss_gnorm_bwd, x, weight, bias, dout, z, groups, eps, center, gate_first, out,
                          workspace)
    M, C, flags, wp, bp, zp = _gnorm_prepare(x, weight, bias, z, groups, center, gate_first)
    _whole(dout, "dout", x.shape, x.dtype, x.device)
    shapes = {"dx": (x.shape, x.dtype), "dz": (x.shape, x.dtype), "dweight": ((C,), torch.float32),
              "dbias": ((C,), torch.float32)}
    present = {"dz": zp is not None, "dweight": wp is not None, "dbias": bp is not None}
    out = dict(out or {})
    for name, (shape, dtype) in shapes.items():
        if not present.get(name, True):
            out[name] = None
        elif out.get(name) is None:
            out[name] = torch.empty(shape, dtype=dtype, device=x.device)
        else:
            _whole(out[name], name, shape, dtype, x.device)
    dt = dtype_id(x)
    workspace, wsb = _workspace(int(lib().ss_gnorm_bwd_workspace_bytes(M, C, groups, dt)), x.device, workspace)
    ptr = {name: None if out[name] is None else out[name].data_ptr() for name in shapes}
    _call("ss_gnorm_bwd", x, x.data_ptr(), wp, bp, zp, dout.data_ptr(), ptr["dx"], ptr["dz"], ptr["dweight"],
          ptr["dbias"], M, C, groups, eps, flags, dt, None if workspace is None else workspace.data_ptr(), wsb)
    return out
