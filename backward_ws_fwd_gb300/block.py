"""Binding of the block operators (include/wsf.h): rotary positions, the top-k
router with its balance loss, and group norm with an activation, channels
last.  Re-exported by the package; like the rest of it, this module marshals
tensors into the C calls.  Shapes and types that the C side cannot see are
checked here (TypeError, ValueError); the rest is checked there (WsfError).
"""
from __future__ import annotations

import ctypes
import math

from . import SIZE_MAX, _check, _dtype_code, _on, _ptr, _scratch, _stream, lib

_vp, _i64, _int, _sz, _f = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t,
                            ctypes.c_float)
_st3 = _i64 * 3
_stp = ctypes.POINTER(_i64)
_ROTARY = [_vp, _stp, _vp, _stp, _i64, _vp, _stp, _vp, _stp, _i64, _vp, _i64, _int, _vp, _f, _int,
           _i64, _i64, _i64, _i64, _int, _vp]
for _fn in (lib.rotary_fwd, lib.rotary_bwd):
    _fn.argtypes, _fn.restype = _ROTARY, _int
lib.router_fwd_workspace_bytes.argtypes, lib.router_fwd_workspace_bytes.restype = [_i64, _i64], _sz
lib.router_fwd.argtypes = [_vp, _i64, _vp, _i64, _int, _vp, _vp, _vp, _vp, _vp, _sz, _i64, _i64,
                           _int, _vp]
lib.router_fwd.restype = _int
lib.router_bwd.argtypes = [_vp, _i64, _vp, _vp, _i64, _int, _vp, _vp, _vp, _i64, _i64, _i64, _int,
                           _vp]
lib.router_bwd.restype = _int
for _fn in (lib.groupnorm_fwd_workspace_bytes, lib.groupnorm_bwd_workspace_bytes):
    _fn.argtypes, _fn.restype = [_i64, _i64, _i64, _i64, _int], _sz
lib.groupnorm_fwd.argtypes = [_vp, _i64, _i64, _vp, _vp, _f, _int, _vp, _i64, _i64, _vp, _vp, _vp,
                              _sz, _i64, _i64, _i64, _i64, _int, _vp]
lib.groupnorm_fwd.restype = _int
lib.groupnorm_bwd.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _vp,
                              _i64, _i64, _vp, _vp, _int, _vp, _sz, _i64, _i64, _i64, _i64, _int,
                              _vp]
lib.groupnorm_bwd.restype = _int


def _want(t, name, dtype, shape, like):
    """t is a contiguous tensor of this type and shape on like's device."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not {like.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _like(t, name, x):
    """t has x's type, shape and device and unit inner stride."""
    if t.dtype != x.dtype:
        raise TypeError(f"{name} must be {x.dtype}, not {t.dtype}")
    if t.shape != x.shape:
        raise ValueError(f"{name} must be {list(x.shape)}, not {list(t.shape)}")
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, not {x.device}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit inner stride")


# ---------------------------------------------------------------------------
# rotary positions

def _strides3(t):
    s = t.stride()
    return _st3(s[0], s[1], s[2]) if len(s) == 4 else _st3(0, s[0], s[1])


def _rotary(call, what, q, k, positions, inv_freq, scale, interleaved, q_out, k_out, stream):
    import torch
    if q.dim() not in (3, 4):
        raise ValueError("heads must be [B, S, H, D] or [T, H, D]")
    B, S = (q.shape[0], q.shape[1]) if q.dim() == 4 else (1, q.shape[0])
    H, D = q.shape[-2:]
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    _like(q, "q", q)
    _like(q_out, "q_out", q)
    R = 2 * inv_freq.numel()
    _want(inv_freq, "inv_freq", torch.float32, (R // 2,), q)
    Hk = 0
    if k is not None:
        if k.shape[:-2] != q.shape[:-2] or k.shape[-1] != D:
            raise ValueError(f"k {list(k.shape)} does not go with q {list(q.shape)}")
        Hk = k.shape[-2]
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        if k.dtype != q.dtype or k.device != q.device:
            raise TypeError("k must have q's type and device")
        _like(k, "k", k)
        _like(k_out, "k_out", k)
    elif k_out is not None:
        raise ValueError("k_out without k")
    pb = {torch.int32: 4, torch.int64: 8}.get(positions.dtype)
    if pb is None:
        raise TypeError(f"positions must be int32 or int64, not {positions.dtype}")
    if positions.device != q.device:
        raise ValueError(f"positions are on {positions.device}, not {q.device}")
    ps = tuple(positions.shape)
    if ps != (S,) and (q.dim() == 3 or ps not in ((B, S), (1, S))):
        raise ValueError(f"positions {list(ps)} do not go with q {list(q.shape)}")
    if S > 1 and positions.stride(-1) != 1:
        raise ValueError("positions must have unit inner stride")
    ldp = positions.stride(0) if ps == (B, S) and len(ps) == 2 and B > 1 else 0
    with _on(q):
        _check(call(_ptr(q), _strides3(q), _ptr(q_out), _strides3(q_out), H, _ptr(k),
                    _strides3(k) if Hk else None, _ptr(k_out), _strides3(k_out) if Hk else None,
                    Hk, _ptr(positions), ldp, pb, _ptr(inv_freq), float(scale), int(interleaved),
                    B, S, D, R, _dtype_code(q), _stream(stream, q.device)), what)
    return q_out, k_out


def rotary_fwd(q, k, positions, inv_freq, scale=1.0, interleaved=False, q_out=None, k_out=None,
               stream=None):
    """Rotary positions of q [B, S, Hq, D] (or [T, Hq, D]) and k (Hk heads, or
    None), any layout of unit inner stride.  positions: int32 or int64 [B, S],
    [S] or [T]; inv_freq: float32 [R/2] (see rotary_frequencies), the first R
    elements of a head are rotated, the others copied.  scale multiplies cos
    and sin.  q_out=q, k_out=k rotates in place.  Returns (yq, yk)."""
    return _rotary(lib.rotary_fwd, "rotary_fwd", q, k, positions, inv_freq, scale, interleaved,
                   q_out, k_out, stream)


def rotary_bwd(dyq, dyk, positions, inv_freq, scale=1.0, interleaved=False, dq=None, dk=None,
               stream=None):
    """The vector-Jacobian product of rotary_fwd: (dq, dk) from (dyq, dyk)."""
    return _rotary(lib.rotary_bwd, "rotary_bwd", dyq, dyk, positions, inv_freq, scale, interleaved,
                   dq, dk, stream)


def rotary_frequencies(R, base=10000.0, scaling=None, factor=1.0, original_length=None, fast=32.0,
                       slow=1.0, device=None):
    """(inv_freq float32 [R/2], scale) for rotary_fwd: base^(-2i/R), and for
    contexts `factor` times longer than the trained ones

    * scaling="linear": every frequency divided by factor;
    * scaling="base": the base grows by factor^(R/(R-2)), which leaves the
      fastest pair alone and divides the slowest by factor;
    * scaling="parts": pairs that turn more than `fast` times over
      `original_length` tokens are left alone, those that turn less than
      `slow` times are divided by factor, those between are blended along the
      pair's index; scale = 0.1·ln(factor) + 1.

    Computed in 64 bits and rounded once."""
    import torch
    if R < 0 or R % 2:
        raise ValueError("R must be even")
    if not factor >= 1.0 or not base > 1.0:
        raise ValueError("factor must be at least 1 and base above 1")
    i = torch.arange(0, R, 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "base":
        base = base * factor ** (R / (R - 2)) if R > 2 else base
    f = base ** (-i / max(R, 1))
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if not original_length or not fast > slow > 0:
            raise ValueError('scaling="parts" needs original_length and fast > slow > 0')

        def index(turns):  # the pair that turns this often over the trained length
            return R * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), R - 1)
        blend = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - blend) + f / factor * blend
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.float().to(device), scale


# ---------------------------------------------------------------------------
# router

def router_fwd_workspace_bytes(T: int, E: int) -> int:
    return lib.router_fwd_workspace_bytes(T, E)


def router_fwd(logits, k, mask=None, renormalize=False, gates=None, ids=None, counts=None,
               loss=None, workspace=None, stream=None):
    """Top-k routing with the balance loss.  logits: [T, E] (unit inner
    stride); mask: bool or uint8 [T], False leaves a row out.  Returns (gates
    float32 [T, k], ids int32 [T, k], counts int32 [E], loss float32 [])."""
    import torch
    T, E = logits.shape
    dev = logits.device
    _like(logits, "logits", logits)
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError("mask must be bool or uint8")
        _want(mask, "mask", mask.dtype, (T,), logits)
    if gates is None:
        gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    else:
        _want(gates, "gates", torch.float32, (T, k), logits)
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    else:
        _want(ids, "ids", torch.int32, (T, k), logits)
    if counts is None:
        counts = torch.empty(E, dtype=torch.int32, device=dev)
    else:
        _want(counts, "counts", torch.int32, (E,), logits)
    if loss is None:
        loss = torch.empty((), dtype=torch.float32, device=dev)
    else:
        _want(loss, "loss", torch.float32, (), logits)
    with _on(logits):
        need = lib.router_fwd_workspace_bytes(T, E)
        if workspace is None and need not in (0, SIZE_MAX):
            workspace = _scratch(need, dev, stream)
        wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(lib.router_fwd(_ptr(logits), logits.stride(0), _ptr(mask), k, int(bool(renormalize)),
                              _ptr(gates), _ptr(ids), _ptr(counts), _ptr(loss), _ptr(workspace),
                              wbytes, T, E, _dtype_code(logits), _stream(stream, dev)),
               "router_fwd")
    return gates, ids, counts, loss


def router_bwd(logits, ids, counts, dgates, dloss, renormalize=False, dlogits=None, stream=None):
    """dlogits of router_fwd from ids and counts as it returned them, dgates
    (float32 [T, k] or None) and dloss (float32 [] or None)."""
    import torch
    T, E = logits.shape
    k = ids.shape[1]
    _like(logits, "logits", logits)
    _want(ids, "ids", torch.int32, (T, k), logits)
    _want(counts, "counts", torch.int32, (E,), logits)
    if dgates is not None:
        _want(dgates, "dgates", torch.float32, (T, k), logits)
    if dloss is not None:
        _want(dloss, "dloss", torch.float32, (), logits)
    if dlogits is None:
        dlogits = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    else:
        _like(dlogits, "dlogits", logits)
    with _on(logits):
        _check(lib.router_bwd(_ptr(logits), logits.stride(0), _ptr(ids), _ptr(counts), k,
                              int(bool(renormalize)), _ptr(dgates), _ptr(dloss), _ptr(dlogits),
                              dlogits.stride(0), T, E, _dtype_code(logits),
                              _stream(stream, logits.device)), "router_bwd")
    return dlogits


# ---------------------------------------------------------------------------
# group norm

ACT_NONE, ACT_SILU = 0, 1
_ACTS = {None: ACT_NONE, "silu": ACT_SILU}


def groupnorm_workspace_bytes(N: int, S: int, C: int, groups: int, dtype, backward: bool) -> int:
    from . import _dtype_code_of_dtype
    code = dtype if isinstance(dtype, int) else _dtype_code_of_dtype(dtype)
    fn = lib.groupnorm_bwd_workspace_bytes if backward else lib.groupnorm_fwd_workspace_bytes
    return fn(N, S, C, groups, code)


def _nsc(x):
    if x.dim() == 3:
        return x.shape
    if x.dim() == 2:
        return x.shape[0], 1, x.shape[1]
    raise ValueError("x must be [N, S, C] or [N, C]")


def _ns_strides(t):
    s = t.stride()
    return (s[0], s[1]) if len(s) == 3 else (s[0], t.shape[1])


def _act(act):
    try:
        return _ACTS[act]
    except (KeyError, TypeError):
        raise ValueError(f"unknown activation {act!r}") from None


def groupnorm_fwd(x, w, b, groups, eps=1e-5, act=None, y=None, mean=None, rstd=None,
                  workspace=None, stream=None):
    """Group norm of x [N, S, C] (or [N, C], S = 1), channels last, over
    `groups` groups of consecutive channels; w, b: float32 [C]; act: None or
    "silu".  Returns (y, mean, rstd), the statistics float32 [N, groups]."""
    import torch
    N, S, C = _nsc(x)
    code, act = _dtype_code(x), _act(act)
    _like(x, "x", x)
    _want(w, "w", torch.float32, (C,), x)
    _want(b, "b", torch.float32, (C,), x)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _like(y, "y", x)
    if mean is None:
        mean = torch.empty((N, groups), dtype=torch.float32, device=x.device)
    else:
        _want(mean, "mean", torch.float32, (N, groups), x)
    if rstd is None:
        rstd = torch.empty((N, groups), dtype=torch.float32, device=x.device)
    else:
        _want(rstd, "rstd", torch.float32, (N, groups), x)
    with _on(x):
        need = lib.groupnorm_fwd_workspace_bytes(N, S, C, groups, code)
        if workspace is None and need not in (0, SIZE_MAX):
            workspace = _scratch(need, x.device, stream)
        wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(lib.groupnorm_fwd(_ptr(x), *_ns_strides(x), _ptr(w), _ptr(b), float(eps), act,
                                 _ptr(y), *_ns_strides(y), _ptr(mean), _ptr(rstd),
                                 _ptr(workspace), wbytes, N, S, C, groups, code,
                                 _stream(stream, x.device)), "groupnorm_fwd")
    return y, mean, rstd


def groupnorm_bwd(x, w, b, mean, rstd, dy, groups, act=None, dx=None, grad_w=None, grad_b=None,
                  accumulate=False, workspace=None, stream=None):
    """dx, grad_w (+)= Σ dz·x̂ and grad_b (+)= Σ dz of groupnorm_fwd, from its
    statistics.  Returns (dx, grad_w, grad_b)."""
    import torch
    N, S, C = _nsc(x)
    code, act = _dtype_code(x), _act(act)
    _like(x, "x", x)
    _like(dy, "dy", x)
    _want(w, "w", torch.float32, (C,), x)
    _want(b, "b", torch.float32, (C,), x)
    _want(mean, "mean", torch.float32, (N, groups), x)
    _want(rstd, "rstd", torch.float32, (N, groups), x)
    if dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _like(dx, "dx", x)
    if grad_w is None:
        grad_w = torch.empty(C, dtype=torch.float32, device=x.device)
    else:
        _want(grad_w, "grad_w", torch.float32, (C,), x)
    if grad_b is None:
        grad_b = torch.empty(C, dtype=torch.float32, device=x.device)
    else:
        _want(grad_b, "grad_b", torch.float32, (C,), x)
    with _on(x):
        need = lib.groupnorm_bwd_workspace_bytes(N, S, C, groups, code)
        if workspace is None and need not in (0, SIZE_MAX):
            workspace = _scratch(need, x.device, stream)
        wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(lib.groupnorm_bwd(_ptr(x), *_ns_strides(x), _ptr(w), _ptr(b), _ptr(mean),
                                 _ptr(rstd), _ptr(dy), *_ns_strides(dy), act, _ptr(dx),
                                 *_ns_strides(dx), _ptr(grad_w), _ptr(grad_b),
                                 int(bool(accumulate)), _ptr(workspace), wbytes, N, S, C, groups,
                                 code, _stream(stream, x.device)), "groupnorm_bwd")
    return dx, grad_w, grad_b
