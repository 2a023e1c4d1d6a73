"""Torch-facing wrappers of the linear attention and block norm entry points.

As in ops.py, torch is used for device memory and streams only, and every wrapper
checks the shape, type and device of every tensor before it takes a pointer.
Activations are float32 or bfloat16 tensors of one dtype; states, decays and norm
weights are float32.  q, k, v and the output gradient may be views with a contiguous
last axis (slices of one projection's output); other tensors are contiguous.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _lib
from .ops import _dt, _ptr, _shape, _stream, _workspace

F32 = torch.float32


def _dims(t, name: str, n: int) -> None:
    if not isinstance(t, torch.Tensor) or t.dim() != n:
        raise ValueError(f"{name} must be a tensor of {n} dimensions")


def _view(t: torch.Tensor, name: str, dtype, device):
    """(pointer, strides) of a view with a contiguous last axis; strides is a ctypes array
    of the element strides of the axes before it (None: packed)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_contiguous() or t.numel() == 0:
        return t.data_ptr(), None
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last axis")
    return t.data_ptr(), (ctypes.c_int64 * (t.dim() - 1))(*t.stride()[:-1])


def _attention_shapes(q, k, v, log_decay, lead, L):
    """Shapes of q, k, v [*lead, heads, width]; returns (H, Hq, Hk, Hv, K, V)."""
    n = len(lead) + (L is not None) + 2
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _dims(t, name, n)
    _dims(log_decay, "log_decay", 1)
    H = log_decay.shape[0]
    head = tuple(lead) + (() if L is None else (L,))
    K, V = q.shape[-1], v.shape[-1]
    _shape(q, "q", head + (q.shape[-2], K))
    _shape(k, "k", head + (k.shape[-2], K))
    _shape(v, "v", head + (v.shape[-2], V))
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t.shape[-2] < 1 or H % t.shape[-2]:
            raise ValueError(f"{name} has {t.shape[-2]} heads, which does not divide log_decay's {H}")
    return H, q.shape[-2], k.shape[-2], v.shape[-2], K, V


def linear_attention_workspace_size(batch, L, H, K, V, dtype=torch.bfloat16) -> int:
    """Bytes of device workspace linear_attention_fwd needs for this shape (0: none)."""
    lib = _lib.load_library()
    dt = _lib.SSM_BF16 if dtype == torch.bfloat16 else _lib.SSM_F32
    return int(lib.ssm_linear_attention_workspace_size(int(batch), int(L), int(H), int(K), int(V), dt))


def linear_attention_bwd_workspace_size(batch, L, H, K, V, dtype=torch.bfloat16, *, Hq=None, Hk=None, Hv=None) -> int:
    """Bytes of device workspace linear_attention_bwd needs (Hq, Hk, Hv: heads of q, k and v, H when None)."""
    lib = _lib.load_library()
    dt = _lib.SSM_BF16 if dtype == torch.bfloat16 else _lib.SSM_F32
    return int(lib.ssm_linear_attention_bwd_workspace_size(int(batch), int(L), int(H), int(Hq or H), int(Hk or H),
                                                           int(Hv or H), int(K), int(V), dt))


def linear_attention_fwd(q, k, v, log_decay, scale=None, *, initial_state=None, lengths=None, out=None,
                         final_state=None, return_final_state=True, workspace=None,
                         stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with a constant decay per head: S_t = exp(log_decay) S_{t-1} + k_t v_t^T,
    o_t = scale q_t S_t.

    q [batch, L, Hq, K], k [batch, L, Hk, K], v [batch, L, Hv, V] (each head count divides
    H; views with a contiguous last axis are fine); log_decay [H] float32; scale defaults
    to K ** -0.5.  `initial_state` [batch, H, K, V] float32 (zero when None); `final_state`
    may be the same tensor (updated in place).  `lengths` [batch] int32: tokens at or past
    a row's length are absent (their outputs are 0).  `workspace`: a device tensor of at
    least linear_attention_workspace_size(...) bytes, or None (allocated here).
    Returns (out [batch, L, H, V], final_state or None).
    """
    lib = _lib.load_library()
    _dims(q, "q", 4)
    batch, L = q.shape[:2]
    H, Hq, Hk, Hv, K, V = _attention_shapes(q, k, v, log_decay, (batch,), L)
    _shape(lengths, "lengths", (batch,))
    _shape(initial_state, "initial_state", (batch, H, K, V))
    _shape(out, "out", (batch, L, H, V))
    _shape(final_state, "final_state", (batch, H, K, V))
    act, dev = q.dtype, q.device
    (qp, qs), (kp, ks), (vp, vs) = (_view(t, n, act, dev) for t, n in ((q, "q"), (k, "k"), (v, "v")))
    if out is None:
        out = torch.empty((batch, L, H, V), dtype=act, device=dev)
    if final_state is None and return_final_state:
        final_state = torch.empty((batch, H, K, V), dtype=F32, device=dev)
    ws_ptr, ws_bytes = _workspace(workspace, linear_attention_workspace_size(batch, L, H, K, V, act), dev)
    _lib.check(lib.ssm_linear_attention_fwd(
        qp, kp, vp, qs, ks, vs, _ptr(log_decay, "log_decay", F32, dev), float(K ** -0.5 if scale is None else scale),
        _ptr(lengths, "lengths", torch.int32, dev), _ptr(initial_state, "initial_state", F32, dev),
        _ptr(out, "out", act, dev), _ptr(final_state, "final_state", F32, dev), batch, L, H, Hq, Hk, Hv, K, V, _dt(q),
        ws_ptr, ws_bytes, _stream(stream)))
    return out, final_state


def linear_attention_bwd(q, k, v, log_decay, dout, scale=None, *, initial_state=None, dfinal_state=None, lengths=None,
                         want_dinitial_state=None, workspace=None, out=None, stream=None) -> dict:
    """Gradients of linear_attention_fwd (same inputs) for the output gradient dout
    [batch, L, H, V] and optionally the final state's, dfinal_state [batch, H, K, V].

    Returns a dict with dq, dk, dv (packed, in the shapes of q, k and v: summed over the
    state heads that share a head) and dinitial_state (None unless an initial state is
    given or want_dinitial_state says so).  log_decay is a constant: it has no gradient.
    `workspace`: a device tensor of at least linear_attention_bwd_workspace_size(...)
    bytes, or None (allocated here); `out` may hold preallocated outputs under the same keys.
    """
    lib = _lib.load_library()
    _dims(q, "q", 4)
    batch, L = q.shape[:2]
    H, Hq, Hk, Hv, K, V = _attention_shapes(q, k, v, log_decay, (batch,), L)
    _shape(dout, "dout", (batch, L, H, V))
    if not isinstance(dout, torch.Tensor):
        raise TypeError("dout must be a torch.Tensor")
    _shape(lengths, "lengths", (batch,))
    _shape(initial_state, "initial_state", (batch, H, K, V))
    _shape(dfinal_state, "dfinal_state", (batch, H, K, V))
    act, dev = q.dtype, q.device
    (qp, qs), (kp, ks), (vp, vs), (dp, ds) = (
        _view(t, n, act, dev) for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")))
    want = initial_state is not None if want_dinitial_state is None else want_dinitial_state
    g = _outputs(out, dev, {"dq": ((batch, L, Hq, K), act, True), "dk": ((batch, L, Hk, K), act, True),
                            "dv": ((batch, L, Hv, V), act, True), "dinitial_state": ((batch, H, K, V), F32, want)})
    ws_ptr, ws_bytes = _workspace(
        workspace, linear_attention_bwd_workspace_size(batch, L, H, K, V, act, Hq=Hq, Hk=Hk, Hv=Hv), dev)
    _lib.check(lib.ssm_linear_attention_bwd(
        qp, kp, vp, dp, qs, ks, vs, ds, _ptr(log_decay, "log_decay", F32, dev),
        float(K ** -0.5 if scale is None else scale), _ptr(lengths, "lengths", torch.int32, dev),
        _ptr(initial_state, "initial_state", F32, dev), _ptr(dfinal_state, "dfinal_state", F32, dev),
        _ptr(g["dq"], "dq", act, dev), _ptr(g["dk"], "dk", act, dev), _ptr(g["dv"], "dv", act, dev),
        _ptr(g["dinitial_state"], "dinitial_state", F32, dev), batch, L, H, Hq, Hk, Hv, K, V, _dt(q),
        ws_ptr, ws_bytes, _stream(stream)))
    return g


def linear_attention_step(state, q_t, k_t, v_t, log_decay, scale=None, *, slots=None, out_state=None, out=None,
                          stream=None) -> torch.Tensor:
    """One token of linear_attention_fwd.  state [states, H, K, V] float32; q_t [batch, Hq, K],
    k_t [batch, Hk, K], v_t [batch, Hv, V].  Updates `out_state` (default: `state`, in place)
    and returns out [batch, H, V].

    `slots` [batch] int32: row b's state is number slots[b] of the pool; a row whose slot
    is outside [0, states) is idle (output 0, no state touched).  No two rows may name one
    slot.  None: row b's state is number b.
    """
    lib = _lib.load_library()
    _dims(state, "state", 4)
    _dims(q_t, "q_t", 3)
    batch, states = q_t.shape[0], state.shape[0]
    H, Hq, Hk, Hv, K, V = _attention_shapes(q_t, k_t, v_t, log_decay, (batch,), None)
    _shape(state, "state", (states, H, K, V))
    _shape(slots, "slots", (batch,))
    _shape(out_state, "out_state", (states, H, K, V))
    _shape(out, "out", (batch, H, V))
    if slots is None and states < batch:
        raise ValueError(f"{batch} rows need as many states, got {states}")
    act, dev = q_t.dtype, state.device
    (qp, qs), (kp, ks), (vp, vs) = (_view(t, n, act, dev) for t, n in ((q_t, "q_t"), (k_t, "k_t"), (v_t, "v_t")))
    if out_state is None:
        out_state = state
    if out is None:
        out = torch.empty((batch, H, V), dtype=act, device=dev)
    _lib.check(lib.ssm_linear_attention_step(
        _ptr(state, "state", F32, dev), _ptr(out_state, "out_state", F32, dev), qp, kp, vp, qs, ks, vs,
        _ptr(log_decay, "log_decay", F32, dev), float(K ** -0.5 if scale is None else scale),
        _ptr(slots, "slots", torch.int32, dev), _ptr(out, "out", act, dev), batch, states, H, Hq, Hk, Hv, K, V,
        _dt(q_t), _stream(stream)))
    return out


def _outputs(given, dev, spec) -> dict:
    """Output tensors by name: the caller's where given (checked), else new ones; None where not computed."""
    got = {}
    for name, (shape, dtype, computed) in spec.items():
        t = (given or {}).get(name)
        if t is not None and computed:
            _shape(t, f"out[{name!r}]", shape)
            if t.dtype != dtype:
                raise TypeError(f"out[{name!r}] must be {dtype}")
            got[name] = t
        else:
            got[name] = torch.empty(shape, dtype=dtype, device=dev) if computed else None
    return got


def _rows(t, name: str, D: int):
    """(pointer, row stride) of [..., D] as rows that lie a constant stride apart."""
    if t is None:
        return None, D
    rows = t.numel() // D if D else 0
    if t.is_contiguous() or rows <= 1:
        if rows == 1 and D > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must have a contiguous last axis")
        return t.data_ptr(), D
    if D > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last axis")
    axes = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n != 1]
    for (_, outer), (n, inner) in zip(axes, axes[1:]):
        if outer != n * inner:
            raise ValueError(f"{name} must have its rows a constant stride apart")
    return t.data_ptr(), axes[-1][1]


def _norm_inputs(x, gate, post_weight, res_scale, pre_weight, groups):
    """Checked (rows shape, D, residual-independent pointers) of a block norm's inputs."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("expected x [..., D]")
    D = x.shape[-1]
    for t, name in ((post_weight, "post_weight"), (res_scale, "res_scale"), (pre_weight, "pre_weight")):
        _shape(t, name, (D,))
    _shape(gate, "gate", x.shape)
    if int(groups) < 1 or D % int(groups):
        raise ValueError(f"groups ({groups}) must divide D ({D})")
    dev = x.device
    for t, name in ((x, "x"), (gate, "gate")):
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must live on the GPU")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
        if t.dtype != x.dtype:
            raise TypeError(f"{name} must be {x.dtype}, got {t.dtype}")
    return x.numel() // D if D else 0, D, dev


def _residual_dtype(dtype, x) -> Tuple[torch.dtype, int]:
    dtype = x.dtype if dtype is None else dtype
    if dtype not in (F32, x.dtype):
        raise TypeError(f"the residual stream must be float32 or {x.dtype}, got {dtype}")
    return dtype, _lib.SSM_F32 if dtype == F32 else _lib.SSM_BF16


def block_norm_fwd(x, residual=None, gate=None, post_weight=None, res_scale=None, pre_weight=None, *, groups=1,
                   eps=1e-5, residual_dtype=None, h=None, y=None, return_h=True,
                   stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """The norms around a block with its gate, residual and residual scale, row by row:

        n = post_weight * x * rsqrt(mean over the column group of x^2 + eps)
        t = n * silu(gate);  h = residual + res_scale * t
        y = pre_weight * h * rsqrt(mean over the row of h^2 + eps)

    each piece only where its argument is given.  x, gate [..., D] (rows may lie a constant
    stride apart); residual, h [..., D] of residual_dtype (the residual's, else x's; float32 or
    x's); the weights [D] float32.  `groups`: column groups of the first norm.  `h` may be the
    residual (updated in place).  Returns (h, y): h None when return_h is False and no h is
    given, y None without pre_weight.
    """
    lib = _lib.load_library()
    rows, D, dev = _norm_inputs(x, gate, post_weight, res_scale, pre_weight, groups)
    _shape(residual, "residual", x.shape)
    _shape(h, "h", x.shape)
    _shape(y, "y", x.shape)
    if residual_dtype is None and (residual is not None or h is not None):
        residual_dtype = (residual if residual is not None else h).dtype
    rdtype, rdt = _residual_dtype(residual_dtype, x)
    if pre_weight is None and y is not None:
        raise ValueError("y is computed only with pre_weight")
    if h is None and (return_h or pre_weight is None):
        h = torch.empty(x.shape, dtype=rdtype, device=dev)
    if y is None and pre_weight is not None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    (xp, xs), (gp, gs) = _rows(x, "x", D), _rows(gate, "gate", D)
    _lib.check(lib.ssm_block_norm_fwd(
        xp, xs, _ptr(residual, "residual", rdtype, dev), gp, gs, _ptr(post_weight, "post_weight", F32, dev),
        _ptr(res_scale, "res_scale", F32, dev), _ptr(pre_weight, "pre_weight", F32, dev), _ptr(h, "h", rdtype, dev),
        _ptr(y, "y", x.dtype, dev), rows, D, int(groups), float(eps), _dt(x), rdt, _stream(stream)))
    return h, y


def block_norm_bwd_workspace_size(rows, D) -> int:
    """Bytes of device workspace block_norm_bwd needs."""
    return int(_lib.load_library().ssm_block_norm_bwd_workspace_size(int(rows), int(D)))


def block_norm_bwd(x, h=None, dy=None, dh=None, gate=None, post_weight=None, res_scale=None, pre_weight=None, *,
                   groups=1, eps=1e-5, residual_dtype=None, workspace=None, out=None, stream=None) -> dict:
    """Gradients of block_norm_fwd (same inputs; `h` is what it returned, needed with pre_weight)
    for dy (the gradient of y, given exactly when pre_weight is) and dh (what reaches h from
    elsewhere; zero when None).

    `residual_dtype`: the residual's dtype when the forward pass had one (then dresidual is
    computed), else None.  Returns a dict with dx, dgate, dresidual, dpost_weight, dres_scale
    and dpre_weight (None where the input is absent).  out["dresidual"] may be dh itself.
    """
    lib = _lib.load_library()
    rows, D, dev = _norm_inputs(x, gate, post_weight, res_scale, pre_weight, groups)
    for t, name in ((h, "h"), (dy, "dy"), (dh, "dh")):
        _shape(t, name, x.shape)
    if (pre_weight is None) != (dy is None):
        raise ValueError("dy is given exactly when pre_weight is")
    if pre_weight is not None and h is None:
        raise ValueError("h (what the forward pass returned) is needed with pre_weight")
    has_residual = residual_dtype is not None
    if residual_dtype is None and (h is not None or dh is not None):
        residual_dtype = (h if h is not None else dh).dtype
    rdtype, rdt = _residual_dtype(residual_dtype, x)
    g = _outputs(out, dev, {"dx": (x.shape, x.dtype, True), "dgate": (x.shape, x.dtype, gate is not None),
                            "dresidual": (x.shape, rdtype, has_residual),
                            "dpost_weight": ((D,), F32, post_weight is not None),
                            "dres_scale": ((D,), F32, res_scale is not None),
                            "dpre_weight": ((D,), F32, pre_weight is not None)})
    ws_ptr, ws_bytes = _workspace(workspace, block_norm_bwd_workspace_size(rows, D), dev)
    (xp, xs), (gp, gs) = _rows(x, "x", D), _rows(gate, "gate", D)
    act = x.dtype
    _lib.check(lib.ssm_block_norm_bwd(
        xp, xs, _ptr(h, "h", rdtype, dev), _ptr(dy, "dy", act, dev), _ptr(dh, "dh", rdtype, dev), gp, gs,
        _ptr(post_weight, "post_weight", F32, dev), _ptr(res_scale, "res_scale", F32, dev),
        _ptr(pre_weight, "pre_weight", F32, dev), _ptr(g["dx"], "dx", act, dev), _ptr(g["dgate"], "dgate", act, dev),
        _ptr(g["dresidual"], "dresidual", rdtype, dev), _ptr(g["dpost_weight"], "dpost_weight", F32, dev),
        _ptr(g["dres_scale"], "dres_scale", F32, dev), _ptr(g["dpre_weight"], "dpre_weight", F32, dev),
        rows, D, int(groups), float(eps), _dt(x), rdt, ws_ptr, ws_bytes, _stream(stream)))
    return g
