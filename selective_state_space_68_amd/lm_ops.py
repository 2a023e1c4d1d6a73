"""Torch-facing wrappers of the linear attention and block norm entry points.

As in ops.py, torch is used for device memory and streams only, and every wrapper
checks the shape, type and device of every tensor before it takes a pointer.
Activations are float32 or bfloat16 tensors of one dtype; states, decays and norm
weights are float32.  q, k, v and the output gradient may be views with a contiguous
last axis (slices of one projection's output); other tensors are contiguous.  `stream=`
is as in ops.py.  Automatic differentiation does not see these calls: a gradient comes from
the _bwd functions, as in the torch.autograd.Functions of examples/linear_attention_lm.py.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import Optional, Tuple

import torch

from . import _lib
from .ops import _elsewhere, _shape, _workspace

F32 = torch.float32
BF16 = torch.bfloat16
_I32 = torch.int32
_Tensor = torch.Tensor

# The checks of a call run before every launch and are most of a small call's time on the
# host, so the passing case is a few comparisons; a failing one goes on to say what is wrong.


def _dt(dtype) -> int:
    if dtype is BF16:
        return _lib.SSM_BF16
    if dtype is F32:
        return _lib.SSM_F32
    raise TypeError(f"activations must be float32 or bfloat16, got {dtype}")


def _dims(t, name: str, n: int) -> None:
    if not isinstance(t, _Tensor) or t.dim() != n:
        raise ValueError(f"{name} must be a tensor of {n} dimensions")


def _is(t, name: str, shape) -> None:
    """_shape for a tuple of ints (None passes)."""
    if t is not None and (not isinstance(t, _Tensor) or t.shape != shape):
        _shape(t, name, shape)


def _device(t, name: str, index: int) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _ptr(t, name: str, dtype, index: int):
    """Pointer of a contiguous tensor of the given type on GPU `index` (None for None)."""
    if t is None:
        return None
    if t.get_device() != index or index < 0:
        _device(t, name, index)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _strides(t, name: str, dtype, index: int):
    """Checks a view with a contiguous last axis; returns a ctypes array of the element
    strides of the axes before it (None: packed)."""
    if t.get_device() != index or index < 0:
        _device(t, name, index)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_contiguous() or t.numel() == 0:
        return None
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last axis")
    return (ctypes.c_int64 * (t.dim() - 1))(*t.stride()[:-1])


def _run(fn, index: int, *args) -> None:
    """Calls fn on GPU `index`'s current stream, with that GPU current."""
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    else:
        status = fn(*args, stream)
    if status:
        _lib.check(status)


def _scratch(workspace, need: int, like):
    """(tensor, pointer, bytes) of the caller's workspace, or of one allocated beside `like`: the
    tensor is held until after the launches, as ops._workspace says."""
    if workspace is None and need == 0:
        return None, None, 0
    return _workspace(workspace, need, like.device)


@lru_cache(maxsize=None)
def _entry(name: str):
    return getattr(_lib.load_library(), name)


def _attention_shapes(q, k, v, log_decay, n: int):
    """Checks q, k, v [..., heads, width] of n dimensions; returns (lead shape, H, Hq, Hk, Hv, K, V)."""
    if not (isinstance(q, _Tensor) and isinstance(k, _Tensor) and isinstance(v, _Tensor) and
            isinstance(log_decay, _Tensor) and q.dim() == k.dim() == v.dim() == n and log_decay.dim() == 1):
        for t, name in ((q, "q"), (k, "k"), (v, "v")):
            _dims(t, name, n)
        _dims(log_decay, "log_decay", 1)
    *lead, Hq, K = q.shape
    Hk, (Hv, V), H = k.shape[-2], v.shape[-2:], log_decay.shape[0]
    _is(k, "k", (*lead, Hk, K))
    _is(v, "v", (*lead, Hv, V))
    for heads, name in ((Hq, "q"), (Hk, "k"), (Hv, "v")):
        if heads < 1 or H % heads:
            raise ValueError(f"{name} has {heads} heads, which does not divide log_decay's {H}")
    return lead, H, Hq, Hk, Hv, K, V


@lru_cache(maxsize=4096)
def linear_attention_workspace_size(batch, L, H, K, V, dtype=BF16) -> int:
    """Bytes of device workspace linear_attention_fwd needs for this shape (0: none)."""
    return int(_entry("ssm_linear_attention_workspace_size")(int(batch), int(L), int(H), int(K), int(V), _dt(dtype)))


@lru_cache(maxsize=4096)
def linear_attention_bwd_workspace_size(batch, L, H, K, V, dtype=BF16, *, Hq=None, Hk=None, Hv=None) -> int:
    """Bytes of device workspace linear_attention_bwd needs (Hq, Hk, Hv: heads of q, k and v, H when None)."""
    return int(_entry("ssm_linear_attention_bwd_workspace_size")(
        int(batch), int(L), int(H), int(Hq or H), int(Hk or H), int(Hv or H), int(K), int(V), _dt(dtype)))


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
    if stream is not None:
        return _elsewhere(linear_attention_fwd, locals())
    (batch, L), H, Hq, Hk, Hv, K, V = _attention_shapes(q, k, v, log_decay, 4)
    states = (batch, H, K, V)
    _is(lengths, "lengths", (batch,))
    _is(initial_state, "initial_state", states)
    _is(out, "out", (batch, L, H, V))
    _is(final_state, "final_state", states)
    act, dev = q.dtype, q.get_device()
    dt = _dt(act)
    qs, ks, vs = _strides(q, "q", act, dev), _strides(k, "k", act, dev), _strides(v, "v", act, dev)
    if out is None:
        out = q.new_empty((batch, L, H, V))
    if final_state is None and return_final_state:
        final_state = q.new_empty(states, dtype=F32)
    ws, ws_ptr, ws_bytes = _scratch(workspace, linear_attention_workspace_size(batch, L, H, K, V, act), q)
    _run(_entry("ssm_linear_attention_fwd"), dev,
         q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, _ptr(log_decay, "log_decay", F32, dev), K ** -0.5 if scale is None else float(scale),
         _ptr(lengths, "lengths", _I32, dev), _ptr(initial_state, "initial_state", F32, dev),
         _ptr(out, "out", act, dev), _ptr(final_state, "final_state", F32, dev), batch, L, H, Hq, Hk, Hv, K, V, dt,
         ws_ptr, ws_bytes)
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
    if stream is not None:
        return _elsewhere(linear_attention_bwd, locals())
    (batch, L), H, Hq, Hk, Hv, K, V = _attention_shapes(q, k, v, log_decay, 4)
    states = (batch, H, K, V)
    if not isinstance(dout, _Tensor):
        raise TypeError("dout must be a torch.Tensor")
    _is(dout, "dout", (batch, L, H, V))
    _is(lengths, "lengths", (batch,))
    _is(initial_state, "initial_state", states)
    _is(dfinal_state, "dfinal_state", states)
    act, dev = q.dtype, q.get_device()
    dt = _dt(act)
    qs, ks, vs = _strides(q, "q", act, dev), _strides(k, "k", act, dev), _strides(v, "v", act, dev)
    ds = _strides(dout, "dout", act, dev)
    want = initial_state is not None if want_dinitial_state is None else want_dinitial_state
    g = _outputs(out, q, {"dq": ((batch, L, Hq, K), act, True), "dk": ((batch, L, Hk, K), act, True),
                            "dv": ((batch, L, Hv, V), act, True), "dinitial_state": (states, F32, want)})
    ws, ws_ptr, ws_bytes = _scratch(
        workspace, linear_attention_bwd_workspace_size(batch, L, H, K, V, act, Hq=Hq, Hk=Hk, Hv=Hv), q)
    _run(_entry("ssm_linear_attention_bwd"), dev,
         q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(), qs, ks, vs, ds, _ptr(log_decay, "log_decay", F32, dev),
         K ** -0.5 if scale is None else float(scale), _ptr(lengths, "lengths", _I32, dev),
         _ptr(initial_state, "initial_state", F32, dev), _ptr(dfinal_state, "dfinal_state", F32, dev),
         _ptr(g["dq"], "dq", act, dev), _ptr(g["dk"], "dk", act, dev), _ptr(g["dv"], "dv", act, dev),
         _ptr(g["dinitial_state"], "dinitial_state", F32, dev), batch, L, H, Hq, Hk, Hv, K, V, dt, ws_ptr, ws_bytes)
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
    if stream is not None:
        return _elsewhere(linear_attention_step, locals())
    (batch,), H, Hq, Hk, Hv, K, V = _attention_shapes(q_t, k_t, v_t, log_decay, 3)
    _dims(state, "state", 4)
    states = state.shape[0]
    _is(state, "state", (states, H, K, V))
    _is(slots, "slots", (batch,))
    _is(out_state, "out_state", state.shape)
    _is(out, "out", (batch, H, V))
    if slots is None and states < batch:
        raise ValueError(f"{batch} rows need as many states, got {states}")
    act, dev = q_t.dtype, state.get_device()
    dt = _dt(act)
    qs, ks, vs = _strides(q_t, "q_t", act, dev), _strides(k_t, "k_t", act, dev), _strides(v_t, "v_t", act, dev)
    state_ptr = _ptr(state, "state", F32, dev)
    if out is None:
        out = q_t.new_empty((batch, H, V))
    _run(_entry("ssm_linear_attention_step"), dev,
         state_ptr, state_ptr if out_state is None else _ptr(out_state, "out_state", F32, dev),
         q_t.data_ptr(), k_t.data_ptr(), v_t.data_ptr(), qs, ks, vs,
         _ptr(log_decay, "log_decay", F32, dev), K ** -0.5 if scale is None else float(scale),
         _ptr(slots, "slots", _I32, dev), _ptr(out, "out", act, dev), batch, states, H, Hq, Hk, Hv, K, V, dt)
    return out


def _outputs(given, like, spec) -> dict:
    """Output tensors by name: the caller's where given (checked), else new ones; None where not computed."""
    got = {}
    for name, (shape, dtype, computed) in spec.items():
        t = (given or {}).get(name)
        if t is not None and computed:
            _is(t, f"out[{name!r}]", tuple(shape))
            if t.dtype != dtype:
                raise TypeError(f"out[{name!r}] must be {dtype}")
            got[name] = t
        else:
            got[name] = like.new_empty(shape, dtype=dtype) if computed else None
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
    """Checks a block norm's inputs; returns (rows, D, the GPU's index)."""
    if not isinstance(x, _Tensor) or x.dim() < 1:
        raise ValueError("expected x [..., D]")
    D = x.shape[-1]
    _is(post_weight, "post_weight", (D,))
    _is(res_scale, "res_scale", (D,))
    _is(pre_weight, "pre_weight", (D,))
    _is(gate, "gate", x.shape)
    if int(groups) < 1 or D % int(groups):
        raise ValueError(f"groups ({groups}) must divide D ({D})")
    dev = x.get_device()
    if dev < 0:
        raise ValueError("x must live on the GPU")
    if gate is not None:
        if gate.get_device() != dev:
            _device(gate, "gate", dev)
        if gate.dtype != x.dtype:
            raise TypeError(f"gate must be {x.dtype}, got {gate.dtype}")
    return x.numel() // D if D else 0, D, dev


def _residual_dtype(dtype, x) -> Tuple[torch.dtype, int]:
    dtype = x.dtype if dtype is None else dtype
    if dtype is not F32 and dtype is not x.dtype:
        raise TypeError(f"the residual stream must be float32 or {x.dtype}, got {dtype}")
    return dtype, _dt(dtype)


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
    if stream is not None:
        return _elsewhere(block_norm_fwd, locals())
    shape = x.shape if isinstance(x, _Tensor) else None
    _is(residual, "residual", shape)
    _is(h, "h", shape)
    _is(y, "y", shape)
    rows, D, dev = _norm_inputs(x, gate, post_weight, res_scale, pre_weight, groups)
    if residual_dtype is None and (residual is not None or h is not None):
        residual_dtype = (residual if residual is not None else h).dtype
    rdtype, rdt = _residual_dtype(residual_dtype, x)
    if pre_weight is None and y is not None:
        raise ValueError("y is computed only with pre_weight")
    if h is None and (return_h or pre_weight is None):
        h = x.new_empty(shape, dtype=rdtype)
    if y is None and pre_weight is not None:
        y = x.new_empty(shape)
    (xp, xs), (gp, gs) = _rows(x, "x", D), _rows(gate, "gate", D)
    act = x.dtype
    _run(_entry("ssm_block_norm_fwd"), dev,
         xp, xs, _ptr(residual, "residual", rdtype, dev), gp, gs, _ptr(post_weight, "post_weight", F32, dev),
         _ptr(res_scale, "res_scale", F32, dev), _ptr(pre_weight, "pre_weight", F32, dev), _ptr(h, "h", rdtype, dev),
         _ptr(y, "y", act, dev), rows, D, int(groups), float(eps), _dt(act), rdt)
    return h, y


@lru_cache(maxsize=4096)
def block_norm_bwd_workspace_size(rows, D) -> int:
    """Bytes of device workspace block_norm_bwd needs."""
    return int(_entry("ssm_block_norm_bwd_workspace_size")(int(rows), int(D)))


def block_norm_bwd(x, h=None, dy=None, dh=None, gate=None, post_weight=None, res_scale=None, pre_weight=None, *,
                   groups=1, eps=1e-5, residual_dtype=None, workspace=None, out=None, stream=None) -> dict:
    """Gradients of block_norm_fwd (same inputs; `h` is what it returned, needed with pre_weight)
    for dy (the gradient of y, given exactly when pre_weight is) and dh (what reaches h from
    elsewhere; zero when None).

    `residual_dtype`: the residual's dtype when the forward pass had one (then dresidual is
    computed), else None.  Returns a dict with dx, dgate, dresidual, dpost_weight, dres_scale
    and dpre_weight (None where the input is absent).  out["dresidual"] may be dh itself.
    """
    if stream is not None:
        return _elsewhere(block_norm_bwd, locals())
    shape = x.shape if isinstance(x, _Tensor) else None
    _is(h, "h", shape)
    _is(dy, "dy", shape)
    _is(dh, "dh", shape)
    if (pre_weight is None) != (dy is None):
        raise ValueError("dy is given exactly when pre_weight is")
    if pre_weight is not None and h is None:
        raise ValueError("h (what the forward pass returned) is needed with pre_weight")
    rows, D, dev = _norm_inputs(x, gate, post_weight, res_scale, pre_weight, groups)
    has_residual = residual_dtype is not None
    if residual_dtype is None and (h is not None or dh is not None):
        residual_dtype = (h if h is not None else dh).dtype
    rdtype, rdt = _residual_dtype(residual_dtype, x)
    g = _outputs(out, x, {"dx": (x.shape, x.dtype, True), "dgate": (x.shape, x.dtype, gate is not None),
                            "dresidual": (x.shape, rdtype, has_residual),
                            "dpost_weight": ((D,), F32, post_weight is not None),
                            "dres_scale": ((D,), F32, res_scale is not None),
                            "dpre_weight": ((D,), F32, pre_weight is not None)})
    ws, ws_ptr, ws_bytes = _scratch(workspace, block_norm_bwd_workspace_size(rows, D), x)
    (xp, xs), (gp, gs) = _rows(x, "x", D), _rows(gate, "gate", D)
    act = x.dtype
    _run(_entry("ssm_block_norm_bwd"), dev,
         xp, xs, _ptr(h, "h", rdtype, dev), _ptr(dy, "dy", act, dev), _ptr(dh, "dh", rdtype, dev), gp, gs,
         _ptr(post_weight, "post_weight", F32, dev), _ptr(res_scale, "res_scale", F32, dev),
         _ptr(pre_weight, "pre_weight", F32, dev), _ptr(g["dx"], "dx", act, dev), _ptr(g["dgate"], "dgate", act, dev),
         _ptr(g["dresidual"], "dresidual", rdtype, dev), _ptr(g["dpost_weight"], "dpost_weight", F32, dev),
         _ptr(g["dres_scale"], "dres_scale", F32, dev), _ptr(g["dpre_weight"], "dpre_weight", F32, dev),
         rows, D, int(groups), float(eps), _dt(act), rdt, ws_ptr, ws_bytes)
    return g
