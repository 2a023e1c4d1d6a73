"""Plain float64 forms (CPU torch) of the linear attention and block norm operators: the
token recurrence and its gradient formulas; the norms row by row and theirs."""
import torch

F64 = torch.float64


def heads(t, H):
    """[..., heads, d] -> [..., H, d]: state head h uses head h // (H / heads)."""
    return t.to(F64).repeat_interleave(H // t.shape[-2], dim=-2)


def share(t, n):
    """[..., H, d] summed over the state heads that share a head -> [..., n, d]."""
    return t.unflatten(-2, (n, -1)).sum(-2)


def attention(q, k, v, log_decay, scale, initial_state=None, lengths=None):
    """(out, final_state) of the recurrence, token by token."""
    B, L = q.shape[:2]
    H, K, V = log_decay.shape[0], q.shape[-1], v.shape[-1]
    q, k, v = (heads(t, H) for t in (q, k, v))
    lam = log_decay.to(F64).exp()
    n = [L] * B if lengths is None else [int(min(max(x, 0), L)) for x in lengths]
    S = torch.zeros(B, H, K, V, dtype=F64) if initial_state is None else initial_state.to(F64).clone()
    out = torch.zeros(B, L, H, V, dtype=F64)
    for b in range(B):
        for t in range(n[b]):
            S[b] = lam[:, None, None] * S[b] + k[b, t, :, :, None] * v[b, t, :, None, :]
            out[b, t] = scale * (q[b, t, :, None, :] @ S[b])[:, 0]
    return out, S


def attention_grad(q, k, v, log_decay, dout, scale, initial_state=None, dfinal_state=None, lengths=None):
    """dict(dq, dk, dv, dinitial_state): the recurrence's gradient, token by token."""
    B, L = q.shape[:2]
    H, K, V = log_decay.shape[0], q.shape[-1], v.shape[-1]
    nq, nk, nv = q.shape[-2], k.shape[-2], v.shape[-2]
    q, k, v = (heads(t, H) for t in (q, k, v))
    do = dout.to(F64)
    lam = log_decay.to(F64).exp()[:, None, None]
    n = [L] * B if lengths is None else [int(min(max(x, 0), L)) for x in lengths]
    dq, dk, dv = (torch.zeros(B, L, H, d, dtype=F64) for d in (K, K, V))
    d0 = torch.zeros(B, H, K, V, dtype=F64)
    for b in range(B):
        S = torch.zeros(H, K, V, dtype=F64) if initial_state is None else initial_state[b].to(F64).clone()
        for t in range(n[b]):
            S = lam * S + k[b, t, :, :, None] * v[b, t, :, None, :]
            dq[b, t] = scale * (S @ do[b, t, :, :, None])[..., 0]
        G = torch.zeros(H, K, V, dtype=F64) if dfinal_state is None else dfinal_state[b].to(F64).clone()
        for t in range(n[b] - 1, -1, -1):
            G = G + scale * q[b, t, :, :, None] * do[b, t, :, None, :]
            dk[b, t] = (G @ v[b, t, :, :, None])[..., 0]
            dv[b, t] = (k[b, t, :, None, :] @ G)[:, 0]
            G = lam * G
        d0[b] = G
    return dict(dq=share(dq, nq), dk=share(dk, nk), dv=share(dv, nv), dinitial_state=d0)


def block_norm(x, residual=None, gate=None, post_weight=None, res_scale=None, pre_weight=None, groups=1, eps=1e-5):
    """(h, y or None)."""
    t = x.to(F64)
    if post_weight is not None:
        parts = t.unflatten(-1, (groups, -1))
        t = (parts / torch.sqrt((parts * parts).mean(-1, keepdim=True) + eps)).flatten(-2) * post_weight.to(F64)
    if gate is not None:
        z = gate.to(F64)
        t = t * z / (1.0 + torch.exp(-z))
    if res_scale is not None:
        t = t * res_scale.to(F64)
    if residual is not None:
        t = t + residual.to(F64)
    y = None
    if pre_weight is not None:
        y = t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps) * pre_weight.to(F64)
    return t, y


def block_norm_grad(x, h, dy, dh, gate=None, post_weight=None, res_scale=None, pre_weight=None, groups=1, eps=1e-5):
    """dict of every gradient by the formulas, with h as given."""
    x = x.to(F64)
    dH = torch.zeros_like(x) if dh is None else dh.to(F64)
    out = {}
    rows = tuple(range(x.dim() - 1))
    if pre_weight is not None:
        hh, dyy, w = h.to(F64), dy.to(F64), pre_weight.to(F64)
        r2 = 1.0 / torch.sqrt((hh * hh).mean(-1, keepdim=True) + eps)
        out["dpre_weight"] = (dyy * hh * r2).sum(rows)
        a = dyy * w
        dH = dH + r2 * (a - hh * r2 * r2 * (a * hh).mean(-1, keepdim=True))
    out["dresidual"] = dH
    xr, r1 = x, None
    if post_weight is not None:
        parts = x.unflatten(-1, (groups, -1))
        r1 = 1.0 / torch.sqrt((parts * parts).mean(-1, keepdim=True) + eps)
        xr = (parts * r1).flatten(-2)
    n = xr if post_weight is None else xr * post_weight.to(F64)
    act, slope = torch.ones_like(x), None
    if gate is not None:
        z = gate.to(F64)
        sg = torch.sigmoid(z)
        act, slope = z * sg, sg + z * sg * (1.0 - sg)
    dt = dH
    if res_scale is not None:
        out["dres_scale"] = (dH * n * act).sum(rows)
        dt = dH * res_scale.to(F64)
    if gate is not None:
        out["dgate"] = dt * n * slope
    dn = dt * act
    if post_weight is not None:
        out["dpost_weight"] = (dn * xr).sum(rows)
        c = (dn * post_weight.to(F64)).unflatten(-1, (groups, -1))
        p = xr.unflatten(-1, (groups, -1))
        dn = (r1 * (c - p * (c * p).mean(-1, keepdim=True))).flatten(-2)
    out["dx"] = dn
    return out
