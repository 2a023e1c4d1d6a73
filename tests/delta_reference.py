"""Plain float64 forms (CPU torch) of the gated delta rule: the token recurrence and its gradient formulas, and inputs
as a layer has them."""
import torch

from lm_reference import heads, share

F64 = torch.float64


def _lengths(B, L, lengths):
    return [L] * B if lengths is None else [int(min(max(x, 0), L)) for x in lengths]


def _live(B, L, lengths):
    n = torch.tensor(_lengths(B, L, lengths))
    return torch.arange(L)[None] < n[:, None]


def _clean(live, *tensors):
    """The tensors with zeros for absent tokens."""
    return [torch.where(live.view(*live.shape, *([1] * (t.dim() - 2))), t.to(F64), torch.zeros((), dtype=F64))
            for t in tensors]


def delta(q, k, v, g, beta, scale, initial_state=None, lengths=None):
    """(out, final_state) of the recurrence, token by token."""
    B, L, H = g.shape
    K, V = q.shape[-1], v.shape[-1]
    live = _live(B, L, lengths)
    q, k, v, g, beta = _clean(live, *(heads(t, H) for t in (q, k, v)), g, beta)
    S = torch.zeros(B, H, K, V, dtype=F64) if initial_state is None else initial_state.to(F64)
    out = torch.zeros(B, L, H, V, dtype=F64)
    for t in range(L):
        on = live[:, t].view(B, 1, 1, 1)
        old = S * g[:, t].exp()[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, None] @ old)[:, :, 0])
        S = torch.where(on, old + k[:, t, :, :, None] * u[:, :, None], S)
        out[:, t] = torch.where(on[..., 0], scale * (q[:, t, :, None] @ S)[:, :, 0], 0.0)
    return out, S


def delta_grad(q, k, v, g, beta, dout, scale, initial_state=None, dfinal_state=None, lengths=None):
    """dict(dq, dk, dv, dg, dbeta, dinitial_state): the recurrence's gradient, token by token."""
    B, L, H = g.shape
    K, V = q.shape[-1], v.shape[-1]
    nq, nk, nv = q.shape[-2], k.shape[-2], v.shape[-2]
    live = _live(B, L, lengths)
    q, k, v, g, beta, do = _clean(live, *(heads(t, H) for t in (q, k, v)), g, beta, dout)
    a = g.exp()[..., None, None]
    S = [torch.zeros(B, H, K, V, dtype=F64) if initial_state is None else initial_state.to(F64)]
    w = torch.zeros(B, L, H, V, dtype=F64)                  # what is wrong under the key: v - a S^T k
    for t in range(L):
        old = S[-1] * a[:, t]
        w[:, t] = v[:, t] - (k[:, t, :, None] @ old)[:, :, 0]
        S.append(old + k[:, t, :, :, None] * (beta[:, t, :, None] * w[:, t])[:, :, None])
    G = torch.zeros(B, H, K, V, dtype=F64) if dfinal_state is None else dfinal_state.to(F64)
    dq, dk, dv = (torch.zeros(B, L, H, d, dtype=F64) for d in (K, K, V))
    dg, db = (torch.zeros(B, L, H, dtype=F64) for _ in range(2))
    for t in range(L - 1, -1, -1):
        old, kt, bt = S[t] * a[:, t], k[:, t], beta[:, t, :, None]
        dq[:, t] = scale * (S[t + 1] @ do[:, t, :, :, None])[..., 0]
        G = G + scale * q[:, t, :, :, None] * do[:, t, :, None]
        du = (kt[:, :, None] @ G)[:, :, 0]
        db[:, t] = (du * w[:, t]).sum(-1)
        dv[:, t] = bt * du
        dk[:, t] = (G @ (bt * w[:, t])[..., None] - old @ dv[:, t, :, :, None])[..., 0]
        G = G - kt[..., None] * dv[:, t, :, None]
        dg[:, t] = torch.where(live[:, t, None], (G * old).sum((-1, -2)), 0.0)
        G = G * a[:, t]
    dq, dk, dv, db = _clean(live, dq, dk, dv, db)
    return dict(dq=share(dq, nq), dk=share(dk, nk), dv=share(dv, nv), dg=dg, dbeta=db, dinitial_state=G)


def inputs(B, L, H, K, V, dtype, heads=None, seed=0, rate=(0.002, 2.0)):
    """dict(q, k, v, g, beta, do), an initial state and a final state's gradient: unit queries and keys with a direction
    in common, decays from slow to fast over the heads."""
    Hq, Hk, Hv = heads or (H, H, H)
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True).clamp(min=1e-6)
    t = dict(q=unit(r(B, L, Hq, K) + 0.3 * r(K)), k=unit(r(B, L, Hk, K) + 0.3 * r(K)), v=r(B, L, Hv, V))
    t = {n: x.to(dtype) for n, x in t.items()}
    t["g"] = -torch.logspace(*torch.log10(torch.tensor(rate)).tolist(), H) * torch.log1p(r(B, L, H).exp())
    t["beta"] = torch.sigmoid(r(B, L, H))
    t["do"] = r(B, L, H, V).to(dtype)
    return t, 0.5 * r(B, H, K, V), r(B, H, K, V)
