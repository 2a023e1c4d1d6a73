"""Plain float64 forms (CPU torch) of the query and key norms with their rotation."""
import torch

F64 = torch.float64


def angles(inv_freq, positions, L):
    """[..., 1, r / 2]: position times frequency."""
    at = torch.arange(L) if positions is None else positions
    return at.to(F64)[..., None, None] * inv_freq.to(F64)


def rotate(n, angle, interleaved):
    """The first 2 * angle.shape[-1] columns of n turned in pairs."""
    r = 2 * angle.shape[-1]
    c, s = angle.cos(), angle.sin()
    a, b = (n[..., 0:r:2], n[..., 1:r:2]) if interleaved else (n[..., :r // 2], n[..., r // 2:r])
    x, y = a * c - b * s, b * c + a * s
    y = torch.stack([x, y], -1).flatten(-2) if interleaved else torch.cat([x, y], -1)
    return torch.cat([y, n[..., r:]], -1)


def qk_norm(x, weight=None, norm="rms", eps=1e-6, inv_freq=None, positions=None, interleaved=False):
    """One of q and k: [batch, L, heads, K] (or [tokens, heads, K])."""
    x = x.to(F64)
    size = x.square().mean(-1, keepdim=True) if norm == "rms" else x.square().sum(-1, keepdim=True)
    n = x / (size + eps).sqrt()
    if weight is not None:
        n = n * weight.to(F64)
    return n if inv_freq is None else rotate(n, angles(inv_freq, positions, x.shape[-3]), interleaved)


def qk_norm_grad(x, dy, weight=None, norm="rms", eps=1e-6, inv_freq=None, positions=None, interleaved=False):
    """(dx, dweight or None)."""
    x, dn = x.to(F64), dy.to(F64)
    if inv_freq is not None:
        dn = rotate(dn, -angles(inv_freq, positions, x.shape[-3]), interleaved)
    mean = (lambda t: t.mean(-1, keepdim=True)) if norm == "rms" else (lambda t: t.sum(-1, keepdim=True))
    r = (mean(x.square()) + eps).rsqrt()
    dw = None
    if weight is not None:
        dw = (dn * x * r).flatten(0, -2).sum(0)
        dn = dn * weight.to(F64)
    return r * (dn - x * r * mean(dn * x * r)), dw
