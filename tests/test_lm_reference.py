"""The float64 forms that the linear attention and block norm tests compare with, checked
by themselves on the CPU: against the quadratic form, automatic differentiation and
differences."""
import pytest
import torch

import lm_reference as ref

F64 = torch.float64


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, dtype=F64)


def _attention_inputs(seed, B=2, L=9, H=4, heads=(4, 2, 1), K=3, V=5):
    gen = torch.Generator().manual_seed(seed)
    q, k = (_rand(gen, B, L, n, K) for n in heads[:2])
    v = _rand(gen, B, L, heads[2], V)
    g = -torch.rand(H, generator=gen, dtype=F64)
    return gen, q, k, v, g, _rand(gen, B, H, K, V)


def test_recurrence_equals_the_quadratic_form():
    _, q, k, v, g, s0 = _attention_inputs(0)
    B, L, H = 2, 9, 4
    out, fin = ref.attention(q, k, v, g, 0.7, s0)
    Q, K, V = (ref.heads(t, H).transpose(1, 2) for t in (q, k, v))
    i = torch.arange(L, dtype=F64)
    off = i[:, None] - i[None]
    M = torch.where(off >= 0, torch.exp(g[:, None, None] * off), 0.0)
    want = ((Q @ K.transpose(-1, -2)) * M) @ V + (Q * torch.exp(g[:, None] * (i + 1))[..., None]) @ s0
    assert torch.allclose(out, 0.7 * want.transpose(1, 2), rtol=1e-12, atol=1e-12)
    w = torch.exp(g[:, None] * (L - 1 - i))
    assert torch.allclose(fin, (K * w[..., None]).transpose(-1, -2) @ V + torch.exp(g * L)[:, None, None] * s0,
                          rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("lengths", [None, (9, 4), (0, 1)])
def test_attention_gradient_against_differentiation_and_differences(lengths):
    gen, q, k, v, g, s0 = _attention_inputs(1)
    do, df = _rand(gen, 2, 9, 4, 5), _rand(gen, 2, 4, 3, 5)
    n = [9, 9] if lengths is None else lengths
    got = ref.attention_grad(q, k, v, g, do, 0.7, s0, df, lengths)

    def loss(q, k, v, s0):                                  # the quadratic form, so that it can be differentiated
        total = 0.0
        for b in range(2):
            L = n[b]
            Q, K, V = (ref.heads(t[b:b + 1, :L], 4).transpose(1, 2)[0] for t in (q, k, v))
            i = torch.arange(L, dtype=F64)
            off = i[:, None] - i[None]
            M = torch.where(off >= 0, torch.exp(g[:, None, None] * off), 0.0)
            o = 0.7 * (((Q @ K.transpose(-1, -2)) * M) @ V + (Q * torch.exp(g[:, None] * (i + 1))[..., None]) @ s0[b])
            w = torch.exp(g[:, None] * (L - 1 - i))
            fin = (K * w[..., None]).transpose(-1, -2) @ V + torch.exp(g * L)[:, None, None] * s0[b]
            total = total + (o.transpose(0, 1) * do[b, :L]).sum() + (fin * df[b]).sum()
        return total

    leaves = [t.clone().requires_grad_() for t in (q, k, v, s0)]
    for name, want in zip(("dq", "dk", "dv", "dinitial_state"), torch.autograd.grad(loss(*leaves), leaves)):
        assert torch.allclose(got[name], want, rtol=1e-10, atol=1e-10), name
    # differences of the recurrence itself: linear in each argument alone, so a step of 1 has no truncation
    f = lambda *a: sum((x * y).sum() for x, y in zip(ref.attention(a[0], a[1], a[2], g, 0.7, a[3], lengths), (do, df)))
    for j, name in enumerate(("dq", "dk", "dv", "dinitial_state")):
        args = [q, k, v, s0]
        d = _rand(gen, *args[j].shape)
        up, down = list(args), list(args)
        up[j], down[j] = args[j] + d, args[j] - d
        diff = float(f(*up) - f(*down)) / 2
        assert diff == pytest.approx(float((got[name] * d).sum()), rel=1e-9, abs=1e-9), name


@pytest.mark.parametrize("parts", ["all", "no_gate", "no_residual", "pre_only", "gated_only"])
def test_block_norm_gradient_against_differentiation_and_differences(parts):
    gen = torch.Generator().manual_seed(2)
    a = dict(x=_rand(gen, 3, 24), residual=_rand(gen, 3, 24), gate=_rand(gen, 3, 24), post_weight=_rand(gen, 24),
             res_scale=_rand(gen, 24), pre_weight=_rand(gen, 24))
    for k in {"all": (), "no_gate": ("gate",), "no_residual": ("residual", "res_scale"),
              "pre_only": ("residual", "gate", "post_weight", "res_scale"),
              "gated_only": ("residual", "res_scale", "pre_weight")}[parts]:
        a[k] = None
    dy, dh = _rand(gen, 3, 24), _rand(gen, 3, 24)
    h, _ = ref.block_norm(**a, groups=3)
    got = ref.block_norm_grad(a["x"], h, dy, dh, a["gate"], a["post_weight"], a["res_scale"], a["pre_weight"], groups=3)

    def loss(**kw):
        h, y = ref.block_norm(**kw, groups=3)
        return (h * dh).sum() + (0.0 if y is None else (y * dy).sum())

    names = [k for k in a if a[k] is not None]
    leaves = {k: a[k].clone().requires_grad_() for k in names}
    grads = torch.autograd.grad(loss(**{**a, **leaves}), [leaves[k] for k in names])
    for k, want in zip(names, grads):
        assert torch.allclose(got["d" + k], want, rtol=1e-10, atol=1e-10), k
        d = _rand(gen, *a[k].shape)
        step = 1e-5                                         # truncation ~1e-10, rounding ~1e-10
        diff = float(loss(**{**a, k: a[k] + step * d}) - loss(**{**a, k: a[k] - step * d})) / (2 * step)
        assert diff == pytest.approx(float((want * d).sum()), rel=1e-6, abs=1e-6), k
