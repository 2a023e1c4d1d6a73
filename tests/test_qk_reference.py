"""Pins of the plain float64 forms that the GPU tests of the query and key norms use."""
import math

import pytest
import torch

import qk_reference as ref

F64 = torch.float64


def _case(K=10, rotary=6, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=F64)
    return r(2, 5, 3, K), r(2, 5, 3, K), r(K), 1.0 / (1.0 + torch.arange(rotary // 2, dtype=F64))


def test_sizes():
    x, _, _, _ = _case()
    assert torch.allclose(ref.qk_norm(x, eps=0.0).square().mean(-1), torch.ones(2, 5, 3, dtype=F64))
    assert torch.allclose(ref.qk_norm(x, norm="l2", eps=0.0).square().sum(-1), torch.ones(2, 5, 3, dtype=F64))


@pytest.mark.parametrize("interleaved", [False, True])
def test_turns(interleaved):
    """Pair i of a unit of its first member goes to (cos, sin); products of queries and keys see differences of positions."""
    freq = torch.tensor([0.5, 2.0], dtype=F64)
    n = torch.zeros(1, 1, 1, 6, dtype=F64)
    n[..., 0] = 1.0
    y = ref.rotate(n, ref.angles(freq, torch.tensor([[3]]), 1), interleaved)[0, 0, 0]
    want = torch.zeros(6, dtype=F64)
    want[0], want[1 if interleaved else 2] = math.cos(1.5), math.sin(1.5)
    assert torch.allclose(y, want)
    x, z, _, freq = _case()
    at = torch.tensor([[7, 8, 9, 10, 11], [0, 1, 2, 3, 4]])
    score = lambda shift: (ref.rotate(x, ref.angles(freq, at + shift, 5), interleaved)[:, :1] *
                           ref.rotate(z, ref.angles(freq, at + shift, 5), interleaved)).sum(-1)
    assert torch.allclose(score(0), score(100))


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_gradient(norm, interleaved, weighted):
    x, dy, w, freq = _case(seed=3)
    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    named = dict(norm=norm, inv_freq=freq, interleaved=interleaved)
    y = ref.qk_norm(xr, wr if weighted else None, **named)
    got = torch.autograd.grad((y * dy).sum(), [xr] + [wr] * weighted)
    dx, dw = ref.qk_norm_grad(x, dy, w if weighted else None, **named)
    assert torch.allclose(dx, got[0], atol=1e-12)
    assert (dw is None) == (not weighted) and (dw is None or torch.allclose(dw, got[1], atol=1e-12))


def test_differences():
    x, dy, w, freq = _case(seed=5)
    way = _case(seed=6)[0]
    loss = lambda h: float((ref.qk_norm(x + h * way, w, inv_freq=freq) * dy).sum())
    slope = (loss(1e-6) - loss(-1e-6)) / 2e-6
    assert abs(slope - float((ref.qk_norm_grad(x, dy, w, inv_freq=freq)[0] * way).sum())) < 1e-6
