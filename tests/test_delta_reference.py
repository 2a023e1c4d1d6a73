"""Pins of the plain float64 forms that the GPU tests of the gated delta rule use: against a state written out as a
product of matrices, automatic differentiation, and differences."""
import pytest
import torch

import delta_reference as ref

F64 = torch.float64


def _case(B=2, L=9, H=4, K=5, V=3, heads=(2, 1, 4), seed=0):
    t, s0, df = ref.inputs(B, L, H, K, V, F64, heads, seed)
    return {n: x.to(F64) for n, x in t.items()}, s0.to(F64), df.to(F64)


def test_products_of_matrices():
    """S_L = sum over t of (product over later s of a_s (I - beta_s k_s k_s^T)) beta_t k_t v_t^T."""
    t, s0, _ = _case(B=1, H=1, heads=(1, 1, 1))
    k, v, a, beta = t["k"][0, :, 0], t["v"][0, :, 0], t["g"][0, :, 0].exp(), t["beta"][0, :, 0]
    S = s0[0, 0].clone()
    eye = torch.eye(5, dtype=F64)
    terms = [S] + [beta[i] * torch.outer(k[i], v[i]) for i in range(9)]
    total = torch.zeros_like(S)
    for i, x in enumerate(terms):
        for s in range(max(i - 1, 0) + (i > 0), 9):
            x = a[s] * (eye - beta[s] * torch.outer(k[s], k[s])) @ x
        total = total + x
    out, S = ref.delta(t["q"], t["k"], t["v"], t["g"], t["beta"], 0.7, s0)
    assert torch.allclose(S[0, 0], total, atol=1e-12)
    assert torch.allclose(out[0, -1, 0], 0.7 * t["q"][0, -1, 0] @ total, atol=1e-12)


def test_orthonormal_keys_replace_values():
    """Unit keys with beta = 1 and no decay: reading a key gives its last value."""
    k = torch.eye(4, dtype=F64)[[0, 1, 0, 2]].view(1, 4, 1, 4)
    v = torch.arange(12, dtype=F64).view(1, 4, 1, 3) + 1
    one, zero = torch.ones(1, 4, 1), torch.zeros(1, 4, 1)
    out, S = ref.delta(k, k, v, zero, one, 1.0)
    assert torch.equal(S[0, 0, 0], v[0, 2, 0]) and torch.equal(S[0, 0, 1], v[0, 1, 0]) and not S[0, 0, 3].any()
    assert torch.equal(out[0, 2, 0], v[0, 2, 0])


@pytest.mark.parametrize("lengths", [None, [4, 9], [0, 1]])
def test_gradient(lengths):
    t, s0, df = _case(seed=3)
    do = t.pop("do")
    leaf = {n: x.clone().requires_grad_() for n, x in t.items()}
    init = s0.clone().requires_grad_()
    out, S = ref.delta(*leaf.values(), 0.3, init, lengths)
    got = torch.autograd.grad((out * do).sum() + (S * df).sum(), [*leaf.values(), init])
    want = ref.delta_grad(*t.values(), do, 0.3, s0, df, lengths)
    assert list(want) == ["d" + n for n in leaf] + ["dinitial_state"]
    for (n, w), x in zip(want.items(), got):
        assert torch.allclose(w, x, atol=1e-11), n


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta"])
def test_differences(name):
    t, s0, df = _case(seed=5)
    do = t.pop("do")
    gen = torch.Generator().manual_seed(1)
    way = torch.randn(t[name].shape, generator=gen, dtype=F64)

    def loss(h):
        x = dict(t)
        x[name] = t[name] + h * way
        out, S = ref.delta(*x.values(), 0.3, s0)
        return float((out * do).sum() + (S * df).sum())

    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    assert abs(slope - float((ref.delta_grad(*t.values(), do, 0.3, s0, df)["d" + name] * way).sum())) < 1e-6 * (1 + abs(slope))


def test_absent_tokens_hold_anything():
    t, s0, df = _case(seed=7)
    clean = {n: x.clone() for n, x in t.items()}
    for x in t.values():
        x[0, 4:] = float("nan")
    do = t.pop("do")
    do_clean = clean.pop("do")
    for x, y in zip(ref.delta(*t.values(), 1.0, s0, [4, 9]), ref.delta(*clean.values(), 1.0, s0, [4, 9])):
        assert torch.equal(x, y)
    want = ref.delta_grad(*clean.values(), do_clean, 1.0, s0, df, [4, 9])
    for n, x in ref.delta_grad(*t.values(), do, 1.0, s0, df, [4, 9]).items():
        assert torch.equal(x, want[n]), n
