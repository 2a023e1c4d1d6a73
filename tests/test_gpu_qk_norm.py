"""GPU parity of the query and key norms with their formulas in float64.

Bounds, value by value against a row's largest value: a row's sum of up to 256 squares, its root, two products, two
angle functions (5e-7: sincospi of a float32 fraction of a turn, 2^-25 of a turn off, and its own rounding) and a sum of two
products are off by at most (256 / 2 + 8) * 2^-24 + 5e-7 = 8.6e-6 in float32, backwards (which has two such sums) twice
that; bfloat16 outputs by 2^-8 of the value more.  Weights' gradients are float32 sums over rows in parts: against the
root of the sum of their terms' squares times the root of the terms that one lane adds in a row (at most 2^12 here),
2^-24 * 64 = 4e-6.
"""
import pytest
import torch

import qk_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = 8.6e-6


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _ssm():
    import selective_state_space_68_amd as ssm
    return ssm


def _check(got, want, what, sums=1):
    got = got.detach().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all()
    if not want.numel():
        return
    bound = sums * TOL * want.abs().amax(-1, keepdim=True) + (2.0 ** -8 if got.dtype == BF16 else 0.0) * want.abs()
    over = (got.double() - want).abs() - bound
    print(f"{what} {tuple(got.shape)} {got.dtype}: {float((got.double() - want).abs().max()):.2e}", flush=True)
    assert float(over.max()) <= 1e-30, (what, float(over.max()))


def _check_weight(got, x, dy, what, **named):
    """The weight's gradient against the size of its terms."""
    K = x.shape[-1]
    _, want = ref.qk_norm_grad(x, dy, torch.ones(K), **named)
    n = ref.qk_norm(x, None, **{**named, "inv_freq": None})
    turned = dy.double()
    if named.get("inv_freq") is not None:
        turned = ref.rotate(turned, -ref.angles(named["inv_freq"], named.get("positions"), x.shape[-3]),
                            named.get("interleaved", False))
    size = (turned * n).flatten(0, -2).square().sum(0).sqrt()
    error = ((got.double().cpu() - want).abs() / size.clamp(min=1e-30)).max()
    print(f"{what}: {float(error):.2e}", flush=True)
    assert float(error) <= 4e-6 + TOL, (what, float(error))


def _case(B, L, Hq, Hk, K, dtype, rotary, seed=0, far=1000):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    t = dict(q=r(B, L, Hq, K).to(dtype), k=(3.0 * r(B, L, Hk, K)).to(dtype), dq=r(B, L, Hq, K).to(dtype),
             dk=r(B, L, Hk, K).to(dtype), qw=1 + 0.3 * r(K), kw=1 + 0.3 * r(K))
    freq = 10000.0 ** (-torch.arange(rotary // 2) * 2.0 / rotary) if rotary else None
    positions = torch.randint(0, far, (B, L), generator=gen, dtype=torch.int32) if rotary else None
    return t, freq, positions


def _on(t):
    return None if t is None else t.cuda()


def _all(t, freq, positions, dtype, norm, interleaved, weighted, eps=1e-6):
    ssm = _ssm()
    d = {n: x.cuda() for n, x in t.items()}
    w = (d["qw"], d["kw"]) if weighted else (None, None)
    named = dict(norm=norm, eps=eps, inv_freq=_on(freq), positions=_on(positions), interleaved=interleaved)
    host = dict(norm=norm, eps=eps, inv_freq=freq, positions=positions, interleaved=interleaved)
    q, k = ssm.qk_norm_fwd(d["q"], d["k"], *w, **named)
    g = ssm.qk_norm_bwd(d["q"], d["k"], d["dq"], d["dk"], *w, **named)
    for n, y in (("q", q), ("k", k)):
        weight = t[n + "w"] if weighted else None
        _check(y, ref.qk_norm(t[n], weight, **host), n)
        dx, _ = ref.qk_norm_grad(t[n], t["d" + n], weight, **host)
        _check(g["d" + n], dx, "d" + n, _times(dx, t, n, weight, host))
        if weighted:
            _check_weight(g[f"d{n}_weight"], t[n], t["d" + n], f"d{n}_weight", **host)
        else:
            assert g[f"d{n}_weight"] is None


def _times(dx, t, n, weight, host):
    """Two sums, times how far the terms of a row's difference, r w dn, may exceed the row's largest value."""
    x, dy = t[n].double(), t["d" + n].double()
    size = x.square().mean(-1, keepdim=True) if host["norm"] == "rms" else x.square().sum(-1, keepdim=True)
    terms = (size + host["eps"]).rsqrt() * dy.abs().amax(-1, keepdim=True) * 2.0 ** 0.5
    terms = terms if weight is None else terms * weight.double().abs().amax()
    return 2 * (terms / dx.abs().amax(-1, keepdim=True).clamp(min=1e-30)).clamp(min=1.0)


SHAPES = [   # batch, L, heads of q and k, K, rotary
    (1, 1, 1, 1, 64, 64),
    (2, 7, 4, 2, 128, 128),
    (1, 33, 3, 3, 128, 64),              # part of the columns
    (2, 5, 2, 1, 80, 0),
    (1, 9, 5, 3, 77, 30),                # one by one
    (3, 4, 2, 2, 100, 100),
    (1, 6, 3, 2, 256, 256),
    (1, 6, 3, 2, 192, 96),
    (2, 3, 2, 1, 255, 254),
    (1, 3, 1, 1, 1, 0),
    (1, 4, 2, 1, 2, 2),
    (2, 300, 9, 3, 96, 8),
    (1, 700, 33, 4, 32, 32),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("norm,interleaved,weighted", [("rms", False, True), ("l2", True, False), ("l2", False, True)])
@pytest.mark.parametrize("B,L,Hq,Hk,K,rotary", SHAPES)
def test_parity(B, L, Hq, Hk, K, rotary, norm, interleaved, weighted, dtype):
    t, freq, positions = _case(B, L, Hq, Hk, K, dtype, rotary, seed=K + L)
    _all(t, freq, positions, dtype, norm, interleaved, weighted)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K", [128, 126])
def test_far_positions(K, dtype):
    """Positions up to 2^31 - 1 and below 0: angles far past what float32 holds."""
    t, freq, _ = _case(1, 6, 2, 1, K, dtype, K, seed=1)
    positions = torch.tensor([[2 ** 31 - 1, 10 ** 6, 131071, 0, -5, -2 ** 31]], dtype=torch.int32)
    _all(t, freq, positions, dtype, "rms", False, True)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forms(dtype):
    """Views of a projection, packed copies, in place, tokens without a batch, queries alone: the same bits."""
    ssm = _ssm()
    gen = torch.Generator("cuda").manual_seed(2)
    z = torch.randn(2, 40, 8, 64, device="cuda", generator=gen).to(dtype)
    q, k = z[:, :, :5], z[:, :, 5:7]
    freq = (1.0 / (1 + torch.arange(16.0))).cuda()
    at = torch.randint(0, 9999, (2, 40), device="cuda", generator=gen, dtype=torch.int32)
    w = 1 + torch.randn(64, device="cuda", generator=gen)
    before = z.clone()
    qo, ko = ssm.qk_norm_fwd(q, k, w, w, inv_freq=freq, positions=at)
    assert torch.equal(z, before)
    qc, kc = q.contiguous(), k.contiguous()
    q2, k2 = ssm.qk_norm_fwd(qc, kc, w, w, inv_freq=freq, positions=at, q_out=qc, k_out=kc)
    assert q2 is qc and torch.equal(qo, q2) and torch.equal(ko, k2)
    q3, none = ssm.qk_norm_fwd(q, None, w, inv_freq=freq, positions=at)
    assert none is None and torch.equal(qo, q3)
    q4, k4 = ssm.qk_norm_fwd(q.flatten(0, 1), k.flatten(0, 1), w, w, inv_freq=freq, positions=at.flatten())
    assert torch.equal(qo.flatten(0, 1), q4) and torch.equal(ko.flatten(0, 1), k4)
    q5, _ = ssm.qk_norm_fwd(q, k, w, w, inv_freq=freq)                          # positions 0..39 in both rows
    q6, _ = ssm.qk_norm_fwd(q, k, w, w, inv_freq=freq, positions=torch.arange(40, device="cuda").int().expand(2, 40).contiguous())
    assert torch.equal(q5, q6)
    dz = torch.randn(2, 40, 8, 64, device="cuda", generator=gen).to(dtype)
    dq, dk = dz[:, :, 1:6], dz[:, :, 6:]
    g = ssm.qk_norm_bwd(q, k, dq, dk, w, w, inv_freq=freq, positions=at)
    dqc, dkc = dq.contiguous(), dk.contiguous()
    g2 = ssm.qk_norm_bwd(q, k, dqc, dkc, w, w, inv_freq=freq, positions=at, out={"dq": dqc, "dk": dkc})
    assert g2["dq"] is dqc and all(torch.equal(g[n], g2[n]) for n in g)
    g3 = ssm.qk_norm_bwd(q, None, dq, None, w, inv_freq=freq, positions=at)
    assert torch.equal(g3["dq"], g["dq"]) and g3["dk"] is None and g3["dk_weight"] is None
    # rows that do not start at pieces of 4 elements give the same values to rounding
    odd = torch.empty(2, 40, 8, 65, device="cuda", dtype=dtype)[..., 1:]
    odd.copy_(z)
    q7, _ = ssm.qk_norm_fwd(odd[:, :, :5], odd[:, :, 5:7], w, w, inv_freq=freq, positions=at)
    _check(q7, qo.double().cpu(), "odd rows")


def test_zero_rows_and_no_tokens():
    ssm = _ssm()
    z = torch.zeros(1, 3, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    q, _ = ssm.qk_norm_fwd(z, z, w, w)
    assert not q.any()
    g = ssm.qk_norm_bwd(z, z, torch.ones_like(z), z, w, w, eps=0.25)
    assert torch.allclose(g["dq"], torch.full_like(z, 2.0)) and not g["dq_weight"].any()
    none = torch.empty(1, 0, 2, 64, device="cuda")
    q, k = ssm.qk_norm_fwd(none, none, w, w)
    assert q.shape == none.shape
    out = {"dq_weight": torch.ones(64, device="cuda"), "dk_weight": torch.ones(64, device="cuda")}
    ssm.qk_norm_bwd(none, none, none, none, w, w, out=out)
    assert not out["dq_weight"].any() and not out["dk_weight"].any()


@pytest.mark.parametrize("K", [64, 50])
def test_small_rows_without_eps(K):
    # a mean square of 10^-38 is below 2^-126; its parts are rounded to 2^-149, so that it is off by 7e-8 more than counted above
    gen = torch.Generator().manual_seed(4)
    q = torch.randn(1, 9, 3, K, generator=gen) * 1e-19
    got, _ = _ssm().qk_norm_fwd(q.cuda(), eps=0.0)
    _check(got, ref.qk_norm(q, None, eps=0.0), "rows of 1e-19", sums=1.01)


def test_gradient_differences():
    """A step of 2^-8 along a direction in float32: the outputs move by the gradient's products, to the step's own square."""
    ssm = _ssm()
    t, freq, positions = _case(1, 5, 2, 1, 64, F32, 32, seed=9)
    d = {n: x.cuda() for n, x in t.items()}
    way = torch.randn(1, 5, 2, 64, generator=torch.Generator().manual_seed(4)).cuda()
    named = dict(inv_freq=freq.cuda(), positions=positions.cuda())
    h = 2.0 ** -8
    f = lambda s: ssm.qk_norm_fwd(d["q"] + s * h * way, d["k"], d["qw"], d["kw"], **named)[0].double()
    slope = ((f(1) - f(-1)) * d["dq"].double()).sum() / (2 * h)
    g = ssm.qk_norm_bwd(d["q"], d["k"], d["dq"], d["dk"], d["qw"], d["kw"], **named)["dq"]
    want = (g.double() * way.double()).sum()
    # central differences: h^2 / 6 times a third derivative, a few |way|^3 / |x|^3 of the outputs: below 2^-16 of |dq| |way|
    assert abs(float(slope - want)) <= 2.0 ** -14 * float(d["dq"].norm() * way.norm())


def test_deterministic():
    ssm = _ssm()
    t, freq, positions = _case(4, 3000, 6, 2, 128, BF16, 128, seed=3)
    d = {n: x.cuda() for n, x in t.items()}
    run = lambda: ssm.qk_norm_bwd(d["q"], d["k"], d["dq"], d["dk"], d["qw"], d["kw"], inv_freq=freq.cuda(), positions=positions.cuda())
    a, b = run(), run()
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_views_past_32_bits_of_elements():
    """Tokens 2^30 elements apart: the bits of packed copies."""
    t, freq, positions = _case(1, 3, 2, 1, 64, BF16, 64, seed=6)
    space = torch.empty(2 ** 31 + 4096, dtype=BF16, device="cuda")

    def far(x, at):
        v = space.as_strided(x.shape, (x[0].numel(), 2 ** 30, x.shape[-1], 1), at)
        return v.copy_(x.cuda())

    q, k, dq, dk = (far(t[n], 512 * i) for i, n in enumerate(("q", "k", "dq", "dk")))
    ssm, named = _ssm(), dict(inv_freq=freq.cuda(), positions=positions.cuda())
    weights = t["qw"].cuda(), t["kw"].cuda()
    for x, y in zip(ssm.qk_norm_fwd(q, k, *weights, **named),
                    ssm.qk_norm_fwd(t["q"].cuda(), t["k"].cuda(), *weights, **named)):
        assert torch.equal(x, y)
    a = ssm.qk_norm_bwd(q, k, dq, dk, *weights, **named)
    b = ssm.qk_norm_bwd(*(t[n].cuda() for n in ("q", "k", "dq", "dk")), *weights, **named)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_outputs_past_32_bits_of_elements():
    L = 2 ** 20 + 33
    q = torch.randn(1, L, 1, 64, device="cuda", dtype=BF16, generator=torch.Generator("cuda").manual_seed(5)).expand(1, L, 32, 64)
    freq = torch.linspace(1.0, 0.001, 32, device="cuda")
    out, _ = _ssm().qk_norm_fwd(q, norm="l2", inv_freq=freq)
    assert out.numel() > 2 ** 31
    for at in (0, 2 ** 19, L - 40):
        pos = torch.arange(at, at + 40, dtype=torch.int32, device="cuda")[None]
        part, _ = _ssm().qk_norm_fwd(q[:, at:at + 40], norm="l2", inv_freq=freq, positions=pos)
        assert torch.equal(part, out[:, at:at + 40])
