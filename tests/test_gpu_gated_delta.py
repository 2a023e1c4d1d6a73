"""GPU parity of the gated delta rule (prompt form, single token) with the token recurrence in float64.

Error of a row (one token's V values of one head; one row of a state): the 2-norm of the difference over the row's own
2-norm plus the root mean square 2-norm of that head's rows.  Bounds, from the roundings on the way:
  float32  a chunk's value is a sum of at most 128 + 64 products, as is each of the three before it in the chain (K E, T X,
           the state), in float32: 4 * 192 * 2^-24 = 4.6e-5 of the terms' size if all roundings agreed, and the square
           root of their number, 4 * sqrt(192) * 2^-24 = 3.3e-6, times the few sizes that a term may exceed its head's
           mean by, as they fall: 2e-5.
  states   float32 from operands of 24 bits (bfloat16 inputs included): the same 2e-5.
  the initial state's gradient is what its first chunk leaves of the gradient that enters it, exp(G_Q) F - K^T (beta
           exp(G) Y) + scale (exp(G) Q)^T D: where the keys are alike the terms cancel (with K = 1 a chunk takes the
           product of 64 factors 1 - beta off F), and float32 sums are good to 2^-24 of their terms, not of what is
           left.  The terms' 2-norms are added to that row's size.
  bfloat16 outputs: rounded by up to 2^-8 of each value, operands of 16 bits before that (2^-16 a product, far below):
           2^-8 * 1.02 + 2e-5.
"""
import pytest
import torch

import delta_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
OUT = {F32: 2e-5, BF16: 2.0 ** -8 * 1.02 + 2e-5}
STATE = 2e-5


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _ssm():
    import selective_state_space_68_amd as ssm
    return ssm


def _first_chunk_terms(t, s0, df, scale):
    """[B, H, K]: the 2-norms of the terms whose sum is the initial state's gradient, row by row."""
    H = t["g"].shape[-1]
    x = {n: ref.heads(t[n], H) if n in "qkv" else t[n].double() for n in t}
    first, rest = ({n: y[:, i] for n, y in x.items()} for i in (slice(0, 64), slice(64, None)))
    state = ref.delta(*(first[n] for n in ("q", "k", "v", "g", "beta")), scale, s0)[1]
    F = ref.delta_grad(*rest.values(), scale, state, df)["dinitial_state"]
    dv = ref.delta_grad(*first.values(), scale, s0, F)["dv"]
    decay = first["g"].cumsum(1).exp()                          # [B, L, H]
    both = first["k"].abs() * dv.norm(dim=-1, keepdim=True) + scale * first["q"].abs() * first["do"].norm(dim=-1, keepdim=True)
    return decay[:, -1, :, None] * F.norm(dim=-1) + (decay[..., None] * both).sum(1)


def _check(got, want, tol, what, more=0.0):
    got, want = got.detach().double().cpu(), want.double()
    assert got.shape == want.shape
    assert torch.isfinite(got).all(), what
    d, r = (got - want).norm(dim=-1), want.norm(dim=-1)
    if d.numel() == 0:
        return
    axes = (0, 1) if d.dim() == 3 and "state" not in what else (0, 2)
    size = r + r.square().mean(axes, keepdim=True).sqrt() + more
    e = float((d / size.clamp(min=1e-30)).max()) if float(d.max()) > 0 else 0.0
    print(f"{what} {tuple(got.shape)}: {e:.2e}", flush=True)
    assert e <= tol, (what, e)


def _cuda(t):
    return {n: x.cuda() for n, x in t.items()}


def _forward(t, s0=None, lengths=None, scale=None, **named):
    d = _cuda(t)
    return _ssm().gated_delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], scale,
                                  initial_state=None if s0 is None else s0.cuda(),
                                  lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda(),
                                  **named)


def _want(t, scale, s0=None, lengths=None):
    return ref.delta(t["q"], t["k"], t["v"], t["g"], t["beta"], scale, s0, lengths)


SHAPES = [   # batch, L, H, K, V, heads of q, k, v
    (1, 1, 1, 64, 64, None),
    (2, 64, 2, 64, 64, None),
    (1, 65, 2, 128, 128, None),
    (2, 200, 4, 64, 128, (4, 2, 2)),
    (1, 130, 6, 128, 64, (2, 6, 3)),
    (2, 77, 3, 72, 40, (1, 1, 3)),       # vectors, tiles partly empty
    (1, 129, 2, 33, 17, None),           # element by element
    (1, 70, 1, 1, 1, None),
    (3, 63, 2, 100, 128, (2, 1, 1)),
    (2, 193, 2, 100, 100, None),         # words
    (1, 140, 3, 34, 98, (3, 1, 1)),
    (2, 300, 2, 128, 50, (1, 2, 2)),
    (1, 1500, 2, 128, 128, None),
    (1, 1100, 2, 100, 36, (1, 2, 2)),
    (1, 1030, 1, 33, 17, None),
    (1, 1200, 2, 96, 128, None),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,H,K,V,heads", SHAPES)
def test_forward(B, L, H, K, V, heads, dtype):
    t, s0, _ = ref.inputs(B, L, H, K, V, dtype, heads, seed=L + K)
    out, fin = _forward(t, s0)
    want, wfin = _want(t, K ** -0.5, s0)
    _check(out, want, OUT[dtype], "out")
    _check(fin, wfin, STATE, "final_state")
    out2, none = _forward(t, scale=0.3, return_final_state=False)
    assert none is None
    _check(out2, _want(t, 0.3)[0], OUT[dtype], "out")


def _gradient(t, s0=None, df=None, lengths=None, scale=None, **named):
    d = _cuda(t)
    return _ssm().gated_delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], scale,
                                  initial_state=None if s0 is None else s0.cuda(),
                                  dfinal_state=None if df is None else df.cuda(),
                                  lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda(),
                                  **named)


def _check_grads(got, want, dtype, terms=0.0):
    """g's and beta's gradients are float32 and a row of theirs is a head's tokens."""
    for n, w in want.items():
        if got[n] is None:
            continue
        if n in ("dg", "dbeta"):
            _check(got[n].transpose(1, 2)[:, :, None], w.transpose(1, 2)[:, :, None], OUT[F32], n)
        else:
            _check(got[n], w, STATE if "state" in n else OUT[dtype], n, terms if "state" in n else 0.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,H,K,V,heads", SHAPES)
def test_gradient(B, L, H, K, V, heads, dtype):
    t, s0, df = ref.inputs(B, L, H, K, V, dtype, heads, seed=L + V)
    got = _gradient(t, s0, df)
    want = ref.delta_grad(*t.values(), K ** -0.5, s0, df)
    assert got.keys() == want.keys()
    _check_grads(got, want, dtype, _first_chunk_terms(t, s0, df, K ** -0.5))
    got = _gradient(t, scale=0.3)
    assert got["dinitial_state"] is None
    _check_grads(got, ref.delta_grad(*t.values(), 0.3), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_absent_tokens_hold_anything(dtype):
    B, L, H, K, V = 6, 150, 3, 64, 72
    lengths = [150, 0, 1, 64, 65, 149]
    t, s0, _ = ref.inputs(B, L, H, K, V, dtype, (3, 1, 1), seed=3)
    absent = torch.arange(L)[None] >= torch.tensor(lengths)[:, None]
    bad = {n: x.clone() for n, x in t.items()}
    for i, x in enumerate(bad.values()):
        x[absent] = (float("nan"), float("inf"), float("-inf"), float("nan"), float("inf"), torch.finfo(dtype).min)[i]
    out, fin = _forward(bad, s0, lengths)
    want, wfin = _want(t, K ** -0.5, s0, lengths)
    _check(out, want, OUT[dtype], "out")
    _check(fin, wfin, STATE, "final_state")
    assert not out.cpu()[absent].any()
    assert torch.equal(fin[1].cpu(), s0[1])                 # no token: the state as it was
    out2, fin2 = _forward(t, s0, [1000, -5, 1, 64, 65, 149])    # clamped to [0, L]
    assert torch.equal(out2, out) and torch.equal(fin2, fin)
    df = torch.randn(B, H, K, V, generator=torch.Generator().manual_seed(2))
    got = _gradient(bad, s0, df, lengths)
    _check_grads(got, ref.delta_grad(*t.values(), K ** -0.5, s0, df, lengths), dtype)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert not got[n].cpu()[absent].any(), n
    assert torch.equal(got["dinitial_state"][1].cpu(), df[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (72, 33)])
def test_step(K, V, dtype):
    """The step from a pool, and the prompt form continued by it, against the recurrence over all tokens."""
    B, L, H = 4, 70, 6
    t, s0, _ = ref.inputs(B, L, H, K, V, dtype, (3, 2, 6), seed=K + V)
    want, wfin = _want(t, K ** -0.5, s0)
    cut = 60
    _, fin = _forward({n: x[:, :cut] for n, x in t.items()}, s0)
    gen = torch.Generator("cuda").manual_seed(1)
    pool = torch.randn(7, H, K, V, device="cuda", generator=gen)
    before = pool.clone()
    slots = torch.tensor([5, 0, 6, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = fin
    for i in range(cut, L):
        d = {n: x[:, i].cuda() for n, x in t.items()}
        out = _ssm().gated_delta_step(pool, d["q"], d["k"], d["v"], d["g"], d["beta"], slots=slots)
        _check(out[:, None], want[:, i:i + 1], OUT[dtype], f"out {i}")
    _check(pool[slots.long()], wfin, STATE, "final_state")
    for i in (1, 3, 4):
        assert torch.equal(pool[i], before[i])
