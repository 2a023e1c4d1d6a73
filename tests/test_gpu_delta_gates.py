"""The gated delta rule's gradient of g where decays are fast: dg_t is a_t times what passes token t, and has to be as
good as that, though the outputs' and values' gradients beside it are of order 1.

The reference is the recurrence in float64.  With P the gradient of the decayed state and S the state before a token,
dg_t = a_t <P, S>.  An error is compared with |dg_t| + a_t |P| |S| / sqrt(K V), the size that the product of such
states has where they point anywhere; in heads of slow decays, whose tokens share their sums, also with the root mean
square of that head's dg.  Bounds: dg_t is a sum of parts that each carry a_t, of the same chains of float32 sums of 64 to
192 products as the other gradients, 2e-5 as derived for those; with bfloat16 activations some operands have two
terms, good to 2^-17 each, and a product of two such leaves out the low terms' product, 2^-18: 2.5 * 2^-17 = 1.9e-5 if
all agreed, so 4e-5.  A decay of 0 has a gradient of exactly 0.
"""
import pytest
import torch

import delta_reference as ref
from lm_reference import heads

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
BOUND = {F32: 2e-5, BF16: 4e-5}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _gradient(t, s0=None, df=None, lengths=None):
    import selective_state_space_68_amd as ssm
    d = {n: x.cuda() for n, x in t.items()}
    return ssm.gated_delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"],
                               initial_state=None if s0 is None else s0.cuda(),
                               dfinal_state=None if df is None else df.cuda(),
                               lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda())


def _want(t, s0=None, df=None, lengths=None):
    """(dg, sizes) [B, L, H] in float64; what absent tokens hold is cleared first."""
    B, L, H = t["g"].shape
    K, V = t["q"].shape[-1], t["v"].shape[-1]
    n = torch.full((B,), L) if lengths is None else torch.tensor(lengths)
    live = torch.arange(L)[None] < n[:, None]
    q, k, v = (torch.where(live[..., None, None], heads(t[x], H), 0.0) for x in "qkv")
    do = torch.where(live[..., None, None], t["do"].double(), 0.0)
    a = torch.where(live[..., None], t["g"].double().exp(), 1.0)[..., None, None]
    beta = torch.where(live[..., None], t["beta"].double(), 0.0)[..., None]
    S = [torch.zeros(B, H, K, V, dtype=torch.float64) if s0 is None else s0.double()]
    for i in range(L):
        old = S[-1] * a[:, i]
        u = beta[:, i] * (v[:, i] - (k[:, i, :, None] @ old)[:, :, 0])
        S.append(old + k[:, i, :, :, None] * u[:, :, None])
    P = torch.zeros(B, H, K, V, dtype=torch.float64) if df is None else df.double()
    dg, size = torch.zeros(B, L, H, dtype=torch.float64), torch.zeros(B, L, H, dtype=torch.float64)
    for i in range(L - 1, -1, -1):
        P = P + K ** -0.5 * q[:, i, :, :, None] * do[:, i, :, None]
        P = P - k[:, i, :, :, None] * (beta[:, i] * (k[:, i, :, None] @ P)[:, :, 0])[:, :, None]
        dg[:, i] = (P * S[i] * a[:, i]).sum((-1, -2)) * live[:, i, None]
        size[:, i] = a[:, i, :, 0, 0] * P.norm(dim=(-1, -2)) * S[i].norm(dim=(-1, -2)) * (K * V) ** -0.5 * live[:, i, None]
        P = P * a[:, i]
    return dg, size + dg.abs()


def _check(got, want, size, tol, what):
    """The worst token's error over its size; where it has none, exactly 0."""
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    none = size < 1e-37
    assert not (got[none].abs() > 1e-37).any(), what
    e = ((got - want).abs() / size.clamp(min=1e-37))[~none]
    if e.numel():
        print(f"{what}: {float(e.max()):.2e}", flush=True)
        assert float(e.max()) <= tol, (what, float(e.max()))
        assert float((want.abs() / size.clamp(min=1e-37))[~none].max()) > 100 * tol      # (zeros would not pass)


RATES = [-0.1, -0.5, -0.69, -0.8, -1.0, -2.0, -5.0, -8.0, -12.0, -20.0]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K,V,L,carried", [(64, 64, 150, True), (128, 128, 200, True), (128, 64, 65, False), (33, 100, 129, True),
                                           (64, 64, 1, True), (100, 36, 65, True), (64, 128, 1100, False)])
def test_one_decay_in_a_head(K, V, L, carried, dtype):
    """A head for each decay, a little different from token to token."""
    H = len(RATES)
    t, s0, df = ref.inputs(1, L, H, K, V, dtype, (H, 1, 2), seed=L + K)
    t["g"] = torch.tensor(RATES) * (0.9 + 0.2 * torch.rand(1, L, H, generator=torch.Generator().manual_seed(L)))
    s0, df = (s0, df) if carried else (None, None)
    want, size = _want(t, s0, df)
    if not carried:
        size[:, 0] = 0.0                                     # (nothing to scale)
    got = _gradient(t, s0, df)["dg"]
    for h, rate in enumerate(RATES):
        if rate > -1.0:                                      # a head's tokens share their sums
            size[:, :, h] += size[:, :, h].square().mean(1, keepdim=True).sqrt() * (size[:, :, h] > 0)
        _check(got[..., h], want[..., h], size[..., h], BOUND[dtype], f"{rate}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("reset", [-3.0, -8.0, -16.0, -30.0, float("-inf")])
@pytest.mark.parametrize("at", [[0], [63], [64], [5, 130], [31, 32, 190], list(range(0, 200, 7))])
def test_resets_in_a_slow_head(at, reset, dtype):
    """The reset's own gradient carries its factor; the others' are those of slow tokens."""
    L, H = 200, 2
    t, s0, df = ref.inputs(1, L, H, 64, 64, dtype, seed=at[0])
    t["g"] = -0.02 * torch.rand(1, L, H, generator=torch.Generator().manual_seed(1))
    t["g"][:, at, 0] = reset
    want, size = _want(t, s0, df)
    got = _gradient(t, s0, df)["dg"]
    rest = [i for i in range(L) if i not in at]
    if reset == float("-inf"):
        assert not got[:, at, 0].any()
    else:
        _check(got[:, at, 0], want[:, at, 0], size[:, at, 0], BOUND[dtype], f"reset {reset}")
    for h, some in ((0, rest), (1, list(range(L)))):
        s = size[:, some, h] + want[:, some, h].square().mean().sqrt()
        _check(got[:, some, h], want[:, some, h], s, BOUND[dtype], f"head {h}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K,V,L,carried", [(64, 64, 150, True), (128, 128, 200, False), (100, 36, 65, True)])
def test_strengths_head_by_head(K, V, L, carried, dtype):
    """beta's gradient, y.w of float32 rows from 24-bit operands in either type, against the size of its own head's."""
    import selective_state_space_68_amd as ssm
    H = len(RATES)
    t, s0, df = ref.inputs(2, L, H, K, V, dtype, (H, 1, 2), seed=L + V)
    t["g"] = torch.tensor(RATES) * (0.9 + 0.2 * torch.rand(2, L, H, generator=torch.Generator().manual_seed(L)))
    s0, df = (s0, df) if carried else (None, None)
    want = ref.delta_grad(*t.values(), K ** -0.5, s0, df)["dbeta"]
    got = ssm.gated_delta_bwd(*(t[n].cuda() for n in ("q", "k", "v", "g", "beta", "do")),
                              initial_state=None if s0 is None else s0.cuda(),
                              dfinal_state=None if df is None else df.cuda())["dbeta"]
    for b in range(2):
        for h, rate in enumerate(RATES):
            size = want[b, :, h].abs() + want[b, :, h].square().mean().sqrt()
            _check(got[b, :, h], want[b, :, h], size, BOUND[F32], f"{b} {rate}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ragged_rows(dtype):
    """Chunks of one token and of none, NaN in absent ones."""
    L, H, lengths = 200, 4, [200, 0, 1, 64, 65, 129]
    t, s0, df = ref.inputs(6, L, H, 64, 64, dtype, seed=3)
    t["g"] = torch.tensor([-0.3, -3.0, -9.0, -15.0]) * (0.9 + 0.2 * torch.rand(6, L, H, generator=torch.Generator().manual_seed(2)))
    absent = torch.arange(L)[None] >= torch.tensor(lengths)[:, None]
    want, size = _want(t, s0, df, lengths)
    for n in t:
        t[n][absent] = float("nan")
    got = _gradient(t, s0, df, lengths)["dg"]
    assert not got.cpu()[absent].any()
    for b in range(6):
        for h in range(H):
            n = lengths[b]
            if n:
                s = size[b, :n, h] + (size[b, :n, h].square().mean().sqrt() if h == 0 else 0.0)
                _check(got[b, :n, h], want[b, :n, h], s, BOUND[dtype], f"{b} {h}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_stretches_of_several_chunks(dtype):
    """Enough heads for kept states to lie several chunks apart; fast and slow chunks in turn in one of them."""
    B, L, H = 8, 1150, 16
    t, s0, df = ref.inputs(B, L, H, 64, 64, dtype, seed=12)
    gen = torch.Generator().manual_seed(3)
    rate = torch.logspace(-3, 1, H)
    t["g"] = -rate * torch.rand(B, L, H, generator=gen)
    t["g"][:, :, 0] = -torch.where(torch.arange(L) // 100 % 2 == 1, 2.0, 0.01) * torch.rand(B, L, generator=gen)
    got = _gradient(t, s0, df)["dg"]
    for b, h in ((0, 0), (0, 4), (3, 8), (3, 10), (7, 12), (7, 13), (7, 15)):
        one = {n: x[b:b + 1, :, h:h + 1] for n, x in t.items()}
        want, size = _want(one, s0[b:b + 1, h:h + 1], df[b:b + 1, h:h + 1])
        size = size + want.square().mean(1, keepdim=True).sqrt()
        _check(got[b:b + 1, :, h:h + 1], want, size, BOUND[dtype], f"{b} {h}")
